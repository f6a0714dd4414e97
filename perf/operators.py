"""Timed cases of the operators that train the layers around the triangle update and the atom
attention: a linear layer with its epilogue, its gradients, the gradients of windowed atom
attention, and activations kept in 8 bits between the forward and the backward.

Every case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run`
makes one pass (the framework's kernels where `own` is true, elementary torch operations in 32
bits otherwise), `work` counts the bytes and operations the pass cannot do without and `exact`
computes the outputs in 64 bits from the definitions.

    linear           y = act(x W^T + b) + r                         x [rows][k], W [n][k]
    linear_backward  D = dy * act'(x W^T + b); dx = D W, dW = D^T x, db = sum of D over rows
                     (x may be held in 8 bits)
    attention_backward  dq, dk, dv, dbias of atom attention, windows of 32 queries x 128 keys
    checkpoint       x -> E4M3 codes with one E8M0 scale per 32 channels -> x
"""
import math

import torch

own = False

BF16 = torch.bfloat16
QW, KW, KOFF, HEAD = 32, 128, 48, 32  # window w: queries 32w .. 32w+31, keys 32w-48 .. 32w+79


def listed():
    return [
        # One short chain's atom features through a gate: the call's latency.
        dict(name="linear_gate_short", op="linear", rows=100, k=128, n=128, act="sigmoid", bias=True, residual=False),
        # A transition's widening projection over every cell of a 768-residue pair representation.
        dict(name="linear_widen_pair768", op="linear", rows=768 * 768, k=128, n=512, act="silu", bias=True,
             residual=False),
        # Its narrowing projection added to the residual stream, 384 residues.
        dict(name="linear_narrow_pair384", op="linear", rows=384 * 384, k=512, n=128, act="none", bias=True,
             residual=True),
        # One row per residue of a four-chain complex, widths that no tile divides.
        dict(name="linear_ragged", op="linear", rows=3605, k=200, n=328, act="relu", bias=True, residual=True),
        # Gradients of a projection of 64 residues' features: the call's latency.
        dict(name="linear_bwd_short", op="linear_backward", rows=64, k=128, n=128, act="none", bias=True, held8=False),
        # Gradients of a gate over the atoms of a training batch.
        dict(name="linear_bwd_gate_atoms", op="linear_backward", rows=8 * 18432, k=128, n=128, act="sigmoid",
             bias=True, held8=False),
        # Gradients of a transition's widening projection whose input was kept in 8 bits.
        dict(name="linear_bwd_widen_held8", op="linear_backward", rows=384 * 384, k=128, n=512, act="silu", bias=True,
             held8=True),
        # Gradients at widths that no tile divides.
        dict(name="linear_bwd_ragged", op="linear_backward", rows=3605, k=328, n=200, act="relu", bias=True,
             held8=False),
        # A small batch of ragged molecules, padded atoms, three heads.
        dict(name="attention_bwd_small", op="attention_backward", batch=2, atoms=1237, heads=3, bias=True, mask="tail"),
        # The atoms of a training batch, four heads, pair bias, 5 % padding.
        dict(name="attention_bwd_batch", op="attention_backward", batch=8, atoms=18432, heads=4, bias=True,
             mask="tail"),
        # The pair representation of a 768-residue crop kept for the backward.
        dict(name="checkpoint_pair768", op="checkpoint", rows=768 * 768, channels=128),
        # A few atoms' features.
        dict(name="checkpoint_short", op="checkpoint", rows=1001, channels=96),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "attention_backward", "checkpoint"])
    if op in ("linear", "linear_backward"):
        held8 = op == "linear_backward" and rng.random() < 0.4
        unit = 32 if held8 else 8
        k = unit * _log(rng, 1, 1024 // unit)
        n = 8 * _log(rng, 1, 128)
        most = max(1, min(600000, int(3e8 / (k + 2 * n)), int(3e10 / (k * n))))
        case = dict(op=op, rows=min(most, _log(rng, 1, 600000)), k=k, n=n,
                    act=rng.choice(["none", "relu", "sigmoid", "silu"]), bias=rng.random() < 0.7)
        if op == "linear":
            case["residual"] = rng.random() < 0.5
        else:
            case["held8"] = held8
        return case
    if op == "attention_backward":
        batch, heads = rng.randint(1, 8), _log(rng, 1, 16)
        atoms = min(_log(rng, 1, 18432), max(1, 500000 // (batch * heads)))
        return dict(op=op, batch=batch, atoms=atoms, heads=heads, bias=rng.random() < 0.7,
                    mask=rng.choice(["none", "tail", "holes"]))
    channels = 32 * _log(rng, 1, 32)
    return dict(op=op, rows=min(_log(rng, 1, 600000), 70000000 // channels), channels=channels)


# ---- inputs -----------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(BF16)


def _features(g, rows, channels):
    """Activations: a scale of its own for each channel, as a residual stream has."""
    s = torch.rand(channels, generator=g, device="cuda") * 1.5 + 0.5
    return (torch.randn(rows, channels, generator=g, device="cuda") * s).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("linear", "linear_backward"):
        rows, k, n = case["rows"], case["k"], case["n"]
        s = dict(op=op, act=case["act"], x=_features(g, rows, k), w=_normal(g, n, k, scale=k ** -0.5),
                 b=_normal(g, n, scale=0.5) if case["bias"] else None)
        if op == "linear":
            s["r"] = _normal(g, rows, n) if case["residual"] else None
        else:
            s["dy"] = _normal(g, rows, n)
            if case["held8"]:
                s["codes"], s["scales"] = _encode(s.pop("x"))
        return s
    if op == "attention_backward":
        B, n, H = case["batch"], case["atoms"], case["heads"]
        s = dict(op=op, bias=None, mask=None)
        s["q"], s["k"], s["v"], s["do"] = (_normal(g, B, n, H, HEAD) for _ in range(4))
        if case["bias"]:
            s["bias"] = _normal(g, B, (n + QW - 1) // QW, H, QW, KW)
        if case["mask"] != "none":
            m = torch.ones(B, n, device="cuda")
            if case["mask"] == "tail":  # a padded batch: each molecule has its own length, 90 to 100 %
                u = torch.rand(B, 1, generator=g, device="cuda")
                m = (torch.arange(n, device="cuda") < (n * (0.9 + 0.1 * u)).ceil()).float()
            else:  # unresolved atoms, and a stretch long enough to leave windows without a key
                m = (torch.rand(B, n, generator=g, device="cuda") > 0.2).float()
                m[:, n // 3:n // 3 + 300] = 0
            s["mask"] = m.to(BF16)
        return s
    return dict(op=op, x=_features(g, case["rows"], case["channels"]))


# ---- the passes -------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "linear":
        return _linear(s["x"], s["w"], s["b"], s["r"], s["act"])
    if op == "linear_backward":
        x = s["x"] if "x" in s else _decode(s["codes"], s["scales"])
        return _linear_backward(x, s["w"], s["b"], s["dy"], s["act"])
    if op == "attention_backward":
        return _attention_backward(s["q"], s["k"], s["v"], s["do"], s["bias"], s["mask"])
    return _decode(*_encode(s["x"]))


def _run_own(s):
    import pair_representation_b200 as tm

    op = s["op"]
    if op == "linear":
        return tm.linear(s["x"], s["w"], bias=s["b"], residual=s["r"], act=s["act"])
    if op == "linear_backward":
        x = s["x"] if "x" in s else tm.Act8(s["codes"], s["scales"])
        dx, dw, db = tm.linear_backward(x, s["w"], s["dy"], bias=s["b"], act=s["act"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "attention_backward":
        dq, dk, dv, dbias = tm.atom_attention_backward(s["q"], s["k"], s["v"], s["do"], bias=s["bias"],
                                                       atom_mask=s["mask"])
        return dict(dq=dq, dk=dk, dv=dv, dbias=dbias)
    return tm.act8_unpack(tm.act8_pack(s["x"]))


def _linear(x, w, b, r, act):
    p = x.float() @ w.float().t()
    if b is not None:
        p += b.float()
    if act == "relu":
        p = torch.clamp_min(p, 0)
    elif act == "sigmoid":
        p = 1 / (1 + torch.exp(-p))
    elif act == "silu":
        p = p / (1 + torch.exp(-p))
    if r is not None:
        p += r.float()
    return p.to(BF16)


def _linear_backward(x, w, b, dy, act):
    x, w, d = x.float(), w.float(), dy.float()
    if act != "none":
        p = x @ w.t()
        if b is not None:
            p += b.float()
        if act == "relu":
            d = d * (p > 0)
        else:
            s = 1 / (1 + torch.exp(-p))
            # 1 - s from exp(-|p|), so that it keeps its digits where s is next to 1
            c = 1 / (1 + torch.exp(p))
            d = d * (s * c) if act == "sigmoid" else d * (s + p * s * c)
    return dict(dx=(d @ w).to(BF16), dw=(d.t() @ x).to(BF16), db=d.sum(0, dtype=torch.float64).to(BF16))


def _windows(t, count):
    """[B, n, ...] -> [B, count, 128, ...]: each window's keys, zeros outside the sequence."""
    B, n = t.shape[:2]
    pad = torch.zeros(B, KOFF + QW * (count - 1) + KW, *t.shape[2:], dtype=torch.float32, device=t.device)
    m = min(n, pad.shape[1] - KOFF)
    pad[:, KOFF:KOFF + m] = t[:, :m].float()
    at = torch.arange(count, device=t.device)[:, None] * QW + torch.arange(KW, device=t.device)
    return pad[:, at]


def _attention_backward(q, k, v, do, bias, mask):
    B, n, H, d = q.shape
    W = (n + QW - 1) // QW
    rows = lambda t: torch.nn.functional.pad(t.float(), (0, 0, 0, 0, 0, W * QW - n)).view(B, W, QW, H, d).transpose(2, 3)  # noqa: E731
    keys = lambda t: _windows(t, W).transpose(2, 3)  # [B, W, H, 128, d]  # noqa: E731
    qw, dow, kw, vw = rows(q), rows(do), keys(k), keys(v)
    valid = _windows(torch.ones(B, n, device=q.device) if mask is None else (mask != 0).float(), W) != 0
    valid = valid[:, :, None, None, :] & (torch.arange(W * QW, device=q.device).view(W, QW) < n)[None, :, None, :, None]
    scale = d ** -0.5
    a = qw @ kw.transpose(-1, -2) * scale
    if bias is not None:
        a = a + bias.float()
    a = torch.where(valid, a, -math.inf)
    top = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    dp = dow @ vw.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = ds @ kw * scale

    def joined(t):
        """Key gradients [B, W, H, 128, d] of the windows, added up where they overlap."""
        t = t.transpose(2, 3).reshape(B, W, KW // QW, QW, H, d)
        parts = [torch.nn.functional.pad(t[:, :, j], (0, 0, 0, 0, 0, 0, j, KW // QW - 1 - j)) for j in range(KW // QW)]
        full = (parts[0] + parts[1] + parts[2] + parts[3]).flatten(1, 2)
        full = full[:, KOFF:KOFF + n]
        return torch.nn.functional.pad(full, (0, 0, 0, 0, 0, n - full.shape[1])).to(BF16)

    return dict(dq=dq.transpose(2, 3).reshape(B, W * QW, H, d)[:, :n].to(BF16).contiguous(),
                dk=joined(ds.transpose(-1, -2) @ qw * scale), dv=joined(p.transpose(-1, -2) @ dow),
                dbias=None if bias is None else ds.to(BF16))


def _power_of_two(e):
    """2^e in 64 bits, from the exponent's bits."""
    return (e.to(torch.int64) + 1023 << 52).view(torch.float64)


def _encode(x):
    """bf16 [rows][channels] -> E4M3 codes (bytes) and E8M0 scales (bytes, one per 32 channels)."""
    v = x.float().view(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    # floor(log2 top) - 8 from the exponent of `top`, at least -127
    e = torch.clamp_min(torch.frexp(top).exponent - 9, -127)
    e = torch.where(top == 0, -127, e)
    q = torch.clamp(v * _power_of_two(-e), -448, 448).float()
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape)
    return codes, (e + 127).to(torch.uint8).squeeze(-1)


def _decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(*scales.shape, 32)
    return (v * _power_of_two(scales.to(torch.int64) - 127)[..., None]).to(BF16).view(codes.shape)


# ---- the least a pass moves and computes ------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, k, n = case["rows"], case["k"], case["n"]
        if op == "linear":
            moved = 2 * (m * k + n * k + m * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0))
            return {"bytes": moved, "flops": 2 * m * n * k}
        x = m * k * 33 / 32 if case["held8"] else 2 * m * k
        moved = x + 2 * (m * n + m * k + 2 * n * k + (2 if case["bias"] else 1) * n)
        return {"bytes": moved, "flops": (4 if case["act"] == "none" else 6) * m * n * k}
    if op == "attention_backward":
        B, n, H = case["batch"], case["atoms"], case["heads"]
        windows = B * H * ((n + QW - 1) // QW)
        moved = 7 * 2 * B * n * H * HEAD + (2 * B * n if case["mask"] != "none" else 0)
        if case["bias"]:
            moved += 2 * 2 * windows * QW * KW
        return {"bytes": moved, "flops": windows * 5 * 2 * QW * KW * HEAD}
    count = case["rows"] * case["channels"]
    return {"bytes": count * (2 + 33 / 32 + 33 / 32 + 2), "flops": 0}


# ---- the definitions, in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if op in ("linear", "linear_backward"):
        if "codes" in s:
            x = _exact_held(s["codes"], s["scales"])
        else:
            x = f64(s["x"])
        w, b = f64(s["w"]), f64(s["b"])
        train = op == "linear_backward"
        if b is None:
            b = torch.zeros(w.shape[0], dtype=torch.float64, device=w.device)
        for t in (x, w, b):
            t.requires_grad_(train)
        y = torch.nn.functional.linear(x, w, b)
        y = dict(none=lambda t: t, relu=torch.relu, sigmoid=torch.sigmoid, silu=torch.nn.functional.silu)[s["act"]](y)
        if train:
            gx, gw, gb = torch.autograd.grad(y, (x, w, b), f64(s["dy"]))
            return dict(dx=gx, dw=gw, db=gb)
        return y if s["r"] is None else y + f64(s["r"])
    if op == "attention_backward":
        return _exact_attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), f64(s["do"]), f64(s["bias"]), s["mask"])
    return _exact_checkpoint(f64(s["x"]))


def _exact_attention(q, k, v, do, bias, mask):
    """The forward window by window of one batch element and head at a time, differentiated."""
    B, n, H, d = q.shape
    W = -(-n // QW)
    out = [torch.zeros_like(t) for t in (q, k, v)] + [None if bias is None else torch.zeros_like(bias)]
    slot = torch.arange(W, device=q.device)[:, None] * QW - KOFF + torch.arange(KW, device=q.device)[None]
    query = torch.arange(W, device=q.device)[:, None] * QW + torch.arange(QW, device=q.device)[None]
    inside, there = (slot >= 0) & (slot < n), query < n
    slot, query = slot.clamp(0, n - 1), query.clamp(0, n - 1)
    for b in range(B):
        ok = inside if mask is None else inside & (mask[b][slot] != 0)
        some = (ok.any(-1)[:, None] & there)[..., None]
        for h in range(H):
            x = [t[b, :, h].clone().requires_grad_() for t in (q, k, v)]
            x += [] if bias is None else [bias[b, :, h].clone().requires_grad_()]
            a = torch.einsum("wqd,wkd->wqk", x[0][query], x[1][slot]) / math.sqrt(d)
            a = a if bias is None else a + x[3]
            a = torch.where(ok[:, None, :] & some, a, torch.where(some, -math.inf, 0.0))
            o = torch.einsum("wqk,wkd->wqd", torch.softmax(a, -1) * some, x[2][slot])
            got = torch.autograd.grad((o * do[b, :, h][query]).sum(), x)
            for t, y in zip(out, got):
                t[b, :, h] = y
    return dict(dq=out[0], dk=out[1], dv=out[2], dbias=out[3])


def _e4m3_values(device):
    """The value of each of the 256 codes: sign, 4 exponent bits with bias 7, 3 mantissa bits."""
    c = torch.arange(256, device=device)
    e, m = (c >> 3 & 15).double(), (c & 7).double()
    size = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _exact_two(e - 7))
    return torch.where(c & 127 == 127, math.nan, torch.where(c > 127, -size, size))


def _exact_two(e):
    return torch.tensor([2.0 ** i for i in range(-200, 200)], dtype=torch.float64, device=e.device)[e.long() + 200]


def _exact_held(codes, scales):
    v = _e4m3_values(codes.device)[codes.long()].view(*scales.shape, 32)
    return (v * _exact_two(scales.long() - 127)[..., None]).view(codes.shape)


def _exact_checkpoint(x):
    v = x.view(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    # frexp: top = m 2^e with m in [1/2, 1)
    size = _exact_two(torch.where(top == 0, -127, (torch.frexp(top).exponent - 1 - 8).clamp_min(-127)))
    u = v / size
    # Spacing of E4M3 next to |u|: 2^(exponent - 3), 2^-9 below 2^-6.
    step = _exact_two(torch.frexp(u.abs().clamp_min(2.0 ** -6)).exponent - 1 - 3)
    return (torch.clamp(torch.round(u / step) * step, -448, 448) * size).view(x.shape)
