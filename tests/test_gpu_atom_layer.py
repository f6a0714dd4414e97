"""The new operators together, as a training step of the atom attention uses them: projections
(linear), the windowed core, the output projection added to the residual stream (linear's
epilogue), and back through linear_backward and atom_attention_backward, with the input
kept as it is or in 8 bits; against float64 autograd of the same layer.

Tolerance. On the way to any gradient a value is rounded to bf16 at most nine times (q, k, v, o, p,
do, ds, dq / dk / dv, and the result; the input itself is exact on both sides), each by at most
u = 2^-8 relative. Roundings are independent, so as root mean squares (u / sqrt(3) each at most) nine
add to sqrt(9 / 3) u = 1.7 u; q and k enter the softmax's exponent, where |logit| of about 1.5 carries
their two roundings into p by as much again, and p enters ds with both signs. 4 u of the norm
covers these sums with a factor of about 2.
"""
import math

import numpy as np
import pytest
import torch

import pair_representation_b200 as tm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TOL = 4 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def reference(x, sd, bias, mask, heads):
    """The layer in float64 torch operations."""
    B, n, c = x.shape
    lin = lambda name, t: torch.nn.functional.linear(t, sd[f"linear_{name}.weight"], sd.get(f"linear_{name}.bias"))  # noqa: E731
    q, k, v = (lin(name, x).view(B, n, heads, 32) for name in "qkv")
    W = -(-n // 32)
    slot = torch.arange(W)[:, None] * 32 - 48 + torch.arange(128)[None]
    ok = ((slot >= 0) & (slot < n))[None].expand(B, W, 128).clone()
    at = slot.clamp(0, n - 1)
    if mask is not None:
        ok &= mask[:, at] != 0
    row = (torch.arange(W)[:, None] * 32 + torch.arange(32)[None]).clamp(max=n - 1)
    a = torch.einsum("bwqhd,bwkhd->bwhqk", q[:, row], k[:, at]) / math.sqrt(32)
    if bias is not None:
        a = a + bias
    some = ok.any(-1)[:, :, None, None, None]
    a = torch.where(ok[:, :, None, None, :], a, torch.where(some, -math.inf, 0.0))
    o = torch.einsum("bwhqk,bwkhd->bwqhd", torch.softmax(a, -1) * some, v[:, at])
    o = o.reshape(B, W * 32, heads * 32)[:, :n]
    return x + lin("o", o)


def make(B, n, c, heads, biases, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    d = heads * 32
    sd = {f"linear_{name}.weight": r(d, c) * c ** -0.5 for name in "qkv"}
    sd["linear_o.weight"] = r(c, d) * d ** -0.5
    if biases:
        sd |= {f"linear_{name}.bias": r(d) * 0.3 for name in "qkv"}
        sd["linear_o.bias"] = r(c) * 0.3
    sd = {k: v.to(torch.bfloat16) for k, v in sd.items()}
    mask = torch.ones(B, n)
    mask[:, n - max(1, n // 15):] = 0
    return r(B, n, c), r(B, n, c), r(B, -(-n // 32), heads, 32, 128), mask.to(torch.bfloat16), sd


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("B,n,c,heads,biases", [(2, 150, 128, 4, True), (1, 333, 64, 2, False), (1, 97, 256, 5, True)])
def test_layer_forward_and_backward(B, n, c, heads, biases, held):
    x, dout, bias, mask, sd = make(B, n, c, heads, biases, seed=n)
    layer = tm.AtomAttention(c, heads).load_state_dict(sd).to(DEV)
    xd = x.to(DEV)
    kept = tm.act8_pack(xd) if held else xd
    y = layer(xd, bias.to(DEV), mask.to(DEV))
    dx, dbias, grads = layer.backward(kept, dout.to(DEV), bias.to(DEV), mask.to(DEV))
    assert tm.device_status(DEV)[0] == 0

    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    ref = reference(x.double(), {k: v.double() for k, v in sd.items()}, bias.double(), mask, heads)
    rel = lambda got, want: (got.double().cpu() - want).norm() / want.norm()  # noqa: E731
    assert rel(y, ref) <= TOL
    # The backward's x: the values that were kept.
    x64 = leaf(tm.act8_unpack(kept).cpu() if held else x)
    sd64, b64 = {k: leaf(v) for k, v in sd.items()}, leaf(bias)
    if not biases:
        sd64 |= {f"linear_{k}.bias": torch.zeros(grads[f"linear_{k}.bias"].numel(), dtype=torch.float64).requires_grad_()
                 for k in "qkvo"}
    out = reference(x64, sd64, b64, mask, heads)
    names = list(sd64)
    want = torch.autograd.grad((out * dout.double()).sum(), [x64, b64] + [sd64[k] for k in names])
    assert rel(dx, want[0]) <= TOL, float(rel(dx, want[0]))
    assert rel(dbias, want[1]) <= TOL, float(rel(dbias, want[1]))
    assert set(grads) == set(names)
    for k, g in zip(names, want[2:]):
        if k == "linear_k.bias":
            # The same shift of every key leaves the softmax as it is: the exact gradient is 0 but for rows
            # without a key, and what is left is the roundings' sum. Small beside dq's rows.
            assert grads[k].double().norm() <= TOL * grads["linear_q.bias"].double().norm() * math.sqrt(B * n)
            continue
        assert rel(grads[k], g) <= TOL, (k, float(rel(grads[k], g)))


def test_step_in_a_graph_on_two_streams():
    """Forward, packing and backward captured once and replayed, while the same layer runs eagerly on
    another stream: every result equals the plain call's, bit for bit."""
    x, dout, bias, mask, sd = make(1, 200, 128, 4, True, seed=5)
    layer = tm.AtomAttention(128, 4).load_state_dict(sd).to(DEV)
    x, dout, bias, mask = (t.to(DEV) for t in (x, dout, bias, mask))

    def step():
        y = layer(x, bias, mask)
        return (y,) + layer.backward(tm.act8_pack(x), dout, bias, mask)

    flat = lambda r: [r[0], r[1], r[2], *(r[3][k] for k in sorted(r[3]))]  # noqa: E731
    ref = [t.clone() for t in flat(step())]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = flat(step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        g.replay()
        with torch.cuda.stream(side):
            eager = flat(step())
    torch.cuda.synchronize()
    for a, b, c in zip(ref, got, eager):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    x, dout, bias, mask, sd = make(1, 64, 128, 4, False, seed=6)
    with pytest.raises(KeyError):
        tm.AtomAttention(128, 4).load_state_dict({k: v for k, v in sd.items() if "_v" not in k})
    with pytest.raises(ValueError):
        tm.AtomAttention(128, 2).load_state_dict(sd)
    layer = tm.AtomAttention(128, 4).load_state_dict(sd).to(DEV)
    with pytest.raises(ValueError):
        layer(x.to(DEV)[0])
    with pytest.raises(ValueError):
        layer(x.to(DEV)[:, :, :64].contiguous())
    with pytest.raises(ValueError):
        layer.backward(x.to(DEV), dout.to(DEV)[:, :10])
