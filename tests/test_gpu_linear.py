"""GPU parity of the linear layer and its gradients (trimul_linear_forward / backward, through the
C ABI) against the float64 oracle (oracle/linear.py).

Tolerances, per element. u = 2^-8 is the largest relative error of one rounding to bf16, e = 2^-23
that of an fp32 operation (the tensor core's sums may truncate). A sum of K products kept in fp32
is off by at most (K + 4) e times the sum of their sizes S.
  forward   p is off by dp = (K + 4) e (S + |b|); an activation's slope is at most 1.1 and its own
            evaluation (hardware exponential and reciprocal, about 2^-21) 2^-19 of its size;
            the residual's addition adds e |r|; then one rounding: u |y|.
  D         dy act'(p): act' has slope at most 1 (0 for identity; relu's inputs here are on a grid
            where p is exact), so D is off by |dy| (dp + 2^-18); rounding D to bf16 adds u |D| for
            sigmoid and silu only.
  dx, dW    sums of these: the D errors times the other factor, summed, plus (K + 4) e of the sizes,
            plus the final rounding.
  db        sums D before its rounding.
"""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from gpu_helpers import as_bf16
from oracle.linear import linear as oracle_linear, linear_backward as oracle_backward

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U, E = 2.0 ** -8, 2.0 ** -23
ACTS = ("none", "relu", "sigmoid", "silu")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def draw(rows, k, n, seed, grid=False):
    rng = np.random.default_rng([rows, k, n, seed])
    if grid:  # multiples of 1/4 and 1/8: every product and sum is exact, p = 0 included
        x = rng.integers(-8, 9, size=(rows, k)) / 4
        w = rng.integers(-8, 9, size=(n, k)) / 8
        b = rng.integers(-8, 9, size=n) / 8
    else:
        x = rng.standard_normal((rows, k)) * rng.uniform(0.5, 2, size=k)
        w = rng.standard_normal((n, k)) / np.sqrt(k)
        b = rng.standard_normal(n)
    return [as_bf16(t) for t in (x, w, b, rng.standard_normal((rows, n)))]


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(torch.bfloat16)


def within(got, ref, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tol
    assert over.max() <= 0, float(over.max())


def check_forward(rows, k, n, act, bias, residual, seed=0):
    x, w, b, r = draw(rows, k, n, seed)
    b, r = (b if bias else None), (r if residual else None)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    y = tm.linear(dev(x), dev(w), bias=dev(b), residual=dev(r), act=act, workspace=ws)
    rc, detail = tm.device_status(ws)
    assert rc == 0, (rc, detail)
    ref = oracle_linear(x, w, b, r, act)
    size = np.abs(x).astype(np.float64) @ np.abs(w).astype(np.float64).T + (0 if b is None else np.abs(b))
    inner = ref if r is None else ref - r
    within(y, ref, U * np.abs(ref) + 1.1 * (k + 4) * E * size + 2.0 ** -19 * np.abs(inner) +
           (0 if r is None else E * np.abs(r)))


SIZES = [(1, 8, 8), (1, 128, 128), (2, 40, 16), (31, 64, 64), (33, 72, 56), (127, 128, 128), (128, 136, 120),
         (129, 256, 264), (257, 320, 512), (300, 512, 128), (1000, 200, 328), (64, 1024, 1024), (2500, 128, 512)]


@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(rows, k, n, act):
    odd = (rows + k) % 3
    check_forward(rows, k, n, act, bias=odd != 0, residual=odd != 1)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_forward_many_rows(bias, residual):
    """More row tiles than SMs: every CTA goes round its ring, its accumulators and its buffers."""
    check_forward(148 * 128 * 2 + 77, 72, 72, "silu", bias, residual)
    check_forward(148 * 128 + 1, 128, 264, "sigmoid", bias, residual)


def test_forward_widest():
    check_forward(200, 64, 10944, "relu", True, True)
    check_forward(130, 72, 16384, "none", True, False)
    check_forward(3, 16384, 40, "none", True, False)


def check_backward(rows, k, n, act, bias=True, held=False, seed=1):
    x, w, b, dy = draw(rows, k, n, seed, grid=act == "relu")
    b = b if bias else None
    xt = dev(x)
    if held:
        a = tm.act8_pack(xt)
        x = tm.act8_unpack(a).float().cpu().numpy()
        if act == "relu":  # 8 bits hold these multiples of 1/4 exactly
            assert np.array_equal(x, xt.float().cpu().numpy())
        xt = a
    need = tm.trimul_linear_backward_workspace_size(rows, k, n, tm.ACTS[act], held)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV)
    dx, dw, db = tm.linear_backward(xt, dev(w), dev(dy), bias=dev(b), act=act, workspace=ws)
    rc, detail = tm.device_status(ws)
    assert rc == 0, (rc, detail)
    rx, rw, rb, D = oracle_backward(x, w, dy, b, act)
    ax, aw, ay, aD = (np.abs(np.asarray(t, np.float64)) for t in (x, w, dy, D))
    smooth = act in ("sigmoid", "silu")
    dD = ay * ((k + 4) * E * (ax @ aw.T + (0 if b is None else np.abs(b))) + 2.0 ** -18) if smooth else np.zeros_like(aD)
    dDr = dD + (U * (aD + dD) if smooth else 0)
    within(dx, rx, U * np.abs(rx) + 1.01 * (dDr @ aw + (n + 4) * E * (aD @ aw)))
    within(dw, rw, U * np.abs(rw) + 1.01 * (dDr.T @ ax + (rows + 4) * E * (aD.T @ ax)))
    within(db, rb, U * np.abs(rb) + 1.01 * (dD.sum(0) + (rows + 4) * E * aD.sum(0)))
    # As whole arrays: the roundings are of random sign, so two of them stay under 1.5 u.
    for got, ref in ((dx, rx), (dw, rw)):
        if ref.size > 64 and np.linalg.norm(ref):
            assert np.linalg.norm(got.double().cpu().numpy() - ref) <= 1.5 * U * np.linalg.norm(ref)


@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_backward(rows, k, n, act):
    check_backward(rows, k, n, act, bias=(rows + n) % 3 != 0)


@pytest.mark.parametrize("rows,k,n", [(1, 32, 8), (5, 64, 24), (129, 96, 136), (1000, 128, 512), (700, 512, 128),
                                      (333, 128, 128)])
@pytest.mark.parametrize("act", ACTS)
def test_backward_from_8_bits(rows, k, n, act):
    check_backward(rows, k, n, act, held=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("held", [True, False])
@pytest.mark.parametrize("k,n", [(128, 128), (96, 200), (64, 264), (128, 392), (128, 512), (160, 72)])
def test_backward_many_rows(k, n, act, held):
    """More row tiles than teams of CTAs, for each way the backward is done."""
    check_backward(148 * 128 + 77, k, n, act, held=held)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_parts_of_the_backward(act):
    """Each gradient alone equals the one of the whole call, bit for bit."""
    x, w, b, dy = (dev(t) for t in draw(500, 96, 160, 2))
    for xx in (x, tm.act8_pack(x)):
        full = tm.linear_backward(xx, w, dy, bias=b, act=act)
        for i in range(3):
            part = tm.linear_backward(xx, w, dy, bias=b, act=act, need_dx=i == 0, need_dw=i == 1, need_db=i == 2)
            assert [t is None for t in part] == [j != i for j in range(3)]
            assert torch.equal(part[i], full[i])
        assert tm.linear_backward(xx, w, dy, act=act, need_dx=False, need_dw=False, need_db=False) == (None,) * 3


def test_equal_calls_give_equal_bits():
    x, w, b, dy = (dev(t) for t in draw(20000, 128, 256, 3))
    for act in ("none", "sigmoid"):
        first = tm.linear_backward(x, w, dy, bias=b, act=act)
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(first, tm.linear_backward(x, w, dy, bias=b, act=act)))


def test_infinities_and_nan():
    """A NaN in a row of x reaches that row of y alone; large and infinite pre-activations end at the
    activation's limits."""
    x, w, b, _ = draw(300, 64, 64, 4)
    x[17, 3] = np.nan
    for act in ACTS:
        y = tm.linear(dev(x), dev(w), bias=dev(b), act=act).float().cpu().numpy()
        assert np.isnan(y[17]).all() and np.isfinite(np.delete(y, 17, 0)).all(), act
    p = np.array([-3e38, -1e5, -200, -90, -80, 0, 80, 200, 1e5, 3e38], np.float32)
    x = np.zeros((len(p), 8), np.float32)
    x[:, 0] = as_bf16(p)
    w = np.eye(8, dtype=np.float32)
    with np.errstate(over="ignore"):
        for act in ACTS:
            y = tm.linear(dev(x), dev(w), act=act).double().cpu().numpy()
            ref = oracle_linear(x, w, act_name=act)
            assert np.isfinite(y).all()
            assert (np.abs(y - ref) <= U * np.abs(ref) + 1e-34).all(), act
            dx, _, _ = tm.linear_backward(dev(x), dev(w), dev(np.ones((len(p), 8))), act=act)
            rx = oracle_backward(x, w, np.ones((len(p), 8)), act_name=act)[0]
            assert (np.abs(dx.double().cpu().numpy() - rx) <= 2.1 * U * np.abs(rx) + 1e-34).all(), act


def test_residual_in_place():
    x, w, b, r = (dev(t) for t in draw(1500, 128, 200, 5))
    ref = tm.linear(x, w, bias=b, residual=r, act="silu")
    got = tm.linear(x, w, bias=b, residual=r, act="silu", out=r)
    assert got is r and torch.equal(got, ref)


@pytest.mark.parametrize("rows,k,n", [(77, 72, 136), (19000, 96, 200), (19000, 128, 392), (77, 160, 72), (19000, 160, 72),
                                      (19000, 72, 520)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_nothing_around_the_outputs_is_written(rows, k, n, act):
    """Outputs and workspace inside larger buffers, the workspace exactly as large as it has to be."""
    x, w, b, dy = (dev(t) for t in draw(rows, k, n, 6))

    def frame(count):
        t = torch.full((count + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
        return t, t[128:128 + count]

    (fy, y), (fx, dx), (fw, dw), (fb, db) = (frame(c) for c in (rows * n, rows * k, n * k, n))
    need = tm.trimul_linear_backward_workspace_size(rows, k, n, tm.ACTS[act])
    fws = torch.full((need + (1 << 20),), 9, dtype=torch.uint8, device=DEV)
    p = tm.LinearParams(rows, k, n, tm.ACTS[act], w.data_ptr(), b.data_ptr(), fws.data_ptr(), need, 0)
    tm.trimul_linear_forward(x, None, p, y)
    tm.trimul_linear_backward(x, None, dy, p, dx, dw, db)
    torch.cuda.synchronize()
    for f, v in ((fy, y), (fx, dx), (fw, dw), (fb, db)):
        assert (f[:128] == 7).all() and (f[128 + v.numel():] == 7).all()
    assert (fws[need:] == 9).all()
    assert torch.equal(y.view(rows, n), tm.linear(x, w, bias=b, act=act))
    for v, t in zip((dx, dw, db), tm.linear_backward(x, w, dy, bias=b, act=act)):
        assert torch.equal(v.view(t.shape), t)


def test_leading_dimensions_empty_batches_streams_and_graphs():
    x, w, b, dy = (dev(t) for t in draw(240, 64, 96, 7))
    y = tm.linear(x, w, bias=b, act="sigmoid")
    assert torch.equal(tm.linear(x.view(4, 5, 12, 64), w, bias=b, act="sigmoid"), y.view(4, 5, 12, 96))
    grads = tm.linear_backward(x, w, dy, bias=b, act="sigmoid")
    got = tm.linear_backward(x.view(4, 60, 64), w, dy.view(4, 60, 96), bias=b, act="sigmoid")
    assert got[0].shape == (4, 60, 64) and all(torch.equal(p.reshape(-1), q.reshape(-1)) for p, q in zip(got, grads))
    assert tm.linear(x[:0], w).shape == (0, 96) and tm.linear(x, w[:0]).shape == (240, 0)
    dx, dw, db = tm.linear_backward(x, w[:0], dy[:, :0].contiguous())
    assert (dx == 0).all() and dx.shape == (240, 64) and dw.shape == (0, 64) and db.shape == (0,)
    dx, dw, db = tm.linear_backward(x[:0], w, dy[:0])
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = tm.linear_backward(x, w, dy, bias=b, act="sigmoid", stream=side)
    y2 = tm.linear(x, w, bias=b, act="sigmoid", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(p, q) for p, q in zip(got, grads))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3 = tm.linear(x, w, bias=b, act="sigmoid")
        got = tm.linear_backward(x, w, dy, bias=b, act="sigmoid")
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, y) and all(torch.equal(p, q) for p, q in zip(got, grads))


@pytest.mark.parametrize("rows,k,n", [(20000, 128, 512), (700, 128, 392), (20000, 320, 136), (90, 128, 128)])
@pytest.mark.parametrize("held", [False, True])
def test_replayed_while_others_run(rows, k, n, held):
    """Each way of the backward captured and replayed, with the forward, while the same calls run eagerly on
    another stream and a second graph of them is replayed: all give the plain call's bits."""
    x, w, b, dy = (dev(t) for t in draw(rows, k, n, 9))
    xx = tm.act8_pack(x) if held else x
    step = lambda: (tm.linear(x, w, bias=b, act="silu"), *tm.linear_backward(xx, w, dy, bias=b, act="silu"))  # noqa: E731
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = step()
    torch.cuda.synchronize()
    for got in (*outs, eager):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_refusals():
    x, w, b, dy = (dev(t) for t in draw(10, 64, 32, 8))
    bad = [lambda: tm.linear(x.float(), w), lambda: tm.linear(x.t(), w), lambda: tm.linear(x, w.t()),
           lambda: tm.linear(x, w, bias=b[:8]), lambda: tm.linear(x, w, act="tanh"),
           lambda: tm.linear(x, w, residual=dy[:5]), lambda: tm.linear(x, w, out=dy[:5]),
           lambda: tm.linear(x.cpu(), w), lambda: tm.linear_backward(x, w, x), lambda: tm.linear_backward(x[:5], w, dy),
           lambda: tm.linear_backward(tm.act8_pack(x[:, :32].contiguous()), w, dy), lambda: tm.act8_pack(x[:, :40]),
           lambda: tm.act8_pack(x[:, :40].contiguous())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    small = torch.zeros(128, dtype=torch.uint8, device=DEV)
    for f in (lambda: tm.linear(x, w, workspace=small), lambda: tm.linear_backward(x, w, dy, workspace=small),
              lambda: tm.linear(x[:, :60].contiguous(), w[:, :60].contiguous()),
              lambda: tm.linear(dy, dev(np.eye(32)), out=dy)):
        with pytest.raises(tm.TrimulError):
            f()


@pytest.mark.parametrize("k,n", [(128, 128), (128, 512), (160, 136)])
def test_relu_sign_under_a_large_bias(k, n):
    """Sums near 1000 that the bias takes back to 0: fp32's rounding is then larger than many p, and the
    gradient is still that of the exact sign. dy is 1 or -1, so db is a whole number under 256 and exact."""
    rng = np.random.default_rng([k, n, 31])
    x, w = rng.standard_normal((500, k)) * 0.01, rng.standard_normal((n, k))
    x[:, 0], w[:, 0] = 1000, 1
    x, w, b = as_bf16(x), as_bf16(w), np.full(n, -1000.0, np.float32)
    dy = rng.choice([-1.0, 1.0], size=(500, n)).astype(np.float32)
    p = x.astype(np.float64) @ w.astype(np.float64).T + b
    assert (np.abs(p) < 1000 * 2.0 ** -23).sum() > 0
    db = tm.linear_backward(dev(x), dev(w), dev(dy), bias=dev(b), act="relu")[2]
    ref = np.where(p > 0, dy, 0).sum(axis=0)
    assert np.abs(ref).max() <= 256
    assert np.array_equal(db.double().cpu().numpy(), ref)


@pytest.mark.parametrize("rows", [1, 300, 3000])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("held", [False, True])
def test_parts_of_the_backward_in_several_products(rows, act, held):
    """Each choice of gradients, where every one is a product of its own: those of the whole call, bit for bit.
    (With act none, db comes with dW's product, whose own result may not be wanted.)"""
    x, w, b, dy = (dev(t) for t in draw(rows, 160, 200, 13))
    xx = tm.act8_pack(x) if held else x
    whole = tm.linear_backward(xx, w, dy, bias=b, act=act)
    for i in range(7):
        need = [bool(i & 1 << j) for j in range(3)]
        ws = torch.zeros(tm.trimul_linear_backward_workspace_size(rows, 160, 200, tm.ACTS[act], held), dtype=torch.uint8,
                         device=DEV)
        part = tm.linear_backward(xx, w, dy, b, act, *need, workspace=ws)
        assert tm.device_status(ws)[0] == 0
        for want, p, q in zip(need, part, whole):
            assert (p is not None) == want and (p is None or torch.equal(p, q))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,k,n", [(37800, 264, 72), (60001, 320, 72), (37800, 72, 520), (19000, 320, 360), (37800, 560, 40),
                                      (60001, 520, 64)])
def test_tall_tiles(rows, k, n, act):
    """Contractions too long for W to stay on chip, over rows enough for tiles of 256: a last one that is cut,
    several rounds of them, several column tiles."""
    check_forward(rows, k, n, act, True, act != "relu")
    check_backward(rows, k, n, act)


@pytest.mark.parametrize("n", [8, 64, 72, 128, 256, 264, 384, 512])
@pytest.mark.parametrize("rows", [100, 20000, 60001])
def test_every_length_of_the_contraction(rows, n):
    """1 to 17 blocks of 64: each place in the ring where a tile may end, with W on chip and streamed, tiles of 128 and
    256 rows. Whole numbers small enough that every sum, the bias with it, is exact in fp32: one rounding."""
    gen = torch.Generator(device=DEV).manual_seed(rows + n)
    whole = lambda *s: torch.randint(-4, 5, s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    b = torch.arange(n, device=DEV).remainder(97).to(torch.bfloat16)
    for blocks in range(1, 18):
        x, w = whole(rows, 64 * blocks), whole(n, 64 * blocks)
        # 1088 products of at most 16 and the bias: under 2^15, exact in fp32 in any order
        ref = torch.nn.functional.linear(x.double(), w.double(), b.double())
        assert torch.equal(tm.linear(x, w, b), ref.to(torch.bfloat16))


@pytest.mark.parametrize("k,n", [(160, 72), (128, 128), (96, 256), (128, 512), (320, 384), (72, 520)])
def test_backward_over_every_number_of_row_blocks(k, n):
    """1 to 20 blocks of 64 rows, and 1 to 4 tiles for each CTA of the form in one pass, all sums exact in fp32 (whole
    numbers up to 4: at most 76001 products of 16, under 2^24): one rounding. relu with a bias that makes p no whole
    number, so that no sign is in doubt."""
    gen = torch.Generator(device=DEV).manual_seed(k + n)
    whole = lambda *s: torch.randint(-4, 5, s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    w, b = whole(n, k), torch.full((n,), 0.5, device=DEV, dtype=torch.bfloat16)
    for rows in [64 * i - i % 3 for i in range(1, 21)] + [19000, 38000, 57000, 76001]:
        x, dy = whole(rows, k), whole(rows, n)
        for act in ("none", "relu"):
            D = dy.double()
            if act == "relu":
                D = D * (x.double() @ w.double().T + 0.5 > 0)
            ref = (D @ w.double(), D.T @ x.double(), D.sum(0))
            for got, want in zip(tm.linear_backward(x, w, dy, b, act), ref):
                assert torch.equal(got, want.to(torch.bfloat16)), (rows, act)
