"""GPU parity of atom attention's gradients (atomattn_backward, through the C ABI) against the
float64 oracle (oracle/atomattn_backward.py).

Tolerances, per element. u = 2^-8 is the largest relative error of one rounding to bf16.
  * p and ds enter the products rounded once: at most u per term, so u times the sum of the
    terms' sizes (the oracle returns those sums); the result is rounded once: u |result|.
  * In fp32: the logits (a sum of 32 products of size up to |q| |k|, plus the bias, off by at
    most 64 2^-24 (|q||k| + |bias|) < 2^-16 here, where |l| < 40) shift p by 2^-16 relative; the
    exponential, the sums over 128 slots and dp add 2^-20 or so relative to their terms. ds =
    p (dp - delta) then is off by up to 2^-15 p (|dp| + sum p |dp|). With E = 2^-15 times
    the largest |dp| (at most the largest |dout| |v| over a row, under 64 here), each
    gradient gets E times the sum of p times the other factor: bounded by E times the
    largest |k| or |q| (under 6) for dq and, four windows of 32 queries sharing a total
    weight under 128, 128 E for dk. These constants are far below u times the sizes for all
    but vanishing gradients: an absolute 2^-9 covers dq and dbias (64 2^-15 = 2^-9),
    and 2^-9 times 6 for dk, whose typical weight per key is about 1.
"""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from gpu_helpers import as_bf16
from oracle.atomattn_backward import atom_attention_backward as oracle_backward

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
ABS = (6 * 2.0 ** -9, 6 * 2.0 ** -9, 2.0 ** -9, 2.0 ** -9)  # dq, dk, dv, dbias
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def draw(B, n, H, seed, bias=True, mask="tail"):
    rng = np.random.default_rng([seed, 22])
    q, k, v, do = (as_bf16(rng.standard_normal((B, n, H, 32))) for _ in range(4))
    b = as_bf16(rng.standard_normal((B, (n + 31) // 32, H, 32, 128))) if bias else None
    m = None
    if mask != "none":
        m = np.ones((B, n), dtype=np.float32)
        if mask == "tail":
            m[:, n - max(1, n // 20):] = 0
            m[:, rng.integers(0, n, size=max(1, n // 50))] = 0
        elif mask == "gap":
            m[:, n // 3:n // 3 + 260] = 0
        elif mask == "zeros":
            m[:] = 0
        elif mask == "one":
            m[:] = 0
            m[:, n // 2] = 1
    return q, k, v, do, b, m


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(torch.bfloat16)


def run(q, k, v, do, b, m):
    ws = torch.zeros(tm.atomattn_workspace_size(), dtype=torch.uint8, device=DEV)
    got = tm.atom_attention_backward(dev(q), dev(k), dev(v), dev(do), dev(b), dev(m), workspace=ws)
    rc, detail = tm.device_status(ws)
    assert rc == 0, (rc, detail)
    return [None if t is None else t.double().cpu().numpy() for t in got]


def check(got, args):
    ref = oracle_backward(*args, sizes=True)
    for name, g, r, size, floor in zip(("dq", "dk", "dv", "dbias"), got, ref[:4], ref[4:], ABS):
        if r is None:
            assert g is None
            continue
        assert np.isfinite(g).all(), name
        over = np.abs(g - r) - (U * np.abs(r) + U * size + floor)
        assert over.max() <= 0, (name, float(over.max()))
        den = np.linalg.norm(r)
        if den:  # and as a whole: two roundings of random sign, each under u / sqrt(3) rms
            assert np.linalg.norm(g - r) <= 1.5 * U * den, (name, np.linalg.norm(g - r) / den)


@pytest.mark.parametrize("mask", ["tail", "none"])
@pytest.mark.parametrize("B,n,H", [(1, 1, 1), (1, 2, 2), (1, 31, 1), (1, 32, 2), (1, 33, 1), (2, 47, 3), (1, 48, 1),
                                   (1, 49, 2), (1, 80, 1), (2, 100, 4), (1, 128, 4), (1, 129, 2), (2, 257, 3),
                                   (1, 1000, 5), (3, 515, 16)])
def test_parity(B, n, H, mask):
    if mask == "tail" and n < 3:
        mask = "zeros"
    args = draw(B, n, H, seed=n + 7 * H, mask=mask)
    check(run(*args), args)


@pytest.mark.parametrize("n", [2049, 2080, 4000])
def test_long_chains(n):
    """Runs of many windows per block, and the ends of sequences inside and on group borders."""
    args = draw(7, n, 16, seed=n)
    check(run(*args), args)


@pytest.mark.parametrize("mask", ["none", "gap", "one"])
@pytest.mark.parametrize("bias", [True, False])
def test_masks(bias, mask):
    args = draw(2, 700, 2, seed=3, bias=bias, mask=mask)
    check(run(*args), args)


def test_all_masked_gives_zero():
    got = run(*draw(1, 200, 2, seed=4, mask="zeros"))
    assert all(np.abs(g).max() == 0.0 for g in got)


def test_one_key_has_no_score_gradient():
    """One valid key: p = 1 and ds = p (dp - dp) = 0, exactly."""
    q, k, v, do, b, m = draw(1, 1, 3, seed=5, mask="none")
    dq, dk, dv, dbias = run(q, k, v, do, b, m)
    assert np.abs(dq).max() == 0 and np.abs(dk).max() == 0 and np.abs(dbias).max() == 0
    assert np.array_equal(dv, do.astype(np.float64))


def test_what_masked_places_hold_does_not_matter():
    q, k, v, do, b, m = draw(2, 300, 2, seed=6, mask="tail")
    clean = run(q, k, v, do, b, m)
    bad = m == 0
    k, v, b = k.copy(), v.copy(), b.copy()
    k[bad] = np.nan
    v[bad] = np.inf
    n, nw = 300, b.shape[1]
    slot = 32 * np.arange(nw)[:, None] - 48 + np.arange(128)[None]
    out = (slot < 0) | (slot >= n)
    inside = np.clip(slot, 0, n - 1)
    for x in range(2):
        off = out | bad[x][inside]
        bx = b[x].transpose(0, 3, 1, 2)  # [window][slot][head][row]
        bx[off] = np.nan
    b[:, -1, :, n % 32:] = np.nan  # rows past the last atom
    dirty = run(q, k, v, do, b, m)
    for x, y in zip(clean, dirty):
        assert np.array_equal(x, y)


def test_bias_of_minus_infinity_and_of_the_lowest_value():
    q, k, v, do, b, m = draw(1, 200, 2, seed=7, mask="none")
    b[0, 2, :, 3] = -np.inf                 # a query whose every logit is -inf
    b[0, 3, :, :, 40:60] = -np.inf          # some slots
    lowest = float(torch.finfo(torch.bfloat16).min)
    b[0, 1, :, :, 10:30] = lowest
    b[0, 4, :, 5] = lowest                  # every slot
    args = (q, k, v, do, b, m)
    got = run(*args)
    assert np.abs(got[0][0, 2 * 32 + 3]).max() == 0 and np.abs(got[3][0, 2, :, 3]).max() == 0
    # Next to the lowest value q k is lost, in fp32 and in float64 alike: p is uniform there.
    check(got, args)


def test_long_logits():
    """Logits of size 100: all weight on a few keys, nothing overflows."""
    q, k, v, do, b, m = draw(1, 150, 2, seed=8)
    b = as_bf16(b * 100)  # the values the kernel is given
    got = run(q, k, v, do, b, m)
    ref = oracle_backward(q, k, v, do, b, m)
    for g, r in zip(got, ref):
        assert np.isfinite(g).all()
        # fp32 logits next to 400 are off by up to 2^-16, p by that relative
        assert np.linalg.norm(g - r) <= 1.5 * U * np.linalg.norm(r)


def test_equal_calls_give_equal_bits():
    args = draw(2, 1237, 3, seed=9)
    x, y = run(*args), run(*args)
    assert all(np.array_equal(a, b) for a, b in zip(x, y))


def test_atoms_behind_the_batch_stay_as_they_were():
    """Outputs inside a larger buffer: nothing around them is written."""
    q, k, v, do, b, m = (dev(t) for t in draw(1, 77, 2, seed=10))
    bufs = [torch.full((t.numel() + 1024,), 7.0, dtype=torch.bfloat16, device=DEV) for t in (q, k, v, b)]
    views = [x[512:512 + t.numel()] for x, t in zip(bufs, (q, k, v, b))]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    p = tm.AtomAttnParams(1, 77, 2, 32, q.data_ptr(), k.data_ptr(), v.data_ptr(), b.data_ptr(), m.data_ptr(),
                          ws.data_ptr(), 256, 0)
    tm.atomattn_backward(p, do, tm.AtomAttnGrads(*(t.data_ptr() for t in views)))
    torch.cuda.synchronize()
    ref = tm.atom_attention_backward(q, k, v, do, b, m)
    for x, w, r in zip(bufs, views, ref):
        assert (x[:512] == 7).all() and (x[512 + w.numel():] == 7).all()
        assert torch.equal(w.view(r.shape), r)


def test_graph_and_other_stream():
    q, k, v, do, b, m = (dev(t) for t in draw(1, 500, 2, seed=11))
    ref = tm.atom_attention_backward(q, k, v, do, b, m)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tm.atom_attention_backward(q, k, v, do, b, m, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = tm.atom_attention_backward(q, k, v, do, b, m)
    for t in got:
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, ref))


@pytest.mark.parametrize("bias", [True, False])
def test_what_queries_without_a_key_hold_does_not_matter(bias):
    """Windows whose every key is masked (padding): q and dout may hold anything."""
    q, k, v, do, b, m = draw(2, 700, 2, seed=12, bias=bias, mask="gap")
    clean = run(q, k, v, do, b, m)
    q, do = q.copy(), do.copy()
    windows = [w for w in range(22) if not m[0, max(0, 32 * w - 48):32 * w + 80].any()]
    assert len(windows) >= 4
    for w, (x, y) in zip(windows, ((np.nan, np.nan), (1.0, np.inf), (np.inf, 1.0), (np.inf, -np.inf))):
        q[:, 32 * w:32 * w + 32], do[:, 32 * w:32 * w + 32] = x, y
    dirty = run(q, k, v, do, b, m)
    for x, y in zip(clean, dirty):
        assert x is None and y is None or np.array_equal(x, y)
