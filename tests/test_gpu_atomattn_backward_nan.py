"""What infinities and NaN of some places of q, v or dout leave of atom attention's gradients: they reach
what the formula takes them to and nothing else. Slots that are not valid and rows past the last atom
hold 0 in dbias whatever the rest is, and a query whose logits are all -inf gives no gradient."""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from oracle.atomattn import key_range
from oracle.atomattn_backward import atom_attention_backward as oracle_backward
from test_gpu_atomattn_backward import ABS, U, draw, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def check(args, lost=()):
    """Finite where the oracle is, and there within the tolerance of tests/test_gpu_atomattn_backward.py. `lost`:
    (query, head) whose logits are not numbers. A softmax over them is not either, nor what it goes into: the
    query's dq, dk and dv of the valid keys of its window, and their slots of dbias. (The oracle takes the
    probabilities of a sum that is not over 0 as 0, which a NaN is not either: these places are set here.)"""
    got = run(*args)
    n, m = args[0].shape[1], args[5][0]
    with np.errstate(all="ignore"):
        ref = oracle_backward(*args, sizes=True)
    for i, h in lost:
        w, off = i // 32, invalid_slots(n, m, i // 32)
        at = np.arange(*key_range(w))[~off]
        ref[0][0, i, h] = ref[1][0, at, h] = ref[2][0, at, h] = np.nan
        ref[3][0, w, h, i % 32][~off] = np.nan
    for name, g, r, size, floor in zip(("dq", "dk", "dv", "dbias"), got, ref[:4], ref[4:], ABS):
        fin = np.isfinite(r)
        assert np.array_equal(np.isfinite(g), fin), (name, int((np.isfinite(g) != fin).sum()))
        over = np.abs(g[fin] - r[fin]) - (U * np.abs(r[fin]) + U * size[fin] + floor)
        assert over.max() <= 0, (name, float(over.max()))
    return got


def invalid_slots(n, m, w):
    at = np.arange(*key_range(w))
    out = (at < 0) | (at >= n)
    return out | (m[np.clip(at, 0, n - 1)] == 0)


@pytest.mark.parametrize("what", ["q", "dout"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_one_query(what, value):
    """A query's q or dout: its window's gradients are lost, but not the slots of dbias that take no part."""
    args = draw(1, 300, 2, seed=31)
    q, k, v, do, b, m = args
    (q if what == "q" else do)[0, 69, 1, 5] = value
    dbias = check(args, [(69, 1)] if what == "q" else [])[3]
    off = invalid_slots(300, m[0], 2)
    assert off.any() and (dbias[0, 2, 1][:, off] == 0).all()


def test_every_query_of_a_window():
    args = draw(1, 300, 2, seed=32)
    q, k, v, do, b, m = args
    q[0, :32], do[0, 40] = np.nan, np.nan
    dbias = check(args, [(i, h) for i in range(32) for h in range(2)])[3]
    for w in (0, 1):
        assert (dbias[0, w][:, :, invalid_slots(300, m[0], w)] == 0).all()


def test_rows_past_the_last_atom():
    """An infinite v meets the missing queries' dout of 0."""
    args = draw(1, 300, 2, seed=33)
    q, k, v, do, b, m = args
    at = int(np.flatnonzero(m[0][:290])[-1])
    v[0, at, 1, 7] = np.inf
    dbias = check(args)[3]
    assert (dbias[0, -1, :, 300 % 32:] == 0).all()


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_query_whose_logits_are_all_minus_infinity(value):
    """Whatever its dout holds. (The rows of dbias that go with it hold 0.)"""
    args = draw(2, 300, 2, seed=34)
    q, k, v, do, b, m = args
    for w, i in ((0, 0), (2, 3), (9, 11)):
        b[:, w, :, i] = -np.inf
    clean = run(*args)
    for w, i in ((0, 0), (2, 3), (9, 11)):
        do[:, 32 * w + i] = value
    dirty = run(*args)
    for x, y in zip(clean, dirty):
        assert np.isfinite(x).all() and np.array_equal(x, y)
