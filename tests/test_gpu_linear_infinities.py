"""Infinities in x or W of a linear layer's backward. Rows past the last and columns past out_features of
a tile are products with zeros, and 0 times infinity is NaN: nothing of them may reach a gradient.

Against the float64 oracle: NaN and infinity stand where the formula has them, and the rest is within
the tolerance of tests/test_gpu_linear.py, here with the sizes of the finite terms only: u = 2^-8 for the
result's rounding, u for D's (sigmoid), and (k + 4) 2^-23 of the sums' sizes for p, dx and dW. The
pre-activations that an infinity makes infinite have slope 0 exactly, and no error.
"""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from gpu_helpers import as_bf16
from oracle.linear import linear_backward as oracle_backward

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U, E = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(torch.bfloat16)


def draw(rows, k, n, seed):
    rng = np.random.default_rng([rows, k, n, seed])
    w = rng.standard_normal((n, k)) / np.sqrt(k)
    return [as_bf16(t) for t in (rng.standard_normal((rows, k)), w, rng.standard_normal(n) / 4,
                                 rng.standard_normal((rows, n)))]


def same_but_for_rounding(got, ref, size):
    got = got.double().cpu().numpy()
    odd = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (int(np.isnan(got).sum()), int(np.isnan(ref).sum()))
    assert np.array_equal(got[odd], ref[odd], equal_nan=True)
    over = np.abs(got - ref)[~odd] - (U * np.abs(ref) + size)[~odd]
    assert over.max() <= 0, float(over.max())


def check(x, w, b, dy, act):
    k, n, rows = w.shape[1], w.shape[0], x.shape[0]
    dx, dw, db = tm.linear_backward(dev(x), dev(w), dev(dy), bias=dev(b), act=act)
    with np.errstate(invalid="ignore"):
        rx, rw, rb, D = oracle_backward(x, w, dy, b, act)
    fin = lambda t: np.where(np.isfinite(t), np.abs(np.asarray(t, np.float64)), 0.0)  # noqa: E731
    ax, aw, aD = fin(x), fin(w), fin(D)
    live = aD > 0  # elsewhere D is 0 exactly, or not a number
    dD = live * fin(dy) * ((k + 4) * E * (ax @ aw.T + fin(b)) + 2.0 ** -18)
    dDr = dD + U * (aD + dD)
    same_but_for_rounding(dx, rx, 1.01 * (dDr @ aw + (n + 4) * E * (aD @ aw)))
    same_but_for_rounding(dw, rw, 1.01 * (dDr.T @ ax + (rows + 4) * E * (aD.T @ ax)))
    same_but_for_rounding(db, rb, 1.01 * (dD.sum(0) + (rows + 4) * E * aD.sum(0)))


@pytest.mark.parametrize("k,n", [(64, 128), (128, 256), (160, 72)])
def test_slope_at_minus_infinity(k, n):
    """Every p is -infinity: sigmoid's slope is 0, so dx, dW and db are 0, exactly."""
    x, w, b, dy = draw(256, k, n, 3)
    b[:] = -np.inf
    dx, dw, db = tm.linear_backward(dev(x), dev(w), dev(dy), bias=dev(b), act="sigmoid")
    assert all((t == 0).all() for t in (dx, dw, db))


# One pass (one column chunk, two, pairs) with columns past out_features, and the several products.
SIZES = [(128, 72), (64, 128), (128, 200), (40, 256), (96, 392), (160, 72), (264, 136)]


@pytest.mark.parametrize("rows", [100, 128, 20000])
@pytest.mark.parametrize("k,n", SIZES)
def test_infinity_in_a_row_of_x(rows, k, n):
    """Every p of the row is infinite and sigmoid's slope there 0: dx of the row is 0."""
    x, w, b, dy = draw(rows, k, n, 1)
    x[rows // 2, 3] = np.inf
    x[rows - 1, 5] = -np.inf
    assert (w[:, [3, 5]] != 0).all()
    check(x, w, b, dy, "sigmoid")


@pytest.mark.parametrize("rows", [100, 128, 20000 + 64])
@pytest.mark.parametrize("k,n", SIZES[:5])
def test_infinity_in_a_row_of_w(rows, k, n):
    """Every p of one column is infinite: its row of dW and its place in db are 0, whatever the number of rows."""
    x, w, b, dy = draw(rows, k, n, 2)
    w[n // 2, 3], w[n - 1, 5] = np.inf, -np.inf
    assert (x[:, [3, 5]] != 0).all()
    check(x, w, b, dy, "sigmoid")


@pytest.mark.parametrize("rows", [100, 128, 20000 + 64])
@pytest.mark.parametrize("k,n", SIZES[5:])
def test_infinity_in_a_row_of_w_several_products(rows, k, n):
    """The same where D is a product of its own."""
    test_infinity_in_a_row_of_w(rows, k, n)
