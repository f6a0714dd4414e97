"""relu's gradient where the sums of p cancel: what is left is far under fp32's rounding of the sums on the
way there, and the gradient is still that of the exact sign. Every factor is chosen so that the gradients'
own sums are exact in fp32 in any order: one rounding, no tolerance."""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from gpu_helpers import as_bf16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(torch.bfloat16)


# One pass (one column chunk, two, pairs) and the several products (W on chip, streamed).
SIZES = [(128, 128), (96, 64), (128, 200), (96, 392), (128, 512), (160, 72), (328, 200), (1024, 136)]


def backward(x, w, dy, b, held):
    xx = dev(x)
    if held:
        xx = tm.act8_pack(xx)
        assert torch.equal(tm.act8_unpack(xx), dev(x))  # 8 bits hold these values
    return tm.linear_backward(xx, dev(w), dev(dy), bias=None if b is None else dev(b), act="relu")


def exact(x, w, dy, b):
    x, w, dy = (torch.from_numpy(np.asarray(t, np.float64)) for t in (x, w, dy))
    p = x @ w.T + (0 if b is None else torch.from_numpy(np.asarray(b, np.float64)))
    D = dy * (p > 0)
    return [t.to(torch.bfloat16) for t in (D @ w, D.T @ x, D.sum(0))]


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("k,n", SIZES)
def test_products_that_cancel(k, n, bias, held):
    """x has 4096 twice and 2^-20 between them, W 1, 1, -1 there: p is the 2^-20 with its sign, and on the way
    the sum is 4096, whose step in fp32 is 2^-11. (Places 0, 40 and 80: different steps of the contraction and
    different blocks of 8-bit scales.) Half of the rows are plain numbers."""
    if held and k % 32:
        pytest.skip("8 bits come in blocks of 32")
    rows = 250
    rng = np.random.default_rng([k, n])
    x = np.zeros((rows, k))
    x[:, 0] = x[:, 80] = 4096
    x[:, 40] = rng.choice([-1, 1], rows) * 2.0 ** -20
    x[::2, 0:96] = rng.integers(-4, 5, ((rows + 1) // 2, 96))
    x[::2, 40] = 0  # dW's column of the small values: them alone, exact
    w = np.zeros((n, k))
    w[:, [0, 40, 80]] = [1, 1, -1]
    w *= rng.choice([-1, 1], (n, 1))
    b = 4096.0 * rng.choice([-1, 1], n) if bias else None
    if bias:  # the bias in the first 4096's place: p = the 2^-20 again
        x[:, 0], w[:, 80] = 0, -np.sign(b) * 1
        w[:, 40] = rng.choice([-1, 1], n)
    dy = rng.choice([-1.0, 1.0], size=(rows, n))
    for got, want in zip(backward(x, w, dy, b, held), exact(x, w, dy, b)):
        assert torch.equal(got.cpu(), want), int((got.cpu() != want).sum())


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("k,n", SIZES)
def test_sums_that_cancel_over_all_features(k, n, held):
    """Features twice, with opposite weights, and four small ones: p is the small ones' sum, 2^-16 of the sums on
    the way, and for many places under their rounding. dy is 1 or -1, so db is a whole number under 256: exact."""
    if held and k % 32:
        pytest.skip("8 bits come in blocks of 32")
    rows, h = 250, k // 2 - 16
    rng = np.random.default_rng([k, n, 5])
    x, w = np.zeros((rows, k)), np.zeros((n, k))
    x[:, :h] = rng.choice([1.0, 1.25, 1.5, 1.75], (rows, h)) * rng.choice([-1, 1], (rows, h))  # 3 bits: 8-bit codes
    x[:, 32 + h:] = x[:, :h]
    x[:, h:h + 4] = rng.choice([1.0, 1.5], (rows, 4)) * 2.0 ** -5
    w[:, :h] = as_bf16(rng.standard_normal((n, h)))
    w[:, 32 + h:] = -w[:, :h]
    w[:, h:h + 4] = as_bf16(rng.standard_normal((n, 4)) * 2.0 ** -17)
    dy = rng.choice([-1.0, 1.0], size=(rows, n))
    p = x @ w.T
    assert (np.abs(p) < 2.0 ** -23 * np.abs(x) @ np.abs(w).T).sum() > 100
    db = backward(x, w, dy, None, held)[2]
    assert torch.equal(db.cpu(), exact(x, w, dy, None)[2])


@pytest.mark.parametrize("scale", [2.0 ** -96, 2.0 ** -40, 2.0 ** 70])
@pytest.mark.parametrize("k,n", [(128, 136), (160, 72)])
def test_small_and_large_rows(k, n, scale):
    """The same cancelling rows times a power of two: neither the squares' underflow nor their overflow hides
    a sign."""
    rows = 200
    rng = np.random.default_rng([k, n, 9])
    x = np.zeros((rows, k))
    x[:, 0] = x[:, 80] = 1
    x[:, 40] = rng.choice([-1, 1], rows) * 2.0 ** -30
    x *= scale
    x[::5] = 0
    w = np.zeros((n, k))
    w[:, [0, 40, 80]] = [1, 1, -1]
    w *= rng.choice([-1, 1], (n, 1))
    w[1::7] = 0
    dy = rng.choice([-1.0, 1.0], size=(rows, n))
    for got, want in zip(backward(x, w, dy, None, False), exact(x, w, dy, None)):
        assert torch.equal(got.cpu(), want), int((got.cpu() != want).sum())
