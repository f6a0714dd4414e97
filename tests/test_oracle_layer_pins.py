"""Pins of the float64 oracles of the linear layer and of atom attention's gradients (CPU):
against central differences of the forwards, and against torch's autograd in float64."""
import numpy as np
import pytest
import torch

from oracle.atomattn import atom_attention
from oracle.atomattn_backward import atom_attention_backward
from oracle.linear import ACTS, linear, linear_backward


def _difference(f, x, step=1e-5):
    """Central differences of the scalar f over the array x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * step)
    return g


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_against_differences(act):
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((5, 4)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    dy = rng.standard_normal((5, 3))
    f = lambda: float((linear(x, w, b, None, act) * dy).sum())  # noqa: E731
    dx, dw, db, _ = linear_backward(x, w, dy, b, act)
    # A central difference is off by step^2 / 6 |f'''| (about 1e-11) and 2^-53 |f| / step (about 1e-10).
    for got, t in ((dx, x), (dw, w), (db, b)):
        assert np.abs(got - _difference(f, t)).max() <= 1e-8


@pytest.mark.parametrize("act", ACTS)
def test_linear_against_torch(act):
    rng = np.random.default_rng(2)
    x, w, b, r = (torch.from_numpy(rng.standard_normal(s)) for s in ((7, 6), (5, 6), (5,), (7, 5)))
    y = torch.nn.functional.linear(x, w, b)
    y = {"none": y, "relu": torch.relu(y), "sigmoid": torch.sigmoid(y), "silu": torch.nn.functional.silu(y)}[act] + r
    assert np.abs(linear(x.numpy(), w.numpy(), b.numpy(), r.numpy(), act) - y.numpy()).max() <= 1e-13


@pytest.mark.parametrize("bias", [True, False])
def test_attention_backward_against_differences(bias):
    rng = np.random.default_rng(3)
    B, n, H = 1, 70, 1
    q, k, v, do = (rng.standard_normal((B, n, H, 32)) for _ in range(4))
    bs = rng.standard_normal((B, 3, H, 32, 128)) if bias else None
    m = (rng.random((B, n)) > 0.3).astype(float)
    m[0, 0] = 0
    f = lambda: float((atom_attention(q, k, v, bs, m) * do).sum())  # noqa: E731
    got = atom_attention_backward(q, k, v, do, bs, m)
    for g, t in zip(got, (q, k, v, bs)):
        if g is None:
            continue
        for _ in range(40):
            i = tuple(rng.integers(0, s) for s in t.shape)
            keep, step = t[i], 1e-4
            t[i] = keep + step
            up = f()
            t[i] = keep - step
            down = f()
            t[i] = keep
            assert abs((up - down) / (2 * step) - g[i]) <= 1e-7, i
    assert (got[1][0, m[0] == 0] == 0).all() and (got[2][0, m[0] == 0] == 0).all()


def test_attention_backward_of_windows_without_a_key():
    rng = np.random.default_rng(4)
    n = 400
    q, k, v, do = (rng.standard_normal((1, n, 2, 32)) for _ in range(4))
    m = np.ones((1, n))
    m[0, 100:330] = 0  # windows 5 and 6 see no valid key
    dq, dk, dv, _ = atom_attention_backward(q, k, v, do, None, m)
    assert (dq[0, 160:224] == 0).all() and np.isfinite(dq).all() and np.isfinite(dk).all() and np.isfinite(dv).all()
    assert np.abs(dq[0, :96]).max() > 0
