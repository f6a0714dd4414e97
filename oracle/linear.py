"""CPU float64 oracle for a linear layer with its epilogue and its gradients (test infrastructure).

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. Formulas in include/linear.h:
y = act(x W^T + b) + r; D = dy act'(x W^T + b), dx = D W, dW = D^T x, db = sum of D.
"""
from __future__ import annotations

import numpy as np

ACTS = ("none", "relu", "sigmoid", "silu")


def _sigmoid(p):
    # e^-|p| in both branches, so that neither end overflows or loses digits
    e = np.exp(-np.abs(p))
    return np.where(p >= 0, 1 / (1 + e), e / (1 + e))


def act(p, name):
    if name == "none":
        return p
    if name == "relu":
        return np.maximum(p, 0)
    s = _sigmoid(p)
    return s if name == "sigmoid" else p * s


def act_slope(p, name):
    if name == "none":
        return np.ones_like(p)
    if name == "relu":
        return (p > 0).astype(np.float64)
    s, c = _sigmoid(p), _sigmoid(-p)
    return s * c if name == "sigmoid" else s + p * s * c


def _pre(x, w, b):
    p = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    return p if b is None else p + np.asarray(b, np.float64)


def linear(x, w, b=None, r=None, act_name="none"):
    y = act(_pre(x, w, b), act_name)
    return y if r is None else y + np.asarray(r, np.float64)


def linear_backward(x, w, dy, b=None, act_name="none"):
    """(dx, dW, db, D)."""
    x, w, dy = (np.asarray(t, np.float64) for t in (x, w, dy))
    D = dy * act_slope(_pre(x, w, b), act_name)
    return D @ w, D.T @ x, D.sum(0), D
