"""CPU float64 oracle for the gradients of windowed atom attention (test infrastructure).

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. The derivative of
``oracle.atomattn.atom_attention`` by reverse accumulation, window by window.
"""
from __future__ import annotations

import numpy as np

from oracle.atomattn import Q_WIN, K_WIN, key_range, n_windows


def atom_attention_backward(q, k, v, dout, bias=None, atom_mask=None, sizes=False):
    """(dq, dk, dv, dbias) of sum(atom_attention(q, k, v, bias, atom_mask) * dout).

    With `sizes`, also the same four sums with every term's size in place of the term
    (|ds| |k| and so on): what a rounding of p and ds to few bits is relative to.
    """
    q, k, v, dout = (np.asarray(t, np.float64) for t in (q, k, v, dout))
    B, n, H, d = q.shape
    scale = 1.0 / np.sqrt(d)
    g = [np.zeros_like(q) for _ in range(3)] + [None if bias is None else np.zeros(np.shape(bias))]
    a = [np.zeros_like(q) for _ in range(3)] + [None if bias is None else np.zeros(np.shape(bias))]
    for b in range(B):
        for w in range(n_windows(n)):
            q0, q1 = Q_WIN * w, min(Q_WIN * (w + 1), n)
            slots = np.arange(*key_range(w))
            valid = (slots >= 0) & (slots < n)
            if atom_mask is not None:
                m = np.zeros(K_WIN, dtype=bool)
                m[valid] = np.asarray(atom_mask[b])[slots[valid]] != 0
                valid = m
            if not valid.any():
                continue
            at = slots[valid]
            l = np.einsum("qhd,khd->hqk", q[b, q0:q1], k[b, at]) * scale
            if bias is not None:
                l = l + np.asarray(bias[b, w], np.float64)[:, : q1 - q0][:, :, valid]
            top = l.max(-1, keepdims=True)
            e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
            total = e.sum(-1, keepdims=True)
            p = np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0)
            dp = np.einsum("qhd,khd->hqk", dout[b, q0:q1], v[b, at])
            ds = p * (dp - (p * dp).sum(-1, keepdims=True))
            for dst, f in ((g, lambda t: t), (a, np.abs)):
                dst[0][b, q0:q1] += np.einsum("hqk,khd->qhd", f(ds), f(k[b, at])) * scale
                dst[1][b, at] += np.einsum("hqk,qhd->khd", f(ds), f(q[b, q0:q1])) * scale
                dst[2][b, at] += np.einsum("hqk,qhd->khd", f(p), f(dout[b, q0:q1]))
                if bias is not None:
                    full = np.zeros((H, q1 - q0, K_WIN))
                    full[:, :, valid] = f(ds)
                    dst[3][b, w][:, : q1 - q0] = full
    return (*g, *a) if sizes else tuple(g)
