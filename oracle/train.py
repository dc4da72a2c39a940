"""Oracle of the training operators around the grouped experts, in float64.

Test infrastructure, like the rest of this package: plain loops over the
definitions, no code shared with the HIP path.
"""
from __future__ import annotations

import numpy as np


def unpermute_backward(dout, y, unpermute_idx, sorted_idx, probs):
    """Gradients of out[t] = sum_k probs[t, k] * y[idx[t, k]]: (dy, written,
    dprobs, bad). ``written`` marks the rows of dy that a slot names; a slot
    whose index is outside [0, min(rows, T*K)), or whose row sorted_idx gives to
    another slot, contributes nothing and makes ``bad`` true (-1 only the
    first)."""
    T, K = probs.shape
    dy = np.zeros(y.shape, np.float64)
    written = np.zeros(y.shape[0], bool)
    dprobs = np.zeros((T, K), np.float64)
    bad = False
    end = min(y.shape[0], T * K)
    for s, p in enumerate(np.asarray(unpermute_idx).reshape(-1)):
        if p == -1:
            continue
        if p < 0 or p >= end or sorted_idx[p] != s:
            bad = True
            continue
        t, k = divmod(s, K)
        dy[p] = np.float64(probs[t, k]) * dout[t]
        written[p] = True
        dprobs[t, k] = np.dot(dout[t], y[p])
    return dy, written, dprobs, bad


def permute_backward(g, unpermute_idx, T, K):
    """dx[t] = sum_k g[idx[t, k]]; (dx, bad)."""
    dx = np.zeros((T, g.shape[1]), np.float64)
    bad = False
    for s, p in enumerate(np.asarray(unpermute_idx).reshape(-1)):
        if 0 <= p < g.shape[0]:
            dx[s // K] += g[p]
        elif p != -1:
            bad = True
    return dx, bad


def newton_schulz(g, coeffs, eps, scale):
    """scale * the iterate after one step for each (a, b, c) of coeffs; g (m, n)."""
    x = np.asarray(g, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coeffs:
        if x.shape[0] <= x.shape[1]:
            p = x @ x.T
            x = a * x + (b * p + c * (p @ p)) @ x
        else:
            p = x.T @ x
            x = a * x + x @ (b * p + c * (p @ p))
    return scale * x
