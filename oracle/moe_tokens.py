"""Oracle of the MoE layer for few tokens, in float64.

Test infrastructure, like the rest of this package: the layer's definition slot
by slot, no code shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

from . import moe


def layer(x, sel, probs, w1, w2, *, ep_rank, num_experts):
    """(out, mag, bad): out (T, H) of this rank's experts, w1 (E_l, H, 2I) and w2
    (E_l, I, H); mag, the same sum with every product's and term's magnitude (the
    scale of rounding errors); bad, whether an id lies outside [0, num_experts)."""
    T, K = sel.shape
    E_l, I = w2.shape[:2]
    out = np.zeros(x.shape, np.float64)
    mag = np.zeros(x.shape, np.float64)
    bad = False
    for t in range(T):
        for k in range(K):
            e = int(sel[t, k])
            if e < 0 or e >= num_experts:
                bad = True
                continue
            e -= ep_rank * E_l
            if e < 0 or e >= E_l:
                continue
            a = x[t] @ w1[e]
            h = moe.swiglu(a[None])[0]
            am = np.abs(x[t]) @ np.abs(w1[e])
            # |dh| <= |silu'| |da_gate| |up| + |silu| |da_up|, |silu'| <= 1.1, |silu(g)| <= |g|
            hm = 1.1 * am[:I] * np.abs(a[I:]) + np.abs(a[:I]) * am[I:] + np.abs(h)
            out[t] += np.float64(probs[t, k]) * (h @ w2[e])
            mag[t] += np.abs(np.float64(probs[t, k])) * (hm @ np.abs(w2[e]))
    return out, mag, bad
