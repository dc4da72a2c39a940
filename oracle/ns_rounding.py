"""How far the fp16 operands of mc2_ns_orthogonalize may take its result from
the exact iterate, in float64. Test infrastructure, like the rest of this
package: no code shared with the HIP path.

The iteration is an odd function f(s) = a s + b s^3 + c s^5 of the singular
values, X = U diag(s) V^T. Written in the basis (U, V), a perturbation E of X
becomes, to first order, entry by entry

  E_ij -> phi+ (E_ij + E_ji) / 2 + phi- (E_ij - E_ji) / 2
  phi+- = (f(s_i) -+ f(s_j)) / (s_i -+ s_j)        (phi+ = f'(s_i) where equal)

and rows outside U's first r columns become p(s_j) E_j, p(s) = f(s) / s. Each
step rounds three matrices to fp16:

  the products' copy of X, which enters through phi - a (the term a X is held
    to more bits; in the last step of the many-launch path it is not: phi);
  A, of which X (b A + c A A) is formed: s_i (b + c (s_i^2 + s_j^2)) per entry
    (a matrix in one workgroup squares a rounded A - mu I and keeps b A in fp32);
  Q, of which X Q is formed: s_i per entry.
"""
from __future__ import annotations

import numpy as np

HALF = 2.0 ** -11  # half a step of fp16, relative
# its root mean square: an error uniform over a step of 2^-10 times a power of
# two, over values whose mantissas' logarithms are uniform (E[x^2] = 1.5 / ln 2)
RMS = 2.0 ** -10 / np.sqrt(12) / np.sqrt(1.5 / np.log(2))


def one_workgroup(m, n):
    """Whether a matrix of this size is iterated by one workgroup: the smaller
    side, padded to 64, at most 128, and at most 64 Ki elements with the larger
    one padded to a power of two times 128."""
    rp, cp = (-(-v // 64) * 64 for v in (min(m, n), max(m, n)))
    rows = 128
    while rows < cp:
        rows *= 2
    return rp <= 128 and rows * rp <= 65536


class _Step:
    """Factors and magnitudes of one step for singular values s."""

    def __init__(self, s, co, one, index, last):
        a, b, c = co
        si, sj, q = s[:, None], s[None, :], s * s
        mu = 0.5 if one and index >= 2 else 0.0

        def phi(sign):
            t = sign * sj
            return a + b * (si ** 2 + si * t + t ** 2) + c * (
                si ** 4 + si ** 3 * t + (si * t) ** 2 + si * t ** 3 + t ** 4)

        self.plus, self.minus = phi(1.0), phi(-1.0)
        self.p = a + b * q + c * q * q
        self.off = 0.0 if last and not one else a  # the part that hi's rounding does not see
        d = q - mu
        self.kappa = c * (d[:, None] + d[None, :]) + (0.0 if one else b)
        self.x2 = (s * s).sum()
        self.a2 = (d * d).sum()
        shift = a + b * mu + c * mu * mu if one else 0.0
        self.q2 = ((self.p - shift) ** 2).sum()


def _values(g, eps):
    g = np.asarray(g, np.float64)
    s = np.linalg.svd(g, compute_uv=False)
    return s / (np.sqrt((g * g).sum()) + eps), min(g.shape), max(g.shape)


def typical(g, coeffs, eps=0.0, one=None):
    """Expected error of the result of g (2-norm of the difference over that of
    the result), with roundings as independent noise spread evenly over each
    matrix. Holds where the singular values are spread over many."""
    s, r, c = _values(g, eps)
    one = one_workgroup(*np.shape(g)) if one is None else one
    sym, anti, perp = np.zeros((r, r)), np.zeros((r, r)), np.zeros(r)
    eye = np.eye(r, dtype=bool)
    for k, co in enumerate(coeffs):
        t = _Step(s, co, one, k, k + 1 == len(coeffs))
        sym, anti, perp = sym * t.plus ** 2, anti * t.minus ** 2, perp * t.p ** 2
        n = RMS ** 2 * t.x2 / (r * c)
        sym += np.where(eye, n, n / 2) * (t.plus - t.off) ** 2
        anti += np.where(eye, 0.0, n / 2) * (t.minus - t.off) ** 2
        perp += (c - r) * n * (t.p - t.off) ** 2
        w = RMS ** 2 / r ** 2 * (t.a2 * t.kappa ** 2 + t.q2)
        sym += w * (s[:, None] + s[None, :]) ** 2 / 4
        anti += w * (s[:, None] - s[None, :]) ** 2 / 4
        s = s * t.p
    return float(np.sqrt((sym + anti).sum() + perp.sum()) / np.linalg.norm(s))


def worst(g, coeffs, eps=0.0, one=None):
    """Bound of the same to first order, every rounding half a step in the worst
    direction. Close where few distinct singular values carry the matrix and
    roundings do not average out."""
    s, r, c = _values(g, eps)
    one = one_workgroup(*np.shape(g)) if one is None else one
    e = 0.0
    for k, co in enumerate(coeffs):
        t = _Step(s, co, one, k, k + 1 == len(coeffs))
        phis = [t.plus, t.minus] if r > 1 else [t.plus]
        phis += [t.p] if c > r else []
        grow = max(np.abs(v).max() for v in phis)
        copy = max(np.abs(v - t.off).max() for v in phis)
        e = grow * e + HALF * (copy * np.sqrt(t.x2)
                               + np.abs(s[:, None] * t.kappa).max() * np.sqrt(t.a2)
                               + np.abs(s).max() * np.sqrt(t.q2))
        s = s * t.p
    return float(e / np.linalg.norm(s))


def _fp16(x):
    return x.astype(np.float16).astype(np.float64)


def emulate(g, coeffs, eps=0.0, one=None, *, rnd=_fp16, keep_lo=True, shift=True):
    """The result before its rounding with the operands rounded as the kernels
    round them and everything else exact. The keywords plant mistakes: another
    rounding of the operands, an iterate without its low half, A held whole in
    the one-workgroup path."""
    x = np.asarray(g, np.float64)
    one = one_workgroup(*x.shape) if one is None else one
    wide = x.shape[0] < x.shape[1]
    x = (x.T if wide else x) / (np.sqrt((x * x).sum()) + eps)
    eye = np.eye(x.shape[1])
    if one:
        for k, (a, b, c) in enumerate(coeffs):
            mu = 0.5 if k >= 2 and shift else 0.0
            hi = rnd(x * 4096) / 4096
            d = hi.T @ hi - mu * eye
            d16 = rnd(d * 512) / 512
            q = rnd(((b + 2 * c * mu) * d + c * d16 @ d16) * 512) / 512
            x = (a * x if keep_lo else a * hi) + (b + c * mu) * mu * hi + hi @ q
    else:
        for k, (a, b, c) in enumerate(coeffs):
            hi = rnd(x * 4096) / 4096
            lo = _fp16((x - hi) * 4096 * 2048) / 4096 / 2048
            m = rnd(hi.T @ hi * 512) / 512
            q = rnd((b * m + c * m @ m + a * eye) * 512) / 512
            x = hi @ q + (a * lo if keep_lo and k + 1 < len(coeffs) else 0.0)
    return x.T if wide else x
