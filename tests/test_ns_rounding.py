"""The error model of the Newton-Schulz orthogonalisation's fp16 operands
(oracle/ns_rounding.py) against an emulation of those operands in float64, and
against planted mistakes; the figures that include/mc2_train.h states."""
import numpy as np
import pytest

from oracle import ns_rounding as nr
from oracle import train as ot

CO = (3.4445, -4.7750, 2.0315)
# What independent roundings give varies by less than this around the expected
# error: the sums behind it run over thousands of entries, but A's and Q's
# roundings fall mostly on their r diagonal entries
SPREAD = 1.4


def rel(x, ref):
    return np.linalg.norm(x - ref) / np.linalg.norm(ref)


def bf16(x):
    i = x.astype(np.float32).view(np.uint32)
    i = (i + 0x7FFF + ((i >> 16) & 1)) & 0xFFFF0000
    return i.astype(np.uint32).view(np.float32).astype(np.float64)


def spread(kind, m, n, seed=0):
    """Matrices whose singular values are spread: full rank, `kind` rows of
    tokens only, or those with 5% of noise."""
    rng = np.random.default_rng(seed)
    if kind == "full":
        return rng.standard_normal((m, n))
    rank = int(kind.split("+")[0])
    g = rng.standard_normal((m, rank)) @ rng.standard_normal((rank, n))
    return g + 0.05 * np.sqrt(rank) * rng.standard_normal((m, n)) if "+" in kind else g


def few(kind, r):
    """Matrices that few or equal singular values carry."""
    rng = np.random.default_rng(r)
    if kind == "identity":
        return np.eye(r)
    if kind == "orthogonal":
        return np.linalg.qr(rng.standard_normal((r, r)))[0]
    g = np.zeros((r, r))
    for i, v in enumerate({"two": (0.6217, 0.7832), "three": (0.6218, 0.6218, 0.4761)}[kind]):
        g[i, i] = v
    return g


SPREAD_CASES = [(k, m, n) for m, n in ((64, 256), (100, 72), (24, 1000), (200, 304), (304, 200))
                for k in ("full", "1", "16", "16+")]
# (case, steps): of a matrix of rank 1, one singular value's error, which does
# not average, stands out until five steps have grown the noise of the others
SPREAD_STEPS = [(*c, s) for c in SPREAD_CASES for s in (2, 5) if s == 5 or c[0] != "1"]
FEW_CASES = [("identity", 4), ("identity", 8), ("identity", 100), ("identity", 319),
             ("identity", 395), ("orthogonal", 27), ("orthogonal", 100), ("orthogonal", 319),
             ("two", 2), ("three", 3), ("two", 200), ("three", 200)]


@pytest.mark.parametrize("kind,m,n,steps", SPREAD_STEPS)
def test_expected_error(kind, m, n, steps):
    g = spread(kind, m, n)
    ref = ot.newton_schulz(g, (CO,) * steps, 0.0, 1.0)
    t = nr.typical(g, (CO,) * steps)
    assert t / SPREAD <= rel(nr.emulate(g, (CO,) * steps), ref) <= t * SPREAD
    if steps == 5:
        assert t * SPREAD <= 3.1e-3  # 2.2e-3 on average over these cases' largest


@pytest.mark.parametrize("kind,r", FEW_CASES)
@pytest.mark.parametrize("steps", [1, 3, 5])
def test_worst_error(kind, r, steps):
    g = few(kind, r)
    e = rel(nr.emulate(g, (CO,) * steps), ot.newton_schulz(g, (CO,) * steps, 0.0, 1.0))
    assert e <= nr.worst(g, (CO,) * steps)
    assert e <= 3.5e-2


def test_scalar_spectra_stay_below_the_stated_worst():
    """Diagonal matrices of r1 values s1 and r2 values s2, every split of the
    norm: both paths' formats stay below 3.5e-2."""
    for one in (False, True):
        for r1, r2 in ((1, 1), (2, 1), (1, 4), (2, 2)):
            t = np.linspace(0.0, np.pi / 2, 20003)[1:-1]
            num = den = 0.0
            for s, r in ((np.cos(t) / np.sqrt(r1), r1), (np.sin(t) / np.sqrt(r2), r2)):
                ref, x = s, s
                for a, b, c in (CO,) * 5:
                    ref = ref * (a + b * ref ** 2 + c * ref ** 4)
                x = _scalar(s, one)
                num, den = num + r * (x - ref) ** 2, den + r * ref ** 2
            w = np.sqrt(num / den).max()
            assert 1e-2 < w <= 3.5e-2, (one, r1, r2, w)


def _scalar(s, one):
    """emulate() for many 1 x 1 matrices at once."""
    h, x = nr._fp16, s
    lo = 0.0
    for k, (a, b, c) in enumerate((CO,) * 5):
        mu = 0.5 if one and k >= 2 else 0.0
        hi = h(x * 4096) / 4096
        if one:
            d = hi * hi - mu
            q = h(((b + 2 * c * mu) * d + c * (h(d * 512) / 512) ** 2) * 512) / 512
            x = a * x + (b + c * mu) * mu * hi + hi * q
        else:
            lo = h((x - hi) * 4096 * 2048) / 4096 / 2048
            m = h(hi * hi * 512) / 512
            x = hi * (h((b * m + c * m * m + a) * 512) / 512) + (a * lo if k < 4 else 0.0)
    return x


@pytest.mark.parametrize("m,n", [(64, 256), (200, 304)])
def test_planted_mistakes_exceed_the_tolerance(m, n):
    """bf16 operands on every input, an iterate without its low half where
    singular values are zero, and A held whole in the one-workgroup path."""
    def over(kind, **kw):
        g = spread(kind, m, n)
        e = rel(nr.emulate(g, (CO,) * 5, **kw), ot.newton_schulz(g, (CO,) * 5, 0.0, 1.0))
        return e > SPREAD * nr.typical(g, (CO,) * 5) + nr.HALF

    for kind in ("full", "1", "16", "16+"):
        assert not over(kind)
        assert over(kind, rnd=bf16)
        if kind != "full":
            assert over(kind, keep_lo=False)
    if nr.one_workgroup(m, n):
        assert over("full", shift=False)
