"""The precision of the Newton-Schulz orthogonalisation, with fp16 output so
that its own error shows, against the float64 oracle. The tolerances come from
oracle/ns_rounding.py, input by input: 1.4 times the expected error of
independent roundings where the singular values are spread (tests/
test_ns_rounding.py derives and checks the factor without a GPU), the bound of
roundings in their worst direction where few or equal ones carry the matrix;
the output's rounding adds half a step of fp16 at most."""
import numpy as np
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import ns_rounding as nr
from oracle import train as ot
from test_ns_rounding import CO, FEW_CASES, SPREAD, SPREAD_STEPS, few, rel, spread

pytestmark = pytest.mark.gpu

F16 = torch.float16


def _error(g, steps):
    g = torch.from_numpy(g).float()
    out = mc2.mc2_ns_orthogonalize(g.cuda(), steps=steps, eps=0.0, out_dtype=F16)
    ref = ot.newton_schulz(g.double().numpy(), (CO,) * steps, 0.0, 1.0)
    return rel(out.double().cpu().numpy(), ref), g.double().numpy()


@pytest.mark.parametrize("kind,m,n,steps", SPREAD_STEPS + [
    ("full", 777, 1001, 5), ("16", 777, 1001, 5), ("16+", 520, 264, 5)])
def test_spread_singular_values(kind, m, n, steps):
    e, g = _error(spread(kind, m, n), steps)
    assert e <= SPREAD * nr.typical(g, (CO,) * steps) + nr.HALF


@pytest.mark.parametrize("kind,r", FEW_CASES)
@pytest.mark.parametrize("steps", [1, 3, 5])
def test_few_or_equal_singular_values(kind, r, steps):
    e, g = _error(few(kind, r), steps)
    assert e <= min(nr.worst(g, (CO,) * steps), 3.5e-2) + nr.HALF


@pytest.mark.parametrize("m,n,ratio", [(64, 256, 1.0), (64, 256, 1e-3), (64, 256, 1e-5),
                                       (200, 304, 1.0), (200, 304, 1e-3), (200, 304, 1e-5),
                                       (4096, 4096, 1e-5)])
def test_norms_below_eps(m, n, ratio):
    """|G| = ratio * eps. At 1e-5 every step multiplies by a alone: the last one's
    singular values are at most a^4 ratio = 1.4e-3, and b s^2 / a 3e-6."""
    g = torch.randn((m, n), generator=torch.Generator().manual_seed(1)).double()
    g = (g / g.norm() * ratio * 1e-3).float()
    out = mc2.mc2_ns_orthogonalize(g.cuda(), eps=1e-3, out_dtype=F16, scale=1.0 / ratio)
    x = g.double().numpy()
    if ratio > 1e-4:
        ref = ot.newton_schulz(x, (CO,) * 5, 1e-3, 1.0 / ratio)
    else:
        ref = CO[0] ** 5 / ratio * x / (np.linalg.norm(x) + 1e-3)
    assert rel(out.double().cpu().numpy(), ref) <= 2.5e-3 + nr.HALF
