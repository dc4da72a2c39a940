"""Calls of the Newton-Schulz orthogonalisation at the edges of what it takes."""
import pytest
import torch

from gemm_collective_core_amd import mc2

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("m,n", [(4, 4), (90, 128), (200, 200), (200, 304), (304, 200)])
@pytest.mark.parametrize("scale", [2e-38, -3e-36, 1e30])
def test_scales_near_the_ends_of_the_range(m, n, scale):
    """The scale is applied to the result, whose entries on the diagonal are near
    1 for a diagonal matrix: two roundings to bf16 lie between the result and the
    scaled result of the call without one, 2^-8 each and 2^-23 for fp32."""
    g = torch.zeros((m, n), device="cuda")
    g.fill_diagonal_(1.0)
    one = mc2.mc2_ns_orthogonalize(g).double().diagonal()
    got = mc2.mc2_ns_orthogonalize(g, scale=scale).double()
    torch.cuda.synchronize()
    assert (one > 0.3).all()
    assert ((got.diagonal() - scale * one).abs() <= 2.1 * 2.0 ** -8 * abs(scale) * one).all()
    got.fill_diagonal_(0)
    assert (got == 0).all()
