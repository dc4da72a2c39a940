"""Calls of the Newton-Schulz orthogonalisation at the edges of what it takes."""
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import ns_rounding as nr
from oracle import train as ot
from test_ns_rounding import SPREAD, rel

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


@pytest.mark.parametrize("B,m,n", [(1, 3, 65536), (60, 64, 1088), (3, 100, 700), (300, 130, 190),
                                   (16, 300, 2000), (5, 2000, 300), (40, 64, 256)])
def test_nothing_behind_the_workspace_is_written(B, m, n):
    """Tiles of every width, in a workspace of exactly the size asked for."""
    g = torch.randn((B, m, n), generator=torch.Generator().manual_seed(9)).cuda()
    ref = mc2.mc2_ns_orthogonalize(g)
    need = mc2.mc2_ns_workspace_size(B, m, n)
    buf = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    out = mc2.mc2_ns_orthogonalize(g, workspace=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 0xAB).all()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    pick = sorted({0, B - 1})
    for b in pick:
        want = ot.newton_schulz(g[b].double().cpu().numpy(), (mc2.MC2_NS_COEFFS,) * 5, 1e-7, 1.0)
        tol = SPREAD * nr.typical(g[b].double().cpu().numpy(), (mc2.MC2_NS_COEFFS,) * 5)
        if min(m, n) >= 48:  # (of three rows, roundings do not average out)
            assert rel(out[b].double().cpu().numpy(), want) <= tol + 2.0 ** -8


def _typical_error(g, out, steps=5):
    co = (mc2.MC2_NS_COEFFS,) * steps
    g = g.double().cpu().numpy()
    e = rel(out.double().cpu().numpy(), ot.newton_schulz(g, co, 1e-7, 1.0))
    assert e <= SPREAD * nr.typical(g, co) + nr.HALF


@pytest.mark.parametrize("B,m,n", [
    # one workgroup a matrix: r padded to 64 and 128, c to 128 .. 1024
    (2, 100, 50), (2, 60, 250), (3, 500, 48), (2, 50, 900), (2, 128, 100), (2, 100, 250),
    (2, 500, 120),
    # tiles of 64; of 128, one and several rounds of them; of 256: every product
    (3, 200, 260), (3, 260, 200), (24, 200, 300), (24, 300, 200), (40, 260, 300), (40, 300, 260),
    (64, 384, 500), (90, 513, 260), (90, 264, 520)])
def test_every_kernel(B, m, n):
    g = torch.randn((B, m, n), generator=torch.Generator().manual_seed(B)).cuda()
    out = mc2.mc2_ns_orthogonalize(g, out_dtype=torch.float16)
    torch.cuda.synchronize()
    for b in sorted({0, B // 2, B - 1}):
        _typical_error(g[b], out[b])


def test_offsets_beyond_32_bits():
    """A stack of more than 2^31 elements."""
    B, m, n = 520, 2048, 2050
    g = torch.randn((B, m, n), generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda")
    assert g.numel() > 2 ** 31
    out = mc2.mc2_ns_orthogonalize(g, steps=1, out_dtype=torch.float16)
    torch.cuda.synchronize()
    for b in (0, B - 1):
        _typical_error(g[b], out[b], 1)
