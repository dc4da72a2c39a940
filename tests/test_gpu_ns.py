"""The Newton-Schulz orthogonalisation against the float64 oracle, through the
C ABI.

Bound: a step rounds three things to fp16, each off by 2^-11 / sqrt(3) of
itself in the root mean square: the products' iterate (enters through Q, whose
eigenvalues reach b^2 / 4c = 2.8), the Gram matrix (enters times |b| = 4.8 or
less) and Q (2.8): sqrt(2.8^2 + 4.8^2 + 2.8^2) * 2.8e-4 = 1.8e-3 of the iterate
a step. A perturbation of an iterate grows by at most |f'| = 1.6 a step where
the singular values have converged (f = a s + b s^3 + c s^5 on [0.7, 1.2]); in
directions whose singular value is still small it grows like the iterate's
own part there. Over five steps, in the root mean square:
1.8e-3 * sqrt(1 + 1.6^2 + 1.6^4 + 1.6^6 + 1.6^8) = 1.5e-2. The result's own
rounding adds 2^-8 (bf16) or 2^-11 (fp16) at most."""
import numpy as np
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import train as ot

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CO = (3.4445, -4.7750, 2.0315)
NS_TOL = 1.5e-2


def _rel(x, ref):
    x = x.double().cpu().numpy()
    return np.linalg.norm(x - ref) / np.linalg.norm(ref)


def _check(g, out, *, coeffs=(CO,) * 5, eps=1e-7, scale=1.0, tol=NS_TOL):
    g3 = g.double().cpu().numpy().reshape(-1, *g.shape[-2:])
    o3 = out.reshape(-1, *out.shape[-2:])
    assert out.shape == g.shape and torch.isfinite(out).all()
    for b in range(len(g3)):
        ref = ot.newton_schulz(g3[b], coeffs, eps, scale)
        if not g3[b].any():
            assert not o3[b].any()
            continue
        r = _rel(o3[b], ref)
        assert r <= tol + torch.finfo(out.dtype).eps / 2, (b, r)


@pytest.mark.parametrize("B,m,n,dt,out", [
    (1, 1, 1, F32, BF), (2, 1, 7, F32, BF), (1, 9, 1, BF, F16), (3, 2, 3, F16, BF),
    (1, 64, 64, F32, BF), (2, 63, 65, F32, BF), (2, 65, 63, BF, BF), (1, 64, 256, F32, F16),
    (5, 100, 72, F16, BF), (8, 264, 272, F32, BF), (1, 272, 264, F32, BF), (3, 129, 130, BF, F16),
    (2, 131, 517, F32, BF), (2, 517, 131, F32, BF), (1, 777, 1001, F32, BF),
    (1, 1001, 777, BF, BF), (16, 384, 256, F32, BF), (2, 512, 1024, F16, F16),
    (1, 1536, 1537, F32, BF), (3, 24, 1000, F32, BF), (40, 136, 200, F32, BF),
    (256, 136, 200, F32, BF), (260, 200, 136, BF, F16), (90, 264, 520, F32, BF),
    (90, 513, 260, F16, BF)])
def test_sizes_and_types(B, m, n, dt, out):
    g = torch.randn((B, m, n), generator=torch.Generator().manual_seed(m * 7 + n)).to(dt).cuda()
    keep = g.clone()
    o = mc2.mc2_ns_orthogonalize(g, out_dtype=out)
    torch.cuda.synchronize()
    assert o.dtype == out and torch.equal(g, keep)
    _check(g, o)


@pytest.mark.parametrize("m,n", [(192, 320), (320, 192), (777, 1001), (60, 250), (500, 120)])
@pytest.mark.parametrize("rank", [1, 16, 100])
def test_rank_deficient(m, n, rank):
    """An expert with fewer tokens than its matrix has rows: the other singular
    values are zero and have to stay there."""
    gen = torch.Generator().manual_seed(rank)
    g = torch.randn((m, rank), generator=gen) @ torch.randn((rank, n), generator=gen)
    _check(g, mc2.mc2_ns_orthogonalize(g.cuda()))


@pytest.mark.parametrize("m,n", [(96, 160), (200, 160), (260, 513)])
def test_a_matrix_of_the_stack_does_not_see_the_others(m, n):
    """Zeros, NaN and infinities beside an ordinary matrix, which gets the bits
    it gets alone."""
    g = torch.randn((4, m, n), generator=torch.Generator().manual_seed(1)).cuda()
    alone = mc2.mc2_ns_orthogonalize(g[1:2].contiguous(), eps=0.0)
    g[0] = 0
    g[2, 5, 7] = float("nan")
    g[3, 1, 2] = float("inf")
    o = mc2.mc2_ns_orthogonalize(g, eps=0.0)
    torch.cuda.synchronize()
    assert (o[0] == 0).all()
    assert torch.equal(o[1:2], alone)
    assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()


@pytest.mark.parametrize("m,n", [(100, 140), (200, 140)])
@pytest.mark.parametrize("mag", [1e-36, 1e-30, 1e-12, 1e12, 1e30, 1e36])
def test_magnitudes(mag, m, n):
    """The norm neither vanishes nor overflows."""
    g = torch.randn((m, n), generator=torch.Generator().manual_seed(2)) * mag
    _check(g, mc2.mc2_ns_orthogonalize(g.cuda(), eps=0.0), eps=0.0)


@pytest.mark.parametrize("m,n", [(90, 150), (150, 200)])
def test_steps_coefficients_eps_scale_and_2d(m, n):
    g = torch.randn((m, n), generator=torch.Generator().manual_seed(3))
    gd = g.cuda()
    for steps in (1, 2, 3):
        _check(g, mc2.mc2_ns_orthogonalize(gd, steps=steps), coeffs=(CO,) * steps)
    own = ((4.0, -6.0, 2.5), (3.0, -3.5, 1.4), (1.875, -1.25, 0.375), (1.875, -1.25, 0.375))
    o = mc2.mc2_ns_orthogonalize(gd, steps=4, coeffs=own, scale=-0.25, eps=20.0)
    _check(g, o, coeffs=own, scale=-0.25, eps=20.0)
    # the cubic iteration: singular values converge to 1
    o = mc2.mc2_ns_orthogonalize(gd, steps=16, coeffs=(1.5, -0.5, 0.0))
    assert (torch.linalg.svdvals(o.float().cpu()) - 1).abs().max() < 0.03
    _check(g, o, coeffs=((1.5, -0.5, 0.0),) * 16)


def test_given_buffers_streams_and_repeats():
    """out and workspace of the caller's (the workspace full of NaN), another
    stream, two calls at once on two streams, out in g's place, the same bits
    every time."""
    gen = torch.Generator().manual_seed(4)
    gs = [torch.randn((3, 200, 136), generator=gen).to(BF).cuda() for _ in range(2)]
    need = mc2.mc2_ns_workspace_size(3, 200, 136)
    ref = [mc2.mc2_ns_orthogonalize(g) for g in gs]
    ws = [torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") for _ in gs]
    outs = [torch.full_like(g, float("nan")) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(3):
        for g, w, o, s in zip(gs, ws, outs, streams):
            with torch.cuda.stream(s):
                assert mc2.mc2_ns_orthogonalize(g, out=o, workspace=w) is o
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        assert torch.equal(r.view(torch.int16), o.view(torch.int16))
    with pytest.raises(mc2.Mc2Error):
        mc2.mc2_ns_orthogonalize(gs[0], workspace=ws[0][:need - 16])
    inplace = gs[0].clone()
    mc2.mc2_ns_orthogonalize(inplace, out=inplace)
    assert torch.equal(inplace.view(torch.int16), ref[0].view(torch.int16))


@pytest.mark.parametrize("B,m,n", [(2, 50, 120), (3, 200, 304), (90, 264, 520)])
def test_captured_and_replayed(B, m, n):
    """Replays of one captured call, with new values, eager calls on the same
    workspace and synchronizations between them, give the eager bits."""
    gen = torch.Generator().manual_seed(5)
    gs = [torch.randn((B, m, n), generator=gen).cuda() for _ in range(2)]
    ws = torch.empty(mc2.mc2_ns_workspace_size(B, m, n), dtype=torch.uint8, device="cuda")
    eager = [mc2.mc2_ns_orthogonalize(g, workspace=ws) for g in gs]
    g, o = gs[0].clone(), torch.empty_like(eager[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mc2.mc2_ns_orthogonalize(g, out=o, workspace=ws)
    for i in (1, 0, 0, 1):
        g.copy_(gs[i])
        o.fill_(3.0)
        mc2.mc2_ns_orthogonalize(gs[1 - i], workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), eager[i].view(torch.int16)), i


@pytest.mark.parametrize("B,m,n", [(1, 3, 65536), (1, 65536, 5), (1, 130, 20000), (65535, 1, 2),
                                   (300, 130, 190), (1, 2500, 2500)])
def test_long_thin_and_many(B, m, n):
    """The largest sides and stacks, and a square matrix wider than a round of
    tiles; some matrices of a large stack stand for all."""
    g = torch.randn((B, m, n), generator=torch.Generator().manual_seed(6)).cuda()
    o = mc2.mc2_ns_orthogonalize(g)
    torch.cuda.synchronize()
    pick = sorted({0, B // 2, B - 1})
    _check(g[pick], o[pick])


@pytest.mark.parametrize("m,n", [(50, 120), (120, 50), (200, 136)])
def test_in_place(m, n):
    g = torch.randn((3, m, n), generator=torch.Generator().manual_seed(7)).to(BF).cuda()
    ref = mc2.mc2_ns_orthogonalize(g)
    assert mc2.mc2_ns_orthogonalize(g, out=g) is g
    assert torch.equal(g.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("m,n", [(50, 120), (200, 136)])
def test_iterates_out_of_range_end_as_such(m, n):
    """Coefficients whose iterates grow without bound: infinities or NaN, and a
    matrix of zeros beside it stays zero."""
    g = torch.randn((2, m, n), generator=torch.Generator().manual_seed(8)).cuda()
    g[1] = 0
    o = mc2.mc2_ns_orthogonalize(g, steps=32, coeffs=(16.0, 16.0, 16.0))
    torch.cuda.synchronize()
    assert not torch.isfinite(o[0]).any() and (o[1] == 0).all()
