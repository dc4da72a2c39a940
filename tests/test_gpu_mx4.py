"""The 4-bit operands on the GPU against their oracle: every code and scale of
the quantisation, every value of its inverse, and the product, in the sizes
where rows, blocks and tiles end inside each other."""
import numpy as np
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import mx4 as ox

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def draw(shape, dtype, seed, spread=3.0):
    """Values over a wide range, with ties of the 4-bit grid among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape, generator=g))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.75, -0.25, -5.0])
    pick = ties[torch.randint(0, len(ties), shape, generator=g)]
    x = torch.where(torch.rand(shape, generator=g) < 0.3, pick, x)
    return x.to(DT[dtype])


def check_quantize(x, trans):
    """Codes, scales and padding of every matrix of x, bit for bit."""
    codes, scales = mc2.mc2_mx4_quantize(x.cuda(), trans=trans)
    xs, cs, ss = (t if t.dim() == 3 else t[None] for t in (x, codes.cpu(), scales.cpu()))
    for m, c, s in zip(xs, cs, ss):
        ref = f64(m)
        pc, ps = ox.pack(*ox.quantize(ref.T if trans else ref))
        np.testing.assert_array_equal(c.numpy(), pc)
        np.testing.assert_array_equal(s.numpy(), ps)
    return codes, scales


SIZES = [(1, 1), (1, 32), (3, 33), (5, 31), (64, 256), (7, 1000), (129, 513), (33, 2047),
         (257, 96), (2, 8200), (300, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", SIZES)
@pytest.mark.parametrize("trans", [False, True])
def test_quantize_bits(rows, k, trans, dtype):
    x = draw((k, rows) if trans else (rows, k), dtype, rows * 7 + k, 1.0 if dtype == "f16" else 3.0)
    check_quantize(x, trans)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_stack(trans, dtype):
    check_quantize(draw((3, 70, 203), dtype, 5), trans)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_special_blocks(trans, dtype):
    """Blocks of zeros, of one NaN or infinity, of the type's smallest and
    largest numbers, and of its subnormals; neighbours are not touched."""
    t = DT[dtype]
    info = torch.finfo(t)
    sub = info.tiny * info.eps
    x = draw((40, 12 * 32), dtype, 9, 0.5)
    v = x.view(40, 12, 32)
    v[:, 1] = 0.0
    v[:, 2, 5] = float("nan")
    v[:, 3, 31] = float("inf")
    v[:, 4, 0] = float("-inf")
    v[:, 5] = 0.0
    v[:, 5, 7] = info.max
    v[:, 6] = torch.where(torch.arange(32) % 2 == 0, sub, -3 * sub).to(t)
    v[:, 7] = 0.0
    v[:, 7, 3] = info.tiny
    v[:, 8] = torch.where(torch.arange(32) % 3 == 0, -0.0, -info.max).to(t)
    v[:, 9] = 0.0
    v[:, 9, 31] = sub
    x = x.t().contiguous() if trans else x
    codes, scales = check_quantize(x, trans)
    back = mc2.mc2_mx4_dequantize(codes, scales, 12 * 32, out_dtype=torch.float32).cpu().view(40, 12, 32)
    assert back[:, 2:5].isnan().all() and back[:, :2].isfinite().all() and back[:, 5:].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [False, True])
def test_dequantize_every_code_and_scale(trans, dtype):
    """All 16 codes at all 256 scales, rounded once to the type."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    pc, ps = ox.pack(codes, scales)
    got = mc2.mc2_mx4_dequantize(torch.from_numpy(pc).cuda(), torch.from_numpy(ps).cuda(), 32,
                                 trans=trans, out_dtype=DT[dtype])
    got = (got.t() if trans else got).cpu()
    want = torch.from_numpy(ox.values(codes, scales, 32)).to(DT[dtype])
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(got[ok].view(torch.int32 if dtype == "f32" else torch.int16),
                       want[ok].view(torch.int32 if dtype == "f32" else torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", SIZES)
@pytest.mark.parametrize("trans", [False, True])
def test_dequantize_sizes(rows, k, trans, dtype):
    """Every element in its place, none written outside the matrix."""
    g = torch.Generator().manual_seed(rows + k)
    nb = ox.blocks(k)
    codes = torch.randint(0, 16, (rows, nb * 32), generator=g, dtype=torch.uint8).numpy()
    scales = torch.randint(120, 133, (rows, nb), generator=g, dtype=torch.uint8).numpy()
    pc, ps = ox.pack(codes, scales)
    shape = (k, rows) if trans else (rows, k)
    buf = torch.full((rows * k + 64,), 99.0, dtype=DT[dtype], device="cuda")
    out = buf[:rows * k].view(shape)
    mc2.mc2_mx4_dequantize(torch.from_numpy(pc).cuda(), torch.from_numpy(ps).cuda(), k,
                           trans=trans, out=out)
    want = torch.from_numpy(ox.values(codes, scales, k)).to(DT[dtype])
    assert torch.equal(out.cpu(), want.t() if trans else want)
    assert (buf[rows * k:] == 99.0).all()


def operand(rows, k, seed, lo=127, hi=129):
    g = torch.Generator().manual_seed(seed)
    nb = ox.blocks(k)
    codes = torch.randint(0, 16, (rows, nb * 32), generator=g, dtype=torch.uint8).numpy()
    codes[:, k:] = 0
    scales = torch.randint(lo, hi, (rows, nb), generator=g, dtype=torch.uint8).numpy()
    pc, ps = ox.pack(codes, scales)
    return (torch.from_numpy(pc).cuda(), torch.from_numpy(ps).cuda()), ox.values(codes, scales, k)


MM = [(1, 32, 8), (1, 8192, 264), (16, 1000, 40), (17, 33, 16), (33, 2048, 136), (64, 513, 24),
      (65, 32, 8), (65, 300, 264), (128, 256, 128), (200, 1416, 392), (513, 2080, 776),
      (130, 4096, 136), (300, 225, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k,n", MM)
@pytest.mark.parametrize("bias", [False, True])
def test_mm_exact(m, k, n, dtype, bias):
    """Scales of 1 and 2: every product is a multiple of 1/4 and every partial
    sum below 2^22 (k * 6 * 6 * 4 < 1.2e6), so that fp32 holds each exactly in
    whatever order, and the output is the exact sum rounded once."""
    a, av = operand(m, k, m + k)
    b, bv = operand(n, k, n + k + 1)
    bt = torch.randint(-64, 64, (n,), generator=torch.Generator().manual_seed(n)).bfloat16()
    out = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0, bias=bt.cuda() if bias else None,
                                  out_dtype=DT[dtype])
    want = torch.from_numpy(ox.mm(av, bv, f64(bt) if bias else None)).to(DT[dtype])
    assert torch.equal(out.cpu(), want)


def test_mm_large_tiles_exact():
    """Enough 256 x 256 tiles for the kernel of many rows, ragged on every side
    (2^22 is out of reach at this k too)."""
    m, k, n = 5003, 1000, 2056
    a, av = operand(m, k, 1)
    b, bv = operand(n, k, 2)
    out = mc2.mc2_mx4_mm_rs_local(*a, *b, k, 1, 0, out_dtype=torch.float32)
    want = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t().contiguous()
    assert torch.equal(out.double(), want)
    for t in (torch.bfloat16, torch.float16):
        got = mc2.mc2_mx4_mm_rs_local(*a, *b, k, 1, 0, out_dtype=t)
        assert torch.equal(got, want.to(t))


@pytest.mark.parametrize("m,k,n", [(40, 4096, 64), (260, 1024, 256), (4200, 512, 2048)])
def test_mm_wide_scales(m, k, n):
    """Scales over 2^-20 .. 2^20: each of the at most k + 8 additions is off by
    at most 2^-23 (a truncated sum; 2^-24 if rounded) of the sum of magnitudes."""
    a, av = operand(m, k, 3, 107, 148)
    b, bv = operand(n, k, 4, 107, 148)
    out = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0, out_dtype=torch.float32)
    av, bv = torch.from_numpy(av).cuda(), torch.from_numpy(bv).cuda()
    ref, mag = av @ bv.t().contiguous(), av.abs() @ bv.abs().t().contiguous()
    assert ((out.double() - ref).abs() <= (k + 8) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("m,n", [(20, 24), (200, 264), (4200, 2048)])
def test_mm_nan_stays_in_its_row_and_column(m, n):
    k = 512
    a, av = operand(m, k, 5)
    b, bv = operand(n, k, 6)
    a[1][m - 2, 3] = 255
    b[1][5, 15] = 255
    out = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0, out_dtype=torch.float32)
    want = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t().contiguous()
    nan = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    nan[m - 2], nan[:, 5] = True, True
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out.double()[~nan], want[~nan])


@pytest.mark.parametrize("op", ["ag", "rs"])
@pytest.mark.parametrize("W,mc,turn", [(2, 30, 0), (4, 250, 3), (8, 700, 0), (4, 1, 1), (2, 513, 7)])
def test_mm_chunks_and_flags(op, W, mc, turn):
    """Every segment's flag is raised, the counters end at zero, and the output
    does not depend on the schedule."""
    m, k, n = W * mc, 416, 520
    a, av = operand(m, k, 7)
    b, bv = operand(n, k, 8)
    want = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t().contiguous()
    segs = W * max(turn, 1)
    flags = torch.zeros(segs, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(segs, dtype=torch.int32, device="cuda")
    f = mc2.mc2_mx4_ag_mm_local if op == "ag" else mc2.mc2_mx4_mm_rs_local
    for epoch, rank in ((3, 0), (4, W - 1)):
        for t in (torch.float32, torch.bfloat16):
            flags.zero_()
            out = f(*a, *b, k, W, rank, out_dtype=t, ready_flags=flags, flag_counters=cnt,
                    epoch=epoch, comm_turn=turn)
            torch.cuda.synchronize()
            assert flags.cpu().tolist() == [epoch] * segs
            assert cnt.cpu().tolist() == [0] * segs
            assert torch.equal(out, want.to(t))


def tiles_of(W, mc, turn, n):
    """Tiles of a call with flags, which always takes the tiled kernel: (rows of a
    tile, whole tiles, tiles that run as two halves)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    sub = max(turn, 1)
    pieces = [mc // sub + (j < mc % sub) for j in range(sub)] * W

    def count(b):
        return sum(-(-p // b) for p in pieces) * -(-n // b)
    if 4 * count(256) <= cus:
        return 128, count(128), 0
    rem = count(256) % cus
    return 256, count(256) - (rem if 2 * rem <= cus else 0), rem if 2 * rem <= cus else 0


# W, rows a chunk, pieces, n, rows of a tile, whether tiles run whole, as halves
TILED = [(1, 1000, 0, 1416, 128, True, False), (8, 1, 0, 24, 128, True, False),
         (4, 130, 3, 264, 128, True, False), (2, 1150, 0, 2056, 256, False, True),
         (1, 3000, 0, 2824, 256, True, False), (2, 1500, 5, 2824, 256, True, False),
         (1, 4400, 0, 4096, 256, True, True), (2, 2200, 0, 4096, 256, True, True),
         (4, 1100, 2, 4000, 256, True, True)]


@pytest.mark.parametrize("W,mc,turn,n,bm,whole,halves", TILED)
@pytest.mark.parametrize("k", [64, 256, 512, 520, 1000])
def test_mm_tiles_exact_with_flags(W, mc, turn, n, bm, whole, halves, k):
    """Every kind of tile, each with one stage of K, whole stages and a last part,
    with and without a bias, in the three output types: the exact sums, every
    segment's flag and counter. (Sums as in test_mm_exact.) Where whole and half
    tiles meet, n_full lies inside a segment."""
    assert tiles_of(W, mc, turn, n)[0] == bm
    assert [v > 0 for v in tiles_of(W, mc, turn, n)[1:]] == [whole, halves]
    m, segs = W * mc, W * max(turn, 1)
    a, av = operand(m, k, k + 1)
    b, bv = operand(n, k, k + 2)
    bias = torch.randint(-64, 64, (n,), generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    ref = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t().contiguous()
    flags, cnt = (torch.zeros(segs, dtype=torch.int32, device="cuda") for _ in range(2))
    f = mc2.mc2_mx4_mm_rs_local if k % 256 else mc2.mc2_mx4_ag_mm_local
    for epoch, (t, bt) in enumerate(((torch.float32, None), (torch.float32, bias),
                                     (torch.bfloat16, bias), (torch.float16, bias)), 1):
        out = f(*a, *b, k, W, W - 1, bias=bt, out_dtype=t, ready_flags=flags, flag_counters=cnt,
                epoch=epoch, comm_turn=turn)
        want = ref if bt is None else ref + bt.double()
        assert torch.equal(out, want.to(t)), t
        assert flags.tolist() == [epoch] * segs and cnt.tolist() == [0] * segs


@pytest.mark.parametrize("sa,sb", [(254, 0), (0, 254), (254, 60), (104, 1), (20, 100), (0, 0),
                                   (253, 127), (254, 254)])
@pytest.mark.parametrize("m", [16, 40, 130])
def test_mm_extreme_scales(m, sa, sb):
    """One product an output, of the largest and smallest powers of two: exact where
    fp32 holds it, its subnormals too, infinite or rounded to nearest past that."""
    k, n = 64, 64
    ops = []
    for rows, s, seed in ((m, sa, 1), (n, sb, 2)):
        codes = np.zeros((rows, k), np.uint8)
        codes[:, 35] = np.random.default_rng(seed).integers(0, 16, rows)
        scales = np.full((rows, 2), s, np.uint8)
        ops.append((*(torch.from_numpy(v).cuda() for v in ox.pack(codes, scales)),
                    ox.values(codes, scales, k)))
    (a, sc_a, av), (b, sc_b, bv) = ops
    flags, cnt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    kw = dict(ready_flags=flags, flag_counters=cnt, epoch=1) if m > 64 else {}  # (flags: tiles)
    out = mc2.mc2_mx4_ag_mm_local(a, sc_a, b, sc_b, k, 1, 0, out_dtype=torch.float32, **kw)
    assert torch.equal(out.cpu(), torch.from_numpy(av @ bv.T).float())
