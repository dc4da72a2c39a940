"""The 4-bit operands where a user's program goes with them: a linear layer's
forward and backward, captured and replayed, operands and outputs beyond 2^31
elements, and one operand in every way of being read."""
import pytest
import torch

from gemm_collective_core_amd import mc2

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(shape, seed, dtype=BF, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def values(op, k):
    return mc2.mc2_mx4_dequantize(*op, k, out_dtype=torch.float32).double()


class Linear:
    """y = Q(x) Q(w)^T, dx = Q(dy) Q(w^T)^T, dw = Q(dy^T) Q(x^T)^T, every buffer kept."""

    def __init__(self, m, k, n):
        def op(rows, c):
            return (torch.empty((rows, mc2.mc2_mx4_row_bytes(c)), dtype=torch.uint8, device="cuda"),
                    torch.empty((rows, mc2.mc2_mx4_scale_bytes(c)), dtype=torch.uint8, device="cuda"))
        self.m, self.k, self.n = m, k, n
        self.x, self.w, self.dy = rnd((m, k), 1), rnd((n, k), 2, std=0.1), rnd((m, n), 3)
        self.qx, self.qw, self.qdy = op(m, k), op(n, k), op(m, n)
        self.qxt, self.qwt, self.qdyt = op(k, m), op(k, n), op(n, m)
        self.y = torch.empty((m, n), dtype=BF, device="cuda")
        self.dx = torch.empty((m, k), dtype=BF, device="cuda")
        self.dw = torch.empty((n, k), dtype=torch.float32, device="cuda")

    def run(self):
        for t, plain, trans in ((self.x, self.qx, self.qxt), (self.w, self.qw, self.qwt),
                                (self.dy, self.qdy, self.qdyt)):
            mc2.mc2_mx4_quantize(t, codes=plain[0], scales=plain[1])
            mc2.mc2_mx4_quantize(t, trans=True, codes=trans[0], scales=trans[1])
        mc2.mc2_mx4_ag_mm_local(*self.qx, *self.qw, self.k, 1, 0, out=self.y)
        mc2.mc2_mx4_mm_rs_local(*self.qdy, *self.qwt, self.n, 1, 0, out=self.dx)
        mc2.mc2_mx4_mm_rs_local(*self.qdyt, *self.qxt, self.m, 1, 0, out=self.dw)

    def outputs(self):
        return [t.clone() for t in (self.y, self.dx, self.dw)]


@pytest.mark.parametrize("m,k,n", [(48, 96, 64), (200, 136, 264), (1000, 520, 776)])
def test_linear_layer_and_its_gradients(m, k, n):
    """Against the formulas in 64 bits on the values that the codes stand for
    (whose derivatives are these products: each output is linear in each
    operand, which a difference of two calls shows for one element)."""
    s = Linear(m, k, n)
    s.run()
    for out, a, b, c in ((s.y, s.qx, s.qw, k), (s.dx, s.qdy, s.qwt, n), (s.dw, s.qdyt, s.qxt, m)):
        av, bv = values(a, c), values(b, c)
        ref, mag = av @ bv.t().contiguous(), av.abs() @ bv.abs().t().contiguous()
        eps = 2.0 ** -8 if out.dtype == BF else 0.0
        # sums of at most c + 8 terms, off by 2^-23 of the magnitudes each, and a rounding
        assert ((out.double() - ref).abs() <= eps * ref.abs() + (c + 8) * 2.0 ** -23 * mag).all()
    # d loss / d w[5, 7] with loss = sum(dy * y): the difference of two forwards
    # in fp32 whose weight differs in that code alone
    dyv, wv = values(s.qdy, n), values(s.qw, k)
    w2 = (s.qw[0].clone(), s.qw[1])
    byte, high = divmod(7, 2)
    code = (w2[0][5, byte] >> (4 if high else 0)) & 15
    w2[0][5, byte] ^= 1 << (4 if high else 0)  # the neighbouring value
    y0, y1 = (mc2.mc2_mx4_ag_mm_local(*s.qx, *w, k, 1, 0, out_dtype=torch.float32).double()
              for w in (s.qw, w2))
    step = values(w2, k)[5, 7] - wv[5, 7]
    assert step != 0, code
    num = (dyv * (y1 - y0)).sum() / step
    ana = (dyv.t().contiguous() @ values(s.qx, k))[5, 7]
    tol = (k + 8) * 2.0 ** -22 * (dyv[:, 5].abs() @ (values(s.qx, k).abs() @ wv[5].abs())) / step.abs()
    assert (num - ana).abs() <= tol


def test_linear_layer_captured_and_replayed():
    s = Linear(200, 136, 264)
    inputs = [(rnd((200, 136), i), rnd((264, 136), i + 10), rnd((200, 264), i + 20)) for i in (4, 5)]

    def load(i):
        for t, v in zip((s.x, s.w, s.dy), inputs[i]):
            t.copy_(v)

    eager = []
    for i in (0, 1):
        load(i)
        s.run()
        eager.append(s.outputs())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in (0, 1, 1, 0):
        load(i)
        for t in (s.y, s.dx, s.dw):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((s.y, s.dx, s.dw), eager[i]):
            assert torch.equal(got, want)


def test_flags_captured_and_replayed():
    m, k, n, W = 800, 300, 520, 4
    a, b = (mc2.mc2_mx4_quantize(rnd((r, k), r)) for r in (m, n))
    want = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0)
    flags = torch.zeros(W, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(W, dtype=torch.int32, device="cuda")
    out = torch.empty_like(want)
    kw = dict(out=out, ready_flags=flags, flag_counters=cnt, epoch=9)
    mc2.mc2_mx4_ag_mm_local(*a, *b, k, W, 1, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mc2.mc2_mx4_ag_mm_local(*a, *b, k, W, 1, **kw)
    for _ in range(3):
        flags.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert flags.tolist() == [9] * W and cnt.tolist() == [0] * W
        assert torch.equal(out, want)


def test_schedules_give_the_same_bits():
    """Chunks, ranks, pieces and flags change no output of the tiled kernel, nor
    does a second call."""
    m, k, n = 1040, 700, 776
    a, b = (mc2.mc2_mx4_quantize(rnd((r, k), r)) for r in (m, n))
    want = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0, out_dtype=torch.float32)
    for W, rank, turn in ((1, 0, 0), (2, 1, 0), (8, 3, 2), (4, 0, 5), (16, 7, 65)):
        for f in (mc2.mc2_mx4_ag_mm_local, mc2.mc2_mx4_mm_rs_local):
            out = f(*a, *b, k, W, rank, comm_turn=turn, out_dtype=torch.float32)
            assert torch.equal(out, want), (W, rank, turn)


@pytest.mark.parametrize("trans", [False, True])
def test_operands_beyond_2_31_elements(trans):
    """70 copies of 1024 rows (columns) of 65536 values, 4.7e9 elements and 2.3e9
    bytes of codes: every copy gets the codes of the first, and they read back."""
    rows, k, copies = 1024, 65536, 70
    base = rnd((k, rows) if trans else (rows, k), 6)
    x = base.repeat(1, copies) if trans else base.repeat(copies, 1)
    c0, s0 = mc2.mc2_mx4_quantize(base, trans=trans)
    c, s = mc2.mc2_mx4_quantize(x, trans=trans)
    assert (c.view(copies, *c0.shape) == c0).all() and (s.view(copies, *s0.shape) == s0).all()
    x.zero_()
    mc2.mc2_mx4_dequantize(c, s, k, trans=trans, out=x)
    back = mc2.mc2_mx4_dequantize(c0, s0, k, trans=trans)
    for i in range(copies):
        part = x[:, i * rows:(i + 1) * rows] if trans else x[i * rows:(i + 1) * rows]
        assert torch.equal(part, back), i


def test_outputs_beyond_2_31_elements():
    """300 copies of 1024 rows against 8192 columns: 2.5e9 outputs."""
    k, n, copies = 64, 8192, 300
    a, b = mc2.mc2_mx4_quantize(rnd((1024, k), 7)), mc2.mc2_mx4_quantize(rnd((n, k), 8))
    big = tuple(t.repeat(copies, 1) for t in a)
    out = mc2.mc2_mx4_ag_mm_local(*big, *b, k, 1, 0)
    want = mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0)
    for i in range(copies):
        assert torch.equal(out[i * 1024:(i + 1) * 1024], want), i


def test_on_another_stream_and_twice_at_once():
    m, k, n = 300, 1000, 264
    pairs = [(mc2.mc2_mx4_quantize(rnd((m, k), i)), mc2.mc2_mx4_quantize(rnd((n, k), i + 5)))
             for i in (1, 2)]
    want = [mc2.mc2_mx4_ag_mm_local(*a, *b, k, 1, 0) for a, b in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(mc2.mc2_mx4_ag_mm_local(*pairs[i][0], *pairs[i][1], k, 1, 0))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(v, w) for v in o)


def test_views_are_refused():
    x = rnd((64, 64), 1)
    with pytest.raises(ValueError, match="contiguous"):
        mc2.mc2_mx4_quantize(x.t())
    c, s = mc2.mc2_mx4_quantize(x)
    with pytest.raises(ValueError, match="contiguous"):
        mc2.mc2_mx4_dequantize(c, s, 64, out=torch.empty((64, 64), dtype=BF, device="cuda").t())
