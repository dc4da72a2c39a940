"""The MoE layer for few tokens against its oracle: exactly, on inputs whose
every intermediate is a small integer, and on drawn ones; and the calls that
decoding makes of it (captured, on another stream, one workspace after
another)."""
import numpy as np
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import moe_tokens as ot

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def f64(t):
    return t.double().cpu().numpy()


def route(g, T, K, E, how):
    if how == "one":  # every slot to one expert
        return torch.full((T, K), E // 2, dtype=torch.int32)
    if how == "dup":  # the same expert several times in a token
        return torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).expand(T, K).contiguous()
    if how == "bad":  # some ids out of range
        s = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
        s.view(-1)[::3] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31, E + 5],
                                       dtype=torch.int32).repeat(T * K)[:len(s.view(-1)[::3])]
        return s
    p = torch.rand((T, E), generator=g) + 0.5 * torch.rand((1, E), generator=g)
    return p.topk(min(K, E), 1).indices.to(torch.int32) if K <= E else torch.randint(
        0, E, (T, K), generator=g, dtype=torch.int32)


def integer_case(T, H, I, E, E_l, K, how, seed):
    """Column 0 of x is 192 and its gate weights +-1, all other x and w1 in {-1,
    0, 1}: a gate is then beyond +-128, where silu is the identity or zero in
    fp32 (exp(-128) < 2^-149), and h = gate * up is an integer of at most 16
    bits, which two bf16 numbers hold. w2 in {-2 .. 2} and powers of two as
    routing weights keep every sum exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    small = lambda *s: torch.randint(-1, 2, s, generator=g).float()  # noqa: E731
    x = small(T, H) * (torch.rand((T, H), generator=g) < min(1.0, 250 / H))
    x[:, 0] = 192
    w1 = small(E_l, H, 2 * I)
    w1[:, 0, :I] = torch.where(torch.rand((E_l, I), generator=g) < 0.7, 1.0, -1.0)
    w1[:, 0, I:] = 0
    w2 = torch.randint(-2, 3, (E_l, I, H), generator=g).float()
    probs = 2.0 ** torch.randint(-2, 2, (T, K), generator=g).float()
    return x.to(BF), route(g, T, K, E, how), probs, w1.to(BF), w2.to(BF)


def own(x, sel, probs, w1, w2, mx4, **kw):
    x, sel, probs, w1, w2 = (t.cuda() for t in (x, sel, probs, w1, w2))
    if mx4:
        (w1, s1), (w2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
        kw.update(w1_scale=s1, w2_scale=s2)
    return mc2.mc2_moe_tokens(x, sel, probs, w1, w2, **kw)


CASES = [
    # T, H, I, E, E_l, K, routing
    (1, 8, 8, 4, 4, 1, "top"), (1, 264, 136, 32, 32, 8, "top"), (2, 72, 40, 8, 8, 2, "top"),
    (1, 136, 72, 8, 8, 4, "dup"), (16, 40, 264, 16, 16, 4, "top"), (16, 264, 72, 6, 3, 5, "one"),
    (17, 136, 136, 8, 8, 2, "one"), (17, 264, 8, 60, 15, 4, "top"), (37, 1416, 200, 32, 8, 6, "top"),
    (64, 264, 136, 128, 128, 8, "top"), (65, 72, 72, 5, 5, 1, "one"), (130, 136, 104, 3, 1, 3, "dup"),
    (256, 72, 40, 16, 16, 16, "top"), (40, 200, 72, 16, 4, 4, "bad"), (3, 2056, 24, 1024, 512, 64, "top"),
    (256, 24, 56, 1, 1, 2, "dup"), (5, 48, 600, 8, 2, 3, "top"),
]


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T,H,I,E,E_l,K,how", CASES)
def test_exact(T, H, I, E, E_l, K, how, mx4):
    case = integer_case(T, H, I, E, E_l, K, how, T * 31 + H)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for rank in range(min(E // E_l, 3)):
        ws = torch.full((mc2.mc2_moe_tokens_workspace_size(T, K, H, I),), 255, dtype=torch.uint8,
                        device="cuda")
        out = own(*case, mx4, ep_rank=rank, num_experts=E, workspace=ws, dev_err=err)
        ref, mag, bad = ot.layer(*(f64(t) if t.dtype != torch.int32 else t.numpy() for t in case),
                                 ep_rank=rank, num_experts=E)
        assert mag.max() < 2.0 ** 38 and np.abs(ref).max() < 2.0 ** 22  # sums stay exact
        want = torch.from_numpy(ref).to(BF)
        off = (out.cpu() != want).nonzero()
        assert len(off) == 0, (rank, len(off), off[:4])
    assert bool(err.item() & mc2.MC2_DEVERR_EXPERT_ID) == (how == "bad")


def drawn(T, H, I, E, E_l, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).to(BF)
    w1 = (0.02 * torch.randn((E_l, H, 2 * I), generator=g)).to(BF)
    w2 = (0.02 * torch.randn((E_l, I, H), generator=g)).to(BF)
    logits = torch.randn((T, E), generator=g)
    probs, sel = torch.softmax(logits, 1).topk(K, 1)
    return x, sel.to(torch.int32), probs.contiguous(), w1, w2


def close(out, ref):
    """One rounding to bf16 (2^-8 of the value at most) on top of errors of the
    32-bit sums and of the 16-bit h, some 2^-16 of the result's size: 2^-12 of
    its root mean square covers them."""
    ref = torch.as_tensor(ref)
    err = (out.double().cpu() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -12 * ref.square().mean().sqrt()).all()


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T,H,I,E,E_l,K", [(1, 512, 264, 16, 16, 4), (20, 264, 392, 8, 4, 3),
                                           (70, 136, 128, 4, 4, 2)])
def test_drawn(T, H, I, E, E_l, K, mx4):
    case = list(drawn(T, H, I, E, E_l, K, 3))
    out = own(*case, mx4, ep_rank=0, num_experts=E)
    if mx4:  # the layer of the weights that the codes stand for
        for i in (3, 4):
            c, s = mc2.mc2_mx4_quantize(case[i].cuda(), trans=True)
            case[i] = mc2.mc2_mx4_dequantize(c, s, case[i].shape[1], trans=True,
                                             out_dtype=torch.float32).cpu()
    ref, _, _ = ot.layer(*(f64(t) if t.dtype != torch.int32 else t.numpy() for t in case),
                         ep_rank=0, num_experts=E)
    close(out, ref)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [3, 40])
def test_faults_stay_where_they_are(T, mx4):
    """NaN and infinities in one token, in experts that no slot names, and in
    the routing weights of slots that are not local reach no other output."""
    H, I, E, E_l, K = 136, 72, 16, 8, 4
    x, sel, probs, w1, w2 = integer_case(T, H, I, E, E_l, K, "top", 5)
    sel = torch.where((sel % 8 == 3), sel + 1, sel)  # experts 3 and 11 are not named
    args = dict(ep_rank=0, num_experts=E)
    base = own(x, sel, probs, w1, w2, mx4, **args).cpu()
    w1[3], w2[3] = float("nan"), float("inf")
    probs = torch.where(sel >= E_l, float("nan"), probs)
    sel[2] = 1
    x[2, 5] = float("nan")
    out = own(x, sel, probs, w1, w2, mx4, **args).cpu()
    assert out[2].isnan().all()
    keep = torch.arange(T) != 2
    assert torch.equal(out[keep], base[keep])
    sel[:] = E - 1  # no slot is local
    assert (own(x, sel, probs, w1, w2, mx4, **args) == 0).all()


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [1, 33])
def test_captured_and_replayed(T, mx4):
    """Replays with other tokens, routing and workspace contents give the eager
    bits, with the program's own eager calls between them."""
    H, I, E, K = 264, 136, 16, 4
    cases = [integer_case(T, H, I, E, E, K, "top", s) for s in (1, 2)]
    x, sel, probs, w1, w2 = (t.cuda() for t in cases[0])
    kw = dict(ep_rank=0, num_experts=E)
    if mx4:
        (w1, s1), (w2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
        kw.update(w1_scale=s1, w2_scale=s2)
    out = torch.empty_like(x)
    ws = torch.empty(mc2.mc2_moe_tokens_workspace_size(T, K, H, I), dtype=torch.uint8, device="cuda")

    def call():
        mc2.mc2_moe_tokens(x, sel, probs, w1, w2, out=out, workspace=ws, **kw)

    def load(c):
        for t, v in zip((x, sel, probs), c):
            t.copy_(v)

    eager = []
    for c in cases:
        load(c)
        call()
        eager.append(out.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in (0, 1, 1, 0):
        load(cases[i])
        ws.fill_(255)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
        call()
        assert torch.equal(out, eager[i])


def test_two_streams_with_a_workspace_each():
    T, H, I, E, K = 24, 264, 136, 16, 4
    cases = [tuple(t.cuda() for t in integer_case(T, H, I, E, E, K, "top", s)) for s in (3, 4)]
    want = [mc2.mc2_moe_tokens(*c, ep_rank=0, num_experts=E) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(20):
        for i, (s, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                outs[i].append(mc2.mc2_moe_tokens(*c, ep_rank=0, num_experts=E))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(v, w) for v in o)


def test_agrees_with_the_path_for_many_tokens():
    """One set of 4-bit expert weights, both ways to use them: this layer on the
    codes, and the grouped path (permute, fc1, fc2, unpermute) on the 16-bit
    weights that they stand for. The grouped path rounds h and y to bf16."""
    T, H, I, E, K = 48, 512, 264, 16, 4
    x, sel, probs, w1, w2 = (t.cuda() for t in drawn(T, H, I, E, E, K, 9))
    (c1, s1), (c2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
    out = mc2.mc2_moe_tokens(x, sel, probs, c1, c2, w1_scale=s1, w2_scale=s2, ep_rank=0,
                             num_experts=E)
    w1 = mc2.mc2_mx4_dequantize(c1, s1, H, trans=True)
    w2 = mc2.mc2_mx4_dequantize(c2, s2, I, trans=True)
    counts = mc2.mc2_moe_histc(sel, E)
    perm, _, uidx, _ = mc2.mc2_moe_permute(x, sel, E)
    kw = dict(ep_rank=0, num_experts=E)
    h = mc2.mc2_gmm_dispatch(perm, counts, counts, w1, **kw)
    buf = torch.zeros((T * K, H), dtype=BF, device="cuda")
    mc2.mc2_gmm_combine(h, counts, counts, w2, buf, **kw)
    many = mc2.mc2_moe_unpermute(buf, uidx, probs)
    # h and y are off by 2^-8 each at most, over sums of hundreds of terms and
    # of K slots, and both outputs by one rounding
    rms = out.double().square().mean().sqrt()
    err = (out.double() - many.double()).abs()
    assert (err <= 2.0 ** -7 * out.double().abs() + 2.0 ** -6 * rms).all()
    assert err.square().mean().sqrt() <= 2.0 ** -8 * 1.5 * rms


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [1, 24])
def test_weights_beyond_2_31_elements(T, mx4):
    """64 equal experts, 2.4e9 elements of w1: the last gives the first's output."""
    H, I, E, K = 4096, 4608, 64, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    w1 = (0.02 * torch.randn((1, H, 2 * I), generator=g, device="cuda")).to(BF)
    w2 = (0.02 * torch.randn((1, I, H), generator=g, device="cuda")).to(BF)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    probs = torch.rand((T, K), generator=g, device="cuda")
    kw = dict(num_experts=E, ep_rank=0)
    if mx4:
        (w1, s1), (w2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
        kw.update(w1_scale=s1.repeat(E, 1, 1), w2_scale=s2.repeat(E, 1, 1))
    w1, w2 = w1.repeat(E, 1, 1), w2.repeat(E, 1, 1)
    outs = [mc2.mc2_moe_tokens(x, torch.full((T, K), e, dtype=torch.int32, device="cuda"), probs,
                               w1, w2, **kw) for e in (0, 31, E - 1)]
    assert outs[0].abs().max() > 0.01
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [40, 48, 61, 256])
def test_a_token_does_not_depend_on_its_place(T, mx4):
    """Many slots of one expert are taken in groups of different sizes, in no
    particular order: a token's bits are the same in every group, so that they are
    the same in every call."""
    H, I, E, K = 1032, 776, 4, 2
    x, _, probs, w1, w2 = (t.cuda() for t in drawn(T, H, I, E, E, K, 17))
    sel = torch.tensor([1, 3], dtype=torch.int32, device="cuda").expand(T, 2).contiguous()
    kw = dict(ep_rank=0, num_experts=E)
    if mx4:
        (w1, s1), (w2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
        kw.update(w1_scale=s1, w2_scale=s2)
    out = mc2.mc2_moe_tokens(x, sel, probs, w1, w2, **kw)
    for shift in (1, T // 2, T - 5):
        got = mc2.mc2_moe_tokens(x.roll(shift, 0), sel, probs.roll(shift, 0), w1, w2, **kw)
        assert torch.equal(got, out.roll(shift, 0)), shift


def wide_h_case(T, I, K, seed):
    """Every h has 24 significant bits, of which fc2's sums need the last. x is 128
    at 0 (the gate, where silu is the identity in fp32) and 1 at three places of
    blocks of their own, whose up weights 2^13, 2^3 and 2^-7 (or 2^-6, 2^-5) make
    h = 2^20 + 2^10 + 1 (2, 4); its neighbour has h = 2^20 + 2^10, and w2 opposite
    signs for the two. Sums are of whole numbers below I * 2^20.1 <= 2^24."""
    g = torch.Generator().manual_seed(seed)
    assert I <= 15
    H, E = 128, 2
    x = torch.zeros((T, H))
    x[:, 0], x[:, 32], x[:, 64], x[:, 96] = 128, 1, 1, 1
    w1 = torch.zeros((E, H, 2 * I))
    w1[:, 0, :I] = 1
    w1[:, 32, I:], w1[:, 64, I:] = 2.0 ** 13, 2.0 ** 3
    w1[:, 96, I::2] = 2.0 ** -torch.randint(5, 8, (E, I // 2), generator=g).float()
    w2 = torch.zeros((E, I, H))
    w2[:, 0::2] = torch.randint(-1, 2, (E, I // 2, H), generator=g).float()
    w2[:, 1::2] = -w2[:, 0::2]
    sel = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    return x.to(BF), sel, torch.ones((T, K)), w1.to(BF), w2.to(BF)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T,K", [(1, 1), (20, 1), (40, 2)])
def test_h_keeps_all_the_bits_of_fp32(T, K, mx4):
    case = wide_h_case(T, 8, K, T)
    out = own(*case, mx4, ep_rank=0, num_experts=2)
    ref, _, _ = ot.layer(*(f64(t) if t.dtype != torch.int32 else t.numpy() for t in case),
                         ep_rank=0, num_experts=2)
    assert np.abs(ref).max() >= 4
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(BF))


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [1, 20])
def test_h_next_to_the_largest_number(T, mx4):
    """h = 2^127 * 511/256, between the largest bf16 number (2^127 * 255/128) and
    fp32's: finite, and so is the output, 2^117 * 511/256 rounded to even, 2^118."""
    x, _, probs, w1, w2 = wide_h_case(T, 8, 1, 1)
    w1[:, 32:, 8:] = 0
    # up = 2^120 * 511/256 = 2^121 - 2^112
    w1[:, 32, 8:], w1[:, 64, 8:] = 2.0 ** 121, -2.0 ** 112
    w2[:] = 0
    w2[:, 3, 5] = 2.0 ** -10
    sel = torch.zeros((T, 1), dtype=torch.int32)
    out = own(x, sel, probs, w1, w2, mx4, ep_rank=0, num_experts=2).cpu()
    want = torch.zeros_like(out)
    want[:, 5] = 2.0 ** 118
    assert torch.equal(out, want)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T,H,I,K", [(3, 40, 72, 1), (20, 136, 136, 1), (40, 72, 264, 2)])
def test_infinite_weights_of_named_experts(T, H, I, K, mx4):
    """Where w2 holds infinities, y is what h @ w2 gives: infinite with the sign of
    the products, NaN where signs differ or h is zero. In 4 bits an infinity is a
    code whose value is past bf16's largest number: 2 held as 4 * 2^-1, its scale
    raised to 2^126."""
    E = 2
    x, sel, probs, w1, w2 = integer_case(T, H, I, E, E, K, "top", 23)
    w1[:, 0, :I] = 1  # silu is the identity
    inf = float("inf")
    w2[:, :, 5:9] = 0
    for e in range(E):
        w2[e, 1 + e, 5] = 2
        w2[e, I - 1, 6] = -2
        w2[e, 3, 7], w2[e, I - 2, 7] = 2, -2
        w2[e, 2::3, 8] = 2
    big = f64(w2)
    big[:, :, 5:9] *= np.where(big[:, :, 5:9] == 0, 1, inf)
    with np.errstate(invalid="ignore"):
        ref, _, _ = ot.layer(f64(x), sel.numpy(), f64(probs), f64(w1), big, ep_rank=0, num_experts=E)
    args = [t.cuda() for t in (x, sel, probs)]
    if mx4:
        (c1, s1), (c2, s2) = (mc2.mc2_mx4_quantize(w.cuda(), trans=True) for w in (w1, w2))
        s2[:, 5:9, :(I + 31) // 32] = 253
        out = mc2.mc2_moe_tokens(*args, c1, c2, w1_scale=s1, w2_scale=s2, ep_rank=0, num_experts=E)
    else:
        out = mc2.mc2_moe_tokens(*args, w1.cuda(), torch.from_numpy(big).to(BF).cuda(), ep_rank=0,
                                 num_experts=E)
    out, want = out.cpu(), torch.from_numpy(ref).to(BF)
    assert want[:, 5:9].isinf().any() and not want[:, 5:9].isfinite().any()
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out[~out.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("mx4,T,H,I,E", [
    # weights, tokens, sizes, experts: strips of fc1 a matrix, groups of K loads a strip
    (True, 60, 72, 200, 512),     # 7 strips of 32 columns, the last of 8; one group
    (True, 16, 72, 200, 512),
    (True, 60, 2056, 200, 512),   # two groups, four for 17 slots or more
    (True, 16, 2056, 232, 400),   # 8 strips
    (False, 60, 72, 136, 1024),   # 3 strips of 64 columns, the last of 8; one group
    (False, 16, 72, 136, 1024),
    (False, 60, 1032, 136, 1024),  # three groups
    (False, 16, 1032, 200, 800),  # 4 strips
])
def test_two_strips_a_workgroup(mx4, T, H, I, E):
    """fc1 with so many workgroups that each takes two neighbouring strips, for
    experts with 1, 11, 16, 17, 28 and 32 slots at a time. Only the experts named
    hold numbers, the others NaN."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    strips = -(-I // (32 if mx4 else 64))
    assert strips * E >= 12 * cus  # the rule of the launch
    Ec, K = 24, 6
    x, _, probs, w1, w2 = integer_case(T, H, I, Ec, Ec, K, "top", T + H)
    g = torch.Generator().manual_seed(H)
    sel = torch.randint(3, Ec, (T, K), generator=g, dtype=torch.int32)
    sel[:, 0] = 0
    sel[:, 4] = torch.where(torch.arange(T) < 17, 1, 2)
    ref, mag, _ = ot.layer(f64(x), sel.numpy(), f64(probs), f64(w1), f64(w2), ep_rank=0,
                           num_experts=Ec)
    assert mag.max() < 2.0 ** 38 and np.abs(ref).max() < 2.0 ** 22
    place = torch.cat([torch.tensor([0, E - 1]), 1 + torch.randperm(E - 2, generator=g)[:Ec - 2]])
    big = []
    for w in (w1, w2):
        b = torch.full((E, *w.shape[1:]), float("nan"), dtype=BF, device="cuda")
        b[place.cuda()] = w.cuda()
        big.append(b)
    out = own(x, place[sel.long()].to(torch.int32), probs, *big, mx4, ep_rank=0, num_experts=E)
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(BF))


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [1, 24])
def test_weights_beyond_2_31_elements_by_the_formula(T, mx4):
    """64 experts, 2.4e9 elements of w1, of which the first and the last hold numbers
    and are named: against the formula in 64 bits."""
    H, I, E = 4096, 4608, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    named = (0, E - 1)
    w1 = torch.full((E, H, 2 * I), float("nan"), dtype=BF, device="cuda")
    w2 = torch.full((E, I, H), float("nan"), dtype=BF, device="cuda")
    for e in named:
        w1[e] = 0.02 * torch.randn((H, 2 * I), generator=g, device="cuda")
        w2[e] = 0.02 * torch.randn((I, H), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    probs = torch.rand((T, 4), generator=g, device="cuda")
    sel = torch.tensor([0, E - 1, 0, E - 1], dtype=torch.int32, device="cuda").expand(T, 4).contiguous()
    kw = dict(num_experts=E, ep_rank=0)
    vals = [(w1[e].double(), w2[e].double()) for e in named]
    if mx4:
        (w1, s1), (w2, s2) = (mc2.mc2_mx4_quantize(w, trans=True) for w in (w1, w2))
        kw.update(w1_scale=s1, w2_scale=s2)
        vals = [tuple(mc2.mc2_mx4_dequantize(w[e], s[e], k, trans=True, out_dtype=torch.float32).double()
                      for w, s, k in ((w1, s1, H), (w2, s2, I))) for e in named]
    out = mc2.mc2_moe_tokens(x, sel, probs, w1, w2, **kw)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for i, (v1, v2) in enumerate(vals):
        a = x.double() @ v1
        y = (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ v2
        ref += probs[:, i::2].double().sum(1, keepdim=True) * y
    assert ref.abs().max() > 0.01
    close(out, ref.cpu())
