"""Gradients of the MoE unpermute and permute against the float64 oracle,
through the C ABI. Bounds: dy is one product, exact in fp64, rounded to the storage
type at once or by way of fp32 (the compiler may fuse the product with an fp16
conversion; both are within half a step and 2^-24); dprobs is an fp32
sum of H exact products, off by at most (H + 8) * 2^-24 of the sum of their
magnitudes; dx is an fp32 sum of K values, (K + 1) * 2^-24 of the sum of their
magnitudes, then half a step of the storage type."""
import numpy as np
import pytest
import torch

from gemm_collective_core_amd import mc2
from oracle import moe as om
from oracle import train as ot

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _routing(T, K, E, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    sel = np.stack([rng.permutation(E)[:K] if K <= E else rng.integers(0, E, K)
                    for _ in range(T)]).astype(np.int32)
    sel[rng.random((T, K)) < drop] = E
    return om.permute(np.zeros((T, 1), np.uint16), sel, E), rng


def _case(T, K, H, E, dt, seed, drop=0.0, rows=None):
    r, _ = _routing(T, K, E, seed, drop)
    g = torch.Generator().manual_seed(seed)
    rows = T * K if rows is None else rows
    return {"idx": torch.from_numpy(r["unpermute_idx"].astype(np.int32)),
            "sidx": torch.from_numpy(r["sorted_idx"].astype(np.int32)),
            "n_valid": int(r["n_valid"]),
            "dout": torch.randn((T, H), generator=g).to(dt),
            "y": torch.randn((rows, H), generator=g).to(dt),
            "probs": torch.rand((T, K), generator=g)}


def _np(t):
    return t.double().cpu().numpy()


def _check_unpermute(c, dy, dprobs, fill, err, bad):
    ref, written, rp, rbad = ot.unpermute_backward(_np(c["dout"]), _np(c["y"]), c["idx"].numpy(),
                                                   c["sidx"].numpy(), c["probs"].numpy())
    assert rbad == bad and bool(err.item() & mc2.MC2_DEVERR_INDEX) == bad
    T, K = c["probs"].shape
    if dy is not None:
        dt = dy.dtype
        got = _np(dy)
        # half a step of the type (of the smallest numbers: half their fixed
        # step), and the fp32 rounding of a product that is not rounded at once
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
        tol = (torch.finfo(dt).eps / 2 + 2.0 ** -24) * np.abs(ref) + tiny
        assert (np.abs(got - ref) <= tol)[written].all()
        assert (got[~written] == fill).all()
    if dprobs is not None:
        mag = np.abs(_np(c["dout"])) @ np.ones(c["dout"].shape[1])
        H = c["dout"].shape[1]
        idx = np.clip(c["idx"].numpy().reshape(T, K), 0, c["y"].shape[0] - 1)
        mag = np.stack([(np.abs(_np(c["dout"])) * np.abs(_np(c["y"])[idx[:, k]])).sum(1)
                        for k in range(K)], 1)
        d = np.abs(_np(dprobs) - rp)
        assert (d <= (H + 8) * 2.0 ** -24 * mag).all(), d.max()
        assert (_np(dprobs)[rp == 0] == 0).all()


CASES = [  # T, K, H, E, dtype, share of slots left out
    (1, 1, 8, 4, BF, 0.0), (5, 3, 64, 4, F16, 0.0), (7, 2, 72, 8, BF, 0.3),
    (33, 8, 128, 16, BF, 0.0), (64, 9, 136, 16, F16, 0.2), (129, 6, 256, 8, BF, 0.0),
    (100, 4, 264, 32, F16, 0.5), (50, 64, 512, 70, BF, 0.1), (41, 8, 520, 16, BF, 0.0),
    (300, 8, 2048, 64, BF, 0.0), (37, 13, 2312, 17, F16, 0.1), (17, 16, 4104, 16, BF, 0.0),
    (6, 2, 64, 4, BF, 1.0)]


@pytest.mark.parametrize("T,K,H,E,dt,drop", CASES)
def test_unpermute_backward(T, K, H, E, dt, drop):
    c = _case(T, K, H, E, dt, 100 + T, drop)
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    for need in ((True, True), (True, False), (False, True)):
        err = _err()
        dy = torch.full_like(d["y"], -3.0) if need[0] else None
        gy, gp = mc2.mc2_moe_unpermute_backward(d["dout"], d["y"], d["idx"], d["sidx"], d["probs"],
                                                dy=dy, need_dy=need[0], need_dprobs=need[1],
                                                dev_err=err)
        torch.cuda.synchronize()
        assert (gy is None) != need[0] and (gp is None) != need[1]
        _check_unpermute(c, gy, gp, -3.0, err, False)


@pytest.mark.parametrize("T,K,H,E,dt,drop", CASES)
def test_permute_backward(T, K, H, E, dt, drop):
    c = _case(T, K, H, E, dt, 200 + T, drop)
    err = _err()
    dx = mc2.mc2_moe_permute_backward(c["y"].cuda(), c["idx"].cuda(), K, dev_err=err)
    ref, bad = ot.permute_backward(_np(c["y"]), c["idx"].numpy(), T, K)
    mag, _ = ot.permute_backward(np.abs(_np(c["y"])), c["idx"].numpy(), T, K)
    assert not bad and err.item() == 0
    tol = torch.finfo(dt).eps / 2 * np.abs(ref) + (K + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -8)
    assert (np.abs(_np(dx) - ref) <= tol).all()


def test_faulty_indices_are_skipped_and_reported():
    T, K, H = 40, 4, 136
    c = _case(T, K, H, 8, BF, 7)
    c["idx"][3] = T * K            # beyond the rows
    c["idx"][10] = -2
    c["idx"][11] = 2 ** 31 - 1
    c["idx"][20] = c["idx"][21]    # two slots name one row: sorted_idx says whose it is
    c["sidx"][c["idx"][30]] = -1   # a row that sorted_idx gives to nobody
    c["sidx"][c["idx"][31]] = 2 ** 31 - 1
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    err = _err()
    dy = torch.full_like(d["y"], 5.0)
    gy, gp = mc2.mc2_moe_unpermute_backward(d["dout"], d["y"], d["idx"], d["sidx"], d["probs"],
                                            dy=dy, dev_err=err)
    torch.cuda.synchronize()
    _check_unpermute(c, gy, gp, 5.0, err, True)
    # without an error word the same rows are skipped
    gy2, _ = mc2.mc2_moe_unpermute_backward(d["dout"], d["y"], d["idx"], d["sidx"], d["probs"],
                                            dy=torch.full_like(d["y"], 5.0))
    assert torch.equal(gy2.view(torch.int16), gy.view(torch.int16))
    err.zero_()
    dx = mc2.mc2_moe_permute_backward(d["y"], d["idx"], K, dev_err=err)
    ref, bad = ot.permute_backward(_np(c["y"]), c["idx"].numpy(), T, K)
    assert bad and err.item() == mc2.MC2_DEVERR_INDEX
    assert (np.abs(_np(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5).all()


@pytest.mark.parametrize("rows", [0, 1, 50, 400])
def test_row_buffers_of_other_sizes(rows):
    """Fewer rows than slots (the slots beyond are skipped and reported), or
    more (the rows behind are left as they were)."""
    T, K, H = 25, 4, 64
    c = _case(T, K, H, 8, F16, 8, rows=rows)
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    err = _err()
    y = d["y"] if rows else torch.empty((0, H), dtype=F16, device="cuda")
    dy = torch.full_like(y, 2.0)
    if rows == 0:  # an empty tensor has no address: nothing to write to
        with pytest.raises(mc2.Mc2Error):
            mc2.mc2_moe_unpermute_backward(d["dout"], y, d["idx"], d["sidx"], d["probs"], dy=dy)
        return
    gy, gp = mc2.mc2_moe_unpermute_backward(d["dout"], y, d["idx"], d["sidx"], d["probs"], dy=dy,
                                            dev_err=err)
    torch.cuda.synchronize()
    _check_unpermute(c, gy, gp, 2.0, err, rows < T * K)


def test_infinities_stay_in_their_rows():
    """A row that no slot reads, a token whose slots are all left out and rows
    of infinities or NaN: only the slots that name them see them."""
    T, K, H = 12, 2, 64
    c = _case(T, K, H, 4, BF, 9)
    c["idx"].view(T, K)[3] = -1                      # token 3 has no slots
    lost = c["sidx"][(c["sidx"] // K) == 3]
    c["sidx"][(c["sidx"] // K) == 3] = -1
    assert len(lost) == K
    gone = [p for p in range(T * K) if c["sidx"][p] < 0]
    c["y"][gone] = float("nan")
    c["dout"][3] = float("inf")
    c["y"][c["idx"][0]] = float("inf")
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    err = _err()
    gy, gp = mc2.mc2_moe_unpermute_backward(d["dout"], d["y"], d["idx"], d["sidx"], d["probs"],
                                            dy=torch.zeros_like(d["y"]), dev_err=err)
    dx = mc2.mc2_moe_permute_backward(d["y"], d["idx"], K)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.isfinite(gy).all() and (gy[gone] == 0).all()
    assert torch.isfinite(gp.view(-1)[1:]).all() and not torch.isfinite(gp.view(-1)[0])
    assert (gp[3] == 0).all() and (dx[3] == 0).all()
    assert torch.isinf(dx[0]).all() and torch.isfinite(dx[1:]).all()


def test_gradients_against_differences():
    """The unpermute is linear in the rows and in the weights, the permute in
    the tokens: <gradient, v> equals the change of <dout, output> along v, up
    to the gradients' own rounding."""
    T, K, H, E = 60, 4, 136, 8
    c = _case(T, K, H, E, BF, 10)
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    gy, gp = mc2.mc2_moe_unpermute_backward(d["dout"], d["y"], d["idx"], d["sidx"], d["probs"])
    dx = mc2.mc2_moe_permute_backward(d["y"], d["idx"], K)
    rng = np.random.default_rng(3)
    idx = c["idx"].numpy().reshape(T, K)
    pr, y, do = _np(c["probs"]), _np(c["y"]), _np(c["dout"])

    def loss(y, pr):
        return sum((do * pr[:, k, None] * y[idx[:, k]]).sum() for k in range(K))

    vy, vp, vx = rng.standard_normal(y.shape), rng.standard_normal(pr.shape), \
        rng.standard_normal((T, H))
    ey = (np.abs(_np(gy)) * np.abs(vy)).sum() * (2.0 ** -8 + 2.0 ** -23)
    assert abs(loss(y + vy, pr) - loss(y, pr) - (_np(gy) * vy).sum()) <= ey
    ep = 1e-4 * np.abs(_np(gp) * vp).sum()
    assert abs(loss(y, pr + vp) - loss(y, pr) - (_np(gp) * vp).sum()) <= ep
    # the permute: sum over rows of y[p] * x[token of p]
    tok = c["sidx"].numpy() // K
    ex = (np.abs(_np(dx)) * np.abs(vx)).sum() * (2.0 ** -8 + 2.0 ** -20)
    assert abs((y * vx[tok]).sum() - (_np(dx) * vx).sum()) <= ex


def test_permute_kernels_indices_fit():
    """With mc2_moe_permute's own outputs, a slot left out and a row buffer of
    T*K rows: exactly the first expert_offsets[E] rows are written."""
    T, K, E, H = 90, 4, 16, 264
    rng = np.random.default_rng(11)
    sel = rng.integers(0, E, (T, K)).astype(np.int32)
    sel[4, 2] = E
    x = torch.randn((T, H)).to(BF).cuda()
    perm, sidx, uidx, offs = mc2.mc2_moe_permute(x, torch.from_numpy(sel).cuda(), E)
    probs = torch.rand((T, K)).cuda()
    err = _err()
    dy = torch.full((T * K, H), 9.0, dtype=BF, device="cuda")
    perm[T * K - 1] = 0  # not written by the permute
    mc2.mc2_moe_unpermute_backward(x, perm, uidx, sidx, probs, dy=dy, dev_err=err)
    n = int(offs[E].item())
    assert n == T * K - 1 and err.item() == 0
    assert (dy[n:] == 9.0).all() and not (dy[:n] == 9.0).all(1).any()


def test_offsets_beyond_32_bits():
    """Row buffers of more than 2^31 elements: rows near the end are found."""
    T, K, H = 131080, 8, 2056
    gen = torch.Generator(device="cuda").manual_seed(12)
    uidx = torch.randperm(T * K, generator=gen, device="cuda")
    sidx = torch.empty_like(uidx)
    sidx[uidx] = torch.arange(T * K, device="cuda")
    u32, s32 = uidx.to(torch.int32), sidx.to(torch.int32)
    y = torch.randn((T * K, H), generator=gen, device="cuda", dtype=BF)
    assert y.numel() > 2 ** 31
    dout = torch.randn((T, H), generator=gen, device="cuda", dtype=BF)
    probs = torch.rand((T, K), generator=gen, device="cuda")
    err = _err()
    dy, dp = mc2.mc2_moe_unpermute_backward(dout, y, u32, s32, probs, dev_err=err)
    dx = mc2.mc2_moe_permute_backward(y, u32, K, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    rows = torch.cat([torch.arange(4, device="cuda"), torch.arange(T * K - 60, T * K, device="cuda")])
    s = sidx[rows]
    d, yr = dout[s // K].double(), y[rows].double()
    ref = probs.view(-1)[s][:, None].double() * d
    assert ((dy[rows].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -24) * ref.abs() + 1e-38).all()
    tol = (H + 8) * 2.0 ** -24 * (d * yr).abs().sum(1)
    assert ((dp.view(-1)[s].double() - (d * yr).sum(1)).abs() <= tol).all()
    t = s // K
    mine = y[uidx.view(T, K)[t]].double()
    tol = 2.0 ** -8 * mine.sum(1).abs() + (K + 1) * 2.0 ** -23 * mine.abs().sum(1)
    assert ((dx[t].double() - mine.sum(1)).abs() <= tol).all()
