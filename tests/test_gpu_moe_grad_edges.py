"""The gradients of the MoE unpermute and permute at the edges of what they
take. Values are small integers and powers of two, so that every result is
exact and compared for equality."""
import pytest
import torch

from gemm_collective_core_amd import mc2

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _ints(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=gen, device="cuda", dtype=torch.int8).to(BF)


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def test_unpermute_backward_of_more_tokens_than_one_launch_holds():
    """2^28 tokens and more: 2^32 threads for both gradients of narrow rows."""
    T, H = 2 ** 28 + 5, 8
    idx = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")  # its own inverse
    dout, y = _ints((T, H), 1), _ints((T, H), 2)
    probs = torch.exp2(_ints((T, 1), 3).float())
    err = _err()
    dy, dp = mc2.mc2_moe_unpermute_backward(dout, y, idx, idx, probs, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    step = 2 ** 26
    for t in range(0, T, step):
        d = dout[t:t + step].float()
        rows = slice(max(T - t - step, 0), T - t)
        assert torch.equal(dy[rows].flip(0).float(), probs[t:t + step] * d)
        assert torch.equal(dp[t:t + step, 0], (d * y[rows].flip(0).float()).sum(1))


def test_permute_backward_of_more_tokens_than_one_launch_holds():
    T, H, rows = 2 ** 29 + 5, 8, 1000
    idx = torch.arange(T, dtype=torch.int32, device="cuda") % rows
    g = _ints((rows, H), 4)
    err = _err()
    dx = mc2.mc2_moe_permute_backward(g, idx, 1, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    step = 2 ** 22  # (torch's own indexing has a smaller limit)
    for t in range(0, T, step):
        assert torch.equal(dx[t:t + step], g[idx[t:t + step].long()])


@pytest.mark.parametrize("named", [False, True])
def test_permute_backward_without_rows(named):
    """A rank whose row buffer is empty: every token's gradient is zero, and a
    slot that names a row all the same is reported."""
    T, K, H = 21, 3, 72
    idx = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    if named:
        idx[17] = 0
    err = _err()
    dx = mc2.mc2_moe_permute_backward(torch.empty((0, H), dtype=BF, device="cuda"), idx, K,
                                      dx=torch.ones((T, H), dtype=BF, device="cuda"), dev_err=err)
    torch.cuda.synchronize()
    assert (dx == 0).all() and err.item() == (mc2.MC2_DEVERR_INDEX if named else 0)


def test_unpermute_backward_without_what_it_does_not_read():
    T, K, H = 40, 4, 136
    idx = torch.randperm(T * K, device="cuda").to(torch.int32)
    sidx = torch.empty_like(idx)
    sidx[idx.long()] = torch.arange(T * K, dtype=torch.int32, device="cuda")
    dout, y = _ints((T, H), 5), _ints((T * K, H), 6)
    probs = torch.exp2(_ints((T, K), 7).float())
    dy, dp = mc2.mc2_moe_unpermute_backward(dout, y, idx, sidx, probs)
    got, none = mc2.mc2_moe_unpermute_backward(dout, None, idx, sidx, probs,
                                               dy=torch.zeros_like(dy), need_dprobs=False)
    assert none is None and torch.equal(got, dy)
    none, got = mc2.mc2_moe_unpermute_backward(dout, y, idx, sidx, None, need_dy=False)
    assert none is None and torch.equal(got, dp)
