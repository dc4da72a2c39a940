"""The binding of the training operators: inputs that a call does not read may
be left out, the others may not. (CPU tensors: a call whose arguments are
accepted ends at the check that they are on the GPU.)"""
import pytest
import torch

from gemm_collective_core_amd import mc2

T, K, H = 10, 4, 64
BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


IDX, PROBS = z(T * K, dtype=torch.int32), z(T, K, dtype=torch.float32)
DOUT, Y = z(T, H), z(T * K, H)


@pytest.mark.parametrize("args,kw,match", [
    ((None, IDX, PROBS), dict(need_dprobs=False, dy=Y), "on the GPU"),
    ((Y, IDX, None), dict(need_dy=False), "on the GPU"),
    ((Y, IDX, None), dict(need_dy=False, dprobs=PROBS), "on the GPU"),
    ((None, IDX, PROBS), dict(need_dprobs=False), "y_full is needed"),
    ((None, IDX, PROBS), dict(dy=Y), "y_full is needed"),
    ((Y, IDX, None), {}, "probs is needed"),
    ((Y, IDX[:-1], None), dict(need_dy=False), "unpermute_idx must hold"),
    ((Y, IDX, None), dict(need_dy=False, dprobs=z(T, K + 1, dtype=torch.float32)),
     "dprobs must have shape"),
    ((None, IDX, PROBS), dict(need_dprobs=False, dy=z(T * K, H + 8)), "dy must have shape"),
    ((z(T * K, H, 1), IDX, PROBS), {}, "probs must be"),
])
def test_unpermute_backward(args, kw, match):
    y, idx, probs = args
    with pytest.raises(ValueError, match=match):
        mc2.mc2_moe_unpermute_backward(DOUT, y, idx, IDX, probs, **kw)


@pytest.mark.parametrize("m,n", [(200, 304), (1100, 64), (130, 20000), (777, 1001), (3, 65536)])
def test_ns_workspace_grows_with_the_batch_alone(m, n):
    """The size is a matter of the sizes, not of how many tiles fill a device."""
    f = mc2.mc2_ns_workspace_size
    one = f(1, m, n)
    for batch in (2, 17, 300, 2000):
        assert f(batch, m, n) == batch * one
    # two iterates, the low half (in whole tiles of at most twice the smaller
    # side), two (r, r) matrices and the partial norms
    rp, cp = (-(-v // 64) * 64 for v in (min(m, n), max(m, n)))
    w = 64 if rp <= 64 else 128 if rp <= 128 else 256
    lo = -(-rp // w) * w * (-(-cp // w) * w)
    assert one <= (2 * rp * cp + lo + 2 * rp * rp) * 2 + 2048
    assert lo <= 2 * rp * cp or cp < w


@pytest.mark.parametrize("m,n", [(1, 2), (64, 256), (1024, 64), (128, 512)])
def test_ns_workspace_of_matrices_in_one_workgroup(m, n):
    """They use none: it does not grow with the batch."""
    f = mc2.mc2_ns_workspace_size
    assert 0 < f(1, m, n) == f(65535, m, n) < 1 << 20
