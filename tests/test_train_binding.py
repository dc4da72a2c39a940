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
