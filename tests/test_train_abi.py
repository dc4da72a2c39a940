"""The entry points of include/mc2_train.h without a GPU: exported, reachable
through mc2.h, and rejecting invalid arguments on the host before any launch
(these calls fail validation, so no device work is ever enqueued); and the
binding's own checks of tensors."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

from conftest import ROOT
from gemm_collective_core_amd import _lib, mc2

HEADER = os.path.join(ROOT, "include", "mc2_train.h")
FAKE = 0x1000  # a non-NULL, 16-byte aligned address that is never dereferenced
MC2_OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_UNSUP, ERR_HIP, ERR_WS, ERR_ALIGN = range(8)
F16, BF16, I8, F32, I32 = range(5)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmc2.so is not built: run `python -m gemm_collective_core_amd.build`")
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(HEADER, encoding="utf-8").read()
    names = re.findall(r"^(?:int|size_t)\s+(mc2_\w+)\(", text, re.M)
    assert sorted(names) == sorted(_lib.TRAIN_SIGNATURES) and len(names) == 4
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("first", ["mc2.h", "mc2_train.h"])
def test_headers_are_plain_c(tmp_path, first):
    """Either header alone declares everything, in C99."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text(f'#include "{first}"\n'
                   "int main(void) { return mc2_ns_workspace_size(1, 64, 64) ? MC2_OK : 1; }\n")
    exe = tmp_path / "use"
    libdir = os.path.dirname(_lib.LIB_PATH)
    res = subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                          os.path.dirname(HEADER), "-I", "/opt/rocm/include", str(src), "-o",
                          str(exe), "-L", libdir, "-lmc2", "-Wl,-rpath," + libdir],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def unperm(lib, **o):
    a = dict(dout=FAKE, y=FAKE, rows=80, idx=FAKE, sidx=FAKE, probs=FAKE, T=10, K=8, H=64, dt=BF16,
             dy=FAKE, dp=FAKE)
    a.update(o)
    return lib.mc2_moe_unpermute_backward(a["dout"], a["y"], a["rows"], a["idx"], a["sidx"],
                                          a["probs"], a["T"], a["K"], a["H"], a["dt"], a["dy"],
                                          a["dp"], None, None)


@pytest.mark.parametrize("over,code", [
    (dict(dout=None), ERR_NULL), (dict(idx=None), ERR_NULL), (dict(sidx=None), ERR_NULL),
    (dict(dy=None, dp=None), ERR_NULL),       # nothing to compute
    (dict(probs=None), ERR_NULL),             # dy needs the weights
    (dict(y=None), ERR_NULL),                 # dprobs needs the rows
    (dict(dt=F32), ERR_DTYPE), (dict(dt=I8), ERR_DTYPE),
    (dict(T=0), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(K=0), ERR_SHAPE),
    (dict(K=65), ERR_SHAPE), (dict(H=0), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE),
    (dict(T=1 << 28, K=8), ERR_SHAPE), (dict(T=1 << 62, K=4), ERR_SHAPE),
    (dict(H=68), ERR_ALIGN), (dict(dout=FAKE + 8), ERR_ALIGN), (dict(y=FAKE + 2), ERR_ALIGN),
    (dict(dy=FAKE + 4), ERR_ALIGN),
])
def test_unpermute_backward_rejects(lib, over, code):
    assert unperm(lib, **over) == code


def test_permute_backward_rejects(lib):
    f = lib.mc2_moe_permute_backward
    assert f(None, 80, FAKE, 10, 8, 64, BF16, FAKE, None, None) == ERR_NULL
    assert f(FAKE, 80, None, 10, 8, 64, BF16, FAKE, None, None) == ERR_NULL
    assert f(FAKE, 80, FAKE, 10, 8, 64, BF16, None, None, None) == ERR_NULL
    assert f(FAKE, 80, FAKE, 10, 8, 64, F32, FAKE, None, None) == ERR_DTYPE
    assert f(FAKE, -1, FAKE, 10, 8, 64, BF16, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE, 80, FAKE, 0, 8, 64, BF16, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE, 80, FAKE, 10, 65, 64, BF16, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE, 80, FAKE, 1 << 62, 4, 64, BF16, FAKE, None, None) == ERR_SHAPE
    assert f(FAKE, 80, FAKE, 10, 8, 60, BF16, FAKE, None, None) == ERR_ALIGN
    assert f(FAKE, 80, FAKE, 10, 8, 64, F16, FAKE + 8, None, None) == ERR_ALIGN


def ns(lib, **o):
    a = dict(g=FAKE, B=2, m=100, n=70, idt=F32, steps=2, co=(3.4445, -4.775, 2.0315) * 2, eps=1e-7,
             scale=1.0, odt=BF16, out=FAKE, ws=FAKE, nb=1 << 40)
    a.update(o)
    co = None if a["co"] is None else (C.c_float * len(a["co"]))(*a["co"])
    return lib.mc2_ns_orthogonalize(a["g"], a["B"], a["m"], a["n"], a["idt"], a["steps"], co,
                                    a["eps"], a["scale"], a["odt"], a["out"], a["ws"], a["nb"], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,code", [
    (dict(g=None), ERR_NULL), (dict(co=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(ws=None), ERR_NULL),
    (dict(idt=I8), ERR_DTYPE), (dict(idt=9), ERR_DTYPE), (dict(odt=F32), ERR_DTYPE),
    (dict(odt=I8), ERR_DTYPE),
    (dict(B=0), ERR_SHAPE), (dict(B=65536), ERR_SHAPE), (dict(m=0), ERR_SHAPE),
    (dict(n=65537), ERR_SHAPE), (dict(steps=0), ERR_SHAPE), (dict(steps=33), ERR_SHAPE),
    (dict(eps=-1.0), ERR_SHAPE), (dict(eps=NAN), ERR_SHAPE), (dict(eps=INF), ERR_SHAPE),
    (dict(scale=NAN), ERR_SHAPE), (dict(scale=-INF), ERR_SHAPE),
    (dict(co=(3.4, -4.7, 2.0, 3.4, NAN, 2.0)), ERR_SHAPE),
    (dict(co=(3.4, -4.7, 2.0, 3.4, -17.0, 2.0)), ERR_SHAPE),
    (dict(g=FAKE + 8), ERR_ALIGN), (dict(out=FAKE + 2), ERR_ALIGN), (dict(ws=FAKE + 8), ERR_ALIGN),
    (dict(nb=1024), ERR_WS),
    (dict(B=65535, m=65536, n=65536), ERR_SHAPE),   # more tiles than a grid holds
])
def test_ns_rejects(lib, over, code):
    assert ns(lib, **over) == code


def test_ns_workspace_size(lib):
    f = lib.mc2_ns_workspace_size
    assert f(0, 64, 64) == f(1, 0, 64) == f(1, 64, 65537) == 0
    # two iterates, their low halves and two (r, r) matrices, padded to 64, in
    # fp16, and the partial norms
    need = 3 * 128 * 192 * 2 + 2 * 128 * 128 * 2
    assert need <= f(1, 100, 130) == f(1, 130, 100) <= need + (64 << 10)
    assert ns(lib, nb=f(2, 100, 70) - 1) == ERR_WS


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def test_binding_checks():
    f32, i32, f16 = torch.float32, torch.int32, torch.float16
    T, K, H = 10, 4, 64
    idx, probs = z(T * K, dtype=i32), z(T, K, dtype=f32)
    dout, y = z(T, H), z(T * K, H)
    U = mc2.mc2_moe_unpermute_backward
    _raises(lambda: U(dout, y, idx, idx, probs), "must be on the GPU")
    _raises(lambda: U(z(T, H, dtype=f32), y, idx, idx, probs), "dout must be one of")
    _raises(lambda: U(dout, z(T * K, H, dtype=f16), idx, idx, probs), "y_full must be")
    _raises(lambda: U(dout, z(T * K, H + 8), idx, idx, probs), "y_full must have shape")
    _raises(lambda: U(dout, y, idx[:-1], idx, probs), "unpermute_idx must hold")
    _raises(lambda: U(dout, y, idx, idx.long(), probs), "sorted_idx must be")
    _raises(lambda: U(dout, y, idx, idx, z(T, K)), "probs must be")
    _raises(lambda: U(dout, y, idx, idx, probs, dy=z(T, H)), "dy must have shape")
    _raises(lambda: U(dout, y, idx, idx, probs, dprobs=z(T, K)), "dprobs must be")
    _raises(lambda: U(dout, y, idx, idx, probs, need_dy=False, need_dprobs=False), "nothing")
    P = mc2.mc2_moe_permute_backward
    _raises(lambda: P(y, idx, K), "must be on the GPU")
    _raises(lambda: P(y, idx, 7), "T \\* topk")
    _raises(lambda: P(y, idx, 0), "T \\* topk")
    _raises(lambda: P(y.float(), idx, K), "dpermuted must be one of")
    _raises(lambda: P(y, idx, K, dx=z(T, H, dtype=f16)), "dx must be")
    N = mc2.mc2_ns_orthogonalize
    _raises(lambda: N(z(3, 8, 8)), "must be on the GPU")
    _raises(lambda: N(z(8)), "g must be")
    _raises(lambda: N(z(8, 8, dtype=torch.float64)), "g must be one of")
    _raises(lambda: N(z(8, 8), out_dtype=f32), "out_dtype")
    _raises(lambda: N(z(8, 8), out=z(8, 8, dtype=f32)), "out_dtype")
    _raises(lambda: N(z(8, 8), out=z(8, 9)), "out must have shape")
    _raises(lambda: N(z(8, 8), coeffs=((1, 2, 3), (4, 5, 6)), steps=3), "coeffs must be")
    _raises(lambda: N(z(8, 8), workspace=z(8, dtype=f32)), "workspace must be")
