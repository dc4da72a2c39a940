"""The entry points of include/mc2_serve.h without a GPU: exported, reachable
through mc2.h, and rejecting invalid arguments on the host before any launch
(these calls fail validation, so no device work is ever enqueued); and the
binding's own checks of tensors."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from conftest import ROOT
from gemm_collective_core_amd import _lib, mc2

HEADER = os.path.join(ROOT, "include", "mc2_serve.h")
FAKE = 0x1000  # a non-NULL, 16-byte aligned address that is never dereferenced
MC2_OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_UNSUP, ERR_HIP, ERR_WS, ERR_ALIGN = range(8)
F16, BF16, I8, F32, I32, MX4 = range(6)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmc2.so is not built: run `python -m gemm_collective_core_amd.build`")
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(HEADER, encoding="utf-8").read()
    names = re.findall(r"^(?:int|size_t)\s+(mc2_\w+)\(", text, re.M)
    assert sorted(names) == sorted(_lib.SERVE_SIGNATURES) and len(names) == 8
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("first", ["mc2.h", "mc2_serve.h"])
def test_headers_are_plain_c(tmp_path, first):
    """Either header alone declares everything, in C99."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text(f'#include "{first}"\n'
                   "int main(void) { return mc2_mx4_row_bytes(33) == 32 ? MC2_OK : 1; }\n")
    exe = tmp_path / "use"
    libdir = os.path.dirname(_lib.LIB_PATH)
    res = subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                          os.path.dirname(HEADER), "-I", "/opt/rocm/include", str(src), "-o",
                          str(exe), "-L", libdir, "-lmc2", "-Wl,-rpath," + libdir],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


@pytest.mark.parametrize("k,row,scale", [(1, 16, 16), (32, 16, 16), (33, 32, 16), (512, 256, 16),
                                         (513, 272, 32), (8192, 4096, 256), (1 << 20, 1 << 19, 1 << 15),
                                         (0, 0, 0), (-5, 0, 0), ((1 << 20) + 1, 0, 0)])
def test_row_sizes(lib, k, row, scale):
    assert lib.mc2_mx4_row_bytes(k) == row and lib.mc2_mx4_scale_bytes(k) == scale
    if k > 0 and row:
        assert mc2._mx4_row(k) == row and mc2._mx4_pitch(k) == scale


def quant(lib, name, **o):
    a = dict(x=FAKE, batch=2, rows=10, k=100, trans=0, dt=BF16, codes=FAKE, scales=FAKE)
    a.update(o)
    if name == "quantize":
        return lib.mc2_mx4_quantize(a["x"], a["batch"], a["rows"], a["k"], a["trans"], a["dt"],
                                    a["codes"], a["scales"], None)
    return lib.mc2_mx4_dequantize(a["codes"], a["scales"], a["batch"], a["rows"], a["k"],
                                  a["trans"], a["dt"], a["x"], None)


@pytest.mark.parametrize("name", ["quantize", "dequantize"])
@pytest.mark.parametrize("over,code", [
    (dict(x=None), ERR_NULL), (dict(codes=None), ERR_NULL), (dict(scales=None), ERR_NULL),
    (dict(dt=I8), ERR_DTYPE), (dict(dt=I32), ERR_DTYPE), (dict(dt=MX4), ERR_DTYPE),
    (dict(batch=0), ERR_SHAPE), (dict(rows=0), ERR_SHAPE), (dict(k=0), ERR_SHAPE),
    (dict(rows=-1), ERR_SHAPE), (dict(k=(1 << 20) + 1), ERR_SHAPE),
    (dict(batch=1 << 20, rows=1 << 20), ERR_SHAPE), (dict(batch=1 << 62, rows=4), ERR_SHAPE),
    (dict(x=FAKE + 8), ERR_ALIGN), (dict(codes=FAKE + 4), ERR_ALIGN),
    (dict(scales=FAKE + 1), ERR_ALIGN),
])
def test_quantize_rejects(lib, name, over, code):
    assert quant(lib, name, **over) == code


def mm(lib, name, **o):
    a = dict(x1=FAKE, s1=FAKE, x2=FAKE, s2=FAKE, m=64, k=100, n=64, W=2, rank=0, bias=None,
             odt=BF16, out=FAKE, flags=None, cnt=None, epoch=0, turn=0)
    a.update(o)
    return getattr(lib, name)(a["x1"], a["s1"], a["x2"], a["s2"], a["m"], a["k"], a["n"], a["W"],
                              a["rank"], a["bias"], a["odt"], a["out"], a["flags"], a["cnt"],
                              a["epoch"], a["turn"], None)


@pytest.mark.parametrize("name", ["mc2_mx4_mm_rs_local", "mc2_mx4_ag_mm_local"])
@pytest.mark.parametrize("over,code", [
    (dict(x1=None), ERR_NULL), (dict(s1=None), ERR_NULL), (dict(x2=None), ERR_NULL),
    (dict(s2=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(m=0), ERR_SHAPE), (dict(m=-4), ERR_SHAPE), (dict(k=0), ERR_SHAPE), (dict(n=0), ERR_SHAPE),
    (dict(m=1 << 62), ERR_SHAPE), (dict(n=(1 << 20) + 8), ERR_SHAPE), (dict(k=1 << 21), ERR_SHAPE),
    (dict(W=3), ERR_SHAPE), (dict(W=0), ERR_SHAPE), (dict(W=64), ERR_SHAPE),
    (dict(rank=2), ERR_SHAPE), (dict(rank=-1), ERR_SHAPE),
    (dict(odt=I8), ERR_DTYPE), (dict(odt=I32), ERR_DTYPE), (dict(odt=MX4), ERR_DTYPE),
    (dict(n=68), ERR_ALIGN), (dict(x1=FAKE + 8), ERR_ALIGN), (dict(s1=FAKE + 4), ERR_ALIGN),
    (dict(x2=FAKE + 2), ERR_ALIGN), (dict(s2=FAKE + 1), ERR_ALIGN), (dict(out=FAKE + 8), ERR_ALIGN),
    (dict(flags=FAKE), ERR_NULL), (dict(cnt=FAKE), ERR_NULL),
    (dict(flags=FAKE, cnt=FAKE, epoch=0), ERR_SHAPE), (dict(turn=-1), ERR_SHAPE),
    (dict(turn=65), ERR_SHAPE),
])
def test_mm_rejects(lib, name, over, code):
    assert mm(lib, name, **over) == code


def test_mm_rs_needs_whole_chunks(lib):
    assert mm(lib, "mc2_mx4_mm_rs_local", m=65) == ERR_SHAPE


def tokens(lib, **o):
    a = dict(x=FAKE, sel=FAKE, probs=FAKE, T=4, K=8, H=64, E=16, rank=0, El=16, dt=BF16, w1=FAKE,
             s1=None, w2=FAKE, s2=None, I=32, out=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(o)
    return lib.mc2_moe_tokens(a["x"], a["sel"], a["probs"], a["T"], a["K"], a["H"], a["E"],
                              a["rank"], a["El"], a["dt"], a["w1"], a["s1"], a["w2"], a["s2"],
                              a["I"], a["out"], a["ws"], a["bytes"], None, None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), ERR_NULL), (dict(sel=None), ERR_NULL), (dict(probs=None), ERR_NULL),
    (dict(w1=None), ERR_NULL), (dict(w2=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(ws=None), ERR_NULL),
    (dict(dt=F16), ERR_DTYPE), (dict(dt=F32), ERR_DTYPE), (dict(dt=I8), ERR_DTYPE),
    (dict(dt=MX4), ERR_NULL),                       # 4-bit weights need their scales
    (dict(dt=MX4, s1=FAKE), ERR_NULL), (dict(s1=FAKE, s2=FAKE), ERR_DTYPE), (dict(s2=FAKE), ERR_DTYPE),
    (dict(T=0), ERR_SHAPE), (dict(T=257), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=65), ERR_SHAPE),
    (dict(T=256, K=17), ERR_SHAPE), (dict(H=0), ERR_SHAPE), (dict(H=65544), ERR_SHAPE),
    (dict(I=0), ERR_SHAPE), (dict(I=65544), ERR_SHAPE), (dict(T=256, K=16, H=65536), ERR_SHAPE),
    (dict(E=0), ERR_SHAPE), (dict(El=0), ERR_SHAPE), (dict(El=17), ERR_SHAPE),
    (dict(rank=1), ERR_SHAPE), (dict(rank=-1), ERR_SHAPE), (dict(E=2000, El=1025), ERR_SHAPE),
    (dict(rank=2 ** 31 - 1, El=1024), ERR_SHAPE),
    (dict(H=68), ERR_ALIGN), (dict(I=36), ERR_ALIGN), (dict(x=FAKE + 8), ERR_ALIGN),
    (dict(w1=FAKE + 2), ERR_ALIGN), (dict(w2=FAKE + 8), ERR_ALIGN), (dict(out=FAKE + 4), ERR_ALIGN),
    (dict(ws=FAKE + 8), ERR_ALIGN), (dict(dt=MX4, s1=FAKE + 1, s2=FAKE), ERR_ALIGN),
    (dict(bytes=64), ERR_WS),
])
def test_tokens_rejects(lib, over, code):
    assert tokens(lib, **over) == code


def test_tokens_workspace(lib):
    f = lib.mc2_moe_tokens_workspace_size
    need = f(4, 8, 64, 32)
    assert tokens(lib, bytes=need - 1) == ERR_WS
    # h as two bf16 and y in fp32 for every slot, and little else
    assert 32 * (32 * 4 + 64 * 4) <= need <= 32 * (32 * 4 + 64 * 4) + 8192
    assert f(0, 8, 64, 32) == f(4, 65, 64, 32) == f(257, 1, 64, 32) == f(4, 8, 0, 32) == 0
    assert f(256, 16, 65536, 8) == 0


def z(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


BF = torch.bfloat16


@pytest.mark.parametrize("call,match", [
    (lambda: mc2.mc2_mx4_quantize(z(4, 4, dtype=torch.int8)), "x must be one of"),
    (lambda: mc2.mc2_mx4_quantize(z(4, dtype=BF)), "a matrix or a stack"),
    (lambda: mc2.mc2_mx4_quantize(z(4, 40, dtype=BF), codes=z(4, 16)), "codes must have shape"),
    (lambda: mc2.mc2_mx4_quantize(z(4, 40, dtype=BF), scales=z(4, 2)), "codes_scale must have shape"),
    (lambda: mc2.mc2_mx4_quantize(z(4, 40, dtype=BF)), "on the GPU"),
    (lambda: mc2.mc2_mx4_quantize(z(40, 4, dtype=BF), trans=True, codes=z(4, 32), scales=z(4, 16)),
     "on the GPU"),
    (lambda: mc2.mc2_mx4_dequantize(z(4, 32), None, 40), "needs codes and scales"),
    (lambda: mc2.mc2_mx4_dequantize(z(4, 32), z(4, 16), 80), "codes must have shape"),
    (lambda: mc2.mc2_mx4_dequantize(z(4, 32), z(4, 16), 40, out_dtype=torch.int8), "out_dtype must be"),
    (lambda: mc2.mc2_mx4_dequantize(z(4, 32), z(4, 16), 40, out=z(40, 4, dtype=BF)), "out must have shape"),
    (lambda: mc2.mc2_mx4_dequantize(z(4, 32), z(4, 16), 40, trans=True, out=z(40, 4, dtype=BF)), "on the GPU"),
    (lambda: mc2.mc2_mx4_ag_mm_local(z(4, 32), z(4, 16), z(8, 32), z(8, 16), 40, 3, 0), "world_size"),
    (lambda: mc2.mc2_mx4_ag_mm_local(z(4, 32), z(4, 16), z(8, 16), z(8, 16), 40, 1, 0), "x2 must have"),
    (lambda: mc2.mc2_mx4_mm_rs_local(z(4, 32), z(4, 16), z(8, 32), z(8, 16), 40, 1, 0,
                                     bias=z(8, dtype=torch.float32)), "bias must be"),
    (lambda: mc2.mc2_mx4_mm_rs_local(z(4, 32), z(4, 16), z(8, 32), z(8, 16), 40, 1, 0,
                                     out=z(4, 9, dtype=BF)), "out must have shape"),
    (lambda: mc2.mc2_mx4_mm_rs_local(z(4, 32), z(4, 16), z(8, 32), z(8, 16), 40, 1, 0), "on the GPU"),
])
def test_mx4_binding(call, match):
    with pytest.raises(ValueError, match=match):
        call()


def moe_args(**o):
    a = dict(x=z(3, 64, dtype=BF), sel=z(3, 2, dtype=torch.int32), probs=z(3, 2, dtype=torch.float32),
             w1=z(4, 64, 48, dtype=BF), w2=z(4, 24, 64, dtype=BF), ep_rank=0, num_experts=4)
    a.update(o)
    return a


@pytest.mark.parametrize("over,match", [
    (dict(), "on the GPU"),
    (dict(sel=z(3, 2, dtype=torch.int64)), "sel must be"), (dict(probs=z(3, 2)), "probs must be"),
    (dict(probs=z(3, 3, dtype=torch.float32)), "probs must have shape"),
    (dict(x=z(3, 64, dtype=torch.float16)), "x must be"), (dict(w1=z(4, 64, 32, dtype=BF)), "w1 must have"),
    (dict(w2=z(5, 24, 64, dtype=BF)), "w2 must have"), (dict(out=z(3, 32, dtype=BF)), "out must have"),
    (dict(w1_scale=z(4, 48, 16)), "go together"),
    (dict(w1=z(4, 48, 32), w1_scale=z(4, 48, 16), w2=z(4, 64, 16), w2_scale=z(4, 64, 16)), "on the GPU"),
    (dict(w1=z(4, 48, 32), w1_scale=z(4, 48, 16), w2=z(4, 64, 32), w2_scale=z(4, 64, 16)), "w2 must have"),
    (dict(workspace=z(64, dtype=torch.int32)), "workspace must be"),
])
def test_moe_binding(over, match):
    with pytest.raises(ValueError, match=match):
        mc2.mc2_moe_tokens(**moe_args(**over))
