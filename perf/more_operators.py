"""What is measured of the 4-bit operators and of the MoE layer for few tokens.

Each operator in its plain form (``own`` false: elementary torch operations in
32 bits) and as the library's entry points compute it (``own`` true):

* ``quantize``: blocks of 32 values to 4-bit floating point with a shared power
  of two (``mc2_mx4_quantize``), and the values it stands for, as
  quantisation-aware training reads them (``mc2_mx4_dequantize``);
* ``dequantize``: 4-bit weights back to 16 bits (``mc2_mx4_dequantize``);
* ``mm``: the product of two operands held in 4 bits, in the chunk schedule of
  the AllGatherMatmul (``mc2_mx4_ag_mm_local``);
* ``moe``: a whole mixture-of-experts layer for few tokens, its weights in bf16
  or in 4 bits (``mc2_moe_tokens``).

4-bit operands are held as ``codes`` (rows, 16 * blocks) uint8, two values a
byte (the even one in the low half), and ``scales`` (rows, blocks rounded up to
16) uint8, the exponent of a block's power of two plus 127; blocks run along k,
the last one of a row filled up with zeros, as are the scales behind the last
block.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# The most that one drawn case may cost: the largest listed cases.
MOST_ELEMENTS = 16384 * 8192
MOST_PRODUCTS = 16384 * 8192 * 3584
MOST_WEIGHTS = 128 * 3 * 2048 * 768


def listed():
    return [
        # the gathered activations of the benchmark's large AllGatherMatmul
        {"name": "quantize_16384x8192_bf16", "op": "quantize", "B": 1, "rows": 16384, "k": 8192,
         "trans": False, "dtype": "bf16"},
        # fc1 weights of the benchmark's 16 local experts, held (H, 2I): blocks run along H
        {"name": "quantize_t_b16_2048x1536_bf16", "op": "quantize", "B": 16, "rows": 1536,
         "k": 2048, "trans": True, "dtype": "bf16"},
        # odd sizes: a gradient in fp32 whose rows are not whole blocks
        {"name": "quantize_777x1001_f32", "op": "quantize", "B": 1, "rows": 777, "k": 1001,
         "trans": False, "dtype": "f32"},
        # the experts' 4-bit weights laid out for the 16-bit grouped path
        {"name": "dequantize_t_b16_2048x1536_bf16", "op": "dequantize", "B": 16, "rows": 1536,
         "k": 2048, "trans": True, "dtype": "bf16"},
        # a small ragged weight: latency counts
        {"name": "dequantize_264x1000_f16", "op": "dequantize", "B": 1, "rows": 264, "k": 1000,
         "trans": False, "dtype": "f16"},
        # the benchmark's large AllGatherMatmul share
        {"name": "mm_16384x8192x3584", "op": "mm", "m": 16384, "k": 8192, "n": 3584, "W": 8,
         "dtype": "bf16", "bias": False},
        # ragged rows and k, fp16 out, with a bias
        {"name": "mm_1000x2056x1416_f16", "op": "mm", "m": 1000, "k": 2056, "n": 1416, "W": 4,
         "dtype": "f16", "bias": True},
        # a batch of decoded tokens through one projection of the large share
        {"name": "mm_64x8192x3584", "op": "mm", "m": 64, "k": 8192, "n": 3584, "W": 1,
         "dtype": "bf16", "bias": False},
        # a single token
        {"name": "mm_1x8192x3584", "op": "mm", "m": 1, "k": 8192, "n": 3584, "W": 1,
         "dtype": "bf16", "bias": False},
        # decoding one sequence through the benchmark's MoE layer, all experts on one GPU
        {"name": "moe_t1_h2048_bf16", "op": "moe", "T": 1, "H": 2048, "I": 768, "E": 128, "E_l": 128,
         "K": 8, "weights": "bf16"},
        # a batch of sequences, weights in 4 bits
        {"name": "moe_t64_h2048_mx4", "op": "moe", "T": 64, "H": 2048, "I": 768, "E": 128,
         "E_l": 128, "K": 8, "weights": "mx4"},
        # a ragged small layer of which this rank holds a quarter of the experts
        {"name": "moe_t37_h1416_bf16_ep4", "op": "moe", "T": 37, "H": 1416, "I": 200, "E": 32,
         "E_l": 8, "K": 6, "weights": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "mm", "mm", "moe", "moe"])
    if op in ("quantize", "dequantize"):
        rows, k = _log_uniform(rng, 1, 16384), _log_uniform(rng, 1, 8192)
        most = max(1, min(16, MOST_ELEMENTS // (rows * k)))
        return {"op": op, "B": rng.randint(1, most), "rows": rows, "k": k,
                "trans": rng.choice([False, True]), "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "mm":
        W = rng.choice([1, 1, 2, 4, 8])
        k, n = _log_uniform(rng, 32, 8192), 8 * _log_uniform(rng, 2, 1024)
        m = min(_log_uniform(rng, 1, 16384), MOST_PRODUCTS // (k * n))
        return {"op": op, "m": max(1, m // W) * W, "k": k, "n": n, "W": W,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "bias": rng.random() < 0.3}
    H, I = 8 * _log_uniform(rng, 16, 512), 8 * _log_uniform(rng, 4, 256)
    E = rng.choice([8, 16, 32, 60, 128])
    while E * 3 * H * I > MOST_WEIGHTS:
        E //= 2
    E = max(E, 1)
    return {"op": op, "T": _log_uniform(rng, 1, 256), "H": H, "I": I, "E": E,
            "E_l": rng.choice([d for d in (E, E, E // 2, E // 4) if d and E % d == 0]),
            "K": rng.randint(1, min(8, E)), "weights": rng.choice(["bf16", "bf16", "mx4"])}


def _pow2(byte):
    """2 ** (byte - 127) in fp32, NaN for 255; byte int32."""
    p = (byte << 23).view(torch.float32)
    p = torch.where(byte == 0, torch.full_like(p, 2.0 ** -127), p)
    return torch.where(byte == 255, torch.full_like(p, math.nan), p)


def _encode(x):
    """codes and scales of x (..., k) in blocks along k, 32-bit operations."""
    k = x.shape[-1]
    nb = -(-k // 32)
    x = torch.nn.functional.pad(x.float(), (0, 32 * nb - k)).unflatten(-1, (nb, 32))
    top = x.abs().amax(-1)
    expo = (top.view(torch.int32) >> 23) & 255  # floor(log2) + 127
    byte = (expo - 2).clamp(min=0)
    byte = torch.where(expo == 255, torch.full_like(byte, 255), byte)
    v = x * ((254 - byte.clamp(max=253)) << 23).view(torch.float32)[..., None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    # the grid's index: halves up to 2, ones up to 4, then 6
    code = torch.where(q <= 2, 2 * q, torch.where(q <= 4, q + 2, q + 1)).to(torch.uint8)
    code = torch.where(torch.signbit(v), code + 8, code)
    code = torch.where((byte == 255)[..., None], torch.zeros_like(code), code)
    code = code.flatten(-2)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.nn.functional.pad(byte.to(torch.uint8), (0, -nb % 16))
    return codes.contiguous(), scales.contiguous()


def _decode(codes, scales, k):
    """The fp32 values (..., k) that codes and scales stand for."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    nb = codes.shape[-1] // 16
    v = v.unflatten(-1, (nb, 32)) * _pow2(scales[..., :nb].int())[..., None]
    return v.flatten(-2)[..., :k]


def _values(g, shape):
    """Activations as a layer meets them: normal, some channels much larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.8 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op == "quantize":
        shape = (case["k"], case["rows"]) if case["trans"] else (case["rows"], case["k"])
        s["x"] = _values(g, (case["B"], *shape)).to(DTYPES[case["dtype"]])
    elif op == "dequantize":
        parts = [_encode(0.02 * torch.randn((case["rows"], case["k"]), generator=g, device="cuda"))
                 for _ in range(case["B"])]
        s["codes"], s["scales"] = (torch.stack(p) for p in zip(*parts))
    elif op == "mm":
        m, k, n = case["m"], case["k"], case["n"]
        s["x1"] = _encode(_values(g, (m, k)))
        s["x2"] = _encode(0.02 * torch.randn((n, k), generator=g, device="cuda"))
        s["bias"] = (torch.randn(n, generator=g, device="cuda").bfloat16() if case["bias"] else None)
    else:
        T, H, I, E, E_l, K = (case[n] for n in ("T", "H", "I", "E", "E_l", "K"))
        logits = torch.randn((T, E), generator=g, device="cuda")
        logits += 0.5 * torch.randn((1, E), generator=g, device="cuda")
        probs, sel = torch.softmax(logits, 1).topk(K, 1)
        s["probs"], s["sel"] = probs.contiguous(), sel.to(torch.int32).contiguous()
        s["rank"] = int(seed) % (E // E_l)
        s["x"] = torch.randn((T, H), generator=g, device="cuda").bfloat16()
        for name, shape in (("w1", (H, 2 * I)), ("w2", (I, H))):
            if case["weights"] == "bf16":
                w = torch.empty((E_l, *shape), dtype=torch.bfloat16, device="cuda")
                for e in range(E_l):
                    w[e] = 0.02 * torch.randn(shape, generator=g, device="cuda")
                s[name] = w
            else:  # blocks along the input of each product
                parts = [_encode(0.02 * torch.randn(shape[::-1], generator=g, device="cuda"))
                         for _ in range(E_l)]
                s[name] = tuple(torch.stack(p) for p in zip(*parts))
    return s


def _run_own(s):
    from gemm_collective_core_amd import mc2
    op = s["op"]
    if op == "quantize":
        codes, scales = mc2.mc2_mx4_quantize(s["x"], trans=s["trans"])
        return mc2.mc2_mx4_dequantize(codes, scales, s["k"], out_dtype=s["x"].dtype)
    if op == "dequantize":
        return mc2.mc2_mx4_dequantize(s["codes"], s["scales"], s["k"], trans=s["trans"],
                                      out_dtype=DTYPES[s["dtype"]])
    if op == "mm":
        return mc2.mc2_mx4_ag_mm_local(*s["x1"], *s["x2"], s["k"], s["W"], 0, bias=s["bias"],
                                       out_dtype=DTYPES[s["dtype"]])
    kw = dict(ep_rank=s["rank"], num_experts=s["E"])
    if s["weights"] == "bf16":
        return mc2.mc2_moe_tokens(s["x"], s["sel"], s["probs"], s["w1"], s["w2"], **kw)
    return mc2.mc2_moe_tokens(s["x"], s["sel"], s["probs"], s["w1"][0], s["w2"][0],
                              w1_scale=s["w1"][1], w2_scale=s["w2"][1], **kw)


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantize":
        x = s["x"].transpose(1, 2).contiguous() if s["trans"] else s["x"]
        return _decode(*_encode(x), s["k"]).to(x.dtype)
    if op == "dequantize":
        v = _decode(s["codes"], s["scales"], s["k"])
        return (v.transpose(1, 2) if s["trans"] else v).to(DTYPES[s["dtype"]]).contiguous()
    if op == "mm":
        out = _decode(*s["x1"], s["k"]) @ _decode(*s["x2"], s["k"]).t().contiguous()
        if s["bias"] is not None:
            out = out + s["bias"].float()
        return out.to(DTYPES[s["dtype"]])
    I, E_l = s["I"], s["E_l"]
    local = s["sel"].long() - s["rank"] * E_l
    mine = (local >= 0) & (local < E_l)
    local = local.clamp(0, E_l - 1)
    x = s["x"].float()
    out = torch.zeros_like(x)
    for k in range(s["K"]):
        if s["weights"] == "bf16":
            w1, w2 = s["w1"][local[:, k]].float(), s["w2"][local[:, k]].float()
        else:
            w1, w2 = (_decode(w[0][local[:, k]], w[1][local[:, k]], n).transpose(1, 2).contiguous()
                      for w, n in ((s["w1"], s["H"]), (s["w2"], I)))
        a = torch.bmm(x[:, None], w1)[:, 0]
        h = a[:, :I] / (1 + torch.exp(-a[:, :I])) * a[:, I:]
        y = torch.bmm(h[:, None], w2)[:, 0]
        out += torch.where(mine[:, k, None], s["probs"][:, k, None] * y, torch.zeros_like(y))
    return out.to(torch.bfloat16)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}.get(case.get("dtype"))
    if op in ("quantize", "dequantize"):
        n = case["B"] * case["rows"] * case["k"]
        # quantize: the input, the 4-bit form written and read, the values
        return ({"bytes": n * (2 * size + 2 * 17 / 32), "flops": 3 * n} if op == "quantize" else
                {"bytes": n * (size + 17 / 32), "flops": n})
    if op == "mm":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": (m + n) * k * 17 / 32 + m * n * size, "flops": 2 * m * n * k}
    T, H, I, E, E_l, K = (case[n] for n in ("T", "H", "I", "E", "E_l", "K"))
    # the experts that T tokens name on average, and the slots that are local
    named, slots = E_l * (1 - (1 - K / E) ** T), T * K * E_l / E
    weight = 3 * H * I * (2 if case["weights"] == "bf16" else 17 / 32)
    return {"bytes": named * weight + T * H * 4 + T * K * 8, "flops": slots * 6 * H * I}


def _exact_values(codes, scales, k):
    """(..., k) in 64 bits from the fields of each 4-bit number: sign, two bits
    of exponent, one of fraction."""
    def value(c):
        c = c.to(torch.int64)
        e, f = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2((e - 1).double()))
        return torch.where(c >= 8, -mag, mag)
    out = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64,
                      device=codes.device)
    out[..., 0::2], out[..., 1::2] = value(codes & 15), value(codes >> 4)
    per_value = scales.double().repeat_interleave(32, -1)[..., :out.shape[-1]]
    return (out * torch.exp2(per_value - 127))[..., :k]


def exact(case, seed):
    """The same from the definitions, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
        # a tie goes to the neighbour whose place in the grid is even
        mids = (grid[1:] + grid[:-1]) / 2
        out = []
        for x in s["x"]:
            x = (x.t() if case["trans"] else x).double()
            pieces = []
            for rows in x.split(2048):
                blocks = torch.nn.functional.pad(rows, (0, -case["k"] % 32)).view(len(rows), -1, 32)
                top = blocks.abs().amax(2, keepdim=True)
                e = (torch.frexp(top)[1] - 3).clamp(-127, 127).double()
                v = blocks / torch.exp2(e)
                lo, hi = (torch.bucketize(v.abs(), mids, right=r) for r in (False, True))
                at = torch.where((lo != hi) & (lo % 2 == 0), lo, hi)
                got = torch.copysign(grid[at], v) * torch.exp2(e)
                pieces.append(torch.where(top > 0, got, blocks).flatten(1)[:, :case["k"]])
            out.append(torch.cat(pieces))
        return torch.stack(out)
    if op == "dequantize":
        v = torch.stack([_exact_values(c, e, case["k"])
                         for c, e in zip(s["codes"], s["scales"])])
        return v.transpose(1, 2).contiguous() if case["trans"] else v
    if op == "mm":
        a, b = (_exact_values(*s[n], case["k"]) for n in ("x1", "x2"))
        out = torch.mm(a, b.t().contiguous())
        return out if s["bias"] is None else out + s["bias"].double()
    I, E_l, first = case["I"], case["E_l"], s["rank"] * case["E_l"]
    x, out = s["x"].double(), torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in range(E_l):
        t, slot = torch.nonzero(s["sel"] == first + e, as_tuple=True)
        if not len(t):
            continue
        if case["weights"] == "bf16":
            w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        else:
            w1 = _exact_values(s["w1"][0][e], s["w1"][1][e], case["H"]).t().contiguous()
            w2 = _exact_values(s["w2"][0][e], s["w2"][1][e], I).t().contiguous()
        a = x[t] @ w1
        h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
        out.index_add_(0, t, s["probs"][t, slot].double()[:, None] * (h @ w2))
    return out
