"""What is measured of the training operators around the grouped experts.

Three operators, each in its plain form (``own`` false: elementary torch
operations in 32 bits) and as the library's entry points compute it (``own``
true):

* ``unpermute_bwd``: the gradient of the weighted return of the routed rows to
  their tokens, with respect to the rows and to the routing weights
  (``mc2_moe_unpermute_backward``);
* ``permute_bwd``: the gradient of the grouping of the token rows by expert
  (``mc2_moe_permute_backward``);
* ``ns``: the orthogonalisation of a stack of weight gradients by Newton-Schulz
  products (``mc2_ns_orthogonalize``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7

# The most that one drawn case may cost: the elements of the routed rows, and
# the products of one matrix stack, of the largest listed cases.
MOST_ROUTED = 32768 * 8 * 2048
MOST_NS = 16 * 1536 * 1536 * (3 * 2048 + 1536)


def listed():
    return [
        # the MoE layer of the benchmark: 32768 tokens, top-8 of 128 experts, bf16
        {"name": "unpermute_bwd_t32768_h2048_k8", "op": "unpermute_bwd", "T": 32768, "H": 2048,
         "K": 8, "E": 128, "drop": 0.0, "dtype": "bf16"},
        # a ragged token count and width, some slots left out by the router's capacity, fp16
        {"name": "unpermute_bwd_t5001_h1416_k6", "op": "unpermute_bwd", "T": 5001, "H": 1416,
         "K": 6, "E": 32, "drop": 0.05, "dtype": "f16"},
        # a small micro-batch (the graph-replay test's layer): latency counts
        {"name": "unpermute_bwd_t900_h256_k4", "op": "unpermute_bwd", "T": 900, "H": 256,
         "K": 4, "E": 32, "drop": 0.0, "dtype": "bf16"},
        # the same layers' grouping of the tokens by expert
        {"name": "permute_bwd_t32768_h2048_k8", "op": "permute_bwd", "T": 32768, "H": 2048,
         "K": 8, "E": 128, "drop": 0.0, "dtype": "bf16"},
        {"name": "permute_bwd_t5001_h1416_k6", "op": "permute_bwd", "T": 5001, "H": 1416,
         "K": 6, "E": 32, "drop": 0.05, "dtype": "f16"},
        {"name": "permute_bwd_t900_h256_k4", "op": "permute_bwd", "T": 900, "H": 256,
         "K": 4, "E": 32, "drop": 0.0, "dtype": "bf16"},
        # fc1 weight gradients of the benchmark's 16 local experts (tall)
        {"name": "ns_b16_2048x1536_f32", "op": "ns", "B": 16, "m": 2048, "n": 1536, "dtype": "f32"},
        # its fc2 weight gradients (wide)
        {"name": "ns_b16_768x2048_f32", "op": "ns", "B": 16, "m": 768, "n": 2048, "dtype": "f32"},
        # one dense weight of a tensor-parallel layer, its momentum kept in bf16
        {"name": "ns_b1_2048x3584_bf16", "op": "ns", "B": 1, "m": 2048, "n": 3584, "dtype": "bf16"},
        # odd sizes: rows that are not whole 16-byte pieces
        {"name": "ns_b3_777x1001_f32", "op": "ns", "B": 3, "m": 777, "n": 1001, "dtype": "f32"},
        # the experts of a small layer (the backward tests' sizes)
        {"name": "ns_b8_264x272_f32", "op": "ns", "B": 8, "m": 264, "n": 272, "dtype": "f32"},
        # one small projection: latency counts
        {"name": "ns_b1_64x256_f32", "op": "ns", "B": 1, "m": 64, "n": 256, "dtype": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["unpermute_bwd", "permute_bwd", "ns", "ns"])
    if op == "ns":
        m, n = _log_uniform(rng, 24, 2400), _log_uniform(rng, 24, 3600)
        r, c = min(m, n), max(m, n)
        most = max(1, min(16, MOST_NS // (r * r * (3 * c + r))))
        return {"op": op, "B": rng.randint(1, most), "m": m, "n": n,
                "dtype": rng.choice(["f32", "f32", "bf16", "f16"])}
    K = rng.randint(1, 10)
    H = 8 * _log_uniform(rng, 8, 512)
    T = _log_uniform(rng, 1, 32768)
    T = max(1, min(T, MOST_ROUTED // (K * H)))
    return {"op": op, "T": T, "H": H, "K": K, "E": rng.choice([16, 32, 60, 128]),
            "drop": rng.choice([0.0, 0.0, 0.1]), "dtype": rng.choice(["bf16", "f16"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    if case["op"] == "ns":
        # Weight gradients as the grouped backward gives them: sums over an
        # expert's tokens of outer products. The experts' token counts are
        # skewed: some have fewer rows than the matrix has, which leaves its
        # other singular values zero, and the last of several has none at all.
        B, m, n = case["B"], case["m"], case["n"]
        r = min(m, n)
        out = torch.zeros((B, m, n), device=dev, dtype=torch.float32)
        share = torch.rand(B, generator=g, device=dev).tolist()
        for b in range(B):
            rows = max(1, int(r * (0.3 + 2.5 * share[b])))
            if B > 4 and b == B - 1:
                continue
            left = torch.randn((m, rows), generator=g, device=dev)
            right = torch.randn((rows, n), generator=g, device=dev)
            right *= torch.exp(0.7 * torch.randn((rows, 1), generator=g, device=dev))
            out[b] = left @ right * 1e-3
        return {"op": "ns", "g": out.to(dt), "scale": 0.2 * math.sqrt(max(m, n))}
    T, H, K, E = case["T"], case["H"], case["K"], case["E"]
    logits = torch.randn((T, E), generator=g, device=dev)
    logits += 0.5 * torch.randn((1, E), generator=g, device=dev)
    probs, sel = torch.softmax(logits, 1).topk(K, 1)
    if case["drop"]:
        sel = torch.where(torch.rand((T, K), generator=g, device=dev) < case["drop"],
                          torch.full_like(sel, E), sel)
    # slots in expert order, ties in slot order, the ones left out behind them
    order = torch.argsort(sel.reshape(-1), stable=True)
    valid = sel.reshape(-1) < E
    place = torch.empty_like(order)
    place[order] = torch.arange(T * K, device=dev)
    s = {"op": case["op"], "K": K,
         "unpermute_idx": torch.where(valid, place, -1).to(torch.int32),
         "sorted_idx": torch.where(valid[order], order, -1).to(torch.int32),
         "rows": torch.randn((T * K, H), generator=g, device=dev, dtype=torch.float32).to(dt)}
    if case["op"] == "unpermute_bwd":
        s["probs"] = probs.contiguous()
        s["dout"] = torch.randn((T, H), generator=g, device=dev).to(dt)
        # rows that no slot names are left as they were
        s["dy"] = torch.zeros((T * K, H), device=dev, dtype=dt)
    return s


def _plain_ns(s):
    x = s["g"].float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    wide = x.shape[1] <= x.shape[2]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    a, b, c = NS_COEFFS
    for _ in range(NS_STEPS):
        p = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * p + c * torch.bmm(p, p), x)
    if not wide:
        x = x.transpose(1, 2)
    return (s["scale"] * x).to(torch.bfloat16).contiguous()


def run(s):
    if own:
        from gemm_collective_core_amd import mc2
        if s["op"] == "ns":
            return mc2.mc2_ns_orthogonalize(s["g"], steps=NS_STEPS, coeffs=NS_COEFFS, eps=NS_EPS,
                                            scale=s["scale"])
        if s["op"] == "permute_bwd":
            return mc2.mc2_moe_permute_backward(s["rows"], s["unpermute_idx"], s["K"])
        return mc2.mc2_moe_unpermute_backward(s["dout"], s["rows"], s["unpermute_idx"],
                                              s["sorted_idx"], s["probs"], dy=s["dy"])
    if s["op"] == "ns":
        return _plain_ns(s)
    rows, K, idx = s["rows"], s["K"], s["unpermute_idx"]
    TK, H = rows.shape
    named = (idx >= 0).view(TK // K, K)
    mine = rows[idx.clamp(min=0)].float().view(TK // K, K, H) * named[:, :, None]
    if s["op"] == "permute_bwd":
        return mine.sum(1).to(rows.dtype)
    dout = s["dout"].float()
    dprobs = (dout[:, None, :] * mine).sum(2)
    slot = s["sorted_idx"]
    token = slot.clamp(min=0)
    dy = s["probs"].view(-1)[token][:, None] * dout[token // K]
    s["dy"].copy_(torch.where((slot >= 0)[:, None], dy, s["dy"].float()))
    return s["dy"], dprobs


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ns":
        B, m, n = case["B"], case["m"], case["n"]
        r, c = min(m, n), max(m, n)
        # each step: the Gram matrix and its square, both symmetric (half of
        # their products), and the product with the iterate
        return {"bytes": B * m * n * (size + 2),
                "flops": NS_STEPS * B * (r * (r + 1) * c + r * r * (r + 1) + 2 * r * r * c)}
    T, H, K = case["T"], case["H"], case["K"]
    kept = T * K * (1 - case["drop"])
    if case["op"] == "permute_bwd":
        return {"bytes": kept * H * 2 + T * K * 4 + T * H * 2, "flops": kept * H}
    return {"bytes": 2 * kept * H * 2 + T * H * 2 + T * K * 16, "flops": 3 * kept * H}


def exact(case, seed):
    """The same from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "ns":
        a, b, c = NS_COEFFS
        out = []
        for x in s["g"].double():
            x = x / (torch.linalg.vector_norm(x) + NS_EPS)
            if x.shape[0] > x.shape[1]:  # from the smaller side: the same polynomial
                for _ in range(NS_STEPS):
                    p = x.t().contiguous() @ x
                    x = x @ (c * (p @ p) + b * p) + a * x
            else:
                for _ in range(NS_STEPS):
                    p = x @ x.t().contiguous()
                    x = (c * (p @ p) + b * p) @ x + a * x
            out.append(x * s["scale"])
        return torch.stack(out)
    K, idx = s["K"], s["unpermute_idx"].long()
    TK, H = s["rows"].shape
    rows = torch.cat([s["rows"].double(), s["rows"].new_zeros((1, H), dtype=torch.float64)])
    if case["op"] == "permute_bwd":
        dx = torch.zeros((TK // K, H), dtype=torch.float64, device=rows.device)
        for k in range(K):  # row -1 is the row of zeros
            dx += rows[idx.view(-1, K)[:, k]]
        return dx
    dout = s["dout"].double()
    dprobs = torch.stack([(dout * rows[idx.view(-1, K)[:, k]]).sum(1) for k in range(K)], 1)
    dy = torch.zeros((TK + 1, H), dtype=torch.float64, device=rows.device)
    for k in range(K):  # the slots left out write to the row behind the last
        dy[idx.view(-1, K)[:, k]] = s["probs"].double()[:, k, None] * dout
    return dy[:TK], dprobs
