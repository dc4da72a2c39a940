"""One training step of the MoE layer through the library: permute, fc1 with
SwiGLU, fc2, unpermute, then every gradient back to the tokens, the routing
weights and the expert weights, and the orthogonalised updates; against torch's
derivation in float64 on the CPU, and replayed from a captured graph."""
import pytest
import torch

import workloads as wl
from gemm_collective_core_amd import mc2
from gpu_util import assert_tol, to_dev, to_f64
from oracle import train as ot

pytestmark = pytest.mark.gpu

T, H, E, K, I = 256, 128, 8, 2, 72


def _inputs(seed):
    return wl.moe_inputs(seed=seed, tokens=T, hidden=H, num_experts=E, topk=K, local_experts=E,
                         inter=I, w_std=0.1)


class Step:
    """The step's buffers, allocated once, as a program that captures it keeps
    them."""

    def __init__(self, d, seed):
        dev = "cuda"
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.x, self.sel, self.probs = to_dev(d["x"], "bf16"), to_dev(d["sel"]), to_dev(d["probs"])
        self.w1, self.w2 = to_dev(d["w1"], "bf16"), to_dev(d["w2"], "bf16")
        self.dout = torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).to(
            torch.bfloat16).cuda()
        self.counts = torch.empty(E, dtype=torch.int32, device=dev)
        self.perm, self.y, self.dy = (torch.zeros((T * K, H), **bf) for _ in range(3))
        self.dperm = torch.zeros((T * K, H), **bf)
        self.sidx, self.uidx = (torch.empty(T * K, dtype=torch.int32, device=dev) for _ in range(2))
        self.offs = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.a, self.h = torch.empty((T * K, 2 * I), **bf), torch.empty((T * K, I), **bf)
        self.out, self.dx = (torch.empty((T, H), **bf) for _ in range(2))
        self.dprobs = torch.empty((T, K), device=dev)
        self.da = torch.empty((T * K, 2 * I), **bf)
        self.dw1, self.dw2 = (torch.empty(w.shape, device=dev) for w in (self.w1, self.w2))
        self.u1, self.u2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        u8 = dict(dtype=torch.uint8, device=dev)
        self.ws = [torch.empty(n, **u8) for n in (
            mc2.mc2_moe_permute_workspace_size(T, K, E),
            mc2.mc2_gmm_backward_workspace_size(T * K, E, I, H),
            mc2.mc2_gmm_backward_workspace_size(T * K, E, H, 2 * I),
            mc2.mc2_ns_workspace_size(E, H, 2 * I), mc2.mc2_ns_workspace_size(E, I, H))]

    def run(self):
        s, kw = self, dict(ep_rank=0, num_experts=E, dev_err=self.err)
        mc2.mc2_moe_histc(s.sel, E, counts=s.counts, dev_err=s.err)
        mc2.mc2_moe_permute(s.x, s.sel, E, permuted=s.perm, sorted_idx=s.sidx,
                            unpermute_idx=s.uidx, expert_offsets=s.offs, workspace=s.ws[0],
                            dev_err=s.err)
        c = s.counts
        mc2.mc2_gmm_dispatch(s.perm, c, c, s.w1, act=mc2.MC2_ACT_NONE, h_out=s.a, **kw)
        mc2.mc2_gmm_dispatch(s.perm, c, c, s.w1, h_out=s.h, **kw)
        mc2.mc2_gmm_combine(s.h, c, c, s.w2, s.y, **kw)
        mc2.mc2_moe_unpermute(s.y, s.uidx, s.probs, out=s.out, dev_err=s.err)
        mc2.mc2_moe_unpermute_backward(s.dout, s.y, s.uidx, s.sidx, s.probs, dy=s.dy,
                                       dprobs=s.dprobs, dev_err=s.err)
        mc2.mc2_gmm_combine_backward(s.dy, c, c, s.w2, s.h, act=mc2.MC2_ACT_SWIGLU, g_saved=s.a,
                                     dgrad_out=s.da, dw2_out=s.dw2, workspace=s.ws[1], **kw)
        mc2.mc2_gmm_dispatch_backward(s.da, c, c, s.w1, s.perm, s.dperm, dw1_out=s.dw1,
                                      workspace=s.ws[2], **kw)
        mc2.mc2_moe_permute_backward(s.dperm, s.uidx, K, dx=s.dx, dev_err=s.err)
        mc2.mc2_ns_orthogonalize(s.dw1, scale=0.2, out=s.u1, workspace=s.ws[3])
        mc2.mc2_ns_orthogonalize(s.dw2, scale=0.2, out=s.u2, workspace=s.ws[4])

    NAMES = ("out", "dx", "dprobs", "dw1", "dw2", "u1", "u2", "dy")

    def results(self):
        return {n: getattr(self, n).clone() for n in self.NAMES}


def test_step_against_float64():
    d = _inputs(61)
    s = Step(d, 1)
    s.run()
    torch.cuda.synchronize()
    assert s.err.item() == 0
    x, w1, w2, probs = (t.double().cpu().requires_grad_() for t in (s.x, s.w1, s.w2, s.probs))
    sel = torch.from_numpy(d["sel"]).long()
    a = torch.einsum("th,tkhi->tki", x, w1[sel])
    h = torch.nn.functional.silu(a[..., :I]) * a[..., I:]
    out = (torch.einsum("tki,tkih->tkh", h, w2[sel]) * probs[..., None]).sum(1)
    out.backward(s.dout.double().cpu())
    for name, ref in (("out", out.detach()), ("dx", x.grad), ("dprobs", probs.grad),
                      ("dw1", w1.grad), ("dw2", w2.grad)):
        # bf16 between the stages: the chain is held to the parity gate, with
        # its absolute term in units of the result
        scale = float(ref.square().mean().sqrt())
        assert_tol(to_f64(getattr(s, name)) / scale, ref.numpy() / scale, name, rtol=3e-2, atol=6e-2)
    for u, g in ((s.u1, s.dw1), (s.u2, s.dw2)):
        for e in range(E):
            ref = ot.newton_schulz(g[e].double().cpu().numpy(), (mc2.MC2_NS_COEFFS,) * 5, 1e-7, 0.2)
            rel = abs(to_f64(u[e]) - ref)
            assert (rel ** 2).sum() ** 0.5 <= 1.9e-2 * (ref ** 2).sum() ** 0.5


def test_step_captured_and_replayed():
    """Every replay gives the eager bits, with new inputs and eager work
    between the replays."""
    ds = [_inputs(s) for s in (62, 63)]
    s = Step(ds[0], 2)

    def load(d):
        for name, dt in (("x", "bf16"), ("sel", None), ("probs", None), ("w1", "bf16"),
                         ("w2", "bf16")):
            getattr(s, name).copy_(to_dev(d[name], dt))

    eager = []
    for d in ds:
        load(d)
        s.run()
        torch.cuda.synchronize()
        eager.append(s.results())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for i in (0, 1, 1, 0):
        load(ds[i])
        for n in s.NAMES:
            getattr(s, n).fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert s.err.item() == 0
        for n, v in s.results().items():
            bits = torch.int16 if v.element_size() == 2 else torch.int32
            assert torch.equal(v.view(bits), eager[i][n].view(bits)), (i, n)
