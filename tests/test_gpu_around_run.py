"""One step of a model around the routed layer, call after call on one stream:
norm with the residual's addition and 8-bit rows, an 8-bit projection with
request adapters beside it, the next norm, the routed layer itself with expert
selection from its logits, and the balance loss with its gradient.  Every stage
is held to what the framework's calls (or fp64 torch) give for its own inputs."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

BF16, F8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
H, E, K_TOP, I, L, R = 512, 16, 4, 256, 6, 16
EPS = 1e-6


class Step:
    def __init__(self, T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.T = T
        self.x, self.res = rn(T, H).to(BF16), rn(T, H).to(BF16)
        self.w1, self.w2 = (1 + 0.1 * rn(H)).to(BF16), (1 + 0.1 * rn(H)).to(BF16)
        proj = (rn(1, H, H) / math.sqrt(H)).to(BF16)
        self.wq, self.ws = torch.empty(1, H, H, dtype=F8, device="cuda"), torch.empty(1, H // 128, H // 128, device="cuda")
        rse.moe_fp8_quantize_weight(proj, self.wq, self.ws)
        self.a, self.b = (rn(L, R, H) / math.sqrt(H)).to(BF16), (rn(L, H, R) * 0.1).to(BF16)
        self.scale = torch.rand(L, generator=g, device="cuda")
        self.ids = torch.randint(-1, L, (T,), generator=g, device="cuda").to(I32)
        self.layer = rse.MoELayer(hidden=H, num_experts=E, top_k=K_TOP, expert_inter=I, shared_inter=0, swiglu_limit=7.0,
                                  routed_scaling_factor=1.0, renormalize=True, router_w=rn(E, H) / math.sqrt(H),
                                  correction_bias=None, w_gate_up=(rn(E, 2 * I, H) / math.sqrt(H)).to(BF16),
                                  w_down=(rn(E, H, I) / math.sqrt(I)).to(BF16), max_tokens=T)
        e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.sum1, self.n1, self.q1, self.s1 = e(T, H), e(T, H), e(T, H, dtype=F8), e(H // 128, T, dtype=torch.float32)
        self.proj, self.y, self.sum2, self.n2, self.out = e(T, H), e(T, H), e(T, H), e(T, H), e(T, H)
        self.plan = e(rse.moe_lora_plan_size(T, L), dtype=torch.uint8)
        self.wsp = e(rse.MOE_BALANCE_WS_BYTES, dtype=torch.uint8)
        rse.moe_workspace_init(self.wsp)
        self.top, self.tw = e(T, K_TOP, dtype=I32), e(T, K_TOP, dtype=torch.float32)
        self.counts, self.tokens = e(1, E, dtype=I32), e(1, dtype=I32)
        self.loss, self.grad = e(1, dtype=torch.float32), e(T, E, dtype=torch.float32)
        self.logits = e(T, E, dtype=torch.float32)

    def run(self):
        rse.moe_lora_plan(self.ids, L, self.plan)
        rse.moe_rmsnorm(self.x, self.w1, EPS, residual=self.res, residual_out=self.sum1, out=self.n1, q=self.q1, scale=self.s1)
        rse.moe_fp8_gemm(self.q1, self.s1, self.wq, self.ws, None, None, self.proj, self.wsp)
        rse.moe_lora(self.n1, self.a, self.b, self.scale, self.plan, self.proj, self.y, self.wsp)
        rse.moe_rmsnorm(self.y, self.w2, EPS, residual=self.sum1, residual_out=self.sum2, out=self.n2)
        self.layer.forward(self.n2, out=self.out, topk_ids=self.top, topk_w=self.tw)
        torch.mm(self.n2.float(), self.layer.tensors["router_w"].t(), out=self.logits)
        rse.moe_balance_loss(self.layer.cfg, self.logits, self.top, self.counts, self.tokens, self.loss, self.wsp,
                             grad_logits=self.grad, coef=0.01)

    def check(self):
        d = lambda t: t.double()  # noqa: E731
        h = (self.x.float() + self.res.float()).to(BF16)
        assert torch.equal(self.sum1, h)
        n = d(h) / (d(h).square().mean(1, keepdim=True) + EPS).sqrt() * d(self.w1)
        # half a bf16 step is 2^-8 of the value at most (7 bits behind the leading one), y's own error 2^-22
        near = ((d(self.n1) - n).abs() <= n.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
        assert bool(near)
        # half an E4M3 step: 2^-4 of the value, or 2^-10 of the scale below the normal range
        sc = d(self.s1).t().repeat_interleave(128, 1)
        wide = d(self.q1) * sc
        near = ((wide - n).abs() <= n.abs() * (2.0 ** -4 + 2.0 ** -21) + sc * 2.0 ** -10).all()
        assert bool(near)
        w = d(self.wq[0]) * torch.kron(d(self.ws[0]), torch.ones(128, 128, dtype=torch.float64, device="cuda"))
        p = wide @ w.t()
        assert float((d(self.proj) - p).norm() / p.norm()) <= 2.0 ** -8
        y = d(self.proj)
        for i in range(L):
            rows = self.ids == i
            y[rows] += float(self.scale[i]) * (d(self.n1[rows]) @ d(self.a[i]).t() @ d(self.b[i]).t())
        assert float((d(self.y) - y).norm() / y.norm()) <= 2.0 ** -8
        assert torch.equal(self.y[self.ids < 0], self.proj[self.ids < 0])
        h2 = (self.y.float() + self.sum1.float()).to(BF16)
        assert torch.equal(self.sum2, h2)
        again = torch.empty_like(self.out)
        self.layer.forward(self.n2, out=again)
        assert torch.equal(again, self.out)
        assert torch.equal(self.counts[0].long(), torch.bincount(self.top.view(-1).long(), minlength=E)) and int(self.tokens) == self.T
        z = d(self.logits).requires_grad_()
        s = torch.sigmoid(z)
        f = d(self.counts[0]) * (E / (K_TOP * self.T))
        loss = 0.01 * ((s / s.sum(1, keepdim=True)).mean(0) * f).sum()
        loss.backward()
        assert abs(float(self.loss) - float(loss.detach())) <= 2.0 ** -17 * float(loss.detach())
        assert float((d(self.grad) - z.grad).norm() / z.grad.norm()) <= 2.0 ** -16
        assert rse.moe_read_device_error(self.wsp) == 0 and self.layer.device_error() == 0


@pytest.mark.parametrize("T", [1, 37, 600])
def test_step(T):
    s = Step(T, T)
    s.run()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("T", [8, 600])
def test_step_in_a_graph(T):
    s = Step(T, 100 + T)
    s.run()                                                       # (the layer's warm-up call)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        s.x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        s.ids.copy_(torch.randint(-1, L, (T,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        s.check()
