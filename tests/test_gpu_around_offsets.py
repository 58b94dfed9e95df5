"""Rows of the adapters, the norm and the balance loss past 2^31 elements of their
tensors (views with wide rows), against the same rows close together."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_balance import config, workspace as balance_workspace
from test_gpu_lora import plan_of, workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

BF16 = torch.bfloat16


def wide(rows, cols, stride, dtype):
    """[rows, cols] whose last rows start past 2^31 elements."""
    assert (rows - 1) * stride > 1 << 31
    if torch.cuda.mem_get_info()[0] < rows * stride * torch.empty((), dtype=dtype).element_size() + (8 << 30):
        pytest.skip("needs more memory")
    return torch.empty(rows * stride, dtype=dtype, device="cuda").view(rows, stride)[:, :cols]


@pytest.mark.parametrize("T", [300, 700])
def test_adapters(T):
    K, N, r, L = 136, 200, 16, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    stride = ((1 << 31) // (T - 2) + 63) // 16 * 16
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    a = (torch.randn(L, r, K, generator=g, device="cuda") / math.sqrt(K)).to(BF16)
    b = torch.randn(L, N, r, generator=g, device="cuda").to(BF16)
    base = torch.randn(T, N, generator=g, device="cuda").to(BF16)
    plan = plan_of(torch.randint(-1, L, (T,), generator=g, device="cuda"), L)
    want = torch.empty_like(base)
    rse.moe_lora(x, a, b, None, plan, base, want, workspace())
    far_x, far = wide(T, K, stride, BF16), wide(T, N, stride, BF16)
    far_x.copy_(x)
    far.copy_(base)
    rse.moe_lora(far_x, a, b, None, plan, far, far, workspace())
    assert torch.equal(far, want)


@pytest.mark.parametrize("rows,dtype", [(300, BF16), (4000, BF16), (300, torch.float32)])
def test_norm(rows, dtype):
    H = 1040
    g = torch.Generator(device="cuda").manual_seed(rows)
    stride = ((1 << 31) // (rows - 2) + 63) // 16 * 16
    x = torch.randn(rows, H, generator=g, device="cuda").to(dtype)
    res = torch.randn(rows, H, generator=g, device="cuda").to(dtype)
    want, sums = torch.empty_like(x), torch.empty_like(x)
    rse.moe_rmsnorm(x, None, 1e-6, residual=res, residual_out=sums, out=want)
    far_x, far_res = wide(rows, H, stride, dtype), wide(rows, H, stride, dtype)
    far_x.copy_(x)
    far_res.copy_(res)
    rse.moe_rmsnorm(far_x, None, 1e-6, residual=far_res, residual_out=far_res, out=far_x)
    assert torch.equal(far_x, want) and torch.equal(far_res, sums)


def test_balance():
    T, E, k = 3000, 40, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    stride = (1 << 31) // (T - 2) + 7
    z = torch.randn(T, E, generator=g, device="cuda").to(BF16)
    ids = z.float().topk(k, dim=1).indices.to(torch.int32)
    far_z, far_g = wide(T, E, stride, BF16), wide(T, E, stride, BF16)
    far_z.copy_(z)
    got = []
    for logits, grad in ((z, torch.empty_like(z)), (far_z, far_g)):
        counts, tokens = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        loss = torch.empty((), device="cuda")
        rse.moe_balance_loss(config(E, k, True), logits, ids, counts, tokens, loss, balance_workspace(), grad_logits=grad, coef=1.0)
        got.append((counts, tokens, loss, grad))
    assert all(torch.equal(p, q) for p, q in zip(*got))
