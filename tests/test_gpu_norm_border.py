"""RMS norm of long, dense rows whose blocks have their largest values within
some fp32 steps of 448 * 2^e, where the scale doubles: fp32 sums of such rows
are off by steps of their own, and the scales have to be those of the exact
rows all the same.  One row a call, copied (its blocks' weights fit it alone)."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import around_oracle as ao

from gpu_util import cuda_available
from test_gpu_norm import BF16, EPS, F16, F32, F8

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def bordering(x, seed):
    """A weight that takes one value of each block to 448 * 2^-4 (1 + j 2^-24), |j| <= 30, and all others below it."""
    g = torch.Generator().manual_seed(seed)
    H = x.shape[1]
    _, y = ao.rmsnorm(x, None, EPS)
    w = torch.full((H,), 2.0 ** -6)
    for b in range(0, H, 128):
        k = b + int(y[0, b:b + 128].abs().argmax())
        j = int(torch.randint(-30, 31, (1,), generator=g))
        w[k] = float(28.0 * (1 + j * 2.0 ** -24) / y[0, k].abs())
    return w


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("H,rows", [(128, 1), (2048, 3), (2048, 9000), (6144, 2), (6144, 1999), (16384, 1), (16384, 1203), (20480, 2),
                                    (32768, 1), (32768, 200)])
def test_scales_of_dense_rows(H, rows, dtype):
    near = 0
    for seed in range(4):
        g = torch.Generator().manual_seed(H + seed)
        x = (torch.randn(1, H, generator=g) * 1.3).to(dtype)
        if seed == 3:
            x = torch.full((1, H), 1.0 + 2.0 ** -6).to(dtype)     # (equal values: every sum rounds the same way)
        w = bordering(x, seed)
        _, y = ao.rmsnorm(x, w, EPS)
        q = torch.zeros(rows, H, dtype=F8, device="cuda")
        s = torch.zeros(H // 128, rows, device="cuda")
        rse.moe_rmsnorm(x.cuda().repeat(rows, 1), w.cuda(), EPS, q=q, scale=s)
        want = ao.norm_scales(y)
        assert bool((s.cpu().double() == want).all())
        assert bool((q.view(torch.uint8) == q[:1].view(torch.uint8)).all())
        top = y.abs().view(-1, 128).amax(1) / 28.0 - 1
        near += int((top.abs() < 2.0 ** -19).sum())
    assert near == 4 * (H // 128)
