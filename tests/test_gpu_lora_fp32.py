"""Adapters of bf16 added to an fp32 result: A x reaches B with all the bits that
fp32 gives it.

Whole numbers, so that every sum is exact: |x| < 2^8, |a| < 2^7 and K = 256 keep
A x below 2^23, and a feature takes one rank with the factor 1, -2 or 0.5."""

import pytest
import torch

from gpu_util import cuda_available
from test_gpu_lora import BF16, F32, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("T", [1, 40, 512, 520, 1300])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 88, 128])
def test_every_bit_of_the_first_product(T, r):
    K, N, L = 256, 2 * r + 5, 3
    g = torch.Generator().manual_seed(T + r)
    x = torch.randint(-255, 256, (T, K), generator=g).to(BF16)
    a = torch.randint(-127, 128, (L, r, K), generator=g).to(BF16)
    factor = torch.tensor([1.0, -2.0, 0.5])[torch.randint(0, 3, (L, N), generator=g)]
    b = torch.zeros(L, N, r)
    which = torch.randint(0, r, (L, N), generator=g)
    b.scatter_(2, which[:, :, None], factor[:, :, None])
    ids = torch.randint(-1, L, (T,), generator=g)
    ids[0] = 0
    out = run(x, a, b.to(BF16), None, ids, None, F32, L).cpu()
    low = torch.einsum("tk,lrk->tlr", x.double(), a.double())
    i = ids.clamp(min=0)
    want = low[torch.arange(T)[:, None], i[:, None], which[i]] * factor[i].double()
    want[ids < 0] = 0
    assert float(low.abs().max()) < 2 ** 23
    assert bool((low.abs() > 2 ** 16).any())                      # more bits than two bf16 values hold
    assert torch.equal(out.double(), want)
