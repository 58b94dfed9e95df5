"""Adapters whose ranks differ much in size, against fp64: what a rank adds to
a feature keeps its bits although another rank, which that feature does not
use, is 2^20 times as large.  The bounds are test_gpu_lora's, element by
element: P is the sum of the feature's own products' magnitudes, so the large
rank has no part in it."""

import pytest
import torch

from oracle import around_oracle as ao

from gpu_util import cuda_available
from test_gpu_lora import BF16, F16, F32, inputs, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("T", [20, 600])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,out_type", [(F16, F16), (F16, F32), (BF16, F32)])
def test_small_ranks_beside_a_large_one(T, r, dtype, out_type):
    K, N, L = 256, 40, 2
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, T + r, none=0.0)
    a = (a.float() * 2.0 ** -8).to(dtype)
    a[:, 3] = (a[:, 3].float() * 2.0 ** 20).to(dtype)             # A x of rank 3 near 2^12, of the others near 2^-8
    b = (b.float() * 2.0 ** 6).to(dtype)
    b[:, :, 3] = 0
    b[:, ::4, 3] = 2.0 ** -6                                      # (every fourth feature uses it)
    base.zero_()
    want, size = ao.lora(x, a, b, scale, ids, base)
    out = run(x, a, b, scale, ids, base, out_type, L).cpu().double()
    half = torch.finfo(out_type).eps / 2
    bound = size * ((K + r) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * half * (1 + 2.0 ** -6) + (2.0 ** -25 if out_type == F16 else 0)
    assert bool(((out - want).abs() <= bound).all()), float(((out - want).abs() / bound).max())


@pytest.mark.parametrize("T", [5, 520])
@pytest.mark.parametrize("up", [2.0 ** 118, 2.0 ** 60, 2.0 ** -60, 2.0 ** -118])
def test_adapter_scales_far_outside_fp16(T, up):
    """scale takes A x to both ends of fp32's range; features of fp32 come back with it."""
    K, N, r, L = 64, 24, 8, 2
    x, a, b, scale, ids, _ = inputs(T, K, N, r, L, F16, F32, T, none=0.0)
    scale = scale * up
    want, size = ao.lora(x, a, b, scale, ids, None)
    out = run(x, a, b, scale, ids, None, F32, L).cpu().double()
    bound = size * ((K + r) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * 2.0 ** -24
    assert bool(((out - want).abs() <= bound).all()), float(((out - want).abs() / bound).max())
