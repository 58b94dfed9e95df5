"""Adapters of ranks on both sides of 64 and as many tiles as take clusters of
eight, four and two, with test_gpu_lora's bounds."""

import pytest

from oracle import around_oracle as ao

from gpu_util import cuda_available
from test_gpu_lora import BF16, F16, F32, check, inputs, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("r", [64, 72, 128])
@pytest.mark.parametrize("T,L", [(2, 25), (16, 16), (20, 20), (34, 40), (40, 30), (90, 60), (200, 100), (512, 130)])
@pytest.mark.parametrize("dtype,out_type", [(BF16, BF16), (F16, F32)])
def test_tiles_and_ranks(T, L, r, dtype, out_type):
    K, N = 328, 138
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, 1000 * T + r)
    want, size = ao.lora(x, a, b, scale, ids, base)
    check(run(x, a, b, scale, ids, base, out_type, L), want, size, K, r)
