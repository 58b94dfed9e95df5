"""An infinity in a token's row: the result is what the formula gives, an infinity
of its sign where every rank and feature agrees on one, whatever the rank is padded
to inside; NaN where signs differ or a factor is 0."""

import math

import pytest
import torch

from gpu_util import cuda_available
from test_gpu_lora import BF16, F16, F32, inputs, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype,out_type", [(BF16, BF16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T", [3, 520])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 88, 128])
def test_sign_of_an_infinity(T, r, dtype, out_type):
    K, N, L = 72, 40, 2
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, T + r, none=0.0)
    a, b = a.abs() + 0.125, b.abs() + 0.125
    b[:, 1::4] = -b[:, 1::4]
    b[:, 2::4, r - 1] = 0
    b[:, 3::4, r // 2] = -b[:, 3::4, r // 2]
    clean = run(x, a, b, scale, ids, base, out_type, L).cpu()
    x[0, 5], x[T - 1, K - 1] = math.inf, -math.inf
    out = run(x, a, b, scale, ids, base, out_type, L).cpu()
    for t, sign in ((0, 1), (T - 1, -1)):
        assert bool((out[t, 0::4] == sign * math.inf).all()) and bool((out[t, 1::4] == -sign * math.inf).all())
        assert bool(torch.isnan(out[t, 2::4]).all()) and bool(torch.isnan(out[t, 3::4]).all())
    assert torch.equal(out[1:T - 1], clean[1:T - 1])
