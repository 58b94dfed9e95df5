"""The adapters' tensor-core kernel when one of its waits runs out: the status
reaches the host, copies and MMAs are waited for, tensor memory is freed, and
the same process goes on computing (no GPU fault is involved: the kernel's
test hook withholds one signal between its own roles)."""

import time

import pytest
import torch

from oracle import around_oracle as ao
from routed_swiglu_experts_b200 import _abi

from gpu_util import cuda_available
from test_gpu_lora import BF16, check, inputs, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def test_timeout_is_reported_and_the_context_survives():
    scratch = torch.zeros(_abi.MOE_SELFTEST_SCRATCH_BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        t0 = time.perf_counter()
        _abi.moe_selftest_pair_timeout(scratch, _abi.MOE_SELFTEST_LORA)
        code = _abi.moe_read_device_error(scratch)
        assert code == _abi.MOE_ERR_DEVICE_TIMEOUT
        assert time.perf_counter() - t0 < 2.0
        assert _abi.moe_read_device_error(scratch) == 0
    for r in (16, 64):
        x, a, b, scale, ids, base = inputs(900, 1000, 300, r, 3, BF16, BF16, r)
        want, size = ao.lora(x, a, b, scale, ids, base)
        check(run(x, a, b, scale, ids, base, BF16, 3), want, size, 1000, r)
