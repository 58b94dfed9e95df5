"""Argument checks of the adapters' timeout hook (no GPU needed)."""

from routed_swiglu_experts_b200 import _abi


def test_hook_checks_its_scratch():
    lib, n = _abi.load_library(), _abi.MOE_SELFTEST_SCRATCH_BYTES
    fake = 1 << 20
    assert lib.moe_selftest_pair_timeout(None, n, _abi.MOE_SELFTEST_LORA, None) == _abi.MOE_ERR_WORKSPACE
    assert lib.moe_selftest_pair_timeout(fake, n - 1, _abi.MOE_SELFTEST_LORA, None) == _abi.MOE_ERR_WORKSPACE
    assert lib.moe_selftest_pair_timeout(fake + 16, n, _abi.MOE_SELFTEST_LORA, None) == _abi.MOE_ERR_INVALID_ARG
    assert lib.moe_selftest_pair_timeout(fake, n, _abi.MOE_SELFTEST_LORA + 1, None) == _abi.MOE_ERR_INVALID_ARG
