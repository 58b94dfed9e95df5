"""moe_lora's out may lie in base's place alone: a product's result over its own
operands is refused (host checks, no GPU).  The operands have places of their
own here, so that each refusal stands alone."""

import pytest

import routed_swiglu_experts_b200 as rse
from routed_swiglu_experts_b200 import _abi

X, A, B, PLAN, WS, OUT = (i << 20 for i in range(1, 7))


@pytest.mark.parametrize("out", [X, A, B])
@pytest.mark.parametrize("T", [4, 1000])
def test_refused(out, T):
    need = rse.moe_lora_plan_size(T, 8)
    got = _abi.load_library().moe_lora(X, _abi.MOE_BF16, 64, A, B, None, T, 64, 64, 16, 8, PLAN, need, None, 64, out, _abi.MOE_BF16,
                                       64, WS, 256, None)
    assert got == _abi.MOE_ERR_INVALID_ARG
