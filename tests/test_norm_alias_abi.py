"""moe_rmsnorm's documented aliases: an output in an input's place has its
type and stride, and no two outputs share a place (host checks, no GPU)."""

import pytest

from routed_swiglu_experts_b200 import _abi

A, B, C, D = (i << 20 for i in range(1, 5))
BAD = _abi.MOE_ERR_INVALID_ARG
F32, BF16 = _abi.MOE_F32, _abi.MOE_BF16


def call(x=A, xs=256, res=None, rs=256, ro=None, ros=256, rt=BF16, w=None, rows=4, out=C, outs=256, q=None, s=None):
    return _abi.load_library().moe_rmsnorm(x, BF16, xs, res, rs, ro, ros, rt, w, BF16, 1e-6, rows, 256, out, outs, q, s, None)


@pytest.mark.parametrize("kw", [
    dict(res=B, ro=B, rs=256, ros=264),                          # the sum in the residual's place, other rows
    dict(res=B, ro=A, xs=264),                                   # ... in x's
    dict(res=B, ro=A, rt=F32),                                   # ... of another type
    dict(out=A, outs=264),                                       # the result in x's place, other rows
    dict(res=B, ro=D, out=B, outs=264),                          # ... in the residual's
    dict(res=B, ro=D, rt=F32, out=B),                            # ... of another type
    dict(res=B, ro=B, out=B),                                    # both results in one place
    dict(res=B, ro=C, out=C),
    dict(res=B, ro=D, w=D), dict(q=C, s=D), dict(q=A, s=D), dict(res=B, ro=B, q=B, s=D, out=None), dict(w=D, q=D, s=B), dict(w=C, out=C),
])
def test_refused(kw):
    assert call(**kw) == BAD
