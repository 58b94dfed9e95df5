"""Argument checks of the norm, the adapters and the balance loss: every
refusal comes from the host, before anything is launched (no GPU needed)."""

import ctypes
import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from routed_swiglu_experts_b200 import _abi

FAKE = 1 << 20
BAD, UNSUP, OK, WS = (_abi.MOE_ERR_INVALID_ARG, _abi.MOE_ERR_UNSUPPORTED, _abi.MOE_OK, _abi.MOE_ERR_WORKSPACE)
F32, BF16, F16 = _abi.MOE_F32, _abi.MOE_BF16, _abi.MOE_F16


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def test_norm_refusals(lib):
    def call(x=FAKE, xt=BF16, xs=256, res=None, rs=256, ro=None, ros=256, rt=BF16, w=FAKE, wt=F32, eps=1e-6, rows=4, H=256,
             out=FAKE, outs=256, q=None, s=None):
        return lib.moe_rmsnorm(x, xt, xs, res, rs, ro, ros, rt, w, wt, eps, rows, H, out, outs, q, s, None)
    assert call(rows=0, x=None, out=None) == OK
    assert call(rows=-1) == BAD
    assert call(rows=1 << 26) == UNSUP
    assert call(xt=3) == BAD
    assert call(H=0) == BAD
    assert call(H=24) == BAD
    assert call(H=_abi.MOE_NORM_MAX_COLUMNS + 16, xs=1 << 20, outs=1 << 20) == UNSUP
    for eps in (0.0, -1e-6, 1e-38, math.inf, math.nan):
        assert call(eps=eps) == BAD
    assert call(x=None) == BAD
    assert call(x=FAKE + 8) == BAD
    assert call(xs=248) == BAD
    assert call(xs=260) == BAD
    assert call(out=None) == BAD                                 # nothing to write
    assert call(out=FAKE + 4) == BAD
    assert call(outs=128) == BAD
    assert call(q=FAKE) == BAD                                   # codes without scales
    assert call(s=FAKE) == BAD
    assert call(q=FAKE + 8, s=FAKE) == BAD
    assert call(q=FAKE, s=FAKE + 2) == BAD
    assert call(res=FAKE) == BAD                                 # a residual without a place for the sum
    assert call(ro=FAKE) == BAD
    assert call(res=FAKE, ro=FAKE, rt=F16) == BAD
    assert call(res=FAKE, ro=FAKE, rs=128) == BAD
    assert call(res=FAKE, ro=FAKE, ros=260) == BAD
    assert call(res=FAKE + 8, ro=FAKE) == BAD
    assert call(res=FAKE, ro=FAKE + 8) == BAD
    assert call(w=FAKE + 8) == BAD
    assert call(wt=F16) == BAD


def test_lora_plan_refusals(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_lora_plan_size(-1, 4, ctypes.byref(n)) == BAD
    assert lib.moe_lora_plan_size(4, 0, ctypes.byref(n)) == BAD
    assert lib.moe_lora_plan_size(4, 4, None) == BAD
    assert lib.moe_lora_plan_size(4, _abi.MOE_MAX_ADAPTERS + 1, ctypes.byref(n)) == UNSUP
    assert lib.moe_lora_plan_size(1 << 22, 4, ctypes.byref(n)) == UNSUP
    assert lib.moe_lora_plan_size(1 << 21, _abi.MOE_MAX_ADAPTERS, ctypes.byref(n)) == OK and n.value > 4 << 21
    need = rse.moe_lora_plan_size(100, 8)

    def call(ids=FAKE, T=100, L=8, plan=FAKE, size=need):
        return lib.moe_lora_plan(ids, T, L, plan, size, None)
    assert call(T=0, ids=None, plan=None, size=0) == OK
    assert call(ids=None) == BAD
    assert call(ids=FAKE + 2) == BAD
    assert call(plan=None) == BAD
    assert call(plan=FAKE + 8) == BAD
    assert call(size=need - 1) == WS
    assert call(L=0) == BAD


def test_lora_refusals(lib):
    need = rse.moe_lora_plan_size(100, 8)

    def call(x=FAKE, xt=BF16, xs=64, a=FAKE, b=FAKE, sc=None, T=100, K=64, N=33, r=16, L=8, plan=FAKE, size=need, base=None,
             bs=33, out=FAKE, ot=BF16, os=33, ws=FAKE, n=256):
        return lib.moe_lora(x, xt, xs, a, b, sc, T, K, N, r, L, plan, size, base, bs, out, ot, os, ws, n, None)
    assert call(T=0, x=None, plan=None, ws=None) == OK
    assert call(T=-1) == BAD
    assert call(T=1 << 22) == UNSUP
    assert call(xt=F32) == BAD
    assert call(ot=F16) == BAD
    assert call(ot=7) == BAD
    assert call(K=60) == BAD
    assert call(K=0) == BAD
    assert call(K=(1 << 30) + 8, xs=1 << 31) == UNSUP
    assert call(N=0) == BAD
    assert call(N=(1 << 30) + 1, os=1 << 31) == UNSUP
    assert call(r=0) == BAD
    assert call(r=12) == BAD
    assert call(r=136) == UNSUP
    assert call(L=0) == BAD
    assert call(L=1025) == UNSUP
    for name in ("x", "a", "b", "plan", "out"):
        assert call(**{name: None}) == BAD
    for name in ("x", "a", "b", "plan"):
        assert call(**{name: FAKE + 8}) == BAD
    assert call(xs=56) == BAD
    assert call(xs=68) == BAD
    assert call(os=32) == BAD
    assert call(base=FAKE + 64, bs=32) == BAD
    assert call(base=FAKE, bs=40) == BAD                         # in place with another stride
    assert call(out=FAKE + 1) == BAD
    assert call(ot=F32, out=FAKE + 2) == BAD
    assert call(base=FAKE + 1) == BAD
    assert call(sc=FAKE + 2) == BAD
    assert call(size=need - 1) == WS
    assert call(ws=None) == WS
    assert call(n=255) == WS
    assert call(ws=FAKE + 16) == BAD


def test_balance_refusals(lib):
    cfg = _abi.make_config(128, 64, 6, 128, 0, 7.0)

    def call(c=cfg, z=FAKE, zt=F32, zs=64, ids=FAKE, off=None, S=1, mask=None, T=4, coef=1.0, up=None, counts=FAKE,
             tokens=FAKE, loss=FAKE, g=FAKE + 4096, gt=F32, gs=64, ws=FAKE, n=_abi.MOE_BALANCE_WS_BYTES):
        return lib.moe_balance_loss(ctypes.byref(c), z, zt, zs, ids, off, S, mask, T, coef, up, counts, tokens, loss, g, gt, gs,
                                    ws, n, None)
    assert call(T=-1) == BAD
    assert call(T=1 << 22) == UNSUP
    assert call(c=_abi.make_config(128, 64, 6, 128, 0, 7.0, score=9)) == BAD
    assert call(zt=4) == BAD
    assert call(gt=BF16) == BAD
    assert call(zt=F16, gt=BF16) == BAD
    assert call(S=0) == BAD
    assert call(S=2) == BAD                                      # sequences without offsets
    assert call(off=FAKE, S=1 << 22) == UNSUP
    assert call(off=FAKE + 2, S=2) == BAD
    assert call(coef=math.inf) == BAD
    assert call(coef=math.nan) == BAD
    for name in ("counts", "tokens", "loss", "z", "ids"):
        assert call(**{name: None}) == BAD
        assert call(**{name: FAKE + 2}) == BAD
    assert call(up=FAKE + 2) == BAD
    assert call(zs=63) == BAD
    assert call(gs=63) == BAD
    assert call(g=FAKE) == BAD                                   # in place
    assert call(g=FAKE + 4098) == BAD
    assert call(ws=None) == WS
    assert call(n=_abi.MOE_BALANCE_WS_BYTES - 1) == WS
    assert call(ws=FAKE + 16) == BAD
    # a score function that the flags do not announce
    plain = _abi.make_config(128, 64, 6, 128, 0, 7.0, score=_abi.MOE_SCORE_SOFTMAX)
    ctypes.c_int32.from_buffer(plain, _abi.moe_config.renormalize.offset).value = 0
    assert call(c=plain) == BAD


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rse.moe_rmsnorm(x, None, 1e-6, out=x)
    with pytest.raises(ValueError, match="float64"):
        rse.moe_rmsnorm(x.double(), None, 1e-6, out=x)
    with pytest.raises(ValueError, match="float32"):
        rse.moe_lora(x.float(), None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="int64"):
        rse.moe_lora_plan(torch.zeros(4, dtype=torch.int64), 2, None)
    cfg = rse.make_config(128, 64, 6, 128, 0, 7.0)
    with pytest.raises(ValueError, match="CUDA"):
        rse.moe_balance_loss(cfg, x, None, None, None, None, None)
    with pytest.raises(rse.MoEError, match="INVALID_ARG"):
        rse.moe_lora_plan_size(4, 0)


def test_new_constants_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ["MOE_LORA_MAX_RANK", "MOE_MAX_ADAPTERS", "MOE_BALANCE_WS_BYTES", "MOE_NORM_MAX_COLUMNS"]
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) {\n' +
                   "".join(f'  printf("%d\\n", (int)({n}));\n' for n in names) + "  return 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "c")], check=True)
    out = subprocess.run([str(tmp_path / "c")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [getattr(_abi, n) for n in names]
