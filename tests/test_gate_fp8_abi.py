"""Argument checks of the selection from logits and of the FP8 calls: every
refusal comes from the host, before anything is launched (no GPU needed)."""

import ctypes

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from routed_swiglu_experts_b200 import _abi

FAKE = 1 << 20
BAD, UNSUP, OK, WS = (_abi.MOE_ERR_INVALID_ARG, _abi.MOE_ERR_UNSUPPORTED, _abi.MOE_OK, _abi.MOE_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def cfg(**kw):
    base = dict(hidden=256, num_experts=64, top_k=6, expert_inter=128, shared_inter=0, swiglu_limit=7.0)
    base.update(kw)
    return _abi.make_config(**base)


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    ({"score": _abi.MOE_SCORE_SOFTMAX}, OK),
    ({"score": 2}, BAD),
    ({"group_score": -1}, BAD),
    ({"num_groups": -1}, BAD),
    ({"num_groups": 1, "top_groups": 99}, OK),            # one group: no groups
    ({"num_groups": 8, "top_groups": 4}, OK),
    ({"num_groups": 8, "top_groups": 4, "group_score": _abi.MOE_GROUP_MAX}, OK),
    ({"num_groups": 8}, BAD),                              # no group kept
    ({"num_groups": 8, "top_groups": 9}, BAD),
    ({"num_groups": 7, "top_groups": 2}, BAD),             # 64 experts in 7 groups
    ({"num_groups": 16, "top_groups": 1}, BAD),            # 6 of 4 experts
    ({"num_groups": 64, "top_groups": 8}, UNSUP),
    ({"expert_format": _abi.MOE_W_FP8_B128}, OK),
    ({"expert_format": _abi.MOE_W_FP8_B128, "swiglu_limit": float("inf")}, OK),
    ({"expert_format": _abi.MOE_W_FP8_B128, "hidden": 200}, UNSUP),
    ({"expert_format": _abi.MOE_W_FP8_B128, "expert_inter": 192}, UNSUP),
])
def test_config(lib, kw, status):
    assert _abi.moe_config_validate(cfg(**kw)) == status


def test_gate_refusals(lib):
    def call(c=None, logits=FAKE, dtype=_abi.MOE_F32, stride=64, bias=None, T=4, ids=FAKE, w=FAKE):
        return lib.moe_gate_topk(ctypes.byref(c or cfg()), logits, dtype, stride, bias, T, ids, w, None)
    assert call(T=0, logits=None, ids=None, w=None) == OK
    assert call(T=-1) == BAD
    assert call(dtype=3) == BAD
    assert call(stride=63) == BAD
    assert call(logits=None) == BAD
    assert call(logits=FAKE + 2) == BAD
    assert call(dtype=_abi.MOE_BF16, logits=FAKE + 1) == BAD
    assert call(ids=None) == BAD
    assert call(w=FAKE + 2) == BAD
    assert call(bias=FAKE + 1) == BAD
    assert call(c=cfg(num_groups=8)) == BAD
    assert call(T=1 << 22) == UNSUP


def test_quantize_refusals(lib):
    def call(x=FAKE, dtype=_abi.MOE_BF16, stride=256, src=None, div=1, rows=4, K=256, q=FAKE, s=FAKE):
        return lib.moe_fp8_quantize(x, dtype, stride, src, div, rows, K, q, s, None)
    assert call(rows=0, x=None, q=None, s=None) == OK
    assert call(rows=-1) == BAD
    assert call(dtype=5) == BAD
    assert call(K=0) == BAD
    assert call(K=24) == BAD
    assert call(stride=128) == BAD
    assert call(stride=260) == BAD                         # rows not 16-byte aligned
    assert call(x=FAKE + 8) == BAD
    assert call(q=FAKE + 8) == BAD
    assert call(s=FAKE + 2) == BAD
    assert call(src=FAKE + 2) == BAD
    assert call(div=0) == BAD
    assert call(x=None) == BAD

    def weight(w=FAKE, dtype=_abi.MOE_F32, G=2, N=100, K=64, q=FAKE, s=FAKE):
        return lib.moe_fp8_quantize_weight(w, dtype, G, N, K, q, s, None)
    assert weight(G=0, w=None) == OK
    assert weight(G=-1) == BAD
    assert weight(N=0) == BAD
    assert weight(K=40) == BAD
    assert weight(dtype=-1) == BAD
    assert weight(w=None) == BAD
    assert weight(q=FAKE + 4) == BAD
    assert weight(G=1 << 20, N=1 << 20, K=1 << 20) == UNSUP


def test_gemm_refusals(lib):
    def call(a=FAKE, sa=FAKE, rows=4, off=FAKE, G=2, w=FAKE, sw=FAKE, N=64, K=64, c=None, out=FAKE, t=_abi.MOE_BF16,
             ws=FAKE, n=256):
        return lib.moe_fp8_gemm(a, sa, rows, off, G, w, sw, N, K, c, out, t, ws, n, None)
    assert call(rows=0, a=None, ws=None) == OK
    assert call(rows=-1) == BAD
    assert call(G=0) == BAD
    assert call(off=None) == BAD                           # two groups without offsets
    assert call(G=2000) == UNSUP
    assert call(N=60) == BAD
    assert call(K=72) == BAD
    assert call(t=_abi.MOE_F16) == BAD
    assert call(a=None) == BAD
    assert call(sw=None) == BAD
    assert call(w=FAKE + 8) == BAD
    assert call(out=FAKE + 4) == BAD
    assert call(sa=FAKE + 2) == BAD
    assert call(c=FAKE + 2) == BAD
    assert call(off=FAKE + 2) == BAD
    assert call(ws=None) == WS
    assert call(n=255) == WS
    assert call(ws=FAKE + 16) == BAD


def test_fp8_layer_needs_its_scales(lib):
    c = cfg(expert_format=_abi.MOE_W_FP8_B128)
    n = _abi.moe_workspace_size(c, 16)

    def call(T=16, ws_bytes=n, **kw):
        w = _abi.make_weights(**{"router_w": FAKE, "w_gate_up": FAKE, "w_down": FAKE, **kw})
        return lib.moe_forward(ctypes.byref(c), ctypes.byref(w), FAKE, T, FAKE, None, None, FAKE, ws_bytes, None)
    assert call() == BAD
    assert call(s_gate_up=FAKE) == BAD
    assert call(s_gate_up=FAKE, s_down=FAKE + 2) == BAD
    assert call(s_gate_up=FAKE, s_down=FAKE + 4, ws_bytes=n - 1) == WS
    assert call(T=0, s_gate_up=FAKE, s_down=FAKE + 4) == OK


def test_binding_refuses_wrong_tensors():
    c = cfg()
    good = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        rse.moe_gate_topk(c, good, None, torch.zeros(3, 6, dtype=torch.int32), torch.zeros(3, 6))
    with pytest.raises(ValueError, match="float64"):
        rse.moe_gate_topk(c, good.double(), None, None, None)
    with pytest.raises(ValueError, match="float64"):
        rse.moe_fp8_quantize(good.double(), None, None)
    with pytest.raises(ValueError, match="missing"):
        rse.moe_fp8_gemm(None, None, None, None, None, None, None, None)
    assert _abi.weight_format(torch.zeros(1, dtype=torch.float8_e4m3fn)) == _abi.MOE_W_FP8_B128


def test_fp8_selftest_argument_checks(lib):
    n = _abi.MOE_SELFTEST_SCRATCH_BYTES
    for kernel in (_abi.MOE_SELFTEST_PAIR_FP8_FEW, _abi.MOE_SELFTEST_PAIR_FP8_WIDE):
        assert lib.moe_selftest_pair_timeout(None, n, kernel, None) == WS
        assert lib.moe_selftest_pair_timeout(FAKE, n - 1, kernel, None) == WS
        assert lib.moe_selftest_pair_timeout(FAKE + 16, n, kernel, None) == BAD
    assert lib.moe_selftest_pair_timeout(FAKE, n, 5, None) == BAD


def test_new_constants_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ["MOE_W_FP8_B128", "MOE_SCORE_SIGMOID", "MOE_SCORE_SOFTMAX", "MOE_GROUP_SUM2", "MOE_GROUP_MAX", "MOE_F32",
             "MOE_BF16", "MOE_F16", "MOE_MAX_GROUPS", "MOE_WS_HEADER_BYTES", "MOE_SELFTEST_PAIR_FP8_FEW",
             "MOE_SELFTEST_PAIR_FP8_WIDE"]
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) {\n' +
                   "".join(f'  printf("%d\\n", (int)({n}));\n' for n in names) + "  return 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "c")], check=True)
    out = subprocess.run([str(tmp_path / "c")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [getattr(_abi, n) for n in names]
