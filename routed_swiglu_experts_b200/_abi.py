"""ctypes binding of ``include/moe.h`` -- argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
plain pointers and sizes; all work runs in the CUDA library.  Tensors are
torch CUDA tensors (device memory and streams are torch's job); ``None``
passes a NULL pointer.  A non-OK status raises ``MoEError``.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5

MOE_W_BF16 = 0
MOE_W_INT4_G128 = 1
MOE_W_NVFP4 = 2
MOE_W_FP8_B128 = 4
MOE_ROUTING_FIELDS = 2
MOE_SCORE_SIGMOID = 0
MOE_SCORE_SOFTMAX = 1
MOE_GROUP_SUM2 = 0
MOE_GROUP_MAX = 1
MOE_F32 = 0
MOE_BF16 = 1
MOE_F16 = 2
MOE_MAX_GROUPS = 32
MOE_WS_HEADER_BYTES = 256
MOE_LORA_MAX_RANK = 128
MOE_MAX_ADAPTERS = 1024
MOE_BALANCE_WS_BYTES = 81920
MOE_NORM_MAX_COLUMNS = 32768
MOE_MAX_TOP_K = 16
MOE_MAX_EXPERTS = 1024
MOE_INT4_MAX_SWIGLU_LIMIT = 255.0

EXPORTED = (
    "moe_status_string", "moe_config_validate", "moe_workspace_size", "moe_workspace_init",
    "moe_router_topk", "moe_permute", "moe_grouped_swiglu_ffn", "moe_grouped_swiglu_ffn_gather", "moe_combine",
    "moe_forward", "moe_forward_ep", "moe_gate_topk", "moe_fp8_quantize", "moe_fp8_quantize_weight", "moe_fp8_gemm",
    "moe_rmsnorm", "moe_lora_plan_size", "moe_lora_plan", "moe_lora", "moe_balance_loss",
    "moe_read_device_error", "moe_permute_no_alloc", "moe_selftest_device_timeout", "moe_selftest_pair_timeout",
)
MOE_NO_ALLOC_MAX_ROWS = 131072
MOE_SELFTEST_SCRATCH_BYTES = 65536
MOE_SELFTEST_PAIR_BF16 = 0
MOE_SELFTEST_PAIR_INT4 = 1
MOE_SELFTEST_PAIR_FP8_FEW = 3
MOE_SELFTEST_PAIR_FP8_WIDE = 4
MOE_SELFTEST_LORA = 6


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_name(status)}")


class moe_config(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("expert_inter", ctypes.c_int32),
        ("shared_inter", ctypes.c_int32),
        ("swiglu_limit", ctypes.c_float),
        ("routed_scaling_factor", ctypes.c_float),
        ("renormalize", ctypes.c_int32),
        ("expert_format", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
    ]

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.renormalize = self.renormalize

    def __setattr__(self, name, value):
        # this struct always has the routing fields
        super().__setattr__(name, value | MOE_ROUTING_FIELDS if name == "renormalize" else value)


class moe_weights(ctypes.Structure):
    _fields_ = [
        ("router_w", ctypes.c_void_p),
        ("correction_bias", ctypes.c_void_p),
        ("w_gate_up", ctypes.c_void_p),
        ("s_gate_up", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p),
        ("s_down", ctypes.c_void_p),
        ("shared_w_gate_up", ctypes.c_void_p),
        ("shared_w_down", ctypes.c_void_p),
        ("g_gate_up", ctypes.c_void_p),
        ("g_down", ctypes.c_void_p),
    ]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library; raise loudly when it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library not found at {path}; build it with "
            "`python -m routed_swiglu_experts_b200.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    F32 = ctypes.c_float
    CFG, W = ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights)
    sig = {
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_config_validate": (ctypes.c_int, [CFG]),
        "moe_workspace_size": (ctypes.c_int, [CFG, I32, ctypes.POINTER(SZ)]),
        "moe_workspace_init": (ctypes.c_int, [P, SZ, P]),
        "moe_router_topk": (ctypes.c_int, [CFG, W, P, I32, P, P, P, SZ, P]),
        "moe_permute": (ctypes.c_int, [CFG, P, P, P, I32, P, P, P, P, P, P, SZ, P]),
        "moe_grouped_swiglu_ffn": (ctypes.c_int, [CFG, W, P, P, P, I32, P, P, P, P, SZ, P]),
        "moe_grouped_swiglu_ffn_gather": (ctypes.c_int, [CFG, W, P, I32, P, P, P, P, P, P, SZ, P]),
        "moe_combine": (ctypes.c_int, [CFG, P, P, P, P, I32, P, P]),
        "moe_forward": (ctypes.c_int, [CFG, W, P, I32, P, P, P, P, SZ, P]),
        "moe_forward_ep": (ctypes.c_int, [CFG, W, I32, I32, P, I32, P, P, P, P, SZ, P]),
        "moe_gate_topk": (ctypes.c_int, [CFG, P, I32, I64, P, I32, P, P, P]),
        "moe_fp8_quantize": (ctypes.c_int, [P, I32, I64, P, I32, I32, I32, P, P, P]),
        "moe_fp8_quantize_weight": (ctypes.c_int, [P, I32, I32, I32, I32, P, P, P]),
        "moe_fp8_gemm": (ctypes.c_int, [P, P, I32, P, I32, P, P, I32, I32, P, P, I32, P, SZ, P]),
        "moe_rmsnorm": (ctypes.c_int, [P, I32, I64, P, I64, P, I64, I32, P, I32, F32, I32, I32, P, I64, P, P, P]),
        "moe_lora_plan_size": (ctypes.c_int, [I32, I32, ctypes.POINTER(SZ)]),
        "moe_lora_plan": (ctypes.c_int, [P, I32, I32, P, SZ, P]),
        "moe_lora": (ctypes.c_int, [P, I32, I64, P, P, P, I32, I32, I32, I32, I32, P, SZ, P, I64, P, I32, I64, P, SZ, P]),
        "moe_balance_loss": (ctypes.c_int, [CFG, P, I32, I64, P, P, I32, P, I32, F32, P, P, P, P, P, I32, I64, P, SZ, P]),
        "moe_read_device_error": (ctypes.c_int, [P, P, ctypes.POINTER(I32)]),
        "moe_selftest_device_timeout": (ctypes.c_int, [P, SZ, P]),
        "moe_selftest_pair_timeout": (ctypes.c_int, [P, SZ, I32, P]),
        "moe_permute_no_alloc": (ctypes.c_int, [CFG, P, P, P, I32, P, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_name(status: int) -> str:
    try:
        return load_library().moe_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, dev: Optional[int] = None) -> Optional[int]:
    if stream is None:
        tt = _tt()
        return tt.stream(tt.device() if dev is None else dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def make_config(hidden, num_experts, top_k, expert_inter, shared_inter, swiglu_limit,
                routed_scaling_factor=1.0, renormalize=False, expert_format=MOE_W_BF16, score=MOE_SCORE_SIGMOID,
                num_groups=0, top_groups=0, group_score=MOE_GROUP_SUM2) -> moe_config:
    return moe_config(int(hidden), int(num_experts), int(top_k), int(expert_inter), int(shared_inter),
                      float(swiglu_limit), float(routed_scaling_factor), int(bool(renormalize)),
                      int(expert_format), int(score), int(num_groups), int(top_groups), int(group_score))


def make_weights(router_w=None, correction_bias=None, w_gate_up=None, s_gate_up=None, w_down=None,
                 s_down=None, shared_w_gate_up=None, shared_w_down=None, g_gate_up=None,
                 g_down=None) -> moe_weights:
    return moe_weights(_ptr(router_w), _ptr(correction_bias), _ptr(w_gate_up), _ptr(s_gate_up),
                       _ptr(w_down), _ptr(s_down), _ptr(shared_w_gate_up), _ptr(shared_w_down),
                       _ptr(g_gate_up), _ptr(g_down))


def weight_format(w_gate_up, g_gate_up=None) -> int:
    """The moe_weight_format of a layer's routed tensors: bf16 weights, E4M3
    weights (torch.float8_e4m3fn, block scales), or uint8 codes -- NVFP4 when
    the per-expert fp32 tensor scales are given, else W4A16."""
    if str(w_gate_up.dtype) == "torch.float8_e4m3fn":
        return MOE_W_FP8_B128
    if g_gate_up is not None:
        return MOE_W_NVFP4
    return MOE_W_INT4_G128 if str(w_gate_up.dtype) == "torch.uint8" else MOE_W_BF16


def check_fp8_weights(where, hidden, inter, experts, *, w_gate_up, w_down, s_gate_up, s_down):
    """The tensors of `experts` FP8 experts: E4M3 codes and fp32 block scales,
    contiguous, of the sizes that the kernels read (they get pointers alone)."""
    import torch
    codes, H, I = (torch.float8_e4m3fn, torch.uint8), hidden, inter
    for name, t, dtypes, n in (("w_gate_up", w_gate_up, codes, 2 * I * H), ("w_down", w_down, codes, H * I),
                               ("s_gate_up", s_gate_up, (torch.float32,), 2 * I // 128 * (H // 128)),
                               ("s_down", s_down, (torch.float32,), H // 128 * (I // 128))):
        if t is None:
            raise ValueError(f"{where}: {name} is missing")
        if t.dtype not in dtypes:
            raise ValueError(f"{where}: {name} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if t.numel() != experts * n:
            raise ValueError(f"{where}: {name} has {t.numel()} elements, expected {experts * n}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")


# ------------------------------------------------------- C entry points ----

def moe_config_validate(cfg: moe_config) -> int:
    return load_library().moe_config_validate(ctypes.byref(cfg))


def moe_workspace_size(cfg: moe_config, max_tokens: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size(ctypes.byref(cfg), int(max_tokens), ctypes.byref(n)),
           "moe_workspace_size")
    return n.value


def moe_workspace_init(ws, stream=None):
    _check(load_library().moe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_workspace_init")


def moe_router_topk(cfg, w, x, T, topk_ids, topk_w, ws, stream=None):
    _check(load_library().moe_router_topk(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), int(T), _ptr(topk_ids),
                                          _ptr(topk_w), _ptr(ws), ws.numel() * ws.element_size(),
                                          _stream(stream)), "moe_router_topk")


def moe_permute(cfg, topk_ids, topk_w, x, T, expert_offsets, row_of, src, w_perm, x_perm, ws, stream=None):
    _check(load_library().moe_permute(ctypes.byref(cfg), _ptr(topk_ids), _ptr(topk_w), _ptr(x), int(T),
                                      _ptr(expert_offsets), _ptr(row_of), _ptr(src), _ptr(w_perm),
                                      _ptr(x_perm), _ptr(ws), ws.numel() * ws.element_size(),
                                      _stream(stream)), "moe_permute")


def moe_grouped_swiglu_ffn(cfg, w, x_perm, expert_offsets, w_perm, T, y_perm, x_shared, shared_out, ws,
                           stream=None):
    _check(load_library().moe_grouped_swiglu_ffn(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(x_perm), _ptr(expert_offsets), _ptr(w_perm), int(T),
        _ptr(y_perm), _ptr(x_shared), _ptr(shared_out), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)), "moe_grouped_swiglu_ffn")


def moe_grouped_swiglu_ffn_gather(cfg, w, x, T, src, expert_offsets, w_perm, y_perm, shared_out, ws, stream=None):
    _check(load_library().moe_grouped_swiglu_ffn_gather(
        ctypes.byref(cfg), ctypes.byref(w), _ptr(x), int(T), _ptr(src), _ptr(expert_offsets), _ptr(w_perm),
        _ptr(y_perm), _ptr(shared_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "moe_grouped_swiglu_ffn_gather")


def moe_combine(cfg, y_perm, row_of, topk_w, shared_out, T, out, stream=None):
    _check(load_library().moe_combine(ctypes.byref(cfg), _ptr(y_perm), _ptr(row_of), _ptr(topk_w),
                                      _ptr(shared_out), int(T), _ptr(out), _stream(stream)), "moe_combine")


def moe_forward(cfg, w, x, T, out, topk_ids_opt, topk_w_opt, ws, stream=None):
    _check(load_library().moe_forward(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), int(T), _ptr(out),
                                      _ptr(topk_ids_opt), _ptr(topk_w_opt), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "moe_forward")


def moe_forward_ep(cfg, w, expert_begin, expert_end, x, T, out_partial, topk_ids_opt, topk_w_opt, ws, stream=None):
    _check(load_library().moe_forward_ep(ctypes.byref(cfg), ctypes.byref(w), int(expert_begin), int(expert_end),
                                         _ptr(x), int(T), _ptr(out_partial), _ptr(topk_ids_opt), _ptr(topk_w_opt),
                                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "moe_forward_ep")


class _Torch:
    """What the checks below look up in torch, once."""

    def __init__(self):
        import torch
        self.types = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
        self.floats = tuple(self.types)
        self.f32 = (torch.float32,)
        self.i32 = (torch.int32,)
        self.u8 = (torch.uint8,)
        self.masks = (torch.bool, torch.uint8)
        # a float type alone, and it or fp32
        self.alone = {t: (t,) for t in self.floats}
        self.or_f32 = {t: (t, torch.float32) for t in self.floats}
        self.halves = (torch.bfloat16, torch.float16)
        self.codes = (torch.float8_e4m3fn, torch.uint8)
        self.outs = (torch.bfloat16, torch.float32)
        # the current device's number, and a device's current stream as its handle alone:
        # building a torch.cuda.Stream around it takes 3 us, so the private look-ups are
        # used where the build has them
        device, stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))
        if not torch.cuda.is_available():
            # no tensor is on the current device (the CPU's number is -1); streams raise torch's error
            self.device, self.stream = lambda: -2, lambda dev: torch.cuda.current_stream().cuda_stream
        elif device is None or stream is None:
            self.device, self.stream = torch.cuda.current_device, lambda dev: torch.cuda.current_stream(dev).cuda_stream
        else:
            self.device, self.stream = device, stream


_torch = None


def _tt() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _want(t, name, dtypes, shape, where, dev, contiguous=True):
    """A tensor argument's element type, shape, layout and device, checked
    before its pointer is passed: the C call sees none of them.  The stream
    and the kernel belong to the current device `dev`, so the tensor must too."""
    if t is None:
        raise ValueError(f"{where}: {name} is missing")
    if (t.dtype in dtypes and (shape is None or t.shape == shape) and t.get_device() == dev
            and (not contiguous or t.is_contiguous())):
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{where}: {name} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} is on {t.device}, expected a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} is on {t.device}, the current device is {dev}")
    raise ValueError(f"{where}: {name} is not contiguous")


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _row_stride(t, name, where):
    """Elements between the rows of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{where}: {name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _rows(t, name, dtypes, shape, where, dev):
    """A 2-D tensor argument whose rows may be strided (shape None: any): the
    checks of _want, and the elements between its rows."""
    if t is not None and t.dtype in dtypes and t.get_device() == dev:
        s = t.shape
        if s == shape or (shape is None and len(s) == 2):
            if t.is_contiguous():
                return s[1]
            st = t.stride()
            if st[1] == 1 or s[1] == 1:
                return st[0] if s[0] > 1 else s[1]
    _want(t, name, dtypes, shape, where, dev, contiguous=False)
    return _row_stride(t, name, where)


def moe_gate_topk(cfg, logits, correction_bias, topk_ids, topk_w, stream=None):
    """Expert selection from logits [T, E] (fp32, bf16 or fp16; rows may be strided)."""
    where, tt = "moe_gate_topk", _tt()
    dev = tt.device()
    _want(logits, "logits", tt.floats, None, where, dev, contiguous=False)
    stride = _row_stride(logits, "logits", where)
    T, E = logits.shape
    if E != cfg.num_experts:
        raise ValueError(f"{where}: logits has {E} columns for {cfg.num_experts} experts")
    if correction_bias is not None:
        _want(correction_bias, "correction_bias", tt.f32, (E,), where, dev)
    shape = (T, cfg.top_k)
    _want(topk_ids, "topk_ids", tt.i32, shape, where, dev)
    _want(topk_w, "topk_w", tt.f32, shape, where, dev)
    _check(load_library().moe_gate_topk(ctypes.byref(cfg), logits.data_ptr(), tt.types[logits.dtype], stride,
                                        _ptr(correction_bias), T, topk_ids.data_ptr(), topk_w.data_ptr(),
                                        _stream(stream, dev)), where)


def moe_fp8_quantize(x, q, scale, src=None, src_div=1, stream=None):
    """Rows x [*, K] to E4M3 codes q [rows, K] and scales [ceil(K/128), rows];
    src int32 [rows]: row r is x[src[r] // src_div]."""
    where, tt = "moe_fp8_quantize", _tt()
    dev = tt.device()
    _want(x, "x", tt.floats, None, where, dev, contiguous=False)
    stride = _row_stride(x, "x", where)
    rows, K = x.shape
    if src is not None:
        rows = src.shape[0]
        _want(src, "src", tt.i32, (rows,), where, dev)
    _want(q, "q", tt.codes, (rows, K), where, dev)
    _want(scale, "scale", tt.f32, (_blocks(K), rows), where, dev)
    _check(load_library().moe_fp8_quantize(x.data_ptr(), tt.types[x.dtype], stride, _ptr(src), int(src_div), rows, K,
                                           q.data_ptr(), scale.data_ptr(), _stream(stream, dev)), where)


def moe_fp8_quantize_weight(w, q, scale, stream=None):
    """Weights w [groups, N, K] to E4M3 codes and scales [groups, ceil(N/128), ceil(K/128)]."""
    where, tt = "moe_fp8_quantize_weight", _tt()
    dev = tt.device()
    _want(w, "w", tt.floats, None, where, dev)
    if w.dim() != 3:
        raise ValueError(f"{where}: w must be [groups, N, K]")
    G, N, K = w.shape
    _want(q, "q", tt.codes, (G, N, K), where, dev)
    _want(scale, "scale", tt.f32, (G, _blocks(N), _blocks(K)), where, dev)
    _check(load_library().moe_fp8_quantize_weight(w.data_ptr(), tt.types[w.dtype], G, N, K, q.data_ptr(),
                                                  scale.data_ptr(), _stream(stream, dev)), where)


def moe_fp8_gemm(a, a_scale, w, w_scale, expert_offsets, row_scale, out, ws, stream=None):
    """out [rows, N] = a [rows, K] times w [groups, N, K] by row groups, E4M3
    codes with block scales (expert_offsets None: one group)."""
    where, tt = "moe_fp8_gemm", _tt()
    dev = tt.device()
    _want(a, "a", tt.codes, None, where, dev)
    _want(w, "w", tt.codes, None, where, dev)
    if a.dim() != 2 or w.dim() != 3 or a.shape[1] != w.shape[2]:
        raise ValueError(f"{where}: a must be [rows, K] and w [groups, N, K]")
    rows, K = a.shape
    G, N, _ = w.shape
    _want(a_scale, "a_scale", tt.f32, (_blocks(K), rows), where, dev)
    _want(w_scale, "w_scale", tt.f32, (G, _blocks(N), _blocks(K)), where, dev)
    if expert_offsets is not None:
        _want(expert_offsets, "expert_offsets", tt.i32, (G + 1,), where, dev)
    if row_scale is not None:
        _want(row_scale, "row_scale", tt.f32, (rows,), where, dev)
    _want(out, "out", tt.outs, (rows, N), where, dev)
    _want(ws, "ws", tt.u8, None, where, dev)
    _check(load_library().moe_fp8_gemm(a.data_ptr(), a_scale.data_ptr(), rows, _ptr(expert_offsets), G, w.data_ptr(),
                                       w_scale.data_ptr(), N, K, _ptr(row_scale), out.data_ptr(), tt.types[out.dtype],
                                       ws.data_ptr(), ws.numel(), _stream(stream, dev)), where)


def moe_rmsnorm(x, weight, eps, residual=None, residual_out=None, out=None, q=None, scale=None, stream=None):
    """RMS norm of rows x [rows, H] (+ residual, the sum written to
    residual_out, which may be residual itself) times weight [H] (None: 1), to
    out (x's type) and/or E4M3 codes q [rows, H] with scale [ceil(H/128), rows].
    Rows of x, residual, residual_out and out may be strided."""
    where, tt = "moe_rmsnorm", _tt()
    dev = tt.device()
    x_stride = _rows(x, "x", tt.floats, None, where, dev)
    shape, dtype = x.shape, x.dtype
    rows, H = shape
    same, types = tt.alone[dtype], tt.or_f32[dtype]
    x_type = res_type = w_type = tt.types[dtype]
    res_ptr = res_out_ptr = w_ptr = out_ptr = q_ptr = scale_ptr = None
    res_stride = res_out_stride = out_stride = H
    if residual is not None or residual_out is not None:
        res_stride = _rows(residual, "residual", types, shape, where, dev)
        res_out_stride = _rows(residual_out, "residual_out", tt.alone[residual.dtype], shape, where, dev)
        res_type, res_ptr, res_out_ptr = tt.types[residual.dtype], residual.data_ptr(), residual_out.data_ptr()
    if weight is not None:
        _want(weight, "weight", types, (H,), where, dev)
        w_type, w_ptr = tt.types[weight.dtype], weight.data_ptr()
    if out is not None:
        out_stride = _rows(out, "out", same, shape, where, dev)
        out_ptr = out.data_ptr()
    if q is not None or scale is not None:
        _want(q, "q", tt.codes, shape, where, dev)
        _want(scale, "scale", tt.f32, (_blocks(H), rows), where, dev)
        q_ptr, scale_ptr = q.data_ptr(), scale.data_ptr()
    _check(load_library().moe_rmsnorm(x.data_ptr(), x_type, x_stride, res_ptr, res_stride, res_out_ptr, res_out_stride, res_type,
                                      w_ptr, w_type, eps, rows, H, out_ptr, out_stride, q_ptr, scale_ptr,
                                      _stream(stream, dev)), where)


def moe_lora_plan_size(T: int, num_adapters: int) -> int:
    """Bytes of a plan for T tokens and num_adapters adapters."""
    n = ctypes.c_size_t(0)
    _check(load_library().moe_lora_plan_size(int(T), int(num_adapters), ctypes.byref(n)), "moe_lora_plan_size")
    return n.value


def moe_lora_plan(adapters, num_adapters, plan, stream=None):
    """The order of a batch by adapter: adapters int32 [T] (-1: none) to plan
    (uint8, moe_lora_plan_size bytes), for every moe_lora call on that batch."""
    where, tt = "moe_lora_plan", _tt()
    dev = tt.device()
    _want(adapters, "adapters", tt.i32, None, where, dev)
    if adapters.dim() != 1:
        raise ValueError(f"{where}: adapters must be [T]")
    _want(plan, "plan", tt.u8, None, where, dev)
    _check(load_library().moe_lora_plan(adapters.data_ptr(), adapters.shape[0], num_adapters, plan.data_ptr(), plan.numel(),
                                        _stream(stream, dev)), where)


def moe_lora(x, a, b, scale, plan, base, out, ws, stream=None):
    """out [T, N] = base [T, N] (None: 0; may be out) + scale [L] * (x [T, K]
    a_l^T) b_l^T by the plan's adapters; a [L, rank, K], b [L, N, rank]."""
    where, tt = "moe_lora", _tt()
    dev = tt.device()
    x_stride = _rows(x, "x", tt.halves, None, where, dev)
    same = tt.alone[x.dtype]
    _want(a, "a", same, None, where, dev)
    _want(b, "b", same, None, where, dev)
    (T, K), a_shape, b_shape = x.shape, a.shape, b.shape
    if len(a_shape) != 3 or len(b_shape) != 3 or a_shape[2] != K or b_shape[0] != a_shape[0] or b_shape[2] != a_shape[1]:
        raise ValueError(f"{where}: a must be [adapters, rank, {K}] and b [adapters, N, rank]")
    L, N, r = b_shape
    scale_ptr = base_ptr = None
    if scale is not None:
        _want(scale, "scale", tt.f32, (L,), where, dev)
        scale_ptr = scale.data_ptr()
    _want(plan, "plan", tt.u8, None, where, dev)
    out_stride = base_stride = _rows(out, "out", tt.or_f32[x.dtype], (T, N), where, dev)
    out_ptr = out.data_ptr()
    if base is out:
        base_ptr = out_ptr
    elif base is not None:
        base_stride = _rows(base, "base", tt.alone[out.dtype], (T, N), where, dev)
        base_ptr = base.data_ptr()
    _want(ws, "ws", tt.u8, None, where, dev)
    _check(load_library().moe_lora(x.data_ptr(), tt.types[x.dtype], x_stride, a.data_ptr(), b.data_ptr(), scale_ptr, T, K,
                                   N, r, L, plan.data_ptr(), plan.numel(), base_ptr, base_stride, out_ptr,
                                   tt.types[out.dtype], out_stride, ws.data_ptr(), ws.numel(), _stream(stream, dev)), where)


def moe_balance_loss(cfg, logits, topk_ids, counts, seq_tokens, loss, ws, grad_logits=None, seq_offsets=None,
                     token_mask=None, coef=1.0, grad_loss=None, stream=None):
    """The router's balance loss (one fp32 value) over logits [T, E] and their
    selection topk_ids [T, k]; counts int32 [S, E] and seq_tokens int32 [S] of
    the sequences seq_offsets int32 [S + 1] (None: one); grad_logits [T, E]
    (the logits' type or fp32) times grad_loss (one fp32 value; None: 1);
    token_mask bool or uint8 [T]: tokens to count."""
    where, tt = "moe_balance_loss", _tt()
    dev = tt.device()
    stride = grad_stride = _rows(logits, "logits", tt.floats, None, where, dev)
    shape, dtype = logits.shape, logits.dtype
    T, E = shape
    if E != cfg.num_experts:
        raise ValueError(f"{where}: logits has {E} columns for {cfg.num_experts} experts")
    _want(topk_ids, "topk_ids", tt.i32, (T, cfg.top_k), where, dev)
    S, offsets_ptr, mask_ptr, up_ptr, grad_ptr = 1, None, None, None, None
    if seq_offsets is not None:
        _want(seq_offsets, "seq_offsets", tt.i32, None, where, dev)
        if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
            raise ValueError(f"{where}: seq_offsets must be [sequences + 1]")
        S, offsets_ptr = seq_offsets.shape[0] - 1, seq_offsets.data_ptr()
    _want(counts, "counts", tt.i32, (S, E), where, dev)
    _want(seq_tokens, "seq_tokens", tt.i32, (S,), where, dev)
    if token_mask is not None:
        _want(token_mask, "token_mask", tt.masks, (T,), where, dev)
        mask_ptr = token_mask.data_ptr()
    _want(loss, "loss", tt.f32, None, where, dev)
    if loss.numel() != 1:
        raise ValueError(f"{where}: loss has {loss.numel()} elements, expected 1")
    if grad_loss is not None:
        _want(grad_loss, "grad_loss", tt.f32, None, where, dev)
        if grad_loss.numel() != 1:
            raise ValueError(f"{where}: grad_loss has {grad_loss.numel()} elements, expected 1")
        up_ptr = grad_loss.data_ptr()
    grad_type = 0
    if grad_logits is not None:
        grad_stride = _rows(grad_logits, "grad_logits", tt.or_f32[dtype], shape, where, dev)
        grad_type, grad_ptr = tt.types[grad_logits.dtype], grad_logits.data_ptr()
    _want(ws, "ws", tt.u8, None, where, dev)
    _check(load_library().moe_balance_loss(
        ctypes.byref(cfg), logits.data_ptr(), tt.types[dtype], stride, topk_ids.data_ptr(), offsets_ptr, S, mask_ptr, T, coef,
        up_ptr, counts.data_ptr(), seq_tokens.data_ptr(), loss.data_ptr(), grad_ptr, grad_type, grad_stride, ws.data_ptr(),
        ws.numel(), _stream(stream, dev)), where)


def moe_permute_no_alloc(cfg, topk_ids, topk_w, x, T, expert_offsets, row_of, src, w_perm, x_perm, stream=None):
    """moe_permute without a workspace (scratch held inside the library)."""
    _check(load_library().moe_permute_no_alloc(ctypes.byref(cfg), _ptr(topk_ids), _ptr(topk_w), _ptr(x), int(T),
                                               _ptr(expert_offsets), _ptr(row_of), _ptr(src), _ptr(w_perm),
                                               _ptr(x_perm), _stream(stream)), "moe_permute_no_alloc")


def moe_read_device_error(ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(load_library().moe_read_device_error(_ptr(ws), _stream(stream), ctypes.byref(code)),
           "moe_read_device_error")
    return code.value


def moe_selftest_device_timeout(scratch, stream=None):
    """Test hook: force the tensor-core kernel's timeout path on a tiny tile
    (the error lands in scratch's error word; read it with
    moe_read_device_error(scratch))."""
    _check(load_library().moe_selftest_device_timeout(_ptr(scratch), scratch.numel() * scratch.element_size(),
                                                      _stream(stream)), "moe_selftest_device_timeout")


def moe_selftest_pair_timeout(scratch, kernel, stream=None):
    """Test hook: force the timeout path of a CTA-pair grouped GEMM
    (one of MOE_SELFTEST_PAIR_*) or of the adapters (MOE_SELFTEST_LORA) on a tiny tile; read the error with moe_read_device_error(scratch)."""
    _check(load_library().moe_selftest_pair_timeout(_ptr(scratch), scratch.numel() * scratch.element_size(),
                                                    int(kernel), _stream(stream)), "moe_selftest_pair_timeout")


def status_strings():
    lib = load_library()
    return {s: lib.moe_status_string(s).decode() for s in range(6)}


INF = math.inf
