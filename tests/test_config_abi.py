"""moe_config grew by four routing fields: a caller built against the header
without them passes a struct that ends before, and only the flag
MOE_ROUTING_FIELDS in renormalize says that they are there (no GPU needed)."""

import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from routed_swiglu_experts_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
SHORT = _abi.moe_config.score.offset  # bytes of the struct before the routing fields


def words(renormalize=1, routing=()):
    """The struct's bytes as a C caller fills them, field by field."""
    n = _abi.moe_config
    c = (ctypes.c_int32 * (ctypes.sizeof(n) // 4))()
    f = ctypes.cast(c, ctypes.POINTER(ctypes.c_float))
    for name, v in dict(hidden=256, num_experts=64, top_k=6, expert_inter=128, shared_inter=0, renormalize=renormalize,
                        expert_format=0).items():
        c[getattr(n, name).offset // 4] = v
    f[n.swiglu_limit.offset // 4] = 7.0
    f[n.routed_scaling_factor.offset // 4] = 2.5
    for i, v in enumerate(routing):
        c[SHORT // 4 + i] = v
    return c


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def call(lib, name, cfg, *args):
    return getattr(lib, name)(ctypes.cast(cfg, ctypes.POINTER(_abi.moe_config)), *args)


GARBAGE = [(-1, -1, -1, -1), (1, 8, 4, 0), (7, 1 << 30, -5, 99), (0, 3, 0, 0)]


@pytest.mark.parametrize("behind", GARBAGE)
def test_what_lies_behind_a_short_struct_is_not_read(lib, behind):
    c = words(1, behind)
    assert call(lib, "moe_config_validate", c) == _abi.MOE_OK
    n, m = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert call(lib, "moe_workspace_size", c, 64, ctypes.byref(n)) == _abi.MOE_OK
    assert call(lib, "moe_workspace_size", words(), 64, ctypes.byref(m)) == _abi.MOE_OK
    assert n.value == m.value
    w = _abi.make_weights(router_w=FAKE, w_gate_up=FAKE, w_down=FAKE)
    assert call(lib, "moe_forward", c, ctypes.byref(w), FAKE, 0, FAKE, None, None, FAKE, n, None) == _abi.MOE_OK
    assert call(lib, "moe_forward_ep", c, ctypes.byref(w), 0, 64, FAKE, 0, FAKE, None, None, FAKE, n, None) == _abi.MOE_OK
    assert call(lib, "moe_router_topk", c, ctypes.byref(w), FAKE, 0, FAKE, FAKE, FAKE, n, None) == _abi.MOE_OK
    assert call(lib, "moe_combine", c, FAKE, FAKE, None, None, 0, FAKE, None) == _abi.MOE_OK
    assert call(lib, "moe_permute_no_alloc", c, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, None) == _abi.MOE_OK


def test_the_flag_brings_the_fields_in(lib):
    two = 1 | _abi.MOE_ROUTING_FIELDS
    assert call(lib, "moe_config_validate", words(two, (1, 8, 4, 1))) == _abi.MOE_OK
    assert call(lib, "moe_config_validate", words(two, (0, 0, 0, 0))) == _abi.MOE_OK
    assert call(lib, "moe_config_validate", words(_abi.MOE_ROUTING_FIELDS, (1, 8, 4, 1))) == _abi.MOE_OK
    for bad in ((2, 0, 0, 0), (0, -1, 0, 0), (0, 8, 9, 0), (0, 8, 4, 2)):
        assert call(lib, "moe_config_validate", words(two, bad)) == _abi.MOE_ERR_INVALID_ARG
    for renormalize in (-1, 4, 5, 7):
        assert call(lib, "moe_config_validate", words(renormalize)) == _abi.MOE_ERR_INVALID_ARG


def test_selection_from_logits_refuses_routing_without_its_flag(lib):
    """The call is younger than the fields, so it may look at them: routing that was set but not announced."""
    for routing in ((1, 0, 0, 0), (0, 8, 4, 0), (0, 0, 0, 1)):
        assert call(lib, "moe_gate_topk", words(1, routing), FAKE, 0, 64, None, 4, FAKE, FAKE, None) == _abi.MOE_ERR_INVALID_ARG
        assert call(lib, "moe_gate_topk", words(3, routing), FAKE, 0, 64, None, 0, FAKE, FAKE, None) == _abi.MOE_OK
    assert call(lib, "moe_gate_topk", words(1), FAKE, 0, 64, None, 0, FAKE, FAKE, None) == _abi.MOE_OK


def test_binding_always_has_the_fields():
    c = _abi.make_config(256, 64, 6, 128, 0, 7.0, num_groups=8, top_groups=9)
    assert _abi.moe_config_validate(c) == _abi.MOE_ERR_INVALID_ARG
    c.top_groups = 4
    c.renormalize = 1
    assert _abi.moe_config_validate(c) == _abi.MOE_OK
    c.score = 2
    assert _abi.moe_config_validate(c) == _abi.MOE_ERR_INVALID_ARG
    c = _abi.moe_config()
    for name, v in dict(hidden=256, num_experts=64, top_k=6, expert_inter=128, swiglu_limit=7.0, num_groups=8).items():
        setattr(c, name, v)
    assert _abi.moe_config_validate(c) == _abi.MOE_ERR_INVALID_ARG  # no group kept
    c = _abi.moe_config(256, 64, 6, 128, 0, 7.0, 1.0, 1, 0, 0, 8, 9, 0)
    assert _abi.moe_config_validate(c) == _abi.MOE_ERR_INVALID_ARG


PAGE = """
import ctypes, mmap, sys
sys.path.insert(0, {root!r})
from routed_swiglu_experts_b200 import _abi
lib, size = _abi.load_library(), mmap.PAGESIZE
libc = ctypes.CDLL(None, use_errno=True)
libc.mmap.restype = ctypes.c_void_p
libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
at = libc.mmap(None, 2 * size, 3, 0x22, -1, 0)
assert libc.mprotect(at + size, size, 0) == 0
at += size - {short}
ctypes.memmove(at, bytes.fromhex({data!r}), {short})
cfg = ctypes.cast(at, ctypes.POINTER(_abi.moe_config))
n = ctypes.c_size_t(0)
print(lib.moe_config_validate(cfg), lib.moe_workspace_size(cfg, 16, ctypes.byref(n)))
"""


@pytest.mark.skipif(not sys.platform.startswith("linux"), reason="mmap flags of Linux")
def test_a_short_struct_may_end_its_page():
    code = PAGE.format(root=ROOT, short=SHORT, data=bytes(words())[:SHORT].hex())
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["0", "0"], (r.returncode, r.stderr[-300:])


def test_flag_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) { printf("%d\\n", MOE_ROUTING_FIELDS); return 0; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "c")], check=True)
    out = subprocess.run([str(tmp_path / "c")], check=True, capture_output=True, text=True).stdout
    assert int(out) == _abi.MOE_ROUTING_FIELDS
