"""What the binding takes from torch: the fast private look-ups where a build
has them, the public ones where it does not (no GPU needed)."""

from types import SimpleNamespace

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from routed_swiglu_experts_b200 import _abi

PRIVATE = ("_cuda_getDevice", "_cuda_getCurrentRawStream")


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    monkeypatch.setattr(_abi, "_torch", None)


def without(monkeypatch, *names):
    for n in names:
        monkeypatch.delattr(torch._C, n, raising=False)


@pytest.mark.parametrize("missing", [PRIVATE[:1], PRIVATE[1:], PRIVATE])
def test_checks_need_no_private_names(monkeypatch, missing):
    without(monkeypatch, *missing)
    cfg = _abi.make_config(256, 64, 6, 128, 0, 7.0)
    z = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        rse.moe_gate_topk(cfg, z, None, torch.zeros(3, 6, dtype=torch.int32), torch.zeros(3, 6))
    with pytest.raises(ValueError, match="float64"):
        rse.moe_fp8_quantize(z.double(), None, None)
    with pytest.raises(ValueError, match="missing"):
        rse.moe_fp8_gemm(None, None, None, None, None, None, None, None)


@pytest.mark.parametrize("missing", [(), PRIVATE])
def test_without_a_gpu_the_stream_raises_torchs_own_error(monkeypatch, missing):
    without(monkeypatch, *missing)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)

    def no_gpu(device=None):
        raise RuntimeError("Found no NVIDIA driver on your system")
    monkeypatch.setattr(torch.cuda, "current_stream", no_gpu)
    with pytest.raises(RuntimeError, match="no NVIDIA driver"):
        _abi._stream(None)
    assert _abi._stream(5) == 5


def test_public_names_stand_in(monkeypatch):
    without(monkeypatch, *PRIVATE)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=70 + device))
    assert _abi._stream(None) == 73
    assert _abi._stream(None, 1) == 71
    assert _abi._stream(SimpleNamespace(cuda_stream=9)) == 9


def test_private_names_are_used_where_there(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch._C, PRIVATE[0], lambda: 2, raising=False)
    monkeypatch.setattr(torch._C, PRIVATE[1], lambda dev: 40 + dev, raising=False)
    assert _abi._stream(None) == 42
