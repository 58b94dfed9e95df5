"""An FP8 layer's tensors are checked for their format when the layer is made:
the C calls see pointers alone (no GPU needed)."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from routed_swiglu_experts_b200 import ep

F8 = torch.float8_e4m3fn


def layer(cls, **kw):
    E, H, I = 4, 256, 128
    t = dict(w_gate_up=torch.zeros(E, 2 * I, H, dtype=F8), w_down=torch.zeros(E, H, I, dtype=F8),
             s_gate_up=torch.zeros(E, 2 * I // 128, H // 128), s_down=torch.zeros(E, H // 128, I // 128))
    t.update(kw)
    return cls(hidden=H, num_experts=E, top_k=2, expert_inter=I, shared_inter=0, swiglu_limit=7.0, routed_scaling_factor=1.0,
               renormalize=True, router_w=torch.zeros(E, H), correction_bias=None, **t)


@pytest.mark.parametrize("cls", [rse.MoELayer, ep.ExpertParallelLayer])
@pytest.mark.parametrize("name,value", [
    ("s_gate_up", torch.zeros(4, 2, 2, dtype=torch.bfloat16)),      # half the bytes that the kernels read
    ("s_gate_up", torch.zeros(4, 2, 2, dtype=torch.uint8)),         # exponents alone
    ("s_gate_up", torch.zeros(4, 2, 1)),
    ("s_down", torch.zeros(4, 1, 1)),
    ("s_down", torch.zeros(4, 2, 1, dtype=torch.float64)),
    ("w_down", torch.zeros(4, 256, 128, dtype=torch.bfloat16)),
    ("w_down", torch.zeros(4, 128, 128, dtype=F8)),
    ("w_gate_up", torch.zeros(4, 128, 256, dtype=F8)),
    ("s_down", torch.zeros(4, 2, 2)[:, :, :1]),                     # not contiguous
])
def test_fp8_layers_refuse_what_is_not_their_format(cls, name, value):
    if cls is ep.ExpertParallelLayer and not value.is_contiguous():
        pytest.skip("the rank's slices are made contiguous")
    with pytest.raises(ValueError, match=name):
        layer(cls, **{name: value})


@pytest.mark.parametrize("cls", [rse.MoELayer, ep.ExpertParallelLayer])
def test_fp8_layers_take_what_is(cls):
    layer(cls)
    layer(cls, w_down=torch.zeros(4, 256, 128, dtype=torch.uint8))
    layer(cls, s_gate_up=torch.zeros(4, 4))
    for rank in range(6):                                           # ranks without experts among them
        if cls is ep.ExpertParallelLayer:
            E, H, I = 4, 256, 128
            ep.ExpertParallelLayer(hidden=H, num_experts=E, top_k=2, expert_inter=I, shared_inter=0, swiglu_limit=7.0,
                                   routed_scaling_factor=1.0, renormalize=True, router_w=torch.zeros(E, H),
                                   correction_bias=None, w_gate_up=torch.zeros(E, 2 * I, H, dtype=F8),
                                   w_down=torch.zeros(E, H, I, dtype=F8), s_gate_up=torch.zeros(E, 2, 2),
                                   s_down=torch.zeros(E, 2, 1), rank=rank, world=6)
