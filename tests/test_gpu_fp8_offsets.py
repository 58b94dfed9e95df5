"""Expert offsets outside the routed rows count as the nearer end in the whole
FP8 feed-forward: in the pass that quantises the rows (blocks of eight, the
last one reaching past them) as in the two products behind it."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_fp8 import fp8_layer

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("T,H,I", [(9, 256, 128), (17, 384, 256), (1501, 512, 512)])  # rows: 27, 51, 4503; few and many rows
@pytest.mark.parametrize("gather", [True, False])
def test_stray_offsets_count_as_the_nearer_end(T, H, I, gather):
    k, E = 3, 4
    R = T * k
    c = fp8_layer(T=T, H=H, E=E, k=k, I=I, seed=T)
    layer, cfg = c.layer, c.layer.cfg
    x = c.x.cuda()
    # 64 rows more than the call owns on either side of what a stray offset could reach
    src = torch.randperm(R, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    src = torch.cat([src, torch.zeros(64, dtype=torch.int32, device="cuda")])
    x_perm = torch.cat([x[(src[:R] // k).long()], torch.full((64, H), 3.0, device="cuda", dtype=torch.bfloat16)])
    cut = [R // 5, R // 5, R // 2]
    outs = []
    for first, last in ((0, R), (0, R + 5), (-3, R + 1), (0, 2 ** 31 - 1)):
        off = torch.tensor([first, *cut, last], dtype=torch.int32, device="cuda")
        y = torch.full((R + 64, H), 7.0, dtype=torch.bfloat16, device="cuda")
        layer.ws[256:].fill_(0x55)          # what the call leaves unwritten is the same each time
        if gather:
            rse.moe_grouped_swiglu_ffn_gather(cfg, layer.w, x, T, src, off, None, y, None, layer.ws)
        else:
            rse.moe_grouped_swiglu_ffn(cfg, layer.w, x_perm, off, None, T, y, None, None, layer.ws)
        outs.append((y, layer.ws.clone()))
        assert layer.device_error() == 0
    for y, ws in outs[1:]:
        assert torch.equal(y, outs[0][0])
        assert torch.equal(ws, outs[0][1])  # codes and scales too: nothing written past their rows
    assert bool((outs[0][0][R:] == 7.0).all())
