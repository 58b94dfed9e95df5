"""The layer's own router with softmax scores or groups of experts selects by
the exact logits x . w: experts and groups whose logits the fp32 product
cannot tell apart come out in the order of the fp64 product, for every token."""

import pytest
import torch

import oracle
import routed_swiglu_experts_b200 as rse
from oracle import gate_fp8_oracle as go
from routed_swiglu_experts_b200 import ep

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

SOFTMAX, MAX = rse.MOE_SCORE_SOFTMAX, rse.MOE_GROUP_MAX
ROUTES = {
    "softmax": dict(score=SOFTMAX),
    "groups": dict(num_groups=4, top_groups=2),
    "groups_max": dict(num_groups=4, top_groups=2, group_score=MAX),
    "softmax_groups": dict(score=SOFTMAX, num_groups=4, top_groups=1),
    "softmax_groups_max": dict(score=SOFTMAX, num_groups=4, top_groups=3, group_score=MAX),
}


def inputs(T, H, E, groups, seed, spread, biased):
    """Experts in close pairs (2 i, 2 i + 1) and groups in close pairs: copies
    with the weights' values off by `spread` of themselves."""
    g = torch.Generator().manual_seed(seed)
    per = E // groups
    base = torch.randn((groups + 1) // 2, (per + 1) // 2, H, generator=g) / H ** 0.5
    w = base.repeat_interleave(2, 0)[:groups].repeat_interleave(2, 1)[:, :per].reshape(E, H)
    w = w * (1 + spread * torch.randn(E, H, generator=g))
    bias = None
    if biased:
        b = torch.rand((groups + 1) // 2, (per + 1) // 2, generator=g) * 0.2 - 0.1
        bias = b.repeat_interleave(2, 0)[:groups].repeat_interleave(2, 1)[:, :per].reshape(E).contiguous()
    return torch.randn(T, H, generator=g).to(torch.bfloat16), w.contiguous(), bias


def route(x, w, bias, k, kw):
    T, H = x.shape
    cfg = rse.make_config(H, w.shape[0], k, 128, 0, 7.0, 2.5, True, **kw)
    ws = torch.empty(rse.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    rse.moe_workspace_init(ws)
    wts = rse.make_weights(router_w=w, correction_bias=bias)
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, k, device="cuda")
    rse.moe_router_topk(cfg, wts, x, T, ids, tw, ws)
    assert rse.moe_read_device_error(ws) == 0
    return ids.cpu().long(), tw.cpu().double()


def check(x, w, bias, k, kw):
    ids, tw = route(x.cuda(), w.cuda(), None if bias is None else bias.cuda(), k, kw)
    z = oracle.router_logits(x, w)
    want, ww = go.gate_select(z, bias, k, 2.5, True, kw.get("score") == SOFTMAX, kw.get("num_groups", 1),
                              kw.get("top_groups", 1), kw.get("group_score") == MAX)
    assert torch.equal(ids, want), f"{int((ids != want).any(1).sum())} of {len(ids)} tokens differ"
    # fp32 logits: off by 1e-6 here, which moves a renormalised weight by 2e-6 of itself
    assert torch.allclose(tw, ww, rtol=2e-5, atol=0)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("name", sorted(ROUTES))
@pytest.mark.parametrize("T,H,E,k", [(1, 256, 16, 3), (200, 2048, 64, 5), (70, 1032, 128, 16), (40, 512, 100, 7), (30, 264, 148, 6)])
def test_close_experts(T, H, E, k, name, biased):
    kw = dict(ROUTES[name])
    if E == 100 and "num_groups" in kw:
        kw["num_groups"] = 5                # 20 experts a group: five lanes
    for spread in (3e-7, 1e-5):
        x, w, bias = inputs(T, H, E, kw.get("num_groups", 1), E + k, spread, biased)
        check(x, w, bias, k, kw)


@pytest.mark.parametrize("name", sorted(ROUTES))
def test_all_experts_close(name):
    """More close experts than the rounds hold (32)."""
    g = torch.Generator().manual_seed(4)
    w = (torch.randn(1, 384, generator=g) / 384 ** 0.5) * (1 + 1e-6 * torch.randn(96, 384, generator=g))
    x = torch.randn(20, 384, generator=g).to(torch.bfloat16)
    for bias in (None, torch.zeros(96)):
        check(x, w, bias, 8, ROUTES[name])


@pytest.mark.parametrize("name", sorted(ROUTES))
def test_large_logits(name):
    """Logits of some 50: their fp32 error grows with them."""
    x, w, bias = inputs(60, 1024, 64, ROUTES[name].get("num_groups", 1), 9, 1e-6, False)
    check(x * 32, w, bias, 5, ROUTES[name])


def test_layer_and_one_rank_take_the_same_route():
    kw = ROUTES["groups"]
    x, w, bias = inputs(150, 256, 16, 4, 2, 1e-6, True)
    g = torch.Generator().manual_seed(5)
    t = dict(router_w=w.cuda(), correction_bias=bias.cuda(),
             w_gate_up=(torch.randn(16, 256, 256, generator=g) / 16).to(torch.bfloat16).cuda(),
             w_down=(torch.randn(16, 256, 128, generator=g) / 11).to(torch.bfloat16).cuda())
    args = dict(hidden=256, num_experts=16, top_k=3, expert_inter=128, shared_inter=0, swiglu_limit=7.0,
                routed_scaling_factor=2.5, renormalize=True, max_tokens=150, **t, **kw)
    z = oracle.router_logits(x, w)
    want, _ = go.gate_select(z, bias, 3, 2.5, True, False, 4, 2)
    for layer in (rse.MoELayer(**args), ep.ExpertParallelLayer(**args)):
        ids = torch.empty(150, 3, dtype=torch.int32, device="cuda")
        tw = torch.empty(150, 3, device="cuda")
        run = layer.forward if isinstance(layer, rse.MoELayer) else layer.forward_partial
        run(x.cuda(), topk_ids=ids, topk_w=tw)
        assert torch.equal(ids.cpu().long(), want)
