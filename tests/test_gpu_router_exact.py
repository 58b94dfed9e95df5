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
    # The weights come from the fp32 logits.  Those are sums of 3 H products, 16 to an addition, whose 3 H / 16
    # roundings (and 32 for the slices) move them by at most 2^-23 of the running sum each: d / 2 with the d below.  A
    # renormalised weight is s_i / sum s: numerator and sum move by d / 2 of themselves each (softmax exactly so,
    # a sigmoid by less), 1e-5 more for the fp32 functions.
    d = (0.75 * x.shape[1] + 64) * 2.0 ** -24 * z.abs().amax(1).clamp(min=1.0)
    assert bool(((tw - ww).abs() <= (1e-5 + d[:, None]) * ww).all())


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


@pytest.mark.parametrize("name", ["softmax", "softmax_groups", "softmax_groups_max"])
def test_softmax_biases_that_meet_the_scores(name):
    """Biases that leave every sum s + b within 1e-9 of a few values, for
    the one token of the call: the softmax's denominator decides as well."""
    g = torch.Generator().manual_seed(31)
    for seed in range(6):
        x = torch.randn(1, 768, generator=g).to(torch.bfloat16)
        w = torch.randn(64, 768, generator=g) / 768 ** 0.5
        s = torch.softmax(oracle.router_logits(x, w), 1)[0]
        level = 0.25 + 0.125 * torch.randint(0, 8, (64,), generator=g)
        bias = (level.double() - s + 1e-9 * torch.randn(64, generator=g).double()).float()
        check(x, w, bias, 6, ROUTES[name])


def test_sigmoid_biases_that_meet_the_scores():
    g = torch.Generator().manual_seed(32)
    for name in ("groups", "groups_max"):
        for seed in range(6):
            x = torch.randn(1, 768, generator=g).to(torch.bfloat16)
            w = torch.randn(64, 768, generator=g) / 768 ** 0.5
            s = torch.sigmoid(oracle.router_logits(x, w))[0]
            level = 1.25 + 0.125 * torch.randint(0, 8, (64,), generator=g)
            bias = (level.double() - s + 1e-9 * torch.randn(64, generator=g).double()).float()
            check(x, w, bias, 6, ROUTES[name])


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("name", sorted(ROUTES))
def test_padded_rows_and_rows_with_nan(name, biased):
    """Rows of zeros tie everywhere: the lowest groups and ids (of the largest
    biases); a NaN row gets valid ids; the rows between are as ever."""
    for E, k in ((64, 6), (148, 5)):
        x, w, bias = inputs(90, 256, E, ROUTES[name].get("num_groups", 1), E, 1e-6, biased)
        x[::3] = 0.0
        check(x, w, bias, k, ROUTES[name])
        x[1, 7] = float("nan")
        ids, _ = route(x.cuda(), w.cuda(), None if bias is None else bias.cuda(), k, ROUTES[name])
        assert 0 <= int(ids.min()) and int(ids.max()) < E and all(len(set(r)) == k for r in ids.tolist())
        z = oracle.router_logits(x[2:], w)
        kw = ROUTES[name]
        want, _ = go.gate_select(z, bias, k, 2.5, True, kw.get("score") == SOFTMAX, kw.get("num_groups", 1),
                                 kw.get("top_groups", 1), kw.get("group_score") == MAX)
        assert torch.equal(ids[2:], want)


def test_many_tokens():
    """More tokens than one pass of the kernels holds, one in twenty a row whose biased scores all meet."""
    g = torch.Generator().manual_seed(41)
    H, E, T = 128, 24, 6000
    w = torch.randn(E, H, generator=g) / H ** 0.5
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    x[::20] = x[0]
    s = torch.softmax(oracle.router_logits(x[:1], w), 1)[0]
    bias = (0.75 - s + 1e-9 * torch.randn(E, generator=g).double()).float()
    check(x, w, bias, 4, ROUTES["softmax"])
    check(x, w, bias, 4, ROUTES["softmax_groups"])


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
