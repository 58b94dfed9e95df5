"""Expert selection from logits against the fp64 oracle: ids bit-exact, on
every type, group layout and degenerate row, and the weights within fp32
rounding.

Weights: a score's relative error is at most (|l - max| + 37 + 8) * 2^-24
(the rounded difference under exp, the softmax sum of at most 32 + 5
additions in a row, and exp, divisions and alpha), below 1e-5 for logits
within 120 of their maximum."""

import math

import pytest
import torch

import moe_inputs
import oracle
import routed_swiglu_experts_b200 as rse
from moe_inputs.configs import LayerConfig
from oracle import gate_fp8_oracle as go
from routed_swiglu_experts_b200 import ep

from gpu_util import cuda_available, gpu_layer

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

RTOL = 1e-5


def config(E, k, softmax=False, groups=1, top=1, group_max=False, renorm=True, alpha=2.5):
    return rse.make_config(128, E, k, 128, 0, 7.0, alpha, renorm,
                           score=rse.MOE_SCORE_SOFTMAX if softmax else rse.MOE_SCORE_SIGMOID, num_groups=groups,
                           top_groups=top, group_score=rse.MOE_GROUP_MAX if group_max else rse.MOE_GROUP_SUM2)


def run(cfg, z, bias):
    T = z.shape[0]
    ids = torch.full((T, cfg.top_k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, cfg.top_k), math.nan, device="cuda")
    rse.moe_gate_topk(cfg, z, bias, ids, w)
    torch.cuda.synchronize()
    return ids.cpu().long(), w.cpu().double()


def check(z, bias, k, softmax=False, groups=1, top=1, group_max=False, renorm=True, alpha=2.5):
    cfg = config(z.shape[1], k, softmax, groups, top, group_max, renorm, alpha)
    ids, w = run(cfg, z.cuda(), None if bias is None else bias.cuda())
    want_ids, want_w = go.gate_select(z, bias, k, alpha, renorm, softmax, groups, top, group_max)
    assert torch.equal(ids, want_ids)
    assert torch.allclose(w, want_w, rtol=RTOL, atol=1e-37)


# E, k, groups, top: lanes with one expert to 32, groups on whole lanes, on
# odd chunks (20 = 5 x 4, 21 = 7 x 3), and a size no chunk divides (37)
SHAPES = [(1, 1, 1, 1), (2, 2, 1, 1), (8, 3, 4, 2), (31, 5, 1, 1), (64, 6, 1, 1), (72, 7, 2, 1), (100, 16, 5, 3),
          (160, 6, 8, 3), (168, 8, 8, 4), (148, 8, 4, 2), (256, 8, 8, 4), (256, 8, 1, 1), (512, 10, 16, 16), (1024, 16, 1, 1),
          (1024, 16, 32, 5), (37, 4, 37 // 37, 1), (64, 2, 32, 1), (6, 6, 3, 3)]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,k,groups,top", SHAPES)
def test_selection_matches_oracle(E, k, groups, top, softmax):
    g = torch.Generator().manual_seed(E * 31 + k)
    for T, biased, group_max, renorm in ((1, True, False, True), (37, False, False, False), (130, True, True, True),
                                         (9, False, True, True)):
        z = torch.randn(T, E, generator=g) * 2
        bias = torch.rand(E, generator=g) * 0.4 - 0.2 if biased else None
        check(z, bias, k, softmax, groups, top, group_max, renorm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types_and_row_strides(dtype):
    g = torch.Generator().manual_seed(3)
    wide = (torch.randn(50, 203, generator=g) * 2).to(dtype)
    bias = torch.rand(96, generator=g) * 0.2
    for at in (0, 1, 8, 107):               # odd offsets: rows aligned to their element only
        z = wide.cuda()[:, at:at + 96]
        ids, w = run(config(96, 6, groups=4, top=2), z, bias.cuda())
        want_ids, want_w = go.gate_select(wide[:, at:at + 96], bias, 6, 2.5, True, groups=4, top_groups=2)
        assert torch.equal(ids, want_ids) and torch.allclose(w, want_w, rtol=RTOL)


def test_ties_and_near_ties_follow_the_exact_order():
    g = torch.Generator().manual_seed(5)
    # bf16 logits: many equal ones; with a zero bias the same order as without
    z = (torch.randn(200, 256, generator=g)).to(torch.bfloat16)
    for bias in (None, torch.zeros(256)):
        for softmax in (False, True):
            check(z, bias, 8, softmax)
            check(z, bias, 8, softmax, groups=8, top=3)
    # biased scores closer than fp32 can tell apart: bias = c - sigmoid(l) rounded to fp32
    z = torch.randn(64, 64, generator=g)
    for row in range(0, 64, 8):
        bias = (0.7 - 1 / (1 + torch.exp(-z[row].double()))).float()
        check(z[row:row + 1], bias, 6)
        check(z[row:row + 1], bias, 6, groups=8, top=4)
    # all logits equal: the lowest ids
    check(torch.zeros(5, 256), None, 8)
    check(torch.zeros(5, 256), torch.zeros(256), 8, groups=8, top=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group_max", [False, True])
def test_close_values_everywhere(group_max, dtype):
    """Logits on a coarse grid and biases of a few 1e-7: most borders, between
    groups, at the k-th place and inside, are closer than fp32 scores can tell."""
    g = torch.Generator().manual_seed(11)
    for E, groups, top, k, grid in ((256, 8, 4, 8, 8), (64, 16, 3, 6, 2), (160, 8, 3, 16, 16), (96, 12, 5, 8, 4),
                                    (256, 32, 20, 8, 1), (1024, 8, 2, 16, 16), (64, 64 // 64, 1, 6, 4)):
        z = ((torch.randn(150, E, generator=g) * grid).round() / grid).to(dtype)
        for width in (1e-7, 3e-6):
            bias = torch.randn(E, generator=g) * width
            check(z, bias, k, groups=groups, top=top, group_max=group_max)
            check(z[:20], bias, k, True, groups, top, group_max)
        check(z, None, k, groups=groups, top=top, group_max=group_max)


def test_more_close_values_than_places():
    """Groups whose sums agree to 1e-8, and 40 experts of one value."""
    g = torch.Generator().manual_seed(12)
    for wide in (3, 40):
        z = torch.randn(1, 256, generator=g)
        target = torch.rand(256, generator=g).double() * 0.3
        target[::32] = 0.9
        target[1::32] = target[2::32] = 0.8
        target[torch.randperm(256, generator=g)[:wide]] = 0.9
        bias = (target - 1 / (1 + torch.exp(-z[0].double()))).float()
        for groups, top in ((1, 1), (8, 4), (8, 1), (16, 9)):
            check(z, bias, 8, groups=groups, top=top)
            check(z, bias, 8, groups=groups, top=top, group_max=True)


def test_saturated_scores_keep_the_order_of_the_logits():
    z = torch.tensor([[200.0, 300.0, 90.0, -200.0, -300.0, 250.0, 0.0, -90.0]])
    check(z, None, 4)
    check(z, None, 8, renorm=False)
    ids, _ = run(config(8, 4, softmax=True), z.cuda(), None)
    assert ids.tolist() == [[1, 5, 0, 2]]


@pytest.mark.parametrize("softmax", [False, True])
def test_masked_experts_and_empty_rows(softmax):
    g = torch.Generator().manual_seed(6)
    z = torch.randn(12, 64, generator=g)
    z[0] = -math.inf                         # nothing left
    z[1, 3:] = -math.inf                     # fewer left than k
    z[2, ::2] = -math.inf
    z[3] = torch.finfo(torch.float32).min
    z[4, 5:] = torch.finfo(torch.float32).min
    check(z, None, 6, softmax)
    check(z, None, 6, softmax, renorm=False)
    check(z, torch.rand(64, generator=g) * 0.1, 6, softmax, groups=4, top=2)


def test_nan_and_infinite_logits_give_valid_ids():
    g = torch.Generator().manual_seed(7)
    z = torch.randn(40, 96, generator=g)
    z[0, 7] = math.nan
    z[1] = math.nan
    z[2, 50:60] = math.inf
    z[3, 9], z[3, 11] = math.nan, math.inf
    for softmax in (False, True):
        for bias in (None, torch.rand(96, generator=g)):
            for groups, top in ((1, 1), (8, 3)):
                cfg = config(96, 8, softmax, groups, top)
                ids, w = run(cfg, z.cuda(), None if bias is None else bias.cuda())
                assert int(ids.min()) >= 0 and int(ids.max()) < 96
                assert all(len(set(r)) == 8 for r in ids.tolist())
                if bias is None and groups == 1:
                    assert ids[0, 0] == 7 and ids[3, :2].tolist() == [9, 11] and ids[1].tolist() == list(range(8))
                # the rows without them are as ever
                want, ww = go.gate_select(z[4:], bias, 8, 2.5, True, softmax, groups, top)
                assert torch.equal(ids[4:], want) and torch.allclose(w[4:], ww, rtol=RTOL)


def test_infinite_bias_switches_experts_off():
    g = torch.Generator().manual_seed(8)
    z = torch.randn(30, 64, generator=g)
    bias = torch.zeros(64)
    bias[::3] = -math.inf
    check(z, bias, 8)
    check(z, bias, 8, groups=8, top=2, group_max=True)


def test_graph_replay_on_a_side_stream():
    g = torch.Generator().manual_seed(9)
    cfg = config(256, 8, groups=8, top=4)
    z = [torch.randn(33, 256, generator=g) for _ in range(2)]
    bias = torch.rand(256, generator=g).cuda() * 0.1
    zin = z[0].cuda()
    ids = torch.empty(33, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(33, 8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rse.moe_gate_topk(cfg, zin, bias, ids, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            rse.moe_gate_topk(cfg, zin, bias, ids, w)
    torch.cuda.current_stream().wait_stream(s)
    for v in z:
        zin.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want, ww = go.gate_select(v, bias.cpu(), 8, 2.5, True, groups=8, top_groups=4)
        assert torch.equal(ids.cpu().long(), want) and torch.allclose(w.cpu().double(), ww, rtol=RTOL)


ROUTED = {"softmax": dict(score=rse.MOE_SCORE_SOFTMAX),
          "groups": dict(num_groups=4, top_groups=2),
          "softmax_groups_max": dict(score=rse.MOE_SCORE_SOFTMAX, num_groups=8, top_groups=3, group_score=rse.MOE_GROUP_MAX)}


@pytest.mark.parametrize("T", [1, 64, 1500])
@pytest.mark.parametrize("name", sorted(ROUTED))
def test_layer_routes_as_configured(name, T):
    """The layer's own router with the same choices: the selection of its
    fp32 logits (near-ties of the fp64 logits within 1e-5 of the border are
    left out), and the whole layer on those ids."""
    kw = ROUTED[name]
    cfg = LayerConfig("routed", T=T, H=256, E=16, k=3, I=128, I_s=64, alpha=2.5, renorm=True)
    inp = moe_inputs.make_layer(cfg, seed=1)
    base = gpu_layer(inp)
    layer = rse.MoELayer(hidden=cfg.H, num_experts=cfg.E, top_k=cfg.k, expert_inter=cfg.I, shared_inter=cfg.I_s,
                         swiglu_limit=cfg.swiglu_limit, routed_scaling_factor=cfg.alpha, renormalize=cfg.renorm,
                         max_tokens=T, **base.tensors, **kw)
    x = inp.x.cuda()
    ids = torch.empty(T, cfg.k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, cfg.k, device="cuda")
    out = layer.forward(x, topk_ids=ids, topk_w=w)
    torch.cuda.synchronize()
    z = oracle.router_logits(inp.x, inp.router_w)
    sel = dict(softmax=kw.get("score") == rse.MOE_SCORE_SOFTMAX, groups=kw.get("num_groups", 1),
               top_groups=kw.get("top_groups", 1), group_max=kw.get("group_score") == rse.MOE_GROUP_MAX)
    want, ww = go.gate_select(z, inp.correction_bias, cfg.k, cfg.alpha, True, **sel)
    same = (ids.cpu().long() == want).all(dim=1)
    # fp32 logits err by about 1e-6 here: some border is that close in few of T * 16 scores
    assert int((~same).sum()) <= T * 16 * 1e-4
    # logits off by 1e-6 move a weight by at most about 2e-6 of itself
    assert torch.allclose(w.cpu().double()[same], ww[same], rtol=2e-5, atol=0)
    res = oracle.moe_forward(inp, ids_override=ids.cpu().long())
    y = torch.zeros(T, cfg.H, dtype=torch.float64) + res.shared
    rows = res.perm.row_of.view(T, cfg.k)
    for j in range(cfg.k):
        y += w.cpu().double()[:, j:j + 1] * res.y_perm[rows[:, j]]
    assert float((out.cpu().double() - y).abs().max()) <= 2e-2 * float(y.abs().max())
    # the staged router call and a one-rank expert-parallel layer take the same route
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    rse.moe_router_topk(layer.cfg, layer.w, x, T, ids2, w2, layer.ws)
    one = ep.ExpertParallelLayer(hidden=cfg.H, num_experts=cfg.E, top_k=cfg.k, expert_inter=cfg.I, shared_inter=cfg.I_s,
                                 swiglu_limit=cfg.swiglu_limit, routed_scaling_factor=cfg.alpha,
                                 renormalize=cfg.renorm, max_tokens=T, **base.tensors, **kw)
    part = one.forward_partial(x)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(part, out)


def test_logits_far_apart():
    """Rows whose offsets pass 32 bits."""
    T, E, stride = 9, 64, 300_000_000
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").as_strided((T, E), (stride, 1))
    wide.copy_(z.cuda())
    ids, w = run(config(E, 6, softmax=True), wide, None)
    want_ids, want_w = go.gate_select(z, None, 6, 2.5, True, True, 1, 1, False)
    assert torch.equal(ids, want_ids)
    assert torch.allclose(w, want_w, rtol=RTOL, atol=1e-37)
