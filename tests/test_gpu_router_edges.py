"""The layer's own router with softmax scores or groups at the ends of its
ranges: one expert, 1024 of them, the shortest rows, equal experts, rows that
overflow, many calls at once."""

import pytest
import torch

import oracle
import routed_swiglu_experts_b200 as rse
from oracle import gate_fp8_oracle as go
from test_gpu_router_exact import MAX, ROUTES, SOFTMAX, check, inputs, route

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,H,E,k,kw", [
    (5, 8, 1, 1, dict(score=SOFTMAX)),
    (3, 8, 2, 1, dict(num_groups=2, top_groups=1)),
    (9, 16, 4, 2, dict(score=SOFTMAX, num_groups=4, top_groups=2)),
    (33, 264, 33, 16, dict(score=SOFTMAX)),
    (21, 136, 1024, 16, dict(score=SOFTMAX)),
    (21, 136, 1024, 16, dict(num_groups=32, top_groups=5)),
    (21, 136, 1024, 16, dict(score=SOFTMAX, num_groups=32, top_groups=20, group_score=MAX)),
    (19, 72, 992, 16, dict(num_groups=31, top_groups=7)),           # 32 experts a group, one lane
    (19, 72, 999, 9, dict(num_groups=27, top_groups=2)),            # 37: no run of lanes
    (19, 72, 999, 9, dict(score=SOFTMAX, num_groups=27, top_groups=2)),
])
def test_shapes(T, H, E, k, kw, biased):
    x, w, bias = inputs(T, H, E, kw.get("num_groups", 1), E, 1e-6, biased)
    check(x, w, bias, k, kw)


@pytest.mark.parametrize("name", sorted(ROUTES))
def test_equal_experts_tie_to_the_lower_id(name):
    g = torch.Generator().manual_seed(6)
    base = torch.randn(8, 512, generator=g) / 512 ** 0.5
    pick = torch.randint(0, 8, (64,), generator=g)
    x = torch.randn(50, 512, generator=g).to(torch.bfloat16)
    z = oracle.router_logits(x, base)[:, pick]          # equal experts: equal logits
    b8 = torch.rand(8, generator=g) * 0.2
    for bias in (None, b8[pick].contiguous()):
        kw = ROUTES[name]
        ids, _ = route(x.cuda(), base[pick].contiguous().cuda(), None if bias is None else bias.cuda(), 6, kw)
        want, _ = go.gate_select(z, bias, 6, 2.5, True, kw.get("score") == SOFTMAX, kw.get("num_groups", 1),
                                 kw.get("top_groups", 1), kw.get("group_score") == MAX)
        assert torch.equal(ids, want)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("name", sorted(ROUTES))
def test_rows_that_overflow_keep_to_themselves(name, biased):
    x, w, bias = inputs(40, 256, 64, ROUTES[name].get("num_groups", 1), 3, 1e-6, biased)
    big = x.clone()
    big[3, 5] = float("inf")
    big[11] = torch.finfo(torch.bfloat16).max
    big[12, 3] = float("-inf")
    dev = None if bias is None else bias.cuda()
    ids, _ = route(big.cuda(), w.cuda(), dev, 6, ROUTES[name])
    clean, _ = route(x.cuda(), w.cuda(), dev, 6, ROUTES[name])
    assert 0 <= int(ids.min()) and int(ids.max()) < 64 and all(len(set(r)) == 6 for r in ids.tolist())
    rest = [t for t in range(40) if t not in (3, 11, 12)]
    assert torch.equal(ids[rest], clean[rest])


def test_two_streams_and_a_graph():
    """Calls in flight at once, a workspace each, and a replayed graph give the ids they give alone."""
    kw = dict(score=SOFTMAX, num_groups=4, top_groups=2)
    sets = []
    for seed in (1, 2):
        x, w, bias = inputs(500, 512, 64, 4, seed, 1e-6, True)
        T, H = x.shape
        cfg = rse.make_config(H, 64, 6, 128, 0, 7.0, 2.5, True, **kw)
        ws = torch.empty(rse.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
        rse.moe_workspace_init(ws)
        dev = (x.cuda(), w.cuda(), bias.cuda())
        ids, tw = torch.empty(T, 6, dtype=torch.int32, device="cuda"), torch.empty(T, 6, device="cuda")
        sets.append((cfg, rse.make_weights(router_w=dev[1], correction_bias=dev[2]), dev[0], T, ids, tw, ws, dev))
    alone = []
    for s in sets:
        rse.moe_router_topk(*s[:7])
        alone.append((s[4].clone(), s[5].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        rse.moe_router_topk(*sets[0][:7])
    for s in sets:
        s[4].fill_(-7)
        s[5].fill_(-7)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            rse.moe_router_topk(*sets[1][:7])
    torch.cuda.synchronize()
    for s, (ids, tw) in zip(sets, alone):
        assert torch.equal(s[4], ids) and torch.equal(s[5], tw)
