"""Request adapters against fp64.

With P the sum of an output's products' magnitudes (|base| among them), an
element's error is at most: K + rank fp32 additions, a last place (2^-23) each,
(K + rank) 2^-23 P; A x carried as two values of x_type, 2^-16 P; half a step of
the output, eps / 2 |out|.
In the 2-norm over a call, where the errors of single additions do not all
point one way and partial sums are no larger than the final ones: 2^-16 for
the split, 2^-23 for each of the K / 16 + rank / 16 steps of a matrix
instruction, 2^-14 covers both for K up to 6144; and eps / 2."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import around_oracle as ao

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def workspace():
    ws = torch.empty(rse.MOE_WS_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    rse.moe_workspace_init(ws)
    return ws


def plan_of(ids, L):
    plan = torch.empty(rse.moe_lora_plan_size(ids.shape[0], L), dtype=torch.uint8, device="cuda")
    rse.moe_lora_plan(ids.to(torch.int32).cuda(), L, plan)
    return plan


def inputs(T, K, N, r, L, dtype, out_type, seed, none=0.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).to(dtype)
    a = (torch.randn(L, r, K, generator=g) / math.sqrt(K)).to(dtype)
    b = torch.randn(L, N, r, generator=g).to(dtype)
    scale = 0.5 + torch.rand(L, generator=g)
    ids = torch.randint(0, L, (T,), generator=g)
    ids[torch.rand(T, generator=g) < none] = -1
    base = torch.randn(T, N, generator=g).to(out_type)
    return x, a, b, scale, ids, base


def check(out, want, size, K, r):
    half = torch.finfo(out.dtype).eps / 2
    got = out.cpu().double()
    err = (got - want).abs()
    bound = size * ((K + r) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * half * (1 + 2.0 ** -6) + (2.0 ** -25 if out.dtype == F16 else 0)
    assert bool((err <= bound).all()), float((err - bound).max())
    norm = float(want.norm())
    assert float((got - want).norm()) <= norm * (2.0 ** -14 + half) + 2.0 ** -25 * math.sqrt(want.numel()), float((got - want).norm()) / norm


def run(x, a, b, scale, ids, base, out_type, L):
    out = torch.full((x.shape[0], b.shape[1]), 7.0, dtype=out_type, device="cuda")
    ws = workspace()
    rse.moe_lora(x.cuda(), a.cuda(), b.cuda(), None if scale is None else scale.cuda(), plan_of(ids, L),
                 None if base is None else base.cuda(), out, ws)
    assert rse.moe_read_device_error(ws) == 0
    return out


@pytest.mark.parametrize("dtype,out_type", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,K,N,r,L", [(1, 8, 1, 8, 1), (1, 6144, 256, 16, 4), (3, 72, 33, 8, 2), (16, 200, 130, 24, 5),
                                       (65, 512, 257, 16, 3), (130, 136, 128, 128, 2), (200, 1000, 300, 40, 7),
                                       (300, 264, 640, 64, 2), (129, 64, 24, 88, 1)])
def test_sizes(T, K, N, r, L, dtype, out_type):
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, T * K + N)
    want, size = ao.lora(x, a, b, scale, ids, base)
    check(run(x, a, b, scale, ids, base, out_type, L), want, size, K, r)


@pytest.mark.parametrize("kind", ["one", "none", "each", "first", "out of range"])
def test_who_has_which_adapter(kind):
    T, K, N, r, L = 150, 128, 96, 16, 150
    x, a, b, scale, _, base = inputs(T, K, N, r, L, BF16, BF16, 4)
    ids = {"one": torch.full((T,), L - 1), "none": torch.full((T,), -1), "each": torch.randperm(T, generator=torch.Generator().manual_seed(1)),
           "first": torch.arange(T).clamp(max=1), "out of range": torch.where(torch.arange(T) % 3 == 0, L, torch.where(torch.arange(T) % 3 == 1, -2 ** 31, 5))}[kind]
    want, size = ao.lora(x, a, b, scale, ids, base)
    out = run(x, a, b, scale, ids, base, BF16, L)
    check(out, want, size, K, r)
    without = (ids < 0) | (ids >= L)
    assert torch.equal(out.cpu()[without], base[without])


def test_plan_orders_tokens_by_adapter():
    g = torch.Generator().manual_seed(2)
    for T, L in ((1, 1), (31, 4), (33, 1), (1000, 7), (5000, 1024), (70000, 3)):
        ids = torch.randint(-1, L, (T,), generator=g)
        plan = plan_of(ids, L).cpu()
        head = plan[:32].view(torch.int32)
        src = plan[32:32 + 4 * T].view(torch.int32).long()
        key = torch.where(ids < 0, L, ids)
        assert torch.equal(src, torch.sort(key, stable=True).indices)
        at = 32 + (4 * T + 15) // 16 * 16
        tiles = plan[at:at + 16 * int(head[3])].view(torch.int32).view(-1, 4).long()
        assert head[1:3].tolist() == [T, L]
        pos = 0
        for adapter, row0, rows, _ in tiles.tolist():
            assert row0 == pos and 1 <= rows <= int(head[4])
            assert bool((key[src[row0:row0 + rows]] == (L if adapter < 0 else adapter)).all())
            pos += rows
        assert pos == T
        # no more tiles than each adapter's rows need
        counts = torch.bincount(key, minlength=L + 1)
        assert len(tiles) == int(((counts + int(head[4]) - 1) // int(head[4])).sum())


def test_without_base_and_without_scale():
    x, a, b, scale, ids, base = inputs(40, 96, 72, 16, 3, BF16, F32, 5)
    for sc, bs in ((None, base), (scale, None), (None, None)):
        want, size = ao.lora(x, a, b, sc, ids, bs)
        out = run(x, a, b, sc, ids, bs, F32, 3)
        check(out, want, size, 96, 16)
        if bs is None:
            assert bool((out.cpu()[ids < 0] == 0).all())


@pytest.mark.parametrize("out_type", [BF16, F32])
def test_in_place_strided_and_untouched_neighbours(out_type):
    x, a, b, scale, ids, base = inputs(37, 120, 51, 8, 4, BF16, out_type, 6)
    want, size = ao.lora(x, a, b, scale, ids, base)
    wide = torch.full((37, 77), 9.0, dtype=out_type, device="cuda")
    view = wide[:, 13:13 + 51]
    view.copy_(base)
    xw = torch.full((37, 200), float("nan"), dtype=BF16, device="cuda")
    xw[:, 16:136] = x.cuda()
    rse.moe_lora(xw[:, 16:136], a.cuda(), b.cuda(), scale.cuda(), plan_of(ids, 4), view, view, workspace())
    check(view, want, size, 120, 8)
    assert bool((wide[:, :13] == 9).all()) and bool((wide[:, 64:] == 9).all())
    # another place, with strides of its own on both sides
    src = torch.full((37, 60), 9.0, dtype=out_type, device="cuda")
    src[:, 2:53] = base.cuda()
    dst = torch.full((37, 90), 9.0, dtype=out_type, device="cuda")
    rse.moe_lora(x.cuda(), a.cuda(), b.cuda(), scale.cuda(), plan_of(ids, 4), src[:, 2:53], dst[:, 5:56], workspace())
    assert torch.equal(dst[:, 5:56], view)
    assert bool((dst[:, :5] == 9).all()) and bool((dst[:, 56:] == 9).all())


def test_a_bad_token_stays_alone():
    x, a, b, scale, ids, base = inputs(50, 128, 64, 16, 2, BF16, BF16, 7, none=0.0)
    x[7, 3], x[20, 5], base[30, 2] = math.nan, math.inf, math.nan
    want, size = ao.lora(x, a, b, scale, ids, base)
    out = run(x, a, b, scale, ids, base, BF16, 2)
    good = torch.ones(50, dtype=torch.bool)
    good[[7, 20, 30]] = False
    check(out[good.cuda()], want[good], size[good], 128, 16)
    assert bool(torch.isnan(out[7]).all()) and not bool(torch.isfinite(out[20]).any())
    fine = torch.ones(64, dtype=torch.bool)
    fine[2] = False
    check(out[30:31, fine.cuda()], want[30:31, fine], size[30:31, fine], 128, 16)
    assert bool(torch.isnan(out[30, 2]))


@pytest.mark.parametrize("out_type", [F16, F32])
def test_fp16_ranges(out_type):
    """A x outside fp16's range, and far below its smallest normal value, while the result is inside."""
    for up in (2.0 ** 10, 2.0 ** -14):
        x, a, b, scale, ids, base = inputs(20, 256, 40, 16, 2, F16, out_type, 8, none=0.0)
        x = (x * 64 * min(up, 1.0)).to(F16)
        a = (a * 16 * max(up, 1.0)).to(F16)
        b = (b * 2.0 ** -10).to(F16)
        scale = scale * (2.0 ** -8 if up > 1 else 2.0 ** 6)
        base.zero_()
        want, size = ao.lora(x, a, b, scale, ids, base)
        assert float(want.abs().max()) < 6e4
        check(run(x, a, b, scale, ids, base, out_type, 2), want, size, 256, 16)


def test_adapters_of_other_tokens_are_not_read():
    """NaN in the adapters that no token has."""
    x, a, b, scale, _, base = inputs(30, 64, 32, 8, 6, BF16, BF16, 9)
    ids = torch.full((30,), 2)
    ids[10:20] = -1
    want, size = ao.lora(x, a, b, scale, ids, base)
    for other in (0, 1, 3, 4, 5):
        a[other], b[other], scale[other] = math.nan, math.nan, math.nan
    x[10:20] = math.nan                                           # nor the rows of tokens without one
    check(run(x, a, b, scale, ids, base, BF16, 6), want, size, 64, 8)


def test_a_plan_for_other_sizes_is_reported():
    x, a, b, scale, ids, base = inputs(24, 64, 32, 8, 4, BF16, BF16, 10)
    other = plan_of(torch.zeros(23), 4)
    plan = torch.zeros(rse.moe_lora_plan_size(24, 4), dtype=torch.uint8, device="cuda")
    plan[:other.numel()] = other[:plan.numel()]
    for p in (plan, torch.zeros_like(plan)):
        ws = workspace()
        out = torch.full((24, 32), 7.0, dtype=BF16, device="cuda")
        rse.moe_lora(x.cuda(), a.cuda(), b.cuda(), scale.cuda(), p, base.cuda(), out, ws)
        assert rse.moe_read_device_error(ws) == rse.MOE_ERR_INVALID_ARG
        assert bool((out == 7).all())


def test_weights_past_32_bits():
    """The last adapter starts past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    L, r, K, N, T = 530, 128, 32768, 256, 5
    g = torch.Generator().manual_seed(3)
    a = torch.zeros(L, r, K, dtype=BF16, device="cuda")
    b = torch.zeros(L, N, r, dtype=BF16, device="cuda")
    a[-1] = (torch.randn(r, K, generator=g) / math.sqrt(K)).to(BF16).cuda()
    b[-1] = torch.randn(N, r, generator=g).to(BF16).cuda()
    x = torch.randn(T, K, generator=g).to(BF16)
    ids = torch.full((T,), L - 1)
    out = torch.empty(T, N, device="cuda")
    rse.moe_lora(x.cuda(), a, b, None, plan_of(ids, L), None, out, workspace())
    want, size = ao.lora(x, a[-1:].cpu(), b[-1:].cpu(), None, torch.zeros(T), None)
    half = 2.0 ** -24
    err = (out.cpu().double() - want).abs()
    assert bool((err <= size * ((K + r) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * half).all())
    assert float(err.norm()) <= float(want.norm()) * 2.0 ** -11       # (K / 16 steps of 2^-23)


def test_same_results_each_time_in_a_graph_and_on_two_streams():
    x, a, b, scale, ids, base = inputs(180, 512, 384, 32, 5, BF16, F32, 12)
    d = [t.cuda() for t in (x, a, b, scale, base)]
    plan, ws = plan_of(ids, 5), workspace()
    want, size = ao.lora(x, a, b, scale, ids, base)
    outs = [torch.empty(180, 384, device="cuda") for _ in range(4)]
    rse.moe_lora(d[0], d[1], d[2], d[3], plan, d[4], outs[0], ws)
    check(outs[0], want, size, 512, 32)
    ids_d = ids.to(torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rse.moe_lora_plan(ids_d, 5, plan)
        rse.moe_lora(d[0], d[1], d[2], d[3], plan, d[4], outs[1], ws)
    for _ in range(3):
        outs[1].zero_()
        graph.replay()
        assert torch.equal(outs[0], outs[1])
    # another batch through the same graph
    ids2 = torch.roll(ids, 50)
    ids_d.copy_(ids2)
    graph.replay()
    want2, size2 = ao.lora(x, a, b, scale, ids2, base)
    check(outs[1], want2, size2, 512, 32)
    plan0 = plan_of(ids, 5)
    streams, wss = [torch.cuda.Stream() for _ in range(2)], [workspace(), workspace()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, wss, outs[2:]):
            rse.moe_lora(d[0], d[1], d[2], d[3], plan0, d[4], o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[0]) and torch.equal(outs[3], outs[0])
