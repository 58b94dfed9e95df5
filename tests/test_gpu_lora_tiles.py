"""Request adapters on batches of more than 512 tokens (tiles of up to 128 of
them), against fp64: the bounds of test_gpu_lora."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import around_oracle as ao

from gpu_util import cuda_available
from test_gpu_lora import BF16, F16, F32, check, inputs, plan_of, run, workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype,out_type", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,K,N,r,L", [(513, 8, 1, 8, 1), (600, 64, 130, 16, 3), (700, 72, 33, 32, 2), (513, 1000, 257, 24, 40),
                                       (900, 520, 1100, 64, 2), (640, 136, 128, 128, 3), (777, 328, 264, 88, 5),
                                       (1300, 200, 520, 16, 600), (2049, 128, 96, 8, 1)])
def test_sizes(T, K, N, r, L, dtype, out_type):
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, T * K + N)
    want, size = ao.lora(x, a, b, scale, ids, base)
    check(run(x, a, b, scale, ids, base, out_type, L), want, size, K, r)


@pytest.mark.parametrize("r", [16, 64, 128])
@pytest.mark.parametrize("kind", ["one", "none", "each", "blocks of 129", "out of range"])
def test_who_has_which_adapter(kind, r):
    T, K, N, L = 650, 192, 200, 650
    x, a, b, scale, _, base = inputs(T, K, N, r, L, BF16, BF16, 4)
    t = torch.arange(T)
    ids = {"one": torch.full((T,), L - 1), "none": torch.full((T,), -1), "each": torch.randperm(T, generator=torch.Generator().manual_seed(1)),
           "blocks of 129": t // 129, "out of range": torch.where(t % 3 == 0, L, torch.where(t % 3 == 1, -2 ** 31, 5))}[kind]
    want, size = ao.lora(x, a, b, scale, ids, base)
    out = run(x, a, b, scale, ids, base, BF16, L)
    check(out, want, size, K, r)
    without = (ids < 0) | (ids >= L)
    assert torch.equal(out.cpu()[without], base[without])


def test_without_base_and_without_scale():
    x, a, b, scale, ids, base = inputs(540, 96, 72, 16, 3, BF16, F32, 5)
    for sc, bs in ((None, base), (scale, None), (None, None)):
        want, size = ao.lora(x, a, b, sc, ids, bs)
        out = run(x, a, b, sc, ids, bs, F32, 3)
        check(out, want, size, 96, 16)
        if bs is None:
            assert bool((out.cpu()[ids < 0] == 0).all())


@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("at", [13, 16])     # rows off 16-byte boundaries, and on them
def test_in_place_strided_and_untouched_neighbours(out_type, at):
    T, N, wide_n = 530, 150, 192
    x, a, b, scale, ids, base = inputs(T, 120, N, 8, 4, BF16, out_type, 6)
    want, size = ao.lora(x, a, b, scale, ids, base)
    wide = torch.full((T, wide_n), 9.0, dtype=out_type, device="cuda")
    view = wide[:, at:at + N]
    view.copy_(base)
    xw = torch.full((T, 200), float("nan"), dtype=BF16, device="cuda")
    xw[:, 16:136] = x.cuda()
    rse.moe_lora(xw[:, 16:136], a.cuda(), b.cuda(), scale.cuda(), plan_of(ids, 4), view, view, workspace())
    check(view, want, size, 120, 8)
    assert bool((wide[:, :at] == 9).all()) and bool((wide[:, at + N:] == 9).all())
    src = torch.full((T, 160), 9.0, dtype=out_type, device="cuda")
    src[:, 8:8 + N] = base.cuda()
    dst = torch.full((T, wide_n), 9.0, dtype=out_type, device="cuda")
    rse.moe_lora(x.cuda(), a.cuda(), b.cuda(), scale.cuda(), plan_of(ids, 4), src[:, 8:8 + N], dst[:, at:at + N], workspace())
    assert torch.equal(dst[:, at:at + N], view)
    assert bool((dst[:, :at] == 9).all()) and bool((dst[:, at + N:] == 9).all())


@pytest.mark.parametrize("r", [16, 64])
def test_a_bad_token_stays_alone(r):
    x, a, b, scale, ids, base = inputs(600, 128, 264, r, 2, BF16, BF16, 7, none=0.0)
    x[7, 3], x[500, 5], base[30, 2] = math.nan, math.inf, math.nan
    want, size = ao.lora(x, a, b, scale, ids, base)
    out = run(x, a, b, scale, ids, base, BF16, 2)
    good = torch.ones(600, dtype=torch.bool)
    good[[7, 500, 30]] = False
    check(out[good.cuda()], want[good], size[good], 128, r)
    assert bool(torch.isnan(out[7]).all()) and not bool(torch.isfinite(out[500]).any())
    fine = torch.ones(264, dtype=torch.bool)
    fine[2] = False
    check(out[30:31, fine.cuda()], want[30:31, fine], size[30:31, fine], 128, r)
    assert bool(torch.isnan(out[30, 2]))


def test_adapters_of_other_tokens_are_not_read():
    x, a, b, scale, _, base = inputs(600, 64, 32, 8, 6, BF16, BF16, 9)
    ids = torch.full((600,), 2)
    ids[100:200] = -1
    want, size = ao.lora(x, a, b, scale, ids, base)
    for other in (0, 1, 3, 4, 5):
        a[other], b[other], scale[other] = math.nan, math.nan, math.nan
    x[100:200] = math.nan
    check(run(x, a, b, scale, ids, base, BF16, 6), want, size, 64, 8)


@pytest.mark.parametrize("out_type", [F16, F32])
def test_fp16_ranges(out_type):
    for up in (2.0 ** 10, 2.0 ** -14):
        x, a, b, scale, ids, base = inputs(520, 256, 40, 16, 2, F16, out_type, 8, none=0.0)
        x = (x * 64 * min(up, 1.0)).to(F16)
        a = (a * 16 * max(up, 1.0)).to(F16)
        b = (b * 2.0 ** -10).to(F16)
        scale = scale * (2.0 ** -8 if up > 1 else 2.0 ** 6)
        base.zero_()
        want, size = ao.lora(x, a, b, scale, ids, base)
        assert float(want.abs().max()) < 6e4
        check(run(x, a, b, scale, ids, base, out_type, 2), want, size, 256, 16)


def test_a_plan_for_other_sizes_is_reported():
    x, a, b, scale, ids, base = inputs(600, 64, 32, 8, 4, BF16, BF16, 10)
    for p in (torch.zeros(rse.moe_lora_plan_size(600, 4), dtype=torch.uint8, device="cuda"), plan_of(torch.zeros(601), 4)):
        ws = workspace()
        out = torch.full((600, 32), 7.0, dtype=BF16, device="cuda")
        rse.moe_lora(x.cuda(), a.cuda(), b.cuda(), scale.cuda(), p, base.cuda(), out, ws)
        assert rse.moe_read_device_error(ws) == rse.MOE_ERR_INVALID_ARG
        assert bool((out == 7).all())


def reference(x, a, b, scale, ids, base):
    """fp64 on the device, adapter by adapter (for sizes that the plain loops take too long on)."""
    out, size = base.double(), base.double().abs()
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i).view(-1)
        if rows.numel():
            xi, ai, bi, c = x[rows].double(), a[i].double(), b[i].double(), float(scale[i])
            out[rows] += c * (xi @ ai.t() @ bi.t())
            size[rows] += c * (xi.abs() @ ai.abs().t() @ bi.abs().t())
    return out, size


@pytest.mark.parametrize("T,K,N,r,L", [(4096, 2048, 1408, 16, 4), (8192, 1024, 2048, 64, 30), (16384, 512, 1000, 32, 100),
                                       (5000, 6144, 640, 128, 9)])
def test_large_batches(T, K, N, r, L):
    """Clusters of every size, several tiles a cluster."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    a = (torch.randn(L, r, K, generator=g, device="cuda") / math.sqrt(K)).to(BF16)
    b = torch.randn(L, N, r, generator=g, device="cuda").to(BF16)
    scale, base = torch.rand(L, generator=g, device="cuda"), torch.randn(T, N, generator=g, device="cuda")
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda")
    want, size = reference(x, a, b, scale, ids, base)
    out, ws = torch.empty_like(base), workspace()
    for _ in range(2):
        out.fill_(7)
        rse.moe_lora(x, a, b, scale, plan_of(ids, L), base, out, ws)
        assert rse.moe_read_device_error(ws) == 0
        check(out, want.cpu(), size.cpu(), K, r)


def test_same_results_each_time_in_a_graph_and_on_two_streams():
    x, a, b, scale, ids, base = inputs(700, 512, 384, 32, 5, BF16, F32, 12)
    d = [t.cuda() for t in (x, a, b, scale, base)]
    plan, ws = plan_of(ids, 5), workspace()
    want, size = ao.lora(x, a, b, scale, ids, base)
    outs = [torch.empty(700, 384, device="cuda") for _ in range(4)]
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


def test_beside_the_layers_tensor_core_kernels_on_another_stream():
    """Blocks of both share SMs, shared memory and tensor memory."""
    g = torch.Generator(device="cuda").manual_seed(5)
    F8 = torch.float8_e4m3fn
    qa = torch.randn(2048, 2048, generator=g, device="cuda").to(F8)
    qw = torch.randn(1, 2048, 2048, generator=g, device="cuda").to(F8)
    sa, sw = torch.ones(16, 2048, device="cuda"), torch.ones(1, 16, 16, device="cuda")
    y, y0 = torch.empty(2048, 2048, device="cuda"), torch.empty(2048, 2048, device="cuda")
    x, a, b, scale, ids, base = (t.cuda() for t in inputs(1500, 1024, 1024, 64, 4, BF16, BF16, 13))
    plan, ws, ws2 = plan_of(ids, 4), workspace(), workspace()
    out, out0 = torch.empty_like(base), torch.empty_like(base)
    rse.moe_lora(x, a, b, scale, plan, base, out0, ws)
    rse.moe_fp8_gemm(qa, sa, qw, sw, None, None, y0, ws2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(30):
        rse.moe_lora(x, a, b, scale, plan, base, out, ws, stream=streams[0])
        rse.moe_fp8_gemm(qa, sa, qw, sw, None, None, y, ws2, stream=streams[1])
    torch.cuda.synchronize()
    assert rse.moe_read_device_error(ws) == 0 and rse.moe_read_device_error(ws2) == 0
    assert torch.equal(out, out0) and torch.equal(y, y0)
