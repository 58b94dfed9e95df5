"""FP8 block-scaled quantisation, products and experts against the fp64 oracle.

Quantisation is exact: codes and scales are compared bit for bit.
Products: with S the sum of the terms' magnitudes, the 128 fp32 additions of a
block leave at most 128 * 2^-23 S (one unit in the last place each, so that a
truncating adder is covered), the scales and the sum over the blocks
(blocks + 4) * 2^-24 S, and the output's rounding 2^-9 * 2 (bf16, half a step
is 2^-8 relative at most) or 2^-24 |out|.
Experts: the framework's layer bar, max|gpu - oracle| <= 2e-2 max|oracle|, and
in the 2-norm 2^-7: half a bf16 step (2^-8) and as much again for activations
whose fp32 value falls on the other side of an E4M3 border than the fp64 one
(one in 2000 of them, off by a step of 2^-3 at most: sqrt(1/2000) / 8 = 2^-8.5)."""

import math
import time
from types import SimpleNamespace

import pytest
import torch

import oracle
import routed_swiglu_experts_b200 as rse
from oracle import gate_fp8_oracle as go
from routed_swiglu_experts_b200 import ep

from gpu_util import cuda_available, rel_err, run_stages

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

F8 = torch.float8_e4m3fn


def codes(q):
    """Code values in fp64 (the dtype's conversion is exact)."""
    return q.cpu().double()


# ------------------------------------------------------------ quantise ------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 128), (17, 144), (5, 512), (9, 1040), (130, 2000)])
def test_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * K)
    x = (torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-20, 10, (rows, 1), generator=g).float())).to(dtype)
    x[0, :16] = 0
    q = torch.empty(rows, K, dtype=F8, device="cuda")
    s = torch.empty((K + 127) // 128, rows, device="cuda")
    rse.moe_fp8_quantize(x.cuda(), q, s)
    want_q, want_s = go.quantize_rows(x)
    assert torch.equal(s.cpu().double(), want_s)
    assert torch.equal(codes(q), want_q)


def test_rows_gathered_from_strided_tokens():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(40, 304, generator=g).to(torch.bfloat16)
    src = torch.randperm(120, generator=g).to(torch.int32)
    for k, at in ((3, 0), (3, 16), (5, 8)):
        n = 40 * k
        src = torch.randperm(n, generator=g).to(torch.int32)
        q = torch.empty(n, 272, dtype=torch.uint8, device="cuda")
        s = torch.empty(3, n, device="cuda")
        rse.moe_fp8_quantize(wide.cuda()[:, at:at + 272], q, s, src=src.cuda(), src_div=k)
        want_q, want_s = go.quantize_rows(wide[:, at:at + 272][(src // k).long()])
        assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q.view(F8)), want_q)


def test_rows_values_at_the_borders():
    # every tie of the grid under scale 1 (a 448 in the block), zeros, the smallest values
    mid = torch.cat([go._MID, -go._MID, go._CODES, torch.tensor([448.0], dtype=torch.float64)]).float()
    x = torch.zeros(4, 512)
    x[0, : mid.numel()] = mid
    x[0, 127::128] = 448.0
    x[2, 5] = 1e-44
    x[3, 128] = torch.finfo(torch.float32).max
    q = torch.empty(4, 512, dtype=F8, device="cuda")
    s = torch.empty(4, 4, device="cuda")
    rse.moe_fp8_quantize(x.cuda(), q, s)
    want_q, want_s = go.quantize_rows(x)
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q), want_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_of_16_bit_values_at_the_borders(dtype):
    """Every finite value of the type in blocks of its own exponent and below the largest one."""
    every = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(dtype)
    every = every[torch.isfinite(every)]
    x = torch.zeros((every.numel() + 125) // 126, 128, dtype=dtype)
    flat = torch.zeros(x.shape[0] * 126, dtype=dtype)
    flat[:every.numel()] = every
    x[:, :126] = flat.view(-1, 126)
    top = x.clone()
    top[::2, 127] = torch.finfo(dtype).max
    top[1::2, 127] = 1.0
    x = torch.cat([x, top], dim=1)
    q = torch.empty(x.shape[0], 256, dtype=F8, device="cuda")
    s = torch.empty(2, x.shape[0], device="cuda")
    rse.moe_fp8_quantize(x.cuda(), q, s)
    want_q, want_s = go.quantize_rows(x)
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q), want_q)


def test_one_row_of_any_stride():
    wide = torch.randn(3, 77, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x = wide.cuda()[:1, :64]
    q = torch.empty(1, 64, dtype=F8, device="cuda")
    s = torch.empty(1, 1, device="cuda")
    rse.moe_fp8_quantize(x, q, s)
    want_q, want_s = go.quantize_rows(wide[:1, :64])
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q), want_q)


def test_rows_with_nan_and_infinity_poison_their_block_only():
    x = torch.randn(3, 384, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    clean_q, clean_s = go.quantize_rows(x)
    x[0, 130] = math.nan
    x[2, 383] = -math.inf
    q = torch.empty(3, 384, dtype=F8, device="cuda")
    s = torch.empty(3, 3, device="cuda")
    rse.moe_fp8_quantize(x.cuda(), q, s)
    bad = torch.zeros(3, 384, dtype=torch.bool)
    bad[0, 128:256] = True
    bad[2, 256:] = True
    assert torch.equal(torch.isnan(codes(q)), bad)
    assert torch.equal(codes(q)[~bad], clean_q[~bad])
    assert float(s[1, 0]) == 1 and float(s[2, 2]) == 1 and torch.equal(s.cpu().double()[0], clean_s[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (2, 128, 128), (3, 200, 144), (1, 129, 400), (2, 56, 1040)])
def test_weights(G, N, K, dtype):
    g = torch.Generator().manual_seed(G * N + K)
    w = (torch.randn(G, N, K, generator=g) / math.sqrt(K)).to(dtype)
    q = torch.empty(G, N, K, dtype=F8, device="cuda")
    s = torch.empty(G, (N + 127) // 128, (K + 127) // 128, device="cuda")
    rse.moe_fp8_quantize_weight(w.cuda(), q, s)
    want_q, want_s = go.quantize_weight(w)
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q), want_q)


# ---------------------------------------------------------------- gemm ------

def header():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    rse.moe_workspace_init(ws)
    return ws


def gemm_inputs(rows, N, K, G, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: (torch.randn(s, generator=g) * 110).clamp(-448, 448).to(F8)  # noqa: E731
    a, w = rnd(rows, K), rnd(G, N, K)
    sa = 2.0 ** torch.randint(-9, 0, ((K + 127) // 128, rows), generator=g).float()
    sw = (0.5 + torch.rand(G, (N + 127) // 128, (K + 127) // 128, generator=g)) / (110 * math.sqrt(K))
    return a, sa * (1 + torch.rand(sa.shape, generator=g)), w, sw, g


def check_gemm(out, want, mag, K, out_dtype):
    blocks = (K + 127) // 128
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    tol = mag * (128 * 2.0 ** -23 + (blocks + 4) * 2.0 ** -24) + want.abs() * half
    off = (out.cpu().double() - want).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol.clamp(min=1e-300)).max()):.2f} of the bound"


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,K", [(1, 8, 16), (1, 256, 128), (3, 136, 144), (16, 512, 256), (17, 264, 400), (64, 128, 2000),
                                      (65, 1000, 640), (255, 392, 1024), (257, 256, 384), (600, 520, 272),
                                      # few tiles: K split over two to four CTA pairs
                                      (1, 6144, 2048), (33, 520, 1552), (16, 136, 1024), (48, 2048, 4096), (130, 264, 1040),
                                      # more tiles of 64 rows than run at once: the form for many rows
                                      (1300, 1032, 400), (1153, 2056, 144), (2100, 1000, 1152), (4900, 136, 128)])
def test_dense_product(rows, N, K, out_dtype):
    a, sa, w, sw, _ = gemm_inputs(rows, N, K, 1, rows + N + K)
    out = torch.full((rows, N), 7.0, dtype=out_dtype, device="cuda")
    ws = header()
    rse.moe_fp8_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), None, None, out, ws)
    want, mag = go.gemm(a.double(), sa, w.double(), sw)
    check_gemm(out, want, mag, K, out_dtype)
    assert rse.moe_read_device_error(ws) == 0
    assert torch.count_nonzero(ws.view(torch.int32)).item() == 0


GROUPS = {
    "empty_and_hot": ([0, 0, 5, 5, 300, 301, 301], 640, 384),
    "one_each": (list(range(41)), 256, 256),
    "ragged": ([0, 31, 95, 96, 223, 480, 1009], 392, 528),
    "many": ([3 * i + (i % 2) for i in range(129)], 128, 128),
    "not_all_rows": ([4, 20, 20, 97], 264, 400),
    "split": ([0, 0, 3, 40, 40, 105], 264, 2064),
    "split_empty": ([0, 0, 0], 128, 2048),
    # the form for many rows: whole and ragged tiles, a CTA without rows, an empty and a hot group
    "wide": ([0, 256, 300, 300, 1500, 1628, 1629, 2300], 1032, 272),
    "wide_not_all_rows": ([7, 200, 2200], 776, 640),
    # ... and tiles of at most 128 rows: 1 to 128, alone and behind whole ones
    "wide_half": ([0, 64, 129, 257, 289, 290, 418, 738, 1122, 1507, 1600], 1032, 400),
}


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_product(name, scaled):
    ends, N, K = GROUPS[name]
    G = len(ends) - 1
    rows = ends[-1] + (9 if name in ("not_all_rows", "split_empty") else 0)
    a, sa, w, sw, g = gemm_inputs(rows, N, K, G, rows)
    c = torch.rand(rows, generator=g) * 2 - 1 if scaled else None
    ws = header()
    for out_dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows, N), 7.0, dtype=out_dtype, device="cuda")
        for _ in range(2):                      # the tile queue is left ready for the next call
            rse.moe_fp8_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), torch.tensor(ends, dtype=torch.int32, device="cuda"),
                             None if c is None else c.cuda(), out, ws)
        want, mag = go.gemm(a.double(), sa, w.double(), sw, ends, c)
        own = ~torch.isnan(want[:, 0])
        check_gemm(out[own.cuda()], want[own], mag[own], K, out_dtype)
        assert bool((out[~own.cuda()] == 7.0).all())   # rows of no group are left as they were
    assert torch.count_nonzero(ws.view(torch.int32)).item() == 0


@pytest.mark.parametrize("rows,N,K,given,held", [
    (60, 264, 400, [-5, 20, 20, 70], [0, 20, 20, 60]),
    (60, 264, 400, [10, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [10, 60, 60, 60]),
    (60, 264, 400, [-2 ** 31, -7, 3, 50], [0, 0, 3, 50]),
    (1500, 776, 272, [-40, 900, 900, 5000], [0, 900, 900, 1500]),
])
def test_offsets_are_held_to_the_rows(rows, N, K, given, held):
    a, sa, w, sw, _ = gemm_inputs(rows + 300, N, K, 3, rows)
    a, sa = a[:rows], sa[:, :rows].contiguous()
    outs = []
    for ends in (given, held):
        out = torch.full((rows, N), 7.0, device="cuda")
        off = torch.tensor(ends, dtype=torch.int64).to(torch.int32).cuda()
        rse.moe_fp8_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), off, None, out, header())
        outs.append(out.cpu())
    assert torch.equal(*outs)


def test_nan_stays_in_its_row():
    a, sa, w, sw, _ = gemm_inputs(40, 256, 256, 1, 3)
    a = a.double()
    a[7, 100] = math.nan
    out = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    rse.moe_fp8_gemm(a.to(F8).cuda(), sa.cuda(), w.cuda(), sw.cuda(), None, None, out, header())
    assert bool(torch.isnan(out[7]).all())
    assert int(torch.isnan(out).sum()) == 256


def test_output_of_more_than_2_31_elements():
    """The last rows of a product whose output's offsets pass 32 bits."""
    rows, N, K = 1_050_001, 2056, 128
    a, sa, w, sw, _ = gemm_inputs(300, N, K, 1, 8)
    big = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    scale = torch.ones(1, rows, device="cuda")
    at = torch.cat([torch.arange(20), torch.arange(rows - 280, rows)])
    big[at.cuda()] = a.view(torch.uint8).cuda()
    scale[:, at.cuda()] = sa.cuda()
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    rse.moe_fp8_gemm(big, scale, w.cuda(), sw.cuda(), None, None, out, header())
    want, mag = go.gemm(a.double(), sa, w.double(), sw)
    check_gemm(out[at.cuda()], want, mag, K, torch.bfloat16)
    assert int(torch.count_nonzero(out[1000:1040])) == 0


def test_rows_and_weights_of_more_than_2_31_elements():
    g = torch.Generator().manual_seed(3)
    part = torch.randn(2, 256, generator=g).to(torch.bfloat16)
    x = torch.empty(3, 1_200_000_000, dtype=torch.bfloat16, device="cuda")    # only what is compared is written
    x[0, :256], x[2, :256] = part[0].cuda(), part[1].cuda()
    q = torch.empty(4, 256, dtype=F8, device="cuda")
    s = torch.empty(2, 4, device="cuda")
    rse.moe_fp8_quantize(x[:, :256], q, s, src=torch.tensor([0, 4, 5, 1], dtype=torch.int32, device="cuda"), src_div=2)
    want_q, want_s = go.quantize_rows(part[[0, 1, 1, 0]])
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(codes(q), want_q)
    del x
    w = torch.zeros(2, 8200, 131072, dtype=torch.bfloat16, device="cuda")
    w[1, -200:, -400:] = torch.randn(200, 400, generator=g).to(torch.bfloat16).cuda()
    q = torch.empty(w.shape, dtype=F8, device="cuda")
    s = torch.empty(2, 65, 1024, device="cuda")
    rse.moe_fp8_quantize_weight(w, q, s)
    want_q, want_s = go.quantize_weight(w[1:, -136:, -512:].cpu())    # rows 8064 on: whole blocks
    assert torch.equal(s[1:, -2:, -4:].cpu().double(), want_s) and torch.equal(codes(q[1:, -136:, -512:]), want_q)


@pytest.mark.parametrize("rows,N,K", [(300, 384, 512), (2300, 1032, 512), (110, 384, 1536)])  # both forms, K split
def test_product_is_deterministic_and_graph_replays_it(rows, N, K):
    a, sa, w, sw, _ = gemm_inputs(rows, N, K, 3, 4)
    dev = [t.cuda() for t in (a, sa, w, sw)]
    off = torch.tensor([0, 100, 101, rows], dtype=torch.int32, device="cuda")
    ws = header()
    first = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    rse.moe_fp8_gemm(*dev, off, None, first, ws)
    again = torch.empty_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        rse.moe_fp8_gemm(*dev, off, None, again, ws)
    for _ in range(3):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, again)


# ---------------------------------------------------------------- layer -----

def fp8_layer(T, H, E, k, I, I_s=0, limit=7.0, seed=0, hot=None, empty=(), **kw):
    """Random inputs of an FP8 layer, its oracle weights and the layer itself."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w1, s1 = go.quantize_weight(rnd(E, 2 * I, H) / math.sqrt(H))
    w2, s2 = go.quantize_weight(rnd(E, H, I) / math.sqrt(I))
    s1, s2 = s1 * (0.7 + torch.rand(s1.shape, generator=g)), s2 * (0.7 + torch.rand(s2.shape, generator=g))
    bias = torch.rand(E, generator=g) * 0.2 - 0.1
    if hot is not None:
        bias[hot] = 5.0
    for e in empty:
        bias[e] = -5.0
    c = SimpleNamespace(x=rnd(T, H).to(torch.bfloat16), router_w=rnd(E, H) / math.sqrt(H), bias=bias, w1=w1, w2=w2,
                        s1=s1.float(), s2=s2.float(), limit=limit, I_s=I_s,
                        sh1=(rnd(2 * I_s, H) / math.sqrt(H)).to(torch.bfloat16) if I_s else None,
                        sh2=(rnd(H, I_s) / math.sqrt(I_s)).to(torch.bfloat16) if I_s else None)
    mv = lambda t: None if t is None else t.cuda()  # noqa: E731
    c.args = dict(hidden=H, num_experts=E, top_k=k, expert_inter=I, shared_inter=I_s, swiglu_limit=limit,
                  routed_scaling_factor=2.5, renormalize=True, router_w=mv(c.router_w), correction_bias=mv(bias),
                  w_gate_up=mv(w1.to(F8)), w_down=mv(w2.to(F8)), s_gate_up=mv(c.s1), s_down=mv(c.s2),
                  shared_w_gate_up=mv(c.sh1), shared_w_down=mv(c.sh2), max_tokens=T, **kw)
    c.layer = rse.MoELayer(**c.args)
    return c


def norm_err(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def layer_oracle(c, offsets, src, w_perm, k):
    y = go.ffn(c.x[(src // k).long()], c.w1, c.s1, c.w2, c.s2, offsets.tolist(), c.limit, w_perm)
    T = c.x.shape[0]
    out = torch.zeros(T, c.x.shape[1], dtype=torch.float64)
    if c.I_s:
        out += oracle.expert_ffn(c.x.double(), c.sh1.double(), c.sh2.double(), c.limit)
    out.index_add_(0, (src // k).long(), y)
    return y, out


LAYERS = {
    "one_token": dict(T=1, H=256, E=8, k=2, I=128, I_s=64),
    "smallest": dict(T=5, H=128, E=2, k=1, I=128),
    "decode": dict(T=32, H=512, E=16, k=4, I=256, I_s=128),
    "hot_expert": dict(T=300, H=256, E=8, k=1, I=128, hot=3),
    "empty_experts": dict(T=150, H=384, E=6, k=2, I=256, I_s=64, empty=(0, 2, 5)),
    "tiles": dict(T=700, H=256, E=3, k=2, I=384),
    "clamped": dict(T=200, H=256, E=4, k=2, I=128, limit=0.5),
    "unclamped": dict(T=200, H=256, E=4, k=2, I=128, limit=math.inf),
    "many_experts": dict(T=40, H=128, E=128, k=16, I=128),
    # the form for many rows on both products
    "wide": dict(T=1500, H=1280, E=3, k=2, I=640, I_s=64),
    "wide_hot": dict(T=1700, H=1024, E=8, k=1, I=512, hot=3),
    "wide_clamped": dict(T=1600, H=1152, E=4, k=2, I=512, limit=0.5),
    "wide_half": dict(T=1500, H=512, E=24, k=2, I=512),
}


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer_matches_oracle(name):
    kw = LAYERS[name]
    c = fp8_layer(**kw)
    k = kw["k"]
    st = run_stages(c.layer, c.x.cuda())
    y, out = layer_oracle(c, st.offsets.cpu(), st.src.cpu(), st.w_perm.cpu(), k)
    for got, want in ((st.y_perm, y), (st.out, out)):
        assert rel_err(got, want) <= 2e-2 and norm_err(got, want) <= 2.0 ** -7, (rel_err(got, want), norm_err(got, want))
    assert torch.equal(st.y_perm, st.y_perm_g)            # gathered rows: the same codes, the same bits
    if c.I_s:
        assert torch.equal(st.shared_out, st.shared_out_g)
    assert torch.equal(c.layer.forward(c.x.cuda()), st.out)
    assert c.layer.device_error() == 0
    assert torch.count_nonzero(c.layer.ws[:256].view(torch.int32)).item() == 0


def test_layer_routes_with_groups_and_replays_in_a_graph():
    """The operators as they are used together: softmax or grouped routing in
    front of FP8 experts, captured once, replayed on other tokens."""
    for kw in (dict(score=rse.MOE_SCORE_SOFTMAX), dict(num_groups=4, top_groups=2)):
        c = fp8_layer(T=96, H=256, E=16, k=4, I=256, I_s=128, **kw)
        other = torch.randn(96, 256, generator=torch.Generator().manual_seed(77)).to(torch.bfloat16)
        x = c.x.cuda()
        ids = torch.empty(96, 4, dtype=torch.int32, device="cuda")
        w = torch.empty(96, 4, device="cuda")
        c.layer.forward(x)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            out = c.layer.forward(x, topk_ids=ids, topk_w=w)
        for tokens in (c.x, other):
            x.copy_(tokens)
            graph.replay()
            torch.cuda.synchronize()
            perm = oracle.permute(ids.cpu(), 16)
            c.x = tokens
            _, want = layer_oracle(c, perm.expert_offsets, perm.src, w.cpu().reshape(-1)[perm.src], 4)
            assert rel_err(out, want) <= 2e-2 and norm_err(out, want) <= 2.0 ** -7
            z = oracle.router_logits(tokens, c.router_w)
            want_ids, _ = go.gate_select(z, c.bias, 4, softmax="score" in kw, groups=kw.get("num_groups", 1),
                                         top_groups=kw.get("top_groups", 1))
            assert int((ids.cpu().long() != want_ids).any(1).sum()) <= 1   # fp32 logits: a border within 1e-6
        assert torch.equal(c.layer.forward(x), out)


@pytest.mark.parametrize("T,world", [(20, 2), (300, 3), (150, 5), (6000, 2)])
def test_expert_parallel_partials_add_up(T, world):
    c = fp8_layer(T=T, H=256, E=4, k=2, I=128, I_s=64)
    full = c.layer.forward(c.x.cuda())
    total = torch.zeros(T, 256, device="cuda")
    for r in range(world):
        part = ep.ExpertParallelLayer(rank=r, world=world, **c.args)
        total += part.forward_partial(c.x.cuda()).float()
        assert _error_free(part)
    # each partial is rounded to bf16 once: world * 2^-8 of the largest value
    assert float((total - full.float()).abs().max()) <= (world + 1) * 2.0 ** -8 * float(full.float().abs().max())


def _error_free(part):
    return rse.moe_read_device_error(part.ws) == 0


@pytest.mark.parametrize("T,H,I", [(64, 256, 128), (1500, 1280, 640)])
def test_nan_token_stays_in_its_rows(T, H, I):
    c = fp8_layer(T=T, H=H, E=4, k=2, I=I)
    clean = c.layer.forward(c.x.cuda())
    x = c.x.clone()
    x[9, 40] = math.nan
    out = c.layer.forward(x.cuda())
    rest = [t for t in range(T) if t != 9]
    assert bool(torch.isnan(out[9]).all()) and torch.equal(out[rest], clean[rest])


def test_two_streams_with_a_workspace_each():
    """Two layers' calls in flight at once give the bits they give alone."""
    a, b = fp8_layer(T=700, H=512, E=8, k=2, I=256, seed=1), fp8_layer(T=40, H=512, E=8, k=4, I=256, seed=2)
    xs = [a.x.cuda(), b.x.cuda()]
    alone = [a.layer.forward(xs[0]), b.layer.forward(xs[1])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(alone[i]) for _ in range(10)] for i in range(2)]
    for n in range(10):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                c.layer.forward(xs[i], out=outs[i][n])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


@pytest.mark.parametrize("kernel", [rse._abi.MOE_SELFTEST_PAIR_FP8_FEW, rse._abi.MOE_SELFTEST_PAIR_FP8_WIDE])
def test_forced_timeout_is_reported_and_context_survives(kernel):
    abi = rse._abi
    scratch = torch.zeros(abi.MOE_SELFTEST_SCRATCH_BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    abi.moe_selftest_pair_timeout(scratch, kernel)
    code = abi.moe_read_device_error(scratch)
    assert code == abi.MOE_ERR_DEVICE_TIMEOUT
    assert time.perf_counter() - t0 < 2.0
    assert torch.count_nonzero(scratch[:256].view(torch.int32)[2:10]).item() == 0   # the tile queue is ready again
    assert abi.moe_read_device_error(scratch) == 0
    # the same kernel goes on computing
    rows, N, K = (40, 256, 256) if kernel == abi.MOE_SELFTEST_PAIR_FP8_FEW else (1300, 1032, 256)
    a, sa, w, sw, _ = gemm_inputs(rows, N, K, 1, 5)
    out = torch.empty(rows, N, device="cuda")
    rse.moe_fp8_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), None, None, out, header())
    want, mag = go.gemm(a.double(), sa, w.double(), sw)
    check_gemm(out, want, mag, K, torch.float32)
