"""RMS norm with the residual's addition and 8-bit rows against fp64.

The sum in the residual's type is exact (one fp32 addition, one rounding) and
compared bit for bit, and so are the scales (taken from fp64 values where fp32
ones could decide otherwise).
y: 1 / rms rounded to fp32, two products: 3 half steps, |y| 3 * 2^-24, 2^-22
with their products.  out: and half a step of its type (and of its smallest
value).  Codes: q * scale is within half an E4M3 step of y, 2^-4 |y| or, below
the normal range, 2^-10 scale, and the error of y."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import around_oracle as ao

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

F8 = torch.float8_e4m3fn
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6
HALF_SMALLEST = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


def check_out(out, y):
    dt = out.dtype
    err = (out.cpu().double() - y).abs()
    bound = y.abs() * (2.0 ** -22 + torch.finfo(dt).eps / 2 * (1 + 2.0 ** -20)) + HALF_SMALLEST[dt]
    assert bool((err <= bound).all()), float((err - bound).max())


def check_codes(q, s, y):
    want = ao.norm_scales(y)
    assert torch.equal(s.cpu().double(), want)
    sc = want.repeat_interleave(128, 0)[:y.shape[1]].t()
    err = (q.view(F8).cpu().double() * sc - y).abs()
    assert bool((err <= y.abs() * (2.0 ** -4 + 2.0 ** -21) + sc * 2.0 ** -10).all())


def run(x, w, residual=None, out=True, quant=True, **kw):
    rows, H = x.shape
    o = torch.full((rows, H), 7.0, dtype=x.dtype, device="cuda") if out else None
    q = torch.zeros(rows, H, dtype=F8, device="cuda") if quant else None
    s = torch.full(((H + 127) // 128, rows), -1.0, device="cuda") if quant else None
    r = torch.full_like(residual, 7.0) if residual is not None else None
    rse.moe_rmsnorm(x, w, kw.get("eps", EPS), residual=residual, residual_out=r, out=o, q=q, scale=s)
    return o, q, s, r


def rows_of(rows, H, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, H, generator=g) * torch.exp2(torch.randint(-8, 6, (rows, 1), generator=g).float())
    return x.to(dtype), g


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,H", [(1, 16), (5, 64), (3, 128), (17, 144), (7, 512), (9, 528), (2, 1040), (33, 2000),
                                    (3, 6144), (2, 16384), (2, 16400), (3, 20480), (1, 32768)])
def test_sizes(rows, H, dtype):
    x, g = rows_of(rows, H, dtype, rows * H)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(dtype)
    o, q, s, _ = run(x.cuda(), w.cuda())
    _, y = ao.rmsnorm(x, w, EPS)
    check_out(o, y)
    check_codes(q, s, y)


@pytest.mark.parametrize("dtype,res_dtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("out,quant", [(True, False), (False, True), (True, True)])
def test_residual(dtype, res_dtype, out, quant):
    x, g = rows_of(19, 1008, dtype, 5)
    res = (torch.randn(19, 1008, generator=g) * 3).to(res_dtype)
    w = 1 + 0.2 * torch.randn(1008, generator=g)
    o, q, s, r = run(x.cuda(), w.cuda(), res.cuda(), out, quant)
    h, y = ao.rmsnorm(x, w, EPS, res)
    assert torch.equal(r.cpu(), h)
    if out:
        check_out(o, y)
    if quant:
        check_codes(q, s, y)


def test_without_weight_and_with_fp32_weight():
    x, g = rows_of(4, 272, BF16, 6)
    for w in (None, torch.randn(272, generator=g), torch.randn(272, generator=g).to(BF16)):
        o, q, s, _ = run(x.cuda(), None if w is None else w.cuda())
        _, y = ao.rmsnorm(x, w, EPS)
        check_out(o, y)
        check_codes(q, s, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows_and_untouched_neighbours(dtype):
    g = torch.Generator().manual_seed(7)
    wide, wres = torch.randn(6, 400, generator=g).to(dtype), torch.randn(6, 352, generator=g).to(dtype)
    big, bsum = torch.full((6, 320), 9.0, dtype=dtype, device="cuda"), torch.full((6, 304), 9.0, dtype=dtype, device="cuda")
    rse.moe_rmsnorm(wide.cuda()[:, 16:16 + 256], None, EPS, residual=wres.cuda()[:, 8:8 + 256], residual_out=bsum[:, 32:32 + 256],
                    out=big[:, 48:48 + 256])
    h, y = ao.rmsnorm(wide[:, 16:272], None, EPS, wres[:, 8:264])
    assert torch.equal(bsum[:, 32:288].cpu(), h)
    check_out(big[:, 48:304], y)
    assert bool((big[:, :48] == 9).all()) and bool((big[:, 304:] == 9).all())
    assert bool((bsum[:, :32] == 9).all()) and bool((bsum[:, 288:] == 9).all())


def test_in_place():
    x, g = rows_of(70, 640, BF16, 8)
    res = torch.randn(70, 640, generator=g).to(BF16)
    h, y = ao.rmsnorm(x, None, EPS, res)
    xd, rd = x.cuda(), res.cuda()
    rse.moe_rmsnorm(xd, None, EPS, residual=rd, residual_out=rd, out=xd)
    assert torch.equal(rd.cpu(), h)
    check_out(xd, y)
    xd, rd = x.cuda(), res.cuda()
    rse.moe_rmsnorm(xd, None, EPS, residual=rd, residual_out=xd, out=rd)     # the other way round
    assert torch.equal(xd.cpu(), h)
    check_out(rd, y)


def test_scales_next_to_the_border():
    """Rows whose largest value is at 448 * 2^e up to fp32's last bits: fp32 alone decides some of them wrongly."""
    g = torch.Generator().manual_seed(9)
    rows, H = 512, 256
    x = torch.randn(rows, H, generator=g)
    step = torch.randint(-6, 7, (rows,), generator=g).double()
    _, y = ao.rmsnorm(x, None, EPS)
    # (a weight that takes the row's largest value next to the border, one row at a time)
    seen = 0
    for r in range(rows):
        k = int(y[r].abs().argmax())
        w = torch.ones(H)
        w[k] = float((1.75 * 2 ** 4 / y[r, k].abs()) * (1 + step[r] * 2.0 ** -25))
        _, q, s, _ = run(x[r:r + 1].cuda(), w.cuda(), out=False)
        _, want = ao.rmsnorm(x[r:r + 1], w, EPS)
        assert torch.equal(s.cpu().double(), ao.norm_scales(want)), r
        seen += abs(float(want.abs().max()) / (1.75 * 2 ** 4) - 1) < 2.0 ** -23
    assert seen > rows // 2


def test_extreme_rows():
    x = torch.zeros(7, 256)
    x[1, 3] = 3e38                       # its square is outside fp32
    x[2] = 3e38
    x[3] = 1e-38                         # and below it: eps decides
    x[4, 255] = math.inf
    x[5, 0] = math.nan
    x[6] = 1.0
    o, q, s, _ = run(x.cuda(), None)
    good = [0, 1, 2, 3, 6]
    _, y = ao.rmsnorm(x[good], None, EPS)
    check_out(o[good], y)
    check_codes(q[good], s[:, good], y)
    assert bool(torch.isnan(o[4, 255])) and bool((o[4, :255] == 0).all())     # inf / inf, and x / inf
    assert bool(torch.isnan(o[5]).all()) and bool(torch.isnan(q[5].float()).all())
    assert float(s[0, 5]) == 1 and float(s[1, 4]) == 1


def test_no_rows_and_one_row_of_any_stride():
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    rse.moe_rmsnorm(e, None, EPS, out=torch.empty_like(e))
    wide = torch.randn(3, 77, generator=torch.Generator().manual_seed(2)).to(BF16)
    o, q, s, _ = run(wide.cuda()[:1, :64], None)
    _, y = ao.rmsnorm(wide[:1, :64], None, EPS)
    check_out(o, y)
    check_codes(q, s, y)


def test_rows_past_32_bits():
    """Offsets of the last rows pass 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    rows, H = (1 << 31) // 16384 + 3, 16384
    x = torch.zeros(rows, H, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, H, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    q = torch.zeros(rows, H, dtype=F8, device="cuda")
    s = torch.zeros(H // 128, rows, device="cuda")
    rse.moe_rmsnorm(x, None, EPS, out=x, q=q, scale=s, residual=None)
    src = torch.randn(3, H, generator=torch.Generator().manual_seed(1)).to(BF16)
    _, y = ao.rmsnorm(src, None, EPS)
    check_out(x[-3:], y)
    check_codes(q[-3:], s[:, -3:], y)


def test_graph_and_another_stream():
    x, g = rows_of(40, 768, BF16, 11)
    xd = x.cuda()
    o, q, s = torch.empty_like(xd), torch.empty(40, 768, dtype=F8, device="cuda"), torch.empty(6, 40, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rse.moe_rmsnorm(xd, None, EPS, out=o, q=q, scale=s)
    for seed in (1, 2):
        new, _ = rows_of(40, 768, BF16, seed)
        xd.copy_(new)
        graph.replay()
        _, y = ao.rmsnorm(new, None, EPS)
        check_out(o, y)
        check_codes(q, s, y)
    rse.moe_rmsnorm(xd, None, EPS, out=o, stream=side)
    side.synchronize()
    check_out(o, y)
