"""RMS norm of enough rows that blocks walk over them, against fp64: the same
bounds as for few rows (test_gpu_norm)."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_norm import BF16, EPS, F16, F32, F8, HALF_SMALLEST

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def exact(x, w, residual=None):
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    y = h.double()
    y = y / (y.square().mean(1, keepdim=True) + float(torch.tensor(EPS))).sqrt()
    return h, y if w is None else y * w.double()


def check(o, q, s, y):
    if o is not None:
        err, half = (o.double() - y).abs(), torch.finfo(o.dtype).eps / 2
        bound = y.abs() * (2.0 ** -22 + half * (1 + 2.0 ** -20)) + HALF_SMALLEST[o.dtype]
        assert bool((err <= bound).all()), float((err - bound).max())
    if q is not None:
        rows, H = y.shape
        amax = torch.nn.functional.pad(y.abs(), (0, -H % 128)).view(rows, -1, 128).amax(2)
        m, e = torch.frexp(amax)
        want = torch.where(amax > 0, torch.exp2((torch.where(m <= 0.875, e - 9, e - 8)).double()), 1.0)
        assert torch.equal(s.double(), want.t())
        sc = want.repeat_interleave(128, 1)[:, :H]
        err = (q.double() - y / sc).abs() * sc
        near = (err <= y.abs() * (2.0 ** -4 + 2.0 ** -21) + sc * 2.0 ** -10).all()
        assert bool(near)


@pytest.mark.parametrize("dtype,res_dtype,w_dtype", [(BF16, None, BF16), (BF16, BF16, BF16), (BF16, BF16, F32), (F16, F16, None),
                                                     (F16, F16, F16), (BF16, F32, BF16), (F32, F32, F32)])
@pytest.mark.parametrize("rows,H", [(40000, 16), (20001, 144), (15000, 256), (12003, 512), (9001, 1008), (9000, 1024), (7001, 2000),
                                    (6003, 2048), (2500, 4112), (1999, 6144), (1203, 16384), (999, 20480)])
def test_many_rows(rows, H, dtype, res_dtype, w_dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + H)
    x = (torch.randn(rows, H, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 5, (rows, 1), generator=g, device="cuda").float())).to(dtype)
    res = None if res_dtype is None else torch.randn(rows, H, generator=g, device="cuda").to(res_dtype)
    w = None if w_dtype is None else (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(w_dtype)
    h, y = exact(x, w, res)
    sums = None if res is None else torch.empty_like(res)
    o = torch.empty_like(x)
    q, s = torch.empty(rows, H, dtype=F8, device="cuda"), torch.empty((H + 127) // 128, rows, device="cuda")
    rse.moe_rmsnorm(x, w, EPS, residual=res, residual_out=sums, out=o, q=q, scale=s)
    check(o, q, s, y)
    if res is not None:
        assert torch.equal(sums, h)
    # codes alone, and in place (the result over x, the sum over the residual)
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    if res is not None:
        rse.moe_rmsnorm(x, w, EPS, residual=res, residual_out=res, out=x)
        assert torch.equal(res, h) and torch.equal(x, o)
    else:
        rse.moe_rmsnorm(x, w, EPS, q=q2, scale=s2)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
        rse.moe_rmsnorm(x, w, EPS, out=x, q=q2, scale=s2)
        assert torch.equal(x, o) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [128, 2048])
def test_many_rows_at_the_scales_border_and_at_the_ends_of_the_range(H, in_place):
    """Rows of one value and zeros (y is sqrt(H) at it, times a weight next to 448 * 2^e), of huge and of tiny values."""
    rows = 6001
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.zeros(rows, H, device="cuda", dtype=BF16)
    at = torch.randint(0, H, (rows,), generator=g, device="cuda")
    x[torch.arange(rows, device="cuda"), at] = torch.exp2(torch.randint(-3, 4, (rows,), generator=g, device="cuda").float()).to(BF16)
    x[3::7] = (torch.randn(x[3::7].shape, generator=g, device="cuda") * 1e38).to(BF16)
    x[5::7] = (torch.randn(x[5::7].shape, generator=g, device="cuda") * 1e-20).to(BF16)
    w = ((448 / 16) / H ** 0.5 * (1 + torch.randint(-6, 7, (H,), generator=g, device="cuda") * 2.0 ** -23)).float()
    _, y = exact(x, w)
    # (some of the huge values are infinities in bf16: NaN at them, as the call says)
    infinite = torch.isinf(x)
    fine = ~infinite.any(1)
    q, s = torch.empty(rows, H, dtype=F8, device="cuda"), torch.empty(H // 128, rows, device="cuda")
    o = x if in_place else torch.empty_like(x)
    rse.moe_rmsnorm(x, w, EPS, out=o, q=q, scale=s)
    check(o[fine], q[fine], s[:, fine], y[fine])
    assert bool(torch.isnan(o[infinite]).all()) and int(fine.sum()) > rows // 2


def test_many_strided_rows_leave_their_neighbours():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(5000, 1200, generator=g, device="cuda").to(BF16)
    big = torch.full((5000, 1104), 9.0, dtype=BF16, device="cuda")
    sums = torch.full((5000, 1064), 9.0, dtype=BF16, device="cuda")
    x, res = wide[:, 8:8 + 1040], wide[:, 160:160 + 1040].clone()
    h, y = exact(x, None, res)
    rse.moe_rmsnorm(x, None, EPS, residual=res, residual_out=sums[:, 16:1056], out=big[:, 40:1080])
    assert torch.equal(sums[:, 16:1056], h)
    check(big[:, 40:1080], None, None, y)
    assert bool((big[:, :40] == 9).all()) and bool((big[:, 1080:] == 9).all())
    assert bool((sums[:, :16] == 9).all()) and bool((sums[:, 1056:] == 9).all())


def test_bad_rows_stay_alone():
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(4000, 1536, generator=g, device="cuda").to(BF16)
    o, q, s = torch.empty_like(x), torch.empty(4000, 1536, dtype=F8, device="cuda"), torch.empty(12, 4000, device="cuda")
    x[1001, 5], x[3999, 1000] = float("nan"), float("inf")
    rse.moe_rmsnorm(x, None, EPS, out=o, q=q, scale=s)
    keep = torch.ones(4000, dtype=torch.bool, device="cuda")
    keep[[1001, 3999]] = False
    _, y = exact(x[keep], None)
    check(o[keep], q[keep], s[:, keep], y)
    assert bool(torch.isnan(o[1001]).all()) and bool(torch.isnan(o[3999, 1000]))


@pytest.mark.parametrize("H", [16, 48, 64, 80, 112, 128])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 7, 9, 31, 1001, 30001])
@pytest.mark.parametrize("x_dtype,res_dtype", [(BF16, None), (F16, F16), (F32, None), (BF16, F32)])
def test_small_rows_lie_side_by_side(rows, H, x_dtype, res_dtype):
    """Several rows to a warp: rows of nothing, of NaN, of fp32's ends and at the scale's border next to ordinary
    ones, and a last warp that is not full."""
    g = torch.Generator(device="cuda").manual_seed(100 * rows + H)
    x = torch.randn(rows, H, generator=g, device="cuda")
    kind = torch.arange(rows, device="cuda") % 6
    x[kind == 1] = 0
    one = torch.zeros(H, device="cuda")
    one[H // 2] = 1
    x[kind == 2] = one
    if x_dtype != F16:
        x[kind == 3] *= 2.0 ** 70
        x[kind == 4] *= 2.0 ** -70
    x = x.to(x_dtype)
    x[kind == 5, 3] = float("nan")
    res = None if res_dtype is None else torch.zeros(rows, H, dtype=res_dtype, device="cuda")
    w = torch.full((H,), 28 / H ** 0.5, device="cuda")
    h, y = exact(x, w, res)
    wide = torch.full((rows + 2, H + 16), 9.0, dtype=x_dtype, device="cuda")
    o = wide[1:rows + 1, 8:H + 8]
    q = torch.full((rows + 2, H), 1.0, device="cuda").to(F8)
    s = torch.full((rows + 2,), 7.0, device="cuda")
    sums = None if res is None else torch.empty_like(res)
    rse.moe_rmsnorm(x, w, EPS, residual=res, residual_out=sums, out=o, q=q[1:rows + 1], scale=s[1:rows + 1].view(1, rows))
    fine = kind != 5
    check(o[fine], q[1:rows + 1][fine], s[1:rows + 1][fine].view(1, -1), y[fine])
    assert bool(torch.isnan(o[~fine]).all())
    if res is not None:
        assert torch.equal(sums[fine], h[fine])
    assert bool((wide[[0, -1]] == 9).all()) and bool((wide[:, :8] == 9).all()) and bool((wide[:, H + 8:] == 9).all())
    assert bool((q[[0, -1]].float() == 1).all()) and bool((s[[0, -1]] == 7).all())
