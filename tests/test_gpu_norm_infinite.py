"""What RMS norm makes of rows with an infinity or a NaN, in every way that its
kernel takes rows (a block each, several to a warp, walked over): NaN at the
infinities and 0 beside them; NaN throughout a row with a NaN.  Codes and scales
follow the block's values.  Other rows are not touched by it."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_norm import BF16, EPS, F16, F32, F8

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype,res_dtype", [(BF16, None), (F16, F16), (F32, None), (BF16, F32)])
@pytest.mark.parametrize("rows,H", [(9, 48), (40000, 64), (7, 112), (30001, 128), (11, 256), (15000, 256), (6, 2000), (7001, 2000),
                                    (6, 6144), (1999, 6144), (6, 20480)])
@pytest.mark.parametrize("out,quant", [(True, True), (True, False), (False, True)])
def test_rows_with_them(rows, H, dtype, res_dtype, out, quant):
    g = torch.Generator(device="cuda").manual_seed(rows + H)
    x = torch.randn(rows, H, generator=g, device="cuda").to(dtype)
    res = None if res_dtype is None else torch.randn(rows, H, generator=g, device="cuda").to(res_dtype)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    clean = dict(x=x.clone(), res=None if res is None else res.clone())
    at, last = H // 2 + 3, rows - 1
    x[1, at] = math.inf
    (x if res is None else res)[2, H - 1] = -math.inf
    x[4, 0], x[4, at] = math.nan, math.inf
    (x if res is None else res)[last, 7] = math.nan
    if res is not None:                                          # an infinity that the addition makes NaN
        x[3, 5], res[3, 5] = math.inf, -math.inf

    def call(x, res):
        o = torch.full((rows, H), 7.0, dtype=dtype, device="cuda") if out else None
        q = torch.zeros(rows, H, device="cuda").to(F8) if quant else None
        s = torch.full(((H + 127) // 128, rows), -1.0, device="cuda") if quant else None
        rse.moe_rmsnorm(x, w, EPS, residual=res, residual_out=None if res is None else torch.empty_like(res), out=o, q=q, scale=s)
        return o, q, s
    o, q, s = call(x, res)
    o0, q0, s0 = call(**clean)
    bad = [1, 2, 4, last] + ([3] if res is not None else [])
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[bad] = False
    nans = torch.zeros(rows, H, dtype=torch.bool, device="cuda")
    nans[1, at] = nans[2, H - 1] = True
    nans[[4, last]] = True
    if res is not None:
        nans[3] = True
    if out:
        assert torch.equal(o[fine], o0[fine])
        assert torch.equal(torch.isnan(o[~fine]), nans[~fine]) and bool((o[~fine][~nans[~fine]] == 0).all())
    if quant:
        assert torch.equal(q[fine].view(torch.uint8), q0[fine].view(torch.uint8)) and torch.equal(s[:, fine], s0[:, fine])
        assert bool((s[:, ~fine] == 1).all())
        blocks = torch.nn.functional.pad(nans, (0, -H % 128)).view(rows, -1, 128).any(2).repeat_interleave(128, 1)[:, :H]
        codes = q.float()
        assert torch.equal(torch.isnan(codes[~fine]), blocks[~fine]) and bool((codes[~fine][~blocks[~fine]] == 0).all())
