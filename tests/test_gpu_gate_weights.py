"""Weights of the expert selection where fp32 scores leave their range:
logits far below 0 (sigmoid) or far below the row's maximum (softmax).

Relative error allowed, 1e-5: where the scores stay normal, the difference
l - max under exp is rounded (70 * 2^-24 at most, in numerator and sum) and exp,
sum and divisions add less than 2^-20; the smaller scores are taken in 64 bits.
Without renormalisation the weight itself may be subnormal: exp is off by two
of its steps there, alpha = 2.5 makes them five, rounded to 2^-149 once more."""

import math

import pytest
import torch

import routed_swiglu_experts_b200 as rse
from oracle import gate_fp8_oracle as go

from gpu_util import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

RTOL, ATOL = 1e-5, 6 * 2.0 ** -149


def check(z, bias, k, softmax, renorm, groups=1, top=1, group_max=False):
    T, E = z.shape
    cfg = rse.make_config(128, E, k, 128, 0, 7.0, 2.5, renorm,
                          score=rse.MOE_SCORE_SOFTMAX if softmax else rse.MOE_SCORE_SIGMOID, num_groups=groups,
                          top_groups=top, group_score=rse.MOE_GROUP_MAX if group_max else rse.MOE_GROUP_SUM2)
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    rse.moe_gate_topk(cfg, z.cuda(), None if bias is None else bias.cuda(), ids, w)
    want_ids, want_w = go.gate_select(z, bias, k, 2.5, renorm, softmax, groups, top, group_max)
    assert torch.equal(ids.cpu().long(), want_ids)
    off = (w.cpu().double() - want_w).abs()
    assert bool((off <= RTOL * want_w + ATOL).all()), (w.cpu()[(off > RTOL * want_w + ATOL).any(1)][0],
                                                       want_w[(off > RTOL * want_w + ATOL).any(1)][0])
    return w.cpu().double()


SHAPES = [(64, 6, 1, 1), (256, 8, 8, 4), (72, 7, 2, 1), (148, 8, 4, 2), (8, 3, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,groups,top", SHAPES)
def test_sigmoid_of_logits_far_below_zero(E, k, groups, top, renorm, dtype):
    g = torch.Generator().manual_seed(E + k)
    # one level a row: around the ends of fp32's normal range (-87.3), of its
    # subnormal one (-103.3), of what exp(-l) holds (-88.7), and far beyond
    level = torch.tensor([-60.0, -69.0, -80.0, -86.0, -87.3, -88.0, -88.8, -95.0, -100.0, -103.0, -104.0, -150.0, -300.0, -650.0])
    z = (level[:, None] + torch.randn(14, E, generator=g)).to(dtype)
    for group_max in (False, True):
        if groups == 1 or group_max:       # sums of such scores are all alike in fp64 too: ties, not weights
            check(z, None, k, False, renorm, groups, top, group_max)
    check(z, torch.rand(E, generator=g), k, False, renorm, groups, top)
    if renorm and groups == 1:
        w = check(torch.full((3, E), -100.0).to(dtype), None, k, False, True)
        assert torch.allclose(w, torch.full_like(w, 2.5 / k), rtol=RTOL)


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_of_logits_far_apart(renorm):
    z = torch.full((3, 64), -200.0)
    z[0, :5] = torch.tensor([-69.0, -75.0, -95.0, -101.0, -110.0])
    z[1, :5] = torch.tensor([40.0, 2.0, -90.0, -100.0, -140.0])
    z[2, 60:] = torch.tensor([-89.0, -88.5, -87.0, -86.0])
    check(z, None, 5, False, renorm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,groups,top", SHAPES)
def test_softmax_of_experts_far_below_the_maximum(E, k, groups, top, renorm, dtype):
    """The bias picks experts that the row's largest logit leaves far behind."""
    g = torch.Generator().manual_seed(E * k)
    depth = torch.tensor([60.0, 69.0, 75.0, 86.0, 88.0, 95.0, 100.0, 110.0, 160.0, 400.0, 700.0])
    z = torch.randn(11, E, generator=g) * 3
    z[:, 0] = depth                        # the maximum, alone in its place
    z = z.to(dtype)
    bias = torch.rand(E, generator=g)
    bias[0] = -3.0
    check(z, bias, k, True, renorm, groups, top)


def test_masked_rows_keep_their_zeros():
    """Masks of the types' lowest values and of -inf leave weight 0, alone or beside others."""
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        z = torch.randn(4, 64, generator=torch.Generator().manual_seed(3)).to(dtype)
        z[0] = torch.finfo(dtype).min
        z[1, 2:] = torch.finfo(dtype).min
        z[2, 1:] = -math.inf
        z[3, 2:40] = -math.inf
        z[3, 1] = -100.0
        check(z, None, 6, False, True)
        check(z, None, 6, False, False)
        check(z, None, 6, True, True)
