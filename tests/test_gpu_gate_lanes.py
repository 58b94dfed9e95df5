"""Close decisions of the expert selection where a group of experts spans a
number of lanes that is no power of two (5 of 4 experts, 3 of 7, 12 of 3), and
where no run of lanes makes up a group (37 experts), on all three types."""

import pytest
import torch

from test_gpu_gate import check, cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

SHAPES = [(100, 5, 3, 16), (100, 5, 1, 6), (168, 8, 4, 8), (72, 2, 1, 7), (148, 4, 2, 8), (74, 2, 1, 9)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group_max", [False, True])
@pytest.mark.parametrize("E,groups,top,k", SHAPES)
def test_close_values(E, groups, top, k, group_max, dtype):
    g = torch.Generator().manual_seed(E + k)
    for grid in (2, 8):
        z = ((torch.randn(60, E, generator=g) * grid).round() / grid).to(dtype)
        check(z, None, k, False, groups, top, group_max)
        check(z[:20], None, k, True, groups, top, group_max)
        for width in (1e-7, 3e-6):
            bias = torch.randn(E, generator=g) * width
            check(z, bias, k, False, groups, top, group_max)
            check(z[:20], bias, k, True, groups, top, group_max)


@pytest.mark.parametrize("E,groups,top,k", SHAPES)
def test_groups_of_one_value(E, groups, top, k):
    """Every group holds the same values, or values 1e-8 apart: the lower groups and ids."""
    g = torch.Generator().manual_seed(E * 7 + k)
    per = E // groups
    z = torch.randn(6, per, generator=g).repeat(1, groups)
    target = torch.rand(per, generator=g).double().repeat(groups) + torch.randn(E, generator=g).double() * 1e-8
    bias = (target - 1 / (1 + torch.exp(-z[0].double()))).float()
    for dtype in (torch.float32, torch.float16):
        check(z.to(dtype), None, k, False, groups, top)
        check(z.to(dtype), None, k, False, groups, top, True)
    check(z[:1], bias, k, False, groups, top)
    check(z[:1], bias, k, False, groups, top, True)
