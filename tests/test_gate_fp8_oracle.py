"""Pins of the oracle of expert selection from logits and of the FP8 block
products: hand-worked selections, the E4M3 grid, and special cases."""

import math

import pytest
import torch

from oracle import gate_fp8_oracle as go


def test_hand_selection_with_groups():
    # groups {0,1} {2,3} {4,5}; sigmoid scores of 0 are 1/2, the bias decides
    bias = torch.tensor([0.4, -0.4, 0.1, 0.1, 0.35, -0.5])
    z = torch.zeros(1, 6)
    # sums of two: 1.0, 1.2, 0.85; largest: 0.9, 0.6, 0.85
    ids, w = go.gate_select(z, bias, 2, groups=3, top_groups=1)
    assert ids.tolist() == [[2, 3]] and w.tolist() == [[0.5, 0.5]]
    ids, _ = go.gate_select(z, bias, 2, groups=3, top_groups=1, group_max=True)
    assert ids.tolist() == [[0, 1]]
    ids, _ = go.gate_select(z, bias, 2, groups=3, top_groups=2, group_max=True)
    assert ids.tolist() == [[0, 4]]
    ids, w = go.gate_select(z, None, 3, alpha=2.0, renorm=True)
    assert ids.tolist() == [[0, 1, 2]] and w[0].tolist() == pytest.approx([2 / 3] * 3)


def test_hand_softmax_and_masked_rows():
    z = torch.tensor([[math.log(1.0), math.log(2.0), math.log(5.0), -math.inf]])
    ids, w = go.gate_select(z, None, 2, softmax=True)
    assert ids.tolist() == [[2, 1]] and w[0].tolist() == pytest.approx([5 / 8, 2 / 8], rel=1e-6)
    ids, w = go.gate_select(torch.full((1, 4), -math.inf), None, 2, softmax=True, renorm=True)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_e4m3_nearest_is_the_library_cast():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float())).clamp(-448, 448)
    mid = torch.cat([go._MID, -go._MID]).float()  # every tie, exact in fp32
    for v in (x, mid):
        assert torch.equal(go.e4m3_nearest(v.double()), v.to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                        (1.7500001, 2.0 ** -7), (0.0, 1.0), (1e-44, 2.0 ** -126)])
def test_block_scale(amax, scale):
    assert go.block_scale(amax) == scale


def test_power_of_two_values_survive_and_products_are_exact():
    a = torch.exp2(torch.randint(-3, 3, (5, 200), generator=torch.Generator().manual_seed(1)).double())
    q, s = go.quantize_rows(a)
    assert torch.equal(go.wide_rows(q, s), a)
    w = torch.randn(2, 130, 200, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    wq, ws = go.quantize_weight(w)
    wide = go.wide_weight(wq, ws)
    assert float(((wide - w).abs() / w.abs().clamp(min=float(w.abs().max()) / 448 * 2 ** -5)).max()) <= 2 ** -4 + 1e-9
    out, _ = go.gemm(q, s, wq, ws, [0, 3, 5])
    assert torch.allclose(out[:3], a[:3] @ wide[0].T) and torch.allclose(out[3:], a[3:] @ wide[1].T)
