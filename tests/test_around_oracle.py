"""The fp64 forms of the norm, the adapters and the balance loss, against
numbers computed by hand, differences and invariances."""

import math

import pytest
import torch

from oracle import around_oracle as ao


def test_norm_of_a_row_by_hand():
    x = torch.tensor([[3.0, 4.0, 0.0, 0.0]])
    h, y = ao.rmsnorm(x, torch.tensor([1.0, 2.0, 1.0, 1.0]), 0.25)
    assert torch.equal(h, x)
    r = 1 / math.sqrt(25 / 4 + 0.25)
    assert torch.allclose(y, torch.tensor([[3 * r, 8 * r, 0, 0]], dtype=torch.float64), rtol=1e-15)


def test_norm_rounds_the_sum_to_the_residual():
    x, res = torch.tensor([[1.0]]).to(torch.bfloat16), torch.tensor([[2.0 ** -9]]).to(torch.bfloat16)
    h, _ = ao.rmsnorm(x, None, 1e-6, res)
    assert h.dtype == torch.bfloat16 and float(h) == 1.0          # a tie: to the even value
    h, _ = ao.rmsnorm(x, None, 1e-6, res.float())
    assert float(h) == 1.0 + 2.0 ** -9


def test_scales_at_the_border():
    y = torch.zeros(3, 128, dtype=torch.float64)
    y[0, 0], y[1, 0], y[2, 0] = 448.0, 448.0 * (1 + 2.0 ** -50), 0.875
    assert ao.norm_scales(y)[0].tolist() == [1.0, 2.0, 2.0 ** -9]


def test_lora_by_hand():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]])
    b = torch.tensor([[[10.0], [0.0]], [[1.0], [-1.0]]])
    out, size = ao.lora(x, a, b, torch.tensor([1.0, 0.5]), torch.tensor([1, -1, 0]), torch.ones(3, 2))
    assert out.tolist() == [[2.0, 0.0], [1.0, 1.0], [51.0, 1.0]]
    assert size.tolist() == [[2.0, 2.0], [1.0, 1.0], [51.0, 1.0]]


@pytest.mark.parametrize("softmax", [False, True])
def test_balance_by_hand(softmax):
    # equal logits: p = 1 / E, so the loss is coef * sum_e f_e / E = coef whatever the ids
    z = torch.zeros(5, 4, dtype=torch.float64)
    ids = torch.tensor([[0, 1], [0, 2], [0, 3], [0, 1], [0, 1]])
    loss, counts, tokens, f = ao.balance(z, ids, softmax, coef=0.5)
    assert abs(float(loss) - 0.5) < 1e-15
    assert counts.tolist() == [[5, 3, 1, 1]] and tokens.tolist() == [5]
    assert torch.allclose(f[0], torch.tensor([2.0, 1.2, 0.4, 0.4], dtype=torch.float64))


def formula_gradient(z, f, counted, n_of, softmax, coef):
    p = ao.balance_scores(z, softmax)
    slope = 1.0 if softmax else torch.sigmoid(-z)
    g = p * (f - (p * f).sum(1, keepdim=True)) * slope
    return g * torch.where(counted, coef / n_of, torch.zeros_like(n_of))[:, None]


@pytest.mark.parametrize("softmax", [False, True])
def test_balance_gradient_against_autograd_and_differences(softmax):
    g = torch.Generator().manual_seed(3)
    T, E, k = 9, 6, 2
    z = torch.randn(T, E, generator=g, dtype=torch.float64, requires_grad=True)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids[4, 1] = -1
    offsets, mask = [1, 4, 4, 8], torch.tensor([1, 1, 0, 1, 1, 1, 1, 0, 1])
    loss, counts, tokens, f = ao.balance(z, ids, softmax, offsets, mask, 0.7)
    assert tokens.tolist() == [2, 0, 3] and int(counts.sum()) == 2 * 5 - 1
    loss.backward()
    counted = torch.tensor([0, 1, 0, 1, 1, 1, 1, 0, 0], dtype=torch.bool)
    n_of = torch.tensor([1, 2, 2, 2, 3, 3, 3, 3, 1], dtype=torch.float64)
    want = formula_gradient(z.detach(), f, counted, n_of, softmax, 0.7 / 2)
    assert torch.allclose(z.grad, want, rtol=1e-12, atol=1e-15)
    at = z.detach()
    for t, e in ((1, 0), (4, 5), (0, 2), (7, 1)):
        d = torch.zeros_like(at)
        d[t, e] = 1e-5
        up, down = (ao.balance(at + s * d, ids, softmax, offsets, mask, 0.7)[0] for s in (1, -1))
        # central differences: an error of h^2 / 6 |f'''| (1e-10) and of 2^-52 / h (1e-11)
        assert abs(float(up - down) / 2e-5 - float(want[t, e])) < 1e-9
