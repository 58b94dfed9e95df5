"""Balance loss where every expert is chosen by every token: f is 1 for all of
them, so the loss is coef times the mean of sum_e p_te = 1, and the gradient
p_j (f_j - sum_e f_e p_e) is 0 for every logit, not a rounding remainder."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_balance import BF16, F16, F32, config, workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("dtype,grad_type", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("T,E,S", [(41, 4, 1), (25, 5, 6), (2600, 2, 1), (4100, 12, 7), (3000, 16, 1), (2400, 3, 300),
                                   (12202, 9, 40), (5000, 16, 4000)])
def test_gradient_is_zero(T, E, S, dtype, grad_type, softmax):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    z = (torch.randn(T, E, generator=g, device="cuda") * 3).to(dtype)
    z[::5] -= 100                                                 # (sigmoids below e^-40 take a way of their own)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1).to(torch.int32)
    mask = torch.rand(T, generator=g, device="cuda") < 0.7
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    counts, tokens = torch.full((S, E), -5, dtype=torch.int32, device="cuda"), torch.full((S,), -5, dtype=torch.int32, device="cuda")
    loss, grad = torch.full((), -5.0, device="cuda"), torch.full((T, E), 7.0, dtype=grad_type, device="cuda")
    ws = workspace()
    rse.moe_balance_loss(config(E, E, softmax), z, ids, counts, tokens, loss, ws, grad_logits=grad,
                         seq_offsets=None if S == 1 else offsets, token_mask=mask, coef=0.5,
                         grad_loss=torch.full((1,), 65536.0, device="cuda"))
    assert rse.moe_read_device_error(ws) == 0
    at = torch.searchsorted(offsets[1:].long(), torch.arange(T, device="cuda"), right=True)
    n = torch.bincount(at[mask], minlength=S)
    assert torch.equal(tokens.long(), n) and torch.equal(counts.long(), n[:, None].expand(S, E))
    assert not bool(grad.any())
    # every d_t is 1; coef / (S' n) in fp32 is off by two roundings of 2^-24
    assert abs(float(loss) - 0.5) <= 0.5 * 2.0 ** -22
