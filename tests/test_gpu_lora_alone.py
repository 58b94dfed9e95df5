"""What a token's result goes by: its own row, adapter and base, and the sizes
of the call.  The other tokens' rows, which adapters they have and where the
token stands leave its bits as they are."""

import pytest
import torch

import routed_swiglu_experts_b200 as rse

from gpu_util import cuda_available
from test_gpu_lora import BF16, F16, F32, inputs, plan_of, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype,out_type", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("T,r,L", [(9, 16, 4), (200, 64, 30), (512, 128, 5), (600, 16, 4), (900, 64, 200), (3000, 128, 3)])
def test_other_tokens_leave_the_bits(T, r, L, dtype, out_type):
    K, N = 1000, 264
    x, a, b, scale, ids, base = inputs(T, K, N, r, L, dtype, out_type, T)
    g = torch.Generator().manual_seed(T + 1)
    ids[0], ids[T // 2], ids[T - 1] = 1, 0, L - 1
    mine = torch.tensor([0, T // 2, T - 1])
    first = run(x, a, b, scale, ids, base, out_type, L).cpu()
    # other rows, other adapters
    x2, ids2, base2 = torch.randn(T, K, generator=g).to(dtype), torch.randint(-1, L, (T,), generator=g), torch.randn(T, N, generator=g).to(out_type)
    x2[mine], ids2[mine], base2[mine] = x[mine], ids[mine], base[mine]
    assert torch.equal(run(x2, a, b, scale, ids2, base2, out_type, L).cpu()[mine], first[mine])
    # every other token on one adapter; the same batch in another order
    ids3 = torch.full((T,), 1)
    ids3[mine] = ids[mine]
    assert torch.equal(run(x2, a, b, scale, ids3, base2, out_type, L).cpu()[mine], first[mine])
    turn = torch.randperm(T, generator=g)
    assert torch.equal(run(x[turn], a, b, scale, ids[turn], base[turn], out_type, L).cpu(), first[turn])
