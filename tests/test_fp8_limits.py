"""FP8 sizes whose index arithmetic would pass 32 bits are refused on the host
(no GPU needed)."""

import pytest

from routed_swiglu_experts_b200 import _abi

FAKE = 1 << 20
BIG = 1 << 30
LAST = (1 << 31) - 16


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


@pytest.mark.parametrize("N,K", [(LAST, 16), (BIG + 16, 16), (16, LAST), (16, BIG + 16), (LAST, LAST)])
def test_weights_past_the_index_range(lib, N, K):
    for groups in (1, 3):
        assert lib.moe_fp8_quantize_weight(FAKE, _abi.MOE_BF16, groups, N, K, FAKE, FAKE, None) == _abi.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows,groups,N,K", [(1, 1, LAST, 16), (1, 1, BIG + 16, 16), (1, 1, 16, LAST), (1, 1, 16, BIG + 16),
                                             (1 << 25, 1, 1 << 28, 16), (1024, 1024, 1 << 29, 16), (1 << 25, 1024, BIG, 16)])
def test_products_past_the_index_range(lib, rows, groups, N, K):
    """More than 2^31 - 1 tiles of 64 rows x 256 columns, or sides past 2^30."""
    assert lib.moe_fp8_gemm(FAKE, FAKE, rows, FAKE, groups, FAKE, FAKE, N, K, None, FAKE, _abi.MOE_BF16, FAKE, 256, None) == \
        _abi.MOE_ERR_UNSUPPORTED
