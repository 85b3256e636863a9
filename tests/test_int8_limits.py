"""Host-side refusals at the INT8 products' limits (no GPU: every call fails validation first, or is a
no-op)."""
import pytest

from test_int8_logprobs_api import G, Q, product, status  # noqa: F401  (Q: the fixture)

LIMIT = (1 << 31) - 256  # columns are counted in 32 bits, rounded up to a tile


@pytest.mark.parametrize("M", [1, 4, 100])
@pytest.mark.parametrize("N", [LIMIT + 1, (1 << 31) - 130, (1 << 31) - 4, (1 << 31) - 1])
def test_product_refuses_columns_past_the_limit(Q, M, N):
    # (A = None: a call that were not refused for its columns ends with another error, not on a GPU)
    assert product(Q, M=M, N=N, ldc=1 << 31, A=None) == Q.QW_ERR_UNSUPPORTED
    assert product(Q, M=M, N=LIMIT, ldc=1 << 31, A=None) == Q.QW_ERR_INVALID_ARG
    with pytest.raises(Q.QwError) as e:
        Q.qgemm_int8_workspace_size(Q.QW_A_BF16, M, N, 64)
    assert e.value.status == Q.QW_ERR_UNSUPPORTED


def test_gated_refuses_columns_past_the_limit(Q):
    def gated(I):
        return status(Q.qgemm_int8_gated, Q.QW_A_BF16, None, 64, None, G, G, None, G, 1 << 30, 4, I, 64, G,
                      1 << 20, None, 0)
    assert gated(LIMIT // 2) == Q.QW_ERR_INVALID_ARG  # (A is null)
    assert gated(LIMIT // 2 + 1) == Q.QW_ERR_UNSUPPORTED
    assert gated((1 << 30) - 1) == Q.QW_ERR_UNSUPPORTED


def test_workspace_size_up_to_the_limit(Q):
    assert Q.qgemm_int8_workspace_size(Q.QW_A_INT8_TOKEN, 16, LIMIT, 64) == 0
