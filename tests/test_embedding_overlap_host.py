"""The embedding and its gradient do not work in place (no GPU needed: refused calls read none of the
addresses)."""
import pytest

A = 1 << 20
INVALID = 1
BF16, FP32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    return rk.load_library()


# a table of 10 rows of 8, 4 tokens
@pytest.mark.parametrize("et,ot,out", [(FP32, FP32, A), (FP32, FP32, A + 10 * 8 * 4 - 4), (BF16, FP32, A + 10 * 8 * 2 - 4),
                                       (FP32, BF16, A - 4 * 8 * 2 + 2), (BF16, BF16, A + 16), (FP32, FP32, A - 4 * 8 * 4 + 4)])
def test_a_lookup_into_its_table_is_refused(lib, et, ot, out):
    assert lib.rk_embedding(1 << 30, None, 0, A, et, 4, 8, 10, 1.0, out, ot, None) == INVALID


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("dt,dE", [(FP32, A), (FP32, A + 4 * 8 * 4 - 4), (BF16, A + 4 * 8 * 2 - 4), (BF16, A - 10 * 8 * 4 + 4)])
def test_a_gradient_over_its_input_is_refused(lib, dt, dE, accumulate):
    assert lib.rk_embedding_bwd(A, dt, 1 << 30, None, 0, 4, 8, 10, 1.0, None, 0, dE, accumulate, 1 << 31, 1 << 24,
                                None) == INVALID
