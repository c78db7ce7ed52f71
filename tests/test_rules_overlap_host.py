"""Results of the sampling rules over the logits: in place, or not at all (no GPU needed: refused calls
read none of the addresses)."""
import ctypes

import pytest

FAKE = 1 << 20
INVALID = 1
BF16, FP32 = 0, 1


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


# rows of 100 columns; (logits' type and stride, out's address, type and stride)
@pytest.mark.parametrize("lt,ld,out,ot,ldo", [
    (FP32, 100, FAKE, BF16, 100),              # the same address, another type
    (BF16, 100, FAKE, FP32, 100),
    (FP32, 100, FAKE, BF16, 200),              # ... with the same stride in bytes
    (FP32, 100, FAKE, FP32, 104),              # another stride
    (BF16, 112, FAKE, BF16, 104),
    (BF16, 100, FAKE + 2, BF16, 100),          # shifted by an element, a row, nearly all of it
    (BF16, 100, FAKE - 2, BF16, 100),
    (BF16, 100, FAKE + 200, BF16, 100),
    (BF16, 100, FAKE + 798, BF16, 100),
    (BF16, 100, FAKE - 798, BF16, 100),
    (FP32, 250, FAKE + 396, FP32, 250),        # side by side, but for one column
    (FP32, 250, FAKE + 604, FP32, 250),
    (FP32, 250, FAKE + 3000 + 396, FP32, 250),  # the last row alone
    (FP32, 250, FAKE - 3000 - 396, FP32, 250),
    (FP32, 250, FAKE + 400, FP32, 249),        # side by side at first, then closer from row to row
    (FP32, 1000, FAKE + 404 + 200, BF16, 1800),  # a later row of one in an earlier one of the other
])
def test_overlapping_results_are_refused(rk, lt, ld, out, ot, ldo):
    lib, s = rk.load_library(), rk._RulesStruct()
    at = ctypes.addressof(s)
    assert lib.rk_logits_rules_apply(FAKE, lt, ld, at, 4, 100, out, ot, ldo, None) == INVALID
    tg = lse = g = 1 << 30
    assert lib.rk_logp_from_logits_rules_bwd(FAKE, lt, ld, tg, None, 0, at, 4, 100, lse, g, out, ot, ldo,
                                             None) == INVALID
    assert lib.rk_logp_from_logits_rules_bwd_lse64(FAKE, lt, ld, tg, None, 0, at, 4, 100, lse, g, out, ot, ldo,
                                                   None) == INVALID
