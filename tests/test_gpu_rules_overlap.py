"""Results of the sampling rules in the buffer that holds the logits: side by side with them they
have the bits of a call apart from it, and what overlaps is refused."""
import pytest
import torch

import rules_plain as rp
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


@pytest.mark.parametrize("V", [9000, 9001])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_side_by_side(rk, dtype, V):
    T = 40
    c = rp.make_case(T, V, dtype=dtype, packed=True, requests=3, bias=2, mask="mixed", history=60, seed=3)
    z, tg, rules = rp.cuda_case(rk, c)
    g = torch.randn(T, device=DEV)
    _, lse = rk.logp_from_logits_rules(z, tg, rules)
    for to in (BF16, FP32):
        x = rk.logits_rules_apply(z, rules, out_dtype=to)
        d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out_dtype=to)
        size = 4 if to == FP32 else 2
        for first in (False, True):  # which of the two comes first in a row
            width = V * (z.element_size() + size) + 12 & ~3  # bytes of a row: room to start the second on 4 bytes
            buf = torch.zeros(T * width, dtype=torch.uint8, device=DEV)
            at = (V * (size if first else z.element_size()) + 3) & ~3
            logits = buf.view(dtype).as_strided((T, V), (width // z.element_size(), 1),
                                                (at if first else 0) // z.element_size())
            out = buf.view(to).as_strided((T, V), (width // size, 1), (0 if first else at) // size)
            logits.copy_(z)
            rk.logits_rules_apply(logits, rules, out=out)
            assert same_bits(out, x) and same_bits(logits, z)
            rk.logp_from_logits_rules_bwd(logits, tg, rules, lse, g, out=out)
            assert same_bits(out, d) and same_bits(logits, z)
    # one behind the other, and a single row in place of itself
    both = torch.empty(2 * T, V, dtype=dtype, device=DEV)
    both[:T] = z
    rk.logits_rules_apply(both[:T], rules, out=both[T:])
    assert same_bits(both[T:], rk.logits_rules_apply(z, rules, out_dtype=dtype))
    one = rk.LogitsRules(temperature=torch.full((1,), 0.7, device=DEV))
    want = rk.logits_rules_apply(z[:1], one, out_dtype=dtype)
    rk.logits_rules_apply(both[:1], one, out=both[:1])
    assert same_bits(both[:1], want)


def test_overlaps_are_refused(rk):
    T, V = 6, 64
    rules = rk.LogitsRules(temperature=torch.full((T,), 0.7, device=DEV))
    buf = torch.zeros(T * V * 4, device=DEV)
    z = buf[:T * V].view(T, V)
    tg = torch.zeros(T, dtype=torch.int64, device=DEV)
    lse, g = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
    for out in (buf[1:1 + T * V].view(T, V), buf[V:V + T * V].view(T, V), buf.as_strided((T, V), (V + 1, 1)),
                buf.view(BF16)[:T * V].view(T, V), buf.view(BF16).as_strided((T, V), (2 * V, 1))):
        with pytest.raises(rk.RkError, match="INVALID"):
            rk.logits_rules_apply(z, rules, out=out)
        for s in (lse, lse.double()):
            with pytest.raises(rk.RkError, match="INVALID"):
                rk.logp_from_logits_rules_bwd(z, tg, rules, s, g, out=out)
    assert not bool(buf.any())
