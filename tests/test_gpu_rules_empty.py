"""A step without requests: the rules of a serving loop whose tensors have no entries."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def tensors(R, V=100):
    i32, i64 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.int64, device=DEV)
    return dict(temperature=torch.ones(R, device=DEV), repetition=torch.ones(R, device=DEV),
                frequency=torch.zeros(R, device=DEV), presence=torch.zeros(R, device=DEV),
                tokens=torch.zeros(0, **i64), token_offsets=torch.zeros(R + 1, **i64),
                prompt_lengths=torch.zeros(R, **i32), bias_ids=torch.zeros(0, **i64),
                bias_values=torch.zeros(0, device=DEV), bias_offsets=torch.zeros(R + 1, **i64),
                mask=torch.zeros(R, (V + 31) // 32, **i32), row_request=torch.arange(R, **i32),
                row_length=torch.zeros(R, **i32), row_mask=torch.full((R,), -1, **i32))


@pytest.mark.parametrize("leave_out", [(), ("row_request",), ("row_request", "row_mask"), ("mask", "row_mask"),
                                       ("tokens", "token_offsets", "prompt_lengths", "row_length"),
                                       ("temperature", "repetition", "frequency", "presence", "prompt_lengths")])
def test_no_requests(rk, leave_out):
    rules = rk.LogitsRules(**{k: v for k, v in tensors(0).items() if k not in leave_out})
    z = torch.empty(0, 100, device=DEV)
    tg = torch.empty(0, dtype=torch.int64, device=DEV)
    assert rk.logits_rules_apply(z, rules).shape == (0, 100)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    assert logp.shape == lse.shape == (0,)
    assert rk.logp_from_logits_rules_bwd(z, tg, rules, lse, logp).shape == (0, 100)
    with pytest.raises(ValueError):
        rk.logits_rules_apply(torch.zeros(1, 100, device=DEV), rules)


def test_no_requests_for_some_rows(rk):
    kw = tensors(0)
    kw.update(row_request=torch.zeros(2, dtype=torch.int32, device=DEV),
              row_length=torch.zeros(2, dtype=torch.int32, device=DEV),
              row_mask=torch.full((2,), -1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        rk.LogitsRules(**kw)
    with pytest.raises(ValueError):  # offsets of no request have one entry
        rk.LogitsRules(**dict(tensors(0), token_offsets=torch.zeros(0, dtype=torch.int64, device=DEV)))


def test_requests_without_tokens_biases_or_rows(rk):
    z = torch.randn(3, 100, device=DEV)
    kw = tensors(3)
    assert torch.equal(rk.logits_rules_apply(z, rk.LogitsRules(**kw)), z)
    for k in ("row_request", "row_length", "row_mask"):
        kw[k] = kw[k][:0]
    assert rk.logits_rules_apply(z[:0], rk.LogitsRules(**kw)).shape == (0, 100)


@pytest.mark.parametrize("V", [1, 33, 9001, 40000])
def test_without_rules_as_the_call_that_knows_none(rk, V):
    # two kernels, and each within its own rounding: the values agree, the last bits need not
    import rules_plain as rp
    T = 20
    z = (torch.randn(T, V, generator=torch.Generator().manual_seed(V)) * 5).bfloat16()
    tg = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1))
    tg[3] = -1
    a = rk.logp_from_logits_rules(z.to(DEV), tg.to(DEV), rk.LogitsRules())
    b = rk.logp_from_logits(z.to(DEV), tg.to(DEV))
    for t in range(T):
        if t == 3:
            assert all(float(v[t]) == 0 for v in a + tuple(b))
            continue
        size = z[t].double().abs().numpy()
        ref = float(torch.logsumexp(z[t].double(), 0))
        k = int(tg[t])
        assert abs(float(a[1][t]) - float(b[1][t])) <= 2 * rp.lse_bound(size, ref)
        assert abs(float(a[0][t]) - float(b[0][t])) <= 2 * rp.logp_bound(size, k, float(z[t, k]) - ref, ref)
