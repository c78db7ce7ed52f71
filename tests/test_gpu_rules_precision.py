"""Logprobs under sampling rules where |logit| / temperature is large: what is small there are
the differences of the logits, and the errors have to be measured against those."""
import numpy as np
import pytest
import torch

import rules_plain as rp
from rules_plain import U

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


def leading(T, V, dtype, size, gap, seed):
    """fp64 copies of logits of spread `size`: in row t, t + 1 columns share the maximum, and as many
    follow it at multiples of `gap` (of the type's step, where that is wider)."""
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * size).to(dtype)
    for t in range(T):
        at = torch.randperm(V, generator=g)[:2 * t + 2]
        top = z[t].max().double()
        z[t, at[:t + 1]] = top.to(dtype)
        z[t, at[t + 1:]] = (top - gap * torch.arange(1, t + 2)).to(dtype)
    return z


# Exponents (z - m) c, c = log2e / tau: the rounding of log2e, of 1 / tau, of their product, of z - m and of
# the last product, five half steps of d = (m - z) / tau; weighed with p they add up to sum p d <= ln V.  (2^(z c
# - fl(m c)) with its factor undone: c's three, one of the difference, and the second order of a residual of at
# most 2^-12, a quarter.)  ex2 4u, the tree of sums at most 28 roundings, log and the last operations 4 + 3 ls.
def sum_bound(V, ls):
    return U * (5 * np.log(V) + 4 + 28 + 4 + 3 * ls)


# logp = (z_t - m) / tau - ls: difference, quotient and the last subtraction
def close_logp_bound(d, V, ls):
    return sum_bound(V, ls) + U * (4 * d + 2 * ls)


# lse = m / tau + ls: quotient and sum, a rounding each
def close_lse_bound(lse, V, ls):
    return sum_bound(V, ls) + U * (2.01 * abs(lse) + ls)


@pytest.mark.parametrize("dtype,size,tau", [
    (BF16, 20.0, 1.0), (BF16, 20.0, 1e-2), (BF16, 20.0, 1e-3), (BF16, 20.0, 1e-4), (BF16, 20.0, 1e-5),
    (BF16, 20.0, 1e-6), (FP32, 20.0, 1e-2), (FP32, 20.0, 1e-3), (FP32, 20.0, 1e-4), (FP32, 20.0, 1e-5),
    (FP32, 20.0, 1e-6), (FP32, 3e6, 1.0), (FP32, 3e7, 1.0), (FP32, 3e8, 1.0), (FP32, 3e8, 1e6), (BF16, 3e8, 1.0),
    (FP32, 1e30, 1.0), (FP32, 1e33, 1.0)])
@pytest.mark.parametrize("shift", [0, 1])
def test_logp_where_the_logits_are_far_from_zero(rk, dtype, size, tau, shift):
    T, V = 24, 9001
    z = leading(T, V, dtype, size, tau, seed=13)
    # half of the rows have a history, whose columns (some lead) only the repetition could change: 1
    c = rp.make_case(T, V, dtype=dtype, history=70, penalties=False, seed=14)
    c.logits = z
    c.kw["tokens"][::5] = z[0].argmax()
    c.kw["temperature"] = torch.full((T,), tau)
    tops = z.double().max(1).values
    c.targets = torch.stack([torch.nonzero(z[t].double() == tops[t])[0, 0] if t % 2 else z[t].double().argsort()[-2 - t]
                             for t in range(T)])
    zg, tg, rules = rp.cuda_case(rk, c, shift)
    logp, lse = rk.logp_from_logits_rules(zg, tg, rules)
    logp, lse = logp.double().cpu().numpy(), lse.double().cpu().numpy()
    t32 = float(c.kw["temperature"][0])
    for t in range(T):
        d = (float(tops[t]) - z[t].double().numpy()) / t32
        ls = float(np.log(np.exp(-d).sum()))
        k = int(c.targets[t])
        assert abs(logp[t] - (-d[k] - ls)) <= close_logp_bound(d[k], V, ls), (t, logp[t], -d[k] - ls)
        ref = float(tops[t]) / t32 + ls
        assert abs(lse[t] - ref) <= close_lse_bound(ref, V, ls), (t, lse[t], ref)
    assert rk.get_device_error() == 0


# p = exp(x - lse): sum_bound for the forward's sum; 1 / tau to 2^-45 of x; of the difference D = x - lse two
# roundings and one in the exponent (log2e: one more); ex2 4u.  Then hot - p and the products with g, 1 / tau.
def close_grad_bound(g, slope, hot, p, x, lse, ls, V):
    D = np.where(p > 0, np.abs(x - lse), 0.0)
    rel = sum_bound(V, ls) + np.abs(x) * 2.0 ** -45 + U * (5 * D + 5)
    return 1.01 * abs(g) * slope * (p * rel + 5 * U * np.abs(hot - p) + 2e-38) + 1e-37


@pytest.mark.parametrize("dtype,size,tau", [
    (BF16, 2.0, 1.0), (BF16, 20.0, 0.1), (BF16, 20.0, 1e-2), (BF16, 20.0, 1e-4), (BF16, 20.0, 1e-6),
    (FP32, 20.0, 1e-2), (FP32, 20.0, 1e-3), (FP32, 20.0, 1e-4), (FP32, 20.0, 1e-5), (FP32, 20.0, 1e-6),
    (FP32, 3e7, 1.0), (BF16, 3e8, 1.0)])
@pytest.mark.parametrize("shift", [0, 1])
def test_gradient_end_to_end_at_low_temperatures(rk, dtype, size, tau, shift):
    T, V = 14, 9001
    c = rp.make_case(T, V, dtype=dtype, history=70, penalties=False, seed=15)
    c.logits = leading(T, V, dtype, size, tau, seed=16)
    c.logits[0, 4000] = c.logits[0].max().abs() * 2  # one token has all there is
    c.kw["tokens"][::5] = c.logits[1].argmax()
    c.kw["temperature"] = torch.full((T,), tau)
    for t in range(T):
        c.targets[t] = c.logits[t].argmax() if t % 2 == 0 else c.logits[t].double().argsort()[-2 - t]
    zg, tg, rules = rp.cuda_case(rk, c, shift)
    g = torch.randn(T, generator=torch.Generator().manual_seed(2))
    logp32, lse32 = rk.logp_from_logits_rules(zg, tg, rules)
    logp, lse = rk.logp_from_logits_rules(zg, tg, rules, lse_dtype=torch.float64)
    assert lse.dtype == torch.float64 and torch.equal(logp, logp32)
    from32 = rk.logp_from_logits_rules_bwd(zg, tg, rules, lse32, g.to(DEV)).double().cpu().numpy()
    got = {d: rk.logp_from_logits_rules_bwd(zg, tg, rules, lse, g.to(DEV), out_dtype=d).double().cpu().numpy()
           for d in (FP32, BF16)}
    lse = lse.cpu().numpy()
    t32 = float(c.kw["temperature"][0])
    for t in range(T):
        x = c.logits[t].double().numpy() / t32
        d = x.max() - x
        ls = float(np.log(np.exp(-d).sum()))
        ref = x.max() + ls
        assert abs(lse[t] - ref) <= sum_bound(V, ls) + abs(ref) * 2.0 ** -50
        p = np.exp(-d - ls)
        hot = np.arange(V) == int(c.targets[t])
        want = float(g[t]) * (hot - p) / t32
        bound = close_grad_bound(float(g[t]), 1 / t32, hot, p, x, ref, ls, V)
        for o, dz in got.items():
            b = bound + rp.half_step(o, np.abs(want) + bound)
            bad = np.abs(dz[t] - want) > b
            assert not bad.any(), (t, o, np.flatnonzero(bad)[:4], dz[t][bad][:4], want[bad][:4])
        # an fp32 lse: its quotient and its sum are rounded
        more = 1.01 * abs(float(g[t])) / t32 * p * np.expm1(2 * U * abs(ref))
        assert np.all(np.abs(from32[t] - want) <= bound * (1 + np.expm1(2 * U * abs(ref))) + more), t
    assert rk.get_device_error() == 0


def test_the_rows_without_a_probability_with_a_64_bit_lse(rk):
    V = 9000
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(1)).to(DEV)
    z[1] = -float("inf")
    z[2, 77] = float("nan")
    z[3] = torch.finfo(FP32).min
    mask = torch.full((6, (V + 31) // 32), -1, dtype=torch.int32, device=DEV)
    mask[4] = 0
    tg = torch.tensor([5, 5, 5, 5, 5, -1], device=DEV)
    rules = rk.LogitsRules(temperature=torch.full((6,), 1.0, device=DEV), mask=mask)
    logp32, lse32 = rk.logp_from_logits_rules(z, tg, rules)
    out = torch.empty(6, dtype=torch.float64, device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules, lse=out)
    assert lse is out and torch.equal(torch.nan_to_num(logp, 7.0), torch.nan_to_num(logp32, 7.0))
    for t, want in ((1, -float("inf")), (4, -float("inf")), (5, 0.0)):
        assert float(lse[t]) == want == float(lse32[t])
    assert torch.isnan(lse[2]) and torch.isnan(lse32[2])
    g = torch.ones(6, device=DEV)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g)
    assert bool((d[[1, 4, 5]] == 0).all()) and bool(d[2].isnan().all())
    # a row at the type's lowest value: every p is 1 / V, not the 1 that a rounded lse leaves
    p = float(np.exp(float(z[3, 0].double()) - float(lse[3])))
    others = torch.arange(V, device=DEV) != 5
    assert p == 1.0  # fp64 rounds ln V away there, too
    assert bool((d[3][others] == -1).all())
    low = rk.LogitsRules(temperature=torch.full((6,), 1e-6, device=DEV))
    lp, ls = rk.logp_from_logits_rules(z, tg, low, lse_dtype=torch.float64)
    # past fp32 the log-sum-exp is an infinity in both
    assert float(ls[3]) == -float("inf") and float(lp[3]) == -float("inf")
    assert bool((rk.logp_from_logits_rules_bwd(z, tg, low, ls, g)[3] == 0).all())


def test_refusals_of_a_64_bit_lse(rk):
    c = rp.make_case(4, 64, seed=2)
    z, tg, rules = rp.cuda_case(rk, c)
    lse, g = torch.zeros(4, dtype=torch.float64, device=DEV), torch.zeros(4, device=DEV)
    for call in (lambda: rk.logp_from_logits_rules(z, tg, rules, lse=lse[:3]),
                 lambda: rk.logp_from_logits_rules(z, tg, rules, lse=lse.cpu()),
                 lambda: rk.logp_from_logits_rules(z, tg, rules, lse=torch.zeros(8, dtype=torch.float64, device=DEV)[::2]),
                 lambda: rk.logp_from_logits_rules(z, tg, rules, lse_dtype=torch.bfloat16),
                 lambda: rk.logp_from_logits_rules(z, tg, rules, lse=lse.half()),
                 lambda: rk.logp_from_logits_rules_bwd(z, tg, rules, lse[:3], g),
                 lambda: rk.logp_from_logits_rules_bwd(z, tg, rules, lse.half(), g),
                 lambda: rk.logp_from_logits_rules_bwd(z, tg, rules, None, g)):
        with pytest.raises((ValueError, TypeError)):
            call()
    lib, vp = rk.load_library(), lse.data_ptr()
    ws = torch.empty(rk.logp_from_logits_rules_workspace_size(4, 64), dtype=torch.uint8, device=DEV)
    assert lib.rk_logp_from_logits_rules_lse64(z.data_ptr(), 0, 64, tg.data_ptr(), None, 0, rules.address, 4, 64,
                                               g.data_ptr(), vp + 4, ws.data_ptr(), ws.numel(), None) == 1
    out = torch.empty(4, 64, device=DEV)
    assert lib.rk_logp_from_logits_rules_bwd_lse64(z.data_ptr(), 0, 64, tg.data_ptr(), None, 0, rules.address, 4, 64,
                                                   vp + 4, g.data_ptr(), out.data_ptr(), 1, 64, None) == 1
    assert lib.rk_logp_from_logits_rules_bwd_lse64(z.data_ptr(), 0, 64, tg.data_ptr(), None, 0, rules.address, 4, 64,
                                                   None, g.data_ptr(), out.data_ptr(), 1, 64, None) == 1


@pytest.mark.parametrize("tau", [1.0, 1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_probabilities_of_the_gradient_add_up_under_all_rules(rk, dtype, tau):
    """Forward and backward take the same y of a touched column, whatever it was rounded to: with the 64-bit lse
    the gradient's probabilities add up to 1 at any temperature."""
    T, V = 60, 20001
    c = rp.make_case(T, V, dtype=dtype, packed=True, requests=4, bias=5, mask="mixed", history=90, seed=33)
    c.kw["repetition"] = torch.ones(4)  # dx/dz is 1 / tau then
    c.kw["temperature"] = torch.full((4,), tau)
    c.logits = c.logits * 8
    hot = c.kw["tokens"][0]
    c.logits[::2, hot] = c.logits.double().abs().max().to(dtype)  # a touched column that leads in every other row
    z, tg, rules = rp.cuda_case(rk, c)
    t32 = float(c.kw["temperature"][0])
    logp, lse = rk.logp_from_logits_rules(z, tg, rules, lse_dtype=torch.float64)
    dz = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.ones(T, device=DEV)).double()
    mask, row_mask = c.kw["mask"], c.kw["row_mask"]
    for t in range(T):
        k = int(c.targets[t])
        allowed = int(row_mask[t]) < 0 or int(mask[t, k // 32]) >> (k % 32) & 1
        left = float(dz[t].sum()) * t32 - (1.0 if allowed else 0.0)  # minus the sum of p; a masked target's 1 is not there
        x = max(abs(float(lse[t])), 1.0) * 4
        # every p to sum_bound + 2^-45 x + 5u (D + 1), sum p D <= ln V + 1; the result's own roundings
        bound = sum_bound(V, np.log(V)) + x * 2.0 ** -45 + 5 * U * (np.log(V) + 3) + 6 * U
        assert abs(left + 1.0) <= 1.01 * bound, (t, left)
    assert rk.get_device_error() == 0
