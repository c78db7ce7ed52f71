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
