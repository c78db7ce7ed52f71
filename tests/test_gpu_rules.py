"""Logits under sampling rules on the GPU against their 64-bit form, and bitwise against
themselves in other layouts."""
import numpy as np
import pytest
import torch

import rules_plain as rp
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


# vocabularies around a group of 8, a mask word, a warp's 1024 and a block's 8192 columns
CASES = {
    "one_column": dict(T=3, V=1),
    "seven": dict(T=5, V=7, bias=2),
    "odd": dict(T=9, V=33, mask="half"),
    "group_edge": dict(T=4, V=1025, bias=1, mask="mixed"),
    "segment": dict(T=6, V=1024, history=200),
    "slice_edge": dict(T=5, V=8193, mask="few"),
    "slices": dict(T=7, V=20001, bias=5, mask="mixed", history=3000),
    "packed": dict(T=150, V=3001, packed=True, requests=6, bias=3),
    "packed_many": dict(T=700, V=1500, packed=True, requests=90, mask="mixed", history=3),
    "packed_long": dict(T=400, V=9000, packed=True, requests=2, history=500),
    "no_history": dict(T=4, V=500, history=-1, mask="half"),
    "empty_history": dict(T=4, V=500, history=0),
    "history_only": dict(T=6, V=700, penalties=False),
    "strided": dict(T=6, V=1001, ld=1008, bias=1, mask="half"),
    "long_history": dict(T=2, V=600, history=20000),
}


def build(name, dtype=BF16):
    return rp.make_case(dtype=dtype, seed=sum(map(ord, name)), **CASES[name])


@pytest.mark.parametrize("out_dtype", [FP32, BF16])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", list(CASES))
def test_apply(rk, name, dtype, out_dtype):
    c = build(name, dtype)
    z, _, rules = rp.cuda_case(rk, c)
    got = rk.logits_rules_apply(z, rules, out_dtype=out_dtype).double().cpu().numpy()
    for t in range(c.T):
        x, _, size = rp.plain_row(c, t)
        dead = np.isneginf(x)
        assert np.array_equal(np.isneginf(got[t]), dead)
        err = np.abs(got[t] - x)[~dead]
        bound = (rp.x_bound(size) + rp.half_step(out_dtype, np.abs(x) + rp.x_bound(size)))[~dead]
        assert np.all(err <= bound + 1e-37), (t, err.max())
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", list(CASES))
def test_logp_and_gradient(rk, name, dtype):
    c = build(name, dtype)
    z, tg, rules = rp.cuda_case(rk, c)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    g = torch.randn(c.T, generator=torch.Generator().manual_seed(7))
    grads = {d: rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g.to(DEV), out_dtype=d)
             .double().cpu().numpy() for d in (FP32, BF16)}
    lp, ls = logp.double().cpu().numpy(), lse.double().cpu().numpy()
    for t in range(c.T):
        x, slope, size = rp.plain_row(c, t)
        ref, k = rp.plain_lse(x), int(c.targets[t])
        if ref == -np.inf:
            assert ls[t] == -np.inf and lp[t] == -np.inf
            assert all(np.all(d[t] == 0) for d in grads.values())
            continue
        assert abs(ls[t] - ref) <= rp.lse_bound(size, ref), (t, ls[t], ref)
        if np.isneginf(x[k]):
            assert lp[t] == -np.inf
        else:
            assert abs(lp[t] - (x[k] - ref)) <= rp.logp_bound(size, k, x[k] - ref, ref)
        p = np.exp(x - ls[t])  # the call's own lse is its input
        want = float(g[t]) * ((np.arange(c.V) == k) - p) * slope
        for d, got in grads.items():
            bound = rp.grad_bound(float(g[t]), slope, size, p)
            bound = bound + rp.half_step(d, np.abs(want) + bound)
            bad = np.abs(got[t] - want) > bound
            assert not bad.any(), (t, d, np.flatnonzero(bad)[:4])
    assert rk.get_device_error() == 0


def test_gradient_against_differences(rk):
    c = rp.make_case(3, 50, dtype=FP32, bias=2, mask="half", history=30, seed=11)
    z, tg, rules = rp.cuda_case(rk, c)
    for t in range(3):  # an allowed target
        tg[t] = int(np.flatnonzero(np.isfinite(rp.plain_row(c, t)[0]))[1])
    c.targets = tg.cpu()
    _, lse = rk.logp_from_logits_rules(z, tg, rules)
    got = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.ones(3, device=DEV)).double().cpu().numpy()
    c.logits = c.logits.double()
    h = 1e-5
    for t in range(3):
        for v in range(50):
            if abs(float(c.logits[t, v])) < 2 * h:
                continue
            d = []
            for s in (h, -h):
                c.logits[t, v] += s
                x, _, _ = rp.plain_row(c, t)
                d.append(x[int(c.targets[t])] - rp.plain_lse(x))
                c.logits[t, v] -= s
            # the quotient itself is good to h^2 and 1e-16 / h; the kernel to some 1e-6
            assert abs((d[0] - d[1]) / (2 * h) - got[t, v]) < 5e-6


@pytest.mark.parametrize("shift", [0, 1, 3, 4])
@pytest.mark.parametrize("ld", [2049, 2056, 2060])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_address_and_stride_change_no_bit(rk, dtype, ld, shift):
    c = rp.make_case(5, 2049, dtype=dtype, ld=ld, bias=2, mask="mixed", seed=4)
    z, tg, rules = rp.cuda_case(rk, c, shift)
    base = z.contiguous()
    g = torch.randn(5, device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    logp0, lse0 = rk.logp_from_logits_rules(base, tg, rules)
    assert same_bits(logp, logp0) and same_bits(lse, lse0)
    assert same_bits(rk.logits_rules_apply(z, rules), rk.logits_rules_apply(base, rules))
    assert same_bits(rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g),
                     rk.logp_from_logits_rules_bwd(base, tg, rules, lse, g))
    for d in (FP32, BF16):  # an output with its own stride and offset; nothing behind the row is written
        buf = torch.full((5 * 2070 + 8,), 7.0, dtype=d, device=DEV)
        out = buf.as_strided((5, 2049), (2070, 1), storage_offset=shift)
        rk.logits_rules_apply(z, rules, out=out)
        assert same_bits(out, rk.logits_rules_apply(base, rules, out_dtype=d))
        rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out=out)
        assert same_bits(out, rk.logp_from_logits_rules_bwd(base, tg, rules, lse, g, out_dtype=d))
        inside = torch.zeros_like(buf, dtype=torch.bool)
        inside.as_strided((5, 2049), (2070, 1), storage_offset=shift).fill_(True)
        assert bool((buf[~inside] == 7.0).all())


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_every_alignment_of_both_kinds_of_slice(rk, dtype, shift):
    # columns of a slice that is spread over the warps, of a whole one that is not, and of a partial one
    V, ld, n = 2 * 8192 + 77, 2 * 8192 + 80, 20
    c = rp.make_case(n, V, dtype=dtype, ld=ld, packed=True, requests=2, bias=2, mask="mixed", history=60, seed=40 + shift)
    c.logits[3, :8300] = -INF
    c.logits[4, 8100:] = torch.finfo(dtype).min
    aligned, tg, rules = rp.cuda_case(rk, c, 0)
    z, _, _ = rp.cuda_case(rk, c, shift)
    assert same_bits(z, aligned)
    g = torch.randn(n, device=DEV)
    logp, lse = rk.logp_from_logits_rules(aligned, tg, rules)
    got = rk.logp_from_logits_rules(z, tg, rules)
    assert same_bits(got[0], logp) and same_bits(got[1], lse)
    for d in (FP32, BF16):
        want = (rk.logits_rules_apply(aligned, rules, out_dtype=d),
                rk.logp_from_logits_rules_bwd(aligned, tg, rules, lse, g, out_dtype=d))
        for to in (shift, 0, 5):
            buf = torch.full((n * (ld + 3) + 8,), 7.0, dtype=d, device=DEV)
            out = buf.as_strided((n, V), (ld + 3, 1), storage_offset=to)
            inside = torch.zeros_like(buf, dtype=torch.bool)
            inside.as_strided((n, V), (ld + 3, 1), storage_offset=to).fill_(True)
            rk.logits_rules_apply(z, rules, out=out)
            assert same_bits(out, want[0])
            rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out=out)
            assert same_bits(out, want[1])
            assert bool((buf[~inside] == 7.0).all())


@pytest.mark.parametrize("V,ld,shift", [(20000, 20000, 0), (9001, 9001, 1), (9001, 9016, 3)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_results_in_place_of_the_logits(rk, dtype, V, ld, shift):
    # histories of some hundred tokens: warps with more touched columns than lanes
    c = rp.make_case(30, V, dtype=dtype, ld=ld, packed=True, requests=3, bias=2, mask="mixed", history=900, seed=70)
    c.kw["tokens"] %= 700
    z, tg, rules = rp.cuda_case(rk, c, shift)
    g = torch.randn(30, device=DEV)
    _, lse = rk.logp_from_logits_rules(z, tg, rules)
    x = rk.logits_rules_apply(z, rules, out_dtype=dtype)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out_dtype=dtype)
    z2, _, _ = rp.cuda_case(rk, c, shift)
    assert rk.logits_rules_apply(z2, rules, out=z2) is z2 and same_bits(z2, x)
    rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out=z)
    assert same_bits(z, d)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_narrow_matrix_at_its_buffers_first_element(rk, dtype):
    # rows of a few bytes: what lies before the tensor is NaN and is not taken for a logit
    for V in (1, 2, 3, 5, 7):
        for shift in range(1, 8):
            buf = torch.full((9 * V + 24,), NAN, dtype=dtype, device=DEV)
            z = buf[shift:shift + 9 * V].view(9, V)
            z.copy_(torch.randn(9, V))
            base = z.clone()
            rules = rk.LogitsRules(temperature=torch.full((1,), 0.7, device=DEV),
                                   row_request=torch.zeros(9, dtype=torch.int32, device=DEV))
            assert same_bits(rk.logits_rules_apply(z, rules), rk.logits_rules_apply(base, rules))
            tg = torch.full((9,), V - 1, device=DEV)
            a, b = rk.logp_from_logits_rules(z, tg, rules), rk.logp_from_logits_rules(base, tg, rules)
            assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and bool(a[0].isfinite().all())


def test_rows_do_not_depend_on_the_batch(rk):
    # a packed batch of prefixes: each row again alone, as a request of its own, and permuted
    c = rp.make_case(260, 9001, packed=True, requests=3, bias=2, mask="mixed", history=40, seed=21)
    z, tg, rules = rp.cuda_case(rk, c)
    g = torch.randn(c.T, device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    x = rk.logits_rules_apply(z, rules)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g)
    perm = torch.randperm(c.T, generator=torch.Generator().manual_seed(1))
    kw = {k: v.to(DEV) for k, v in c.kw.items()}
    for rows in (perm, torch.tensor([0]), torch.tensor([137, 5]), torch.arange(40, 160)):
        at = rows.to(DEV)
        sub = dict(kw)
        for k in ("row_request", "row_length", "row_mask"):
            sub[k] = kw[k][at].contiguous()
        rr = rk.LogitsRules(**sub)
        lp, ls = rk.logp_from_logits_rules(z[at].contiguous(), tg[at], rr)
        assert same_bits(lp, logp[at]) and same_bits(ls, lse[at])
        assert same_bits(rk.logits_rules_apply(z[at].contiguous(), rr), x[at])
        assert same_bits(rk.logp_from_logits_rules_bwd(z[at].contiguous(), tg[at], rr, ls, g[at]), d[at])
    for t in (3, 100, 259):  # the prefix as a request of its own
        r, L = int(c.kw["row_request"][t]), int(c.kw["row_length"][t])
        a, b = int(c.kw["token_offsets"][r]), int(c.kw["bias_offsets"][r])
        one = dict(tokens=kw["tokens"][a:a + L].clone(), token_offsets=torch.tensor([0, L], device=DEV),
                   bias_ids=kw["bias_ids"][b:b + 2].clone(), bias_values=kw["bias_values"][b:b + 2].clone(),
                   bias_offsets=torch.tensor([0, 2], device=DEV), mask=kw["mask"][t:t + 1].clone(),
                   row_mask=torch.tensor([0 if t % 3 else -1], dtype=torch.int32, device=DEV),
                   **{k: kw[k][r:r + 1].clone() for k in ("temperature", "repetition", "frequency", "presence",
                                                           "prompt_lengths")})
        lp, ls = rk.logp_from_logits_rules(z[t:t + 1].contiguous(), tg[t:t + 1], rk.LogitsRules(**one))
        assert same_bits(lp, logp[t:t + 1]) and same_bits(ls, lse[t:t + 1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("ld", [9000, 9003])
def test_touched_columns_that_lead(rk, dtype, ld):
    # the largest logits are touched ones that the rules push down by a little or by a lot, at
    # ordinary and at very low temperatures, one of them or a hundred: their raw terms must
    # leave no trace in the sum
    V, T = 9000, 24
    c = rp.make_case(T, V, dtype=dtype, history=200, bias=1, mask="mixed", ld=ld, seed=77)
    c.logits = c.logits.clone()
    for t in range(T):
        a, b = int(c.kw["token_offsets"][t]), int(c.kw["token_offsets"][t + 1])
        hot = c.kw["tokens"][a:b].unique()[: 1 if t % 3 else 100]
        c.logits[t, hot] += [12.0, 30.0, 90.0][t % 3]
        c.kw["bias_ids"][t] = int(hot[0]) if len(hot) else 5
        c.kw["bias_values"][t] = [-8.0, -100.0, -float("inf")][t // 3 % 3]
        c.kw["temperature"][t] = [1.0, 0.7, 0.01, 50.0][t % 4]
    z, tg, rules = rp.cuda_case(rk, c)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    for t in range(T):
        x, _, size = rp.plain_row(c, t)
        size = np.where(np.isfinite(size), size, 0.0)
        ref = rp.plain_lse(x)
        assert abs(float(lse[t]) - ref) <= rp.lse_bound(size, ref), t
        k = int(c.targets[t])
        if np.isfinite(x[k]):
            assert abs(float(logp[t]) - (x[k] - ref)) <= rp.logp_bound(size, k, x[k] - ref, ref)


def test_history_that_jumps_and_shrinks(rk):
    # rows of one request whose lengths grow by one, by many, stay, and go back
    c = rp.make_case(12, 5000, packed=True, requests=1, history=4000, bias=1, seed=5)
    n = int(c.kw["token_offsets"][1])
    c.kw["row_length"] = torch.tensor([0, 1, 2, 40, 40, 3900, n, 7, 8, 9, n + 50, -3], dtype=torch.int32)
    z, tg, rules = rp.cuda_case(rk, c)
    x = rk.logits_rules_apply(z, rules).double().cpu().numpy()
    _, lse = rk.logp_from_logits_rules(z, tg, rules)
    for t in range(12):
        ref, _, size = rp.plain_row(c, t)
        assert np.all(np.abs(x[t] - ref) <= rp.x_bound(size))
        assert abs(float(lse[t]) - rp.plain_lse(ref)) <= rp.lse_bound(size, rp.plain_lse(ref))


def test_masked_places_never_matter(rk):
    c = rp.make_case(6, 2500, mask="half", bias=2, seed=8)
    z, tg, rules = rp.cuda_case(rk, c)
    bits = torch.tensor(np.unpackbits(c.kw["mask"].numpy().view(np.uint8), axis=1, bitorder="little")[:, :2500])
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    g = torch.randn(6, device=DEV)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g)
    x = rk.logits_rules_apply(z, rules)
    for value in (NAN, INF, -INF, torch.finfo(BF16).min):
        z2 = torch.where(bits.to(DEV) == 1, z, torch.tensor(value, dtype=BF16, device=DEV))
        lp2, ls2 = rk.logp_from_logits_rules(z2, tg, rules)
        assert same_bits(lp2, logp) and same_bits(ls2, lse)
        assert same_bits(rk.logits_rules_apply(z2, rules), x)
        assert same_bits(rk.logp_from_logits_rules_bwd(z2, tg, rules, lse, g), d)


def test_values_at_the_edges_of_the_type(rk):
    V = 1300
    z = torch.zeros(5, V, dtype=BF16)
    z[0] = -INF          # every logit -inf: as if nothing were left
    z[1, 5] = NAN        # an allowed NaN
    z[2] = torch.finfo(BF16).min
    z[2, 7] = 0.0        # all but one at the type's lowest value
    z[3, ::2] = -INF
    z[4, 3] = INF
    z, tg = z.to(DEV), torch.full((5,), 7, device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rk.LogitsRules())
    assert lse[0] == -INF and logp[0] == -INF
    assert torch.isnan(lse[1]) and torch.isnan(logp[1])
    assert lse[2] == 0 and logp[2] == 0
    assert abs(float(lse[3]) - np.log(650)) < 1e-5 and abs(float(logp[3]) + np.log(650)) < 1e-5
    assert torch.isnan(logp[4])
    d = rk.logp_from_logits_rules_bwd(z, tg, rk.LogitsRules(), lse, torch.ones(5, device=DEV))
    assert bool((d[0] == 0).all()) and bool(torch.isnan(d[1]).all())
    assert bool((d[2] == 0).all())
    assert bool((d[3, ::2] == 0).all()) and abs(float(d[3, 7]) - (1 - 1 / 650)) < 1e-6


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_row_at_the_lowest_value_of_its_type(rk, dtype):
    # lse = lowest + ln V, which rounds to lowest: every p is exp(0) of that rounded lse
    V = 2100
    z = torch.full((2, V), torch.finfo(dtype).min, dtype=dtype, device=DEV)
    tg = torch.tensor([7, 2099], device=DEV)
    for kw in (dict(), dict(temperature=torch.ones(2, device=DEV), presence=torch.ones(2, device=DEV),
                            tokens=torch.tensor([7, 8], device=DEV), token_offsets=torch.tensor([0, 1, 2], device=DEV))):
        rules = rk.LogitsRules(**kw)
        logp, lse = rk.logp_from_logits_rules(z, tg, rules)
        assert bool((lse == torch.finfo(dtype).min).all())
        assert bool((logp + np.log(V) < 1e-5).all()) and bool((logp + np.log(V) > -1e-5).all())
        d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.ones(2, device=DEV))
        assert d[0, 7] == 0 and d[1, 2099] == 0 and d[0, 9] == -1 and bool(torch.isfinite(d).all())
        assert bool((rk.logits_rules_apply(z, rules) == torch.finfo(dtype).min).all())


def test_a_mask_that_leaves_nothing_and_a_bias_of_minus_infinity(rk):
    V = 9000
    mask = torch.full((3, (V + 31) // 32), 0, dtype=torch.int32)
    mask[1, 8] = 1 << 3       # token 259 alone
    mask[2, :] = -1
    kw = dict(mask=mask.to(DEV), bias_ids=torch.tensor([4, 4, 9], device=DEV),
              bias_values=torch.tensor([5.0, -INF, 2.0], device=DEV),
              bias_offsets=torch.tensor([0, 0, 0, 3], device=DEV))
    z = torch.randn(3, V, device=DEV)
    tg = torch.tensor([0, 259, 4], device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rk.LogitsRules(**kw))
    assert lse[0] == -INF and logp[0] == -INF
    one = np.abs(z[1].double().cpu().numpy())[259:260]
    assert abs(float(lse[1]) - float(z[1, 259])) <= rp.lse_bound(one, one[0])
    assert -rp.logp_bound(one, 0, 0.0, one[0]) <= float(logp[1]) <= 0   # never above 0
    assert logp[2] == -INF and torch.isfinite(lse[2])   # banned by the last of its two biases
    d = rk.logp_from_logits_rules_bwd(z, tg, rk.LogitsRules(**kw), lse, torch.ones(3, device=DEV))
    assert bool((d[0] == 0).all()) and bool((d[1, torch.arange(V) != 259] == 0).all())
    assert abs(float(d[1, 259])) <= rp.grad_bound(1.0, 1.0, one[0], 1.0) + rp.lse_bound(one, one[0])
    x = rk.logits_rules_apply(z, rk.LogitsRules(**kw))
    assert x[2, 4] == -INF and x[2, 9] == z[2, 9] + 2 and bool((x[0] == -INF).all())


def test_padding_rows(rk):
    c = rp.make_case(40, 1200, packed=True, requests=4, bias=1, seed=9)
    pad = torch.tensor([0, 1, 17, 39])
    c.kw["row_request"][pad] = -1
    z, tg, rules = rp.cuda_case(rk, c)
    z[pad] = NAN
    tg[5] = -100
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    out = torch.full((40, 1200), 3.0, device=DEV)
    rk.logits_rules_apply(z, rules, out=out)
    assert bool((out[pad] == 3.0).all()) and not bool((out[2] == 3.0).all())
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.full((40,), 1.0, device=DEV))
    for t in [5] + pad.tolist():
        assert logp[t] == 0 and lse[t] == 0 and bool((d[t] == 0).all())
    # cu_seqlens bounds the active rows in the same way
    cu = torch.tensor([3, 20, 30], dtype=torch.int32, device=DEV)
    lp2, ls2 = rk.logp_from_logits_rules(z, tg, rules, cu)
    assert bool((lp2[:3] == 0).all()) and bool((lp2[30:] == 0).all())
    assert same_bits(lp2[3:30], logp[3:30]) and same_bits(ls2[3:30], lse[3:30])
    d2 = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.full((40,), 1.0, device=DEV), cu)
    assert bool((d2[:3] == 0).all()) and same_bits(d2[3:30], d[3:30])
    assert rk.get_device_error() == 0


def test_unusable_rules_give_nan_and_the_error_word(rk):
    # every fault sits in one row or request; the bounds checks of the kernel turn it into NaN
    def call(change, rows, bit):
        c = rp.make_case(8, 1100, packed=True, requests=4, bias=2, mask="mixed", history=6, seed=12)
        c.kw["row_request"] = torch.tensor([0, 0, 1, 1, 2, 2, 3, 3], dtype=torch.int32)
        c.kw["row_length"] = torch.tensor([0, 1] * 4, dtype=torch.int32)
        good = rp.cuda_case(rk, c)
        ok_logp, ok_lse = rk.logp_from_logits_rules(*good)
        assert rk.get_device_error() == 0
        change(c)
        z, tg, rules = rp.cuda_case(rk, c)
        logp, lse = rk.logp_from_logits_rules(z, tg, rules)
        assert rk.get_device_error() == bit
        x = rk.logits_rules_apply(z, rules)
        d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.ones(8, device=DEV))
        assert rk.get_device_error() == bit
        for t in range(8):
            if t in rows:
                assert torch.isnan(logp[t]) and torch.isnan(lse[t]) and bool(torch.isnan(d[t]).all())
                if bit == rk.DEVERR_RULES:
                    assert bool(torch.isnan(x[t]).all())
            else:
                assert same_bits(logp[t:t + 1], ok_logp[t:t + 1]) and not bool(torch.isnan(d[t]).any())

    def put(name, at, v):
        def f(c):
            c.kw[name][at] = v
        return f
    R = rk.DEVERR_RULES
    call(put("row_request", 2, 4), [2], R)
    call(put("row_request", 2, -7), [2], R)
    call(put("row_request", 2, 2 ** 31 - 1), [2], R)
    call(put("row_mask", 4, 8), [4], R)
    for v in (0.0, -1.0, NAN, INF, 1e-7, 1e7):
        call(put("temperature", 1, v), [2, 3], R)
        call(put("repetition", 3, v), [6, 7], R)
    call(put("token_offsets", 0, -1), [0, 1], R)
    call(put("token_offsets", 4, 2 ** 40), [6, 7], R)
    call(put("bias_offsets", 4, 9), [6, 7], R)

    def crossed(c):
        c.kw["token_offsets"][1] = c.kw["token_offsets"][2] + 1
    call(crossed, [2, 3], R)

    def target(c):
        c.targets[3] = 1100
    call(target, [3], rk.DEVERR_TARGET_RANGE)


def test_too_many_biases(rk):
    z = torch.randn(2, 70000, device=DEV)
    tg = torch.zeros(2, dtype=torch.int64, device=DEV)
    for n, bit in ((65534, 0), (65535, rk.DEVERR_RULES)):
        rules = rk.LogitsRules(bias_ids=torch.arange(n, device=DEV), bias_values=torch.arange(n, device=DEV) * 1e-3,
                               bias_offsets=torch.tensor([0, n, n], device=DEV))
        x = rk.logits_rules_apply(z, rules)
        assert rk.get_device_error() == bit
        assert same_bits(x[1], z[1])
        if bit:
            assert bool(torch.isnan(x[0]).all())
        else:
            assert same_bits(x[0, :n], z[0, :n] + torch.arange(n, device=DEV) * 1e-3) and same_bits(x[0, n:], z[0, n:])


def test_ids_outside_the_vocabulary_are_passed_over(rk):
    c = rp.make_case(6, 1030, history=12, bias=3, seed=14)
    n = c.kw["tokens"].numel()
    c.kw["tokens"][:: 3] = torch.tensor([-1, 1030, 1 << 40, -(1 << 40), 1031, 5000] * n)[: len(range(0, n, 3))]
    c.kw["bias_ids"][::4] = 1030
    c.kw["bias_ids"][1] = -5
    z, tg, rules = rp.cuda_case(rk, c)
    x = rk.logits_rules_apply(z, rules).double().cpu().numpy()
    for t in range(6):
        ref, _, size = rp.plain_row(c, t)
        assert np.all(np.abs(x[t] - ref) <= rp.x_bound(size))
    assert rk.get_device_error() == 0


def test_no_rows(rk):
    z = torch.empty(0, 100, dtype=BF16, device=DEV)
    tg = torch.empty(0, dtype=torch.int64, device=DEV)
    e = torch.empty(0, device=DEV)
    r = rk.LogitsRules()
    assert rk.logits_rules_apply(z, r).shape == (0, 100)
    assert rk.logp_from_logits_rules(z, tg, r)[0].shape == (0,)
    assert rk.logp_from_logits_rules_bwd(z, tg, r, e, e).shape == (0, 100)


def test_offsets_past_32_bits(rk):
    # 40000 rows of 60000 columns are 2.4e9 logits: the last rows against the same rows alone
    T, V = 40000, 60000
    z = torch.empty(T, V, dtype=BF16, device=DEV)
    z[:8] = torch.randn(8, V, device=DEV)
    z[-8:] = z[:8]
    z[8:-8] = 0
    tg = torch.full((T,), -1, device=DEV)
    tg[-8:] = torch.arange(8, device=DEV) * 7000
    rules = rk.LogitsRules(temperature=torch.full((1,), 0.7, device=DEV),
                           row_request=torch.zeros(T, dtype=torch.int32, device=DEV))
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    small = rk.LogitsRules(temperature=torch.full((1,), 0.7, device=DEV),
                           row_request=torch.zeros(8, dtype=torch.int32, device=DEV))
    lp, ls = rk.logp_from_logits_rules(z[:8].contiguous(), tg[-8:].contiguous(), small)
    assert same_bits(logp[-8:], lp) and same_bits(lse[-8:], ls) and bool((logp[:-8] == 0).all())
    g = torch.ones(T, device=DEV)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, out_dtype=BF16)
    want = rk.logp_from_logits_rules_bwd(z[:8].contiguous(), tg[-8:].contiguous(), small, ls, g[:8],
                                         out_dtype=BF16)
    assert same_bits(d[-8:], want) and bool((d[:8] == 0).all())
    x = rk.logits_rules_apply(z, rules, out_dtype=BF16)
    assert same_bits(x[-8:], x[:8]) and not bool((x[:8] == 0).all())


def test_on_another_stream_and_in_a_graph(rk):
    c = rp.make_case(30, 20000, packed=True, requests=3, bias=2, mask="mixed", seed=31)
    z, tg, _ = rp.cuda_case(rk, c)
    kw = {k: v.to(DEV) for k, v in c.kw.items()}
    rules = rk.LogitsRules(**kw)
    g = torch.randn(30, device=DEV)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    x = rk.logits_rules_apply(z, rules)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(rk.logp_from_logits_rules_workspace_size(30, 20000), dtype=torch.uint8, device=DEV)
    out = [torch.empty(30, device=DEV), torch.empty(30, device=DEV), torch.empty_like(x), torch.empty_like(d)]

    def step(stream):
        rk.logp_from_logits_rules(z, tg, rules, out=out[0], lse=out[1], workspace=ws, stream=stream)
        rk.logits_rules_apply(z, rules, out=out[2], stream=stream)
        rk.logp_from_logits_rules_bwd(z, tg, rules, out[1], g, out=out[3], stream=stream)
    step(side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(out, (logp, lse, x, d)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    # new logits, tokens, lengths and masks in the captured tensors
    c2 = rp.make_case(30, 20000, packed=True, requests=3, bias=2, mask="mixed", seed=32)
    z2, tg2, rules2 = rp.cuda_case(rk, c2)
    n = min(kw["tokens"].numel(), c2.kw["tokens"].numel())
    z.copy_(z2)
    kw["tokens"][:n] = c2.kw["tokens"][:n].to(DEV)
    kw["mask"].copy_(c2.kw["mask"])
    kw["row_length"] -= 1
    for _ in range(2):
        [o.fill_(NAN) for o in out]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        logp, lse = rk.logp_from_logits_rules(z, tg, rules)
        want = (logp, lse, rk.logits_rules_apply(z, rules), rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g))
        assert all(same_bits(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_what_is_not_a_number_in_an_allowed_place(rk, dtype, bad):
    # in a touched column (9), a plain one, and the last; rows 0 and 4 have none, row 5 masks it
    c = rp.make_case(6, 9001, dtype=dtype, mask="half", seed=77)
    for t, v in ((1, 9), (2, 5000), (3, 9000), (5, 5001)):
        c.logits[t, v] = bad
        c.kw["mask"][t, v // 32] |= torch.tensor(1 << 31, dtype=torch.int64).to(torch.int32) if v % 32 == 31 else 1 << v % 32
    c.kw["mask"][5, 5001 // 32] &= ~(1 << 5001 % 32)
    c.kw["tokens"][c.kw["token_offsets"][1]:c.kw["token_offsets"][2]] = 9
    z, tg, rules = rp.cuda_case(rk, c)
    logp, lse = rk.logp_from_logits_rules(z, tg, rules)
    d = rk.logp_from_logits_rules_bwd(z, tg, rules, lse, torch.ones(6, device=DEV))
    sick = torch.tensor([False, True, True, True, False, False], device=DEV)
    assert bool((logp.isnan() == sick).all()) and bool((lse.isnan() == sick).all())
    assert bool(d[sick].isnan().all()) and bool(d[~sick].isfinite().all())


def test_calls_on_two_streams_at_once(rk):
    cases = [rp.make_case(200, 40000, packed=True, requests=3, bias=2, mask="mixed", seed=s) for s in (80, 81)]
    args = [rp.cuda_case(rk, c) for c in cases]
    ids = torch.randint(0, 3000, (9000,), device=DEV)
    d = torch.randn(9000, 256, device=DEV)
    want = [rk.logp_from_logits_rules(*a[:2], a[2]) + (rk.embedding_bwd(d, ids, 3000 + i),) for i, a in enumerate(args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [[], []]
        for i, (a, st) in enumerate(zip(args, streams)):
            got[i] = rk.logp_from_logits_rules(*a[:2], a[2], stream=st) + (rk.embedding_bwd(d, ids, 3000 + i, stream=st),)
        torch.cuda.synchronize()
        assert all(same_bits(x, y) for g, w in zip(got, want) for x, y in zip(g, w))


@pytest.mark.parametrize("bias", [0, 1])
@pytest.mark.parametrize("history", [0, 1, 2])
def test_requests_without_a_history_between_others(rk, history, bias):
    # several rows to a block, each of a request of its own, many with no token and no bias
    c = rp.make_case(200, 30000, history=history, bias=bias, seed=50 + history)
    if bias:  # every third request has the biases
        n = [1 if r % 3 == 0 else 0 for r in range(200)]
        c.kw["bias_offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]))
    c.kw["tokens"] %= 5
    z, _, rules = rp.cuda_case(rk, c)
    x = rk.logits_rules_apply(z, rules).double().cpu().numpy()
    for t in range(200):
        want, _, size = rp.plain_row(c, t)
        assert np.all(np.abs(x[t] - want) <= rp.x_bound(size) + 1e-37), t
    # the same as rows of packed sequences of three, whose first has seen nothing
    rq = torch.arange(200, dtype=torch.int32) // 3
    ln = torch.arange(200, dtype=torch.int32) % 3
    c.kw.update(row_request=rq, row_length=ln)
    z, tg, rules = rp.cuda_case(rk, c)
    x = rk.logits_rules_apply(z, rules).double().cpu().numpy()
    for t in range(200):
        want, _, size = rp.plain_row(c, t)
        assert np.all(np.abs(x[t] - want) <= rp.x_bound(size) + 1e-37), t


def test_memory_made_by_a_call_is_its_streams(rk):
    """What a call on a side stream allocates does not come out of the current stream's
    freed memory, which work on that stream may still be using."""
    c = rp.make_case(6, 3000, seed=3)
    z, tg, rules = rp.cuda_case(rk, c)
    lse, g = torch.zeros(6, device=DEV), torch.zeros(6, device=DEV)
    E = torch.randn(50, 64, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for call in (lambda s: rk.logits_rules_apply(z, rules, stream=s),
                 lambda s: rk.logp_from_logits_rules(z, tg, rules, stream=s),
                 lambda s: rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g, stream=s),
                 lambda s: rk.embedding(tg % 50, E, stream=s),
                 lambda s: rk.embedding_bwd(E[:6], tg % 50, 50, stream=s)):
        torch.cuda.empty_cache()
        freed = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (24, 512, 1024, 1 << 14, 72000, 1 << 18) * 4]
        places = {f.data_ptr() for f in freed}
        del freed
        res = call(side)
        res = res if isinstance(res, tuple) else (res,)
        assert not places & {r.data_ptr() for r in res}
        side.synchronize()
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        assert all(same_bits(a, b) for a, b in zip(res, want))


def test_binding_refusals(rk):
    c = rp.make_case(4, 64, mask="half", seed=2)
    z, tg, rules = rp.cuda_case(rk, c)
    kw = {k: v.to(DEV) for k, v in c.kw.items()}
    for bad in (dict(temperature=kw["temperature"][:3]), dict(temperature=kw["temperature"].double()),
                dict(token_offsets=kw["token_offsets"][:4]), dict(mask=kw["mask"][:3]),
                dict(tokens=kw["tokens"].int()), dict(row_length=kw["prompt_lengths"][:3]),
                dict(mask=kw["mask"].t().contiguous().t()), dict(mask=kw["mask"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            rk.LogitsRules(**{**kw, **bad})
    for half in (("tokens",), ("token_offsets",), ("prompt_lengths",), ("row_length",), ("row_mask",)):
        with pytest.raises(ValueError):
            rk.LogitsRules(**{k: kw.get(k, torch.zeros(4, dtype=torch.int32, device=DEV)) for k in half})
    with pytest.raises(ValueError):
        rk.LogitsRules(bias_ids=torch.zeros(4, dtype=torch.int64, device=DEV))
    lse, g = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    for call in (lambda: rk.logits_rules_apply(z[:3], rules), lambda: rk.logits_rules_apply(z.half(), rules),
                 lambda: rk.logits_rules_apply(z[:, ::2], rules),
                 lambda: rk.logits_rules_apply(z[:, :32].contiguous(), rules),
                 lambda: rk.logits_rules_apply(z, None),
                 lambda: rk.logits_rules_apply(z, rules, out=torch.empty(4, 63, device=DEV)),
                 lambda: rk.logits_rules_apply(z, rules, out_dtype=torch.float16),
                 lambda: rk.logits_rules_apply(z[:1].expand(4, 64), rules),
                 lambda: rk.logp_from_logits_rules(z, tg[:3], rules),
                 lambda: rk.logp_from_logits_rules(z, tg.int(), rules),
                 lambda: rk.logp_from_logits_rules(z, tg, rules, workspace=torch.empty(8, device=DEV)),
                 lambda: rk.logp_from_logits_rules_bwd(z, tg, rules, lse[:3], g),
                 lambda: rk.logp_from_logits_rules_bwd(z, tg, rules, lse, g.double())):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(rk.RkError, match="WORKSPACE"):
        rk.logp_from_logits_rules(z, tg, rules, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
