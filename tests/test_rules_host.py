"""The 64-bit forms of the sampling rules against facts other than themselves, and what the
binding and the C ABI refuse before anything is launched (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import rules_plain as rp


# ---- the plain form ----

def test_without_rules_it_is_log_softmax():
    c = rp.make_case(5, 37, penalties=False, history=-1, seed=1)
    for t in range(5):
        x, slope, _ = rp.plain_row(c, t)
        z = c.logits[t].double()
        assert np.array_equal(x, z.numpy()) and np.all(slope == 1)
        assert abs(rp.plain_lse(x) - float(torch.logsumexp(z, 0))) < 1e-13


def test_one_token_by_hand():
    # z = [2, -2, 1], token 0 in the prompt, token 1 produced twice, token 2 never
    c = rp.Case(torch.tensor([[2.0, -2.0, 1.0]]), torch.tensor([0]),
                dict(temperature=torch.tensor([0.5]), repetition=torch.tensor([2.0]),
                     frequency=torch.tensor([0.25]), presence=torch.tensor([0.125]),
                     tokens=torch.tensor([0, 1, 1]), token_offsets=torch.tensor([0, 3]),
                     prompt_lengths=torch.tensor([1], dtype=torch.int32)), 3)
    x, slope, _ = rp.plain_row(c, 0)
    assert x.tolist() == [2.0, 2 * (-4 - 0.5 - 0.125), 2.0]
    assert slope.tolist() == [1.0, 4.0, 2.0]


def test_the_slope_is_the_difference_quotient_of_logp():
    c = rp.make_case(4, 29, dtype=torch.float32, bias=3, mask="half", seed=3)
    c.logits = c.logits.double()
    for t in range(4):
        x, slope, _ = rp.plain_row(c, t)
        allowed = np.flatnonzero(np.isfinite(x))
        tgt = int(allowed[0])
        p = np.exp(x - rp.plain_lse(x))
        grad = ((np.arange(29) == tgt) - p) * slope
        h = 1e-6
        for v in range(29):
            if abs(float(c.logits[t, v])) < 10 * h:
                continue
            d = []
            for s in (h, -h):
                c.logits[t, v] += s
                xx, _, _ = rp.plain_row(c, t)
                d.append(xx[tgt] - rp.plain_lse(xx))
                c.logits[t, v] -= s
            assert abs((d[0] - d[1]) / (2 * h) - grad[v]) < 1e-7


def test_the_embedding_gradient_is_the_transposed_lookup():
    rng = np.random.RandomState(0)
    ids = rng.randint(-1, 9, 50)
    d = torch.randn(50, 4, dtype=torch.float64)
    dE, _, count = rp.plain_embedding_bwd(d, ids, 9, 2.0)
    onehot = (ids[:, None] == np.arange(9)).astype(float)
    assert np.allclose(dE, 2.0 * onehot.T @ d.numpy(), atol=1e-12)
    assert count.tolist() == onehot.sum(0).astype(int).tolist()


# ---- refusals of the C ABI ----

@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


FAKE = 4096  # an address that a refused call never reads
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def rules_struct(rk, **kw):
    s = rk._RulesStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def apply_status(rk, s, T=4, V=100, logits=FAKE, lt=0, ld=100, out=FAKE, ot=1, ldo=100):
    return rk.load_library().rk_logits_rules_apply(logits, lt, ld, ctypes.addressof(s), T, V, out, ot,
                                                   ldo, None)


def test_apply_refusals(rk):
    s = rules_struct(rk)
    assert apply_status(rk, s, T=0) == OK
    for bad in (dict(T=-1), dict(V=0), dict(lt=2), dict(ot=-1), dict(logits=None), dict(out=None),
                dict(ld=99), dict(ldo=99), dict(logits=FAKE + 1), dict(out=FAKE + 2)):
        assert apply_status(rk, s, **bad) == INVALID, bad
    assert apply_status(rk, s, V=1 << 31, ld=1 << 31, ldo=1 << 31) == UNSUPPORTED
    assert apply_status(rk, s, T=1 << 31) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(num_requests=-1), dict(temperature=FAKE), dict(tokens=FAKE, token_offsets=FAKE),
    dict(num_requests=4, tokens=FAKE), dict(num_requests=4, prompt_lengths=FAKE),
    dict(num_requests=4, bias_ids=FAKE), dict(num_requests=4, bias_ids=FAKE, bias_values=FAKE),
    dict(num_requests=3, temperature=FAKE),     # 4 rows, no row_request
    dict(mask=FAKE, mask_rows=3),               # 4 rows, no row_mask
    dict(num_requests=4, num_tokens=-1), dict(num_bias=-1), dict(mask_rows=-1),
])
def test_rules_refusals(rk, kw):
    s = rules_struct(rk, **kw)
    assert apply_status(rk, s) == INVALID
    lib = rk.load_library()
    big = 1 << 30
    assert lib.rk_logp_from_logits_rules(FAKE, 0, 100, FAKE, None, 0, ctypes.addressof(s), 4, 100, FAKE,
                                         None, FAKE, big, None) == INVALID
    assert lib.rk_logp_from_logits_rules_bwd(FAKE, 0, 100, FAKE, None, 0, ctypes.addressof(s), 4, 100,
                                             FAKE, FAKE, FAKE, 1, 100, None) == INVALID


def test_logp_refusals(rk):
    lib = rk.load_library()
    s = rules_struct(rk)
    size = rk.logp_from_logits_rules_workspace_size
    assert size(0, 100) == 0
    # eight (max, sum) pairs per 8192 columns and the target's logit, per row
    assert size(300, 9000) == (300 * 16 * 8 + 300 * 4 + 255) // 256 * 256

    def logp(T=4, V=100, z=FAKE, ty=0, ld=100, tg=FAKE, cu=None, ns=0, rules=ctypes.addressof(s),
             out=FAKE, ws=FAKE, wb=1 << 20):
        return lib.rk_logp_from_logits_rules(z, ty, ld, tg, cu, ns, rules, T, V, out, None, ws, wb, None)

    def bwd(T=4, V=100, z=FAKE, ty=0, ld=100, tg=FAKE, lse=FAKE, g=FAKE, out=FAKE, ot=0, ldo=100,
            rules=ctypes.addressof(s)):
        return lib.rk_logp_from_logits_rules_bwd(z, ty, ld, tg, None, 0, rules, T, V, lse, g, out, ot,
                                                 ldo, None)
    assert logp(T=0) == OK and bwd(T=0) == OK
    for bad in (dict(T=-1), dict(V=0), dict(z=None), dict(tg=None), dict(out=None), dict(ld=99),
                dict(ty=7), dict(cu=FAKE, ns=-1), dict(rules=None), dict(z=FAKE + 1), dict(ws=FAKE + 8)):
        assert logp(**bad) == INVALID, bad
    assert logp(ws=None) == WORKSPACE and logp(wb=8) == WORKSPACE
    for bad in (dict(T=-1), dict(V=0), dict(z=None), dict(tg=None), dict(lse=None), dict(g=None),
                dict(out=None), dict(ldo=99), dict(ot=3), dict(rules=None), dict(out=FAKE + 1)):
        assert bwd(**bad) == INVALID, bad


def test_embedding_refusals(rk):
    lib = rk.load_library()

    def fwd(T=4, H=8, V=10, ids=FAKE, cu=None, ns=0, E=FAKE, et=0, out=FAKE, ot=1):
        return lib.rk_embedding(ids, cu, ns, E, et, T, H, V, 1.0, out, ot, None)

    def bwd(T=4, H=8, V=10, d=FAKE, dt=0, ids=FAKE, order=None, n=0, dE=FAKE, acc=0, ws=FAKE,
            wb=1 << 24):
        return lib.rk_embedding_bwd(d, dt, ids, None, 0, T, H, V, 1.0, order, n, dE, acc, ws, wb, None)
    assert fwd(T=0) == OK
    for bad in (dict(T=-1), dict(H=0), dict(V=0), dict(ids=None), dict(E=None), dict(out=None),
                dict(et=2), dict(ot=2), dict(E=FAKE + 1), dict(out=FAKE + 2), dict(cu=FAKE, ns=-1)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(V=1 << 31) == UNSUPPORTED and fwd(H=1 << 31) == UNSUPPORTED
    for bad in (dict(T=-1), dict(H=0), dict(V=0), dict(d=None), dict(dt=5), dict(ids=None),
                dict(dE=None), dict(acc=2), dict(order=FAKE, n=-1), dict(dE=FAKE + 2), dict(ws=FAKE + 8)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(ws=None) == WORKSPACE and bwd(wb=16) == WORKSPACE
    assert bwd(V=(1 << 31) - 1) == UNSUPPORTED
    assert rk.embedding_bwd_workspace_size(0, 8, 10) == 0


# ---- refusals of the binding ----

def test_binding_refuses_cpu_tensors(rk):
    c = rp.make_case(3, 40)
    with pytest.raises(ValueError, match="CUDA"):
        rk.LogitsRules(**c.kw)
    with pytest.raises(ValueError, match="CUDA"):
        rk.logits_rules_apply(c.logits, rk.LogitsRules())
    with pytest.raises(ValueError, match="CUDA"):
        rk.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        rk.embedding_bwd(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), 4)
