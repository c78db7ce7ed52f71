"""The embedding lookup and its gradient on the GPU against their 64-bit forms, in other
layouts, and in a step with the operators around them."""
import numpy as np
import pytest
import torch

import rules_plain as rp
from helpers import same_bits
from invariant_rl_logprob_gb300 import synth

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


def ids_like(T, V, seed, hot=0.5):
    """Ids of which a share falls on a few tokens, and some are padding."""
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(0, V, (T,), generator=g)
    b = torch.randint(0, min(V, 3), (T,), generator=g)
    ids = torch.where(torch.rand(T, generator=g) < hot, b, a)
    ids[torch.rand(T, generator=g) < 0.1] = -1
    return ids


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (5, 9, 7), (64, 100, 8), (33, 50, 1000), (300, 1000, 264), (7, 20, 4097)])
def test_lookup_is_the_rounded_product(rk, T, V, H, dtype, out_dtype):
    ids = ids_like(T, V, seed=T + H)
    E = torch.randn(V, H, generator=torch.Generator().manual_seed(1)).to(dtype)
    got = rk.embedding(ids.to(DEV), E.to(DEV), scale=1.7, out_dtype=out_dtype)
    want = torch.where((ids >= 0)[:, None], E[ids.clamp(min=0)].float() * torch.tensor(1.7), 0.0).to(out_dtype)
    assert same_bits(got, want)
    assert rk.get_device_error() == 0


def test_lookup_rows(rk):
    E = torch.randn(50, 24, device=DEV)
    ids = torch.tensor([3, 50, -1, 49, 1 << 40, 0], device=DEV)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    out = rk.embedding(ids, E, cu)
    assert rk.get_device_error() == rk.DEVERR_TARGET_RANGE
    assert bool(torch.isnan(out[1]).all()) and bool((out[2] == 0).all()) and bool((out[4:] == 0).all())
    assert same_bits(out[0], E[3]) and same_bits(out[3], E[49])
    # an unaligned table and output give the same bits
    buf = torch.empty(50 * 24 + 1, device=DEV)
    E2 = buf[1:].view(50, 24)
    E2.copy_(E)
    out2 = torch.empty(6 * 24 + 1, device=DEV)[1:].view(6, 24)
    ids[4] = -1
    ids[1] = 7
    assert same_bits(rk.embedding(ids, E2, out=out2), rk.embedding(ids, E))
    assert rk.embedding(ids[:0], E).shape == (0, 24)


# ids of no, one and many pieces; sorts of one to three passes, in one block, by tiles whose
# blocks scan the counts, and by tiles with a scan of its own (131072 tokens and more)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,V,H,hot", [(1, 1, 1, 0.0), (3, 5, 7, 0.5), (100, 511, 64, 0.5), (700, 512, 16, 0.9),
                                       (1000, 70000, 8, 0.4), (5000, 300000, 24, 0.5), (9000, 40, 9, 0.0),
                                       (4097, 3, 40, 0.0), (333, 1000, 1030, 0.3), (8192, 600, 8, 0.2),
                                       (8193, 600, 8, 0.2), (140000, 900, 4, 0.1), (9000, 600000, 8, 0.1)])
def test_gradient(rk, T, V, H, hot, dtype):
    ids = ids_like(T, V, seed=T, hot=hot)
    g = torch.Generator().manual_seed(T + 1)
    d = torch.randn(T, H, generator=g).to(dtype)
    old = torch.randn(V, H, generator=g)
    want, mag, count = rp.plain_embedding_bwd(d, ids.numpy(), V, 0.75)
    got = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, scale=0.75).double().cpu().numpy()
    # between a row and its id's total: at most 32 additions in its piece, then one per
    # piece; one product with the scale
    adds = (np.minimum(count, 32) + (count + 31) // 32 + 2)[:, None]
    bound = adds * rp.U * 1.01 * mag
    assert np.all(np.abs(got - want) <= bound)
    assert np.all(got[count == 0] == 0)
    dE = old.to(DEV)
    assert rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, scale=0.75, dE=dE, accumulate=True) is dE
    total = old.double().numpy() + want
    assert np.all(np.abs(dE.double().cpu().numpy() - total) <= bound + rp.U * 1.01 * (np.abs(total) + bound))
    assert same_bits(dE[torch.tensor(count == 0)], old[torch.tensor(count == 0)])
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("T", [9001, 140000])
def test_a_sort_of_four_passes(rk, T):
    V = (1 << 27) + 3
    g = torch.Generator().manual_seed(T)
    some = torch.cat([torch.randint(0, V, (T // 3,), generator=g), torch.tensor([0, V - 1, 1 << 26])])
    ids = some[torch.randint(0, some.numel(), (T,), generator=g)]
    d = torch.randn(T, 1, generator=g)
    dE = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V)
    u, where = ids.unique(return_inverse=True)
    want, mag = torch.zeros(len(u), dtype=torch.float64), torch.zeros(len(u), dtype=torch.float64)
    want.index_add_(0, where, d[:, 0].double())
    mag.index_add_(0, where, d[:, 0].double().abs())
    # fewer than 40 rows an id: 32 additions in a piece, one more per piece, the scale
    assert int(torch.bincount(where).max()) < 40
    assert bool(((dE[u.to(DEV), 0].cpu().double() - want).abs() <= 36 * rp.U * 1.01 * mag).all())
    dE[u.to(DEV)] = 0
    assert not bool(dE.any())


def test_one_token_for_every_row(rk):
    T, H = 70001, 16
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(3))
    got = rk.embedding_bwd(d.to(DEV), torch.full((T,), 5, device=DEV), 9).double().cpu()
    pieces = (T + 31) // 32
    bound = (32 + pieces + 2) * rp.U * 1.01 * d.double().abs().sum(0)
    assert bool(((got[5] - d.double().sum(0)).abs() <= bound).all())
    assert bool((got[torch.arange(9) != 5] == 0).all())


def test_gradient_does_not_depend_on_the_layout(rk):
    T, V, H = 3000, 700, 72
    ids = ids_like(T, V, seed=5)
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(6)).to(BF16)
    base = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V)
    # the same tokens in the same canonical order from other places, between padding and NaN rows
    g = torch.Generator().manual_seed(7)
    P = 5000
    place = torch.randperm(P, generator=g)[:T]
    ids2 = torch.full((P,), -1)
    d2 = torch.full((P, H), float("nan"), dtype=BF16)
    ids2[place], d2[place] = ids, d
    got = rk.embedding_bwd(d2.to(DEV), ids2.to(DEV), V, row_order=place.to(DEV))
    assert same_bits(got, base)
    # out-of-range entries of the order are skipped; cu_seqlens bounds the rows
    order = torch.cat([torch.tensor([-1, P, 1 << 40]), place, torch.tensor([-(1 << 40)])])
    assert same_bits(rk.embedding_bwd(d2.to(DEV), ids2.to(DEV), V, row_order=order.to(DEV)), base)
    lead = 13
    ids3 = torch.cat([torch.zeros(lead, dtype=torch.int64), ids, torch.ones(5, dtype=torch.int64)])
    d3 = torch.cat([torch.full((lead, H), float("nan")), d.float(), torch.full((5, H), float("nan"))]).to(BF16)
    cu = torch.tensor([lead, lead + 100, lead + T], dtype=torch.int32, device=DEV)
    assert same_bits(rk.embedding_bwd(d3.to(DEV), ids3.to(DEV), V, cu), base)
    # an id's row does not depend on the other ids
    keep = (ids == 1) | (ids == 2)
    only = rk.embedding_bwd(d.to(DEV), torch.where(keep, ids, -1).to(DEV), V)
    assert same_bits(only[1:3], base[1:3])
    other = rk.embedding_bwd(d.to(DEV), torch.where(keep, ids, 0).to(DEV), V)
    assert same_bits(other[1:3], base[1:3])
    # an unaligned gradient
    buf = torch.empty(T * H + 1, dtype=BF16, device=DEV)[1:].view(T, H)
    buf.copy_(d)
    assert same_bits(rk.embedding_bwd(buf, ids.to(DEV), V), base)
    dE = torch.empty(V * H + 1, device=DEV)[1:].view(V, H)
    assert same_bits(rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, dE=dE), base)
    assert rk.get_device_error() == 0


def test_rows_named_twice_and_ids_out_of_range(rk):
    d = torch.randn(4, 8, device=DEV)
    ids = torch.tensor([2, 9, 2, 1], device=DEV)
    got = rk.embedding_bwd(d, ids, 3, row_order=torch.tensor([0, 3, 0, 1], device=DEV))
    assert rk.get_device_error() == rk.DEVERR_TARGET_RANGE
    assert same_bits(got[2], d[0] + d[0]) and same_bits(got[1], d[3]) and bool((got[0] == 0).all())


def test_no_tokens(rk):
    dE = torch.full((6, 10), 2.0, device=DEV)
    none = torch.empty(0, 10, device=DEV)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    rk.embedding_bwd(none, ids, 6, dE=dE, accumulate=True)
    assert bool((dE == 2).all())
    rk.embedding_bwd(none, ids, 6, dE=dE)
    assert bool((dE == 0).all())
    d = torch.randn(5, 10, device=DEV)
    for kw in (dict(ids=torch.full((5,), -1, device=DEV)),
               dict(ids=torch.zeros(5, dtype=torch.int64, device=DEV), row_order=ids)):
        dE.fill_(2.0)
        rk.embedding_bwd(d, kw["ids"], 6, row_order=kw.get("row_order"), dE=dE, accumulate=True)
        assert bool((dE == 2).all())
        assert bool((rk.embedding_bwd(d, kw["ids"], 6, row_order=kw.get("row_order")) == 0).all())


def test_offsets_past_32_bits(rk):
    V, H, T = 300000, 8192, 40   # 2.46e9 elements
    E = torch.zeros(V, H, dtype=BF16, device=DEV)
    E[-1] = torch.randn(H, device=DEV)
    ids = torch.full((T,), V - 1, device=DEV)
    assert same_bits(rk.embedding(ids, E), E[-1:].expand(T, H))
    del E
    d = torch.randn(T, H, device=DEV)
    dE = rk.embedding_bwd(d, ids, V)
    want = rk.embedding_bwd(d, torch.zeros(T, dtype=torch.int64, device=DEV), 1)
    assert same_bits(dE[-1], want[0]) and bool((dE[:-1] == 0).all())


def test_on_another_stream_and_in_a_graph(rk):
    T, V, H = 2000, 900, 64
    ids, d = ids_like(T, V, 9).to(DEV), torch.randn(T, H, device=DEV)
    base = rk.embedding_bwd(d, ids, V)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(rk.embedding_bwd_workspace_size(T, H, V), dtype=torch.uint8, device=DEV)
    dE, out = torch.zeros(V, H, device=DEV), torch.empty(T, H, device=DEV)
    torch.cuda.synchronize()
    rk.embedding_bwd(d, ids, V, dE=dE, workspace=ws, stream=side)
    side.synchronize()
    assert same_bits(dE, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rk.embedding_bwd(d, ids, V, dE=dE, workspace=ws, stream=side)
        rk.embedding(ids, dE, out=out, scale=0.5, stream=side)
    ids.copy_(ids_like(T, V, 10))
    d.normal_()
    for _ in range(2):
        ws.fill_(255)
        dE.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = rk.embedding_bwd(d, ids, V)
        assert same_bits(dE, want) and same_bits(out, rk.embedding(ids, want, scale=0.5))


def test_binding_refusals(rk):
    E, ids, d = torch.zeros(5, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(3, 8, device=DEV)
    for call in (lambda: rk.embedding(ids.int(), E), lambda: rk.embedding(ids, E.half()), lambda: rk.embedding(ids, E.t()),
                 lambda: rk.embedding(ids, E, out=torch.empty(3, 7, device=DEV)),
                 lambda: rk.embedding_bwd(d, ids[:2], 5), lambda: rk.embedding_bwd(d, ids, 5, accumulate=True),
                 lambda: rk.embedding_bwd(d, ids, 5, dE=torch.empty(4, 8, device=DEV)),
                 lambda: rk.embedding_bwd(d, ids, 5, dE=torch.empty(5, 8, dtype=BF16, device=DEV)),
                 lambda: rk.embedding_bwd(d, ids, 5, row_order=ids.int())):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(rk.RkError, match="WORKSPACE"):
        rk.embedding_bwd(d, ids, 5, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_decode_then_score_then_tied_gradient(rk):
    """A decoding loop (lm_head, rules, greedy pick, embedding of the pick) and the training
    step on what it produced: the logprob the loop saw comes back bit for bit from the packed
    batch, and both halves of a tied weight's gradient go into one tensor."""
    H, V, R, steps = 128, 3000, 5, 12
    gen = synth.generator(3)
    W = synth.normal_bf16(gen, (V, H), 0.05).to(DEV)
    mix = synth.normal_bf16(gen, (H, H), 0.1).to(DEV)
    prompts = [3, 1, 6, 2, 4]
    first = torch.randint(0, V, (sum(prompts),), generator=gen).split(prompts)
    tokens = torch.zeros(R, 32, dtype=torch.int64, device=DEV)   # room for each request's tokens
    for r in range(R):
        tokens[r, :prompts[r]] = first[r].to(DEV)
    kw = dict(temperature=torch.tensor([0.7, 1.0, 0.9, 1.2, 0.8], device=DEV),
              repetition=torch.tensor([1.1, 1.3, 1.0, 1.2, 1.05], device=DEV),
              frequency=torch.full((R,), 0.3, device=DEV), presence=torch.full((R,), 0.2, device=DEV),
              tokens=tokens.view(-1), token_offsets=torch.arange(R + 1, device=DEV) * 32,
              prompt_lengths=torch.tensor(prompts, dtype=torch.int32, device=DEV))
    length = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    rules = rk.LogitsRules(**kw, row_length=length)
    rows = torch.arange(R, device=DEV)
    hs, picks, seen = [], [], []
    last = tokens[rows, length.long() - 1]
    for _ in range(steps):
        h = rk.embedding(last, W, scale=H ** 0.5) @ mix
        z = rk.lm_head(h, W)
        x = rk.logits_rules_apply(z, rules)
        last = x.argmax(1)
        logp, _ = rk.logp_from_logits_rules(z, last, rules)
        assert bool((logp <= 0).all()) and not bool((x == z).all())
        hs.append(h)
        picks.append(last)
        seen.append(logp)
        tokens[rows, length.long()] = last
        length += 1
    # packed by request, each row with its prefix
    order = [(s, r) for r in range(R) for s in range(steps)]
    h = torch.stack([hs[s][r] for s, r in order])
    tg = torch.stack([picks[s][r] for s, r in order])
    want = torch.stack([seen[s][r] for s, r in order])
    packed = rk.LogitsRules(**kw, row_request=torch.tensor([r for _, r in order], dtype=torch.int32, device=DEV),
                            row_length=torch.tensor([prompts[r] + s for s, r in order], dtype=torch.int32, device=DEV))
    z = rk.lm_head(h, W)
    logp, lse = rk.logp_from_logits_rules(z, tg, packed)
    assert same_bits(logp, want)
    loss = rk.grpo_token_loss(logp, want, torch.ones_like(logp), tg)
    dz = rk.logp_from_logits_rules_bwd(z, tg, packed, lse, loss["grad"])
    dh = dz @ W.float()
    inputs = torch.stack([tokens[r, prompts[r] + s - 1] for s, r in order])
    demb = (dh @ mix.float().t()).to(BF16)
    dW = dz.t() @ h.float()
    ref = dW.double().cpu().numpy()
    more, mag, count = rp.plain_embedding_bwd(demb.cpu(), inputs.cpu().numpy(), V, H ** 0.5)
    got = rk.embedding_bwd(demb, inputs, V, scale=H ** 0.5, dE=dW, accumulate=True).double().cpu().numpy()
    bound = (count + 4)[:, None] * rp.U * mag + 1.01 * rp.U * np.abs(ref + more)
    assert np.all(np.abs(got - (ref + more)) <= bound)
    assert rk.get_device_error() == 0
