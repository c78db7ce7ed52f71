"""The preference loss on the GPU against its 64-bit form, in other layouts, in one cluster and
over the whole device, on other streams and in graphs."""
import numpy as np
import pytest
import torch

import preference_plain as pp
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def run(rk, c, **kw):
    args, named = c.to(DEV).args()
    return rk.preference_loss(*args, **named, **kw)


def check(got, want, bound):
    for name, w, b in zip(("loss", "grad", "logratio"), want, bound):
        d = np.abs(got[name].double().cpu().numpy() - w)
        assert np.all(d <= b), (name, float((d - b).max()))


LENGTHS = {
    "one": [1], "pair": [3, 5], "short": [0, 1, 2, 0, 0, 7, 8, 9, 0], "runs": [8, 16, 24, 8], "long": [5000, 1, 3001],
    "empty": [3] + [0] * 700 + [2] + [0] * 600 + [9, 0, 30],
    "many": [(7 * i) % 13 for i in range(900)], "mixed": [1000, 40, 0, 2047, 256, 255, 257, 31, 33, 1024],
}


@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.25), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("ref,margin,average", [(True, False, False), (False, True, True), (True, True, True)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_against_64_bits(rk, name, ref, margin, average, kind, smoothing):
    lengths = LENGTHS[name]
    for P, beta, scale in ((1, 2.0, 1.0), (len(lengths) * 2, 0.125, 0.25)):
        c = pp.make_case(lengths, P, ref=ref, margin=margin, lead=3, trail=5, seed=len(name) + P)
        kw = dict(kind=kind, beta=beta, average=average, scale=scale)
        want, bound = pp.plain(c, smoothing=smoothing, **kw)
        check(run(rk, c, label_smoothing=smoothing, **kw), want, bound)
    assert rk.get_device_error() == 0


def test_many_pairs_and_sequences(rk):
    """More sequences than are searched in shared memory, and one that nearly every pair names."""
    for Q, P in ((9000, 4000), (300, 5000), (20000, 300)):
        c = pp.make_case([(5 * i) % 7 if Q < 20000 else (i % 997 == 5) * 11 for i in range(Q)], P, seed=Q)
        c.chosen[::2] = 17
        c.rejected[5] = 17
        c.chosen[5] = 17
        want, bound = pp.plain(c)
        check(run(rk, c, beta=0.125), want, bound)
    assert rk.get_device_error() == 0


def test_pairs_that_are_none(rk):
    c = pp.make_case([10, 20, 30], 6, seed=3)
    c.chosen = torch.tensor([0, -1, 2, 3, 1, 1], dtype=torch.int32)
    c.rejected = torch.tensor([1, 0, -7, 0, 1, 2], dtype=torch.int32)
    got = run(rk, c, beta=0.125)
    assert rk.get_device_error() == rk.DEVERR_RULES
    assert bool(torch.isnan(got["loss"][3])) and got["loss"][1] == 0 and got["loss"][2] == 0
    # the pair out of range is as good as none elsewhere
    c.chosen[3] = -1
    want, bound = pp.plain(c, beta=0.125)
    got["loss"][3] = 0
    check(got, want, bound)
    # a sequence against itself: log 2, and no gradient of its own
    alone = pp.make_case([10], 1, seed=3)
    got = run(rk, alone)
    assert abs(float(got["loss"]) - np.log(2)) < 1e-6 and not bool(got["grad"].any())
    assert rk.get_device_error() == 0


def test_nothing(rk):
    empty = lambda t: torch.empty(0, dtype=t, device=DEV)  # noqa: E731
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = rk.preference_loss(empty(torch.float32), empty(torch.int64), cu, empty(torch.int32), empty(torch.int32))
    assert all(got[k].numel() == 0 for k in got)
    # no pairs, no sequences, no tokens
    for lengths, P in (([5, 9], 0), ([], 0), ([0, 0], 2)):
        c = pp.make_case(lengths, P, trail=4)
        got = run(rk, c, beta=0.125)
        want, bound = pp.plain(c)
        check(got, want, bound)
    c = pp.make_case([4, 4], 1, share=0.0)
    check(run(rk, c, beta=0.125, average=True), *pp.plain(c, average=True))
    assert rk.get_device_error() == 0


def layouts(c, g):
    """The same sequences packed behind rows of their own, padded left and right, with gaps of
    inactive rows inside."""
    cu = c.cu.tolist()
    Q = len(cu) - 1
    out = []
    for side in ("packed", "right", "left", "gaps"):
        width = max(cu[i + 1] - cu[i] for i in range(Q)) + 37
        rows, marks, at = [], [0], 0
        for q in range(Q):
            n = cu[q + 1] - cu[q]
            idx = torch.arange(cu[q], cu[q + 1])
            none = lambda k: torch.full((k,), -1, dtype=torch.int64)  # noqa: E731
            if side == "right":
                idx = torch.cat([idx, none(width - n)])
            elif side == "left":
                idx = torch.cat([none(width - n), idx])
            elif side == "gaps":
                place = torch.randperm(width, generator=g)[:n].sort().values
                full = none(width)
                full[place] = idx
                idx = full
            rows.append(idx)
            at += len(idx)
            marks.append(at)
        idx = torch.cat(rows)
        take = lambda t, fill: torch.where(idx >= 0, t[idx.clamp(min=0)], torch.tensor(fill, dtype=t.dtype))  # noqa: E731
        out.append((idx, pp.Case(take(c.logp, float("nan")), None if c.ref is None else take(c.ref, float("inf")),
                                 take(c.targets, -100), torch.tensor(marks, dtype=torch.int32), c.chosen, c.rejected,
                                 c.margin)))
    return out


@pytest.mark.parametrize("average", [False, True])
def test_layouts_have_the_same_bits(rk, average):
    g = torch.Generator().manual_seed(1)
    c = pp.make_case([300, 1, 77, 2500, 640], 7, seed=5)
    base = run(rk, c, average=average)
    for idx, other in layouts(c, g):
        got = run(rk, other, average=average)
        assert same_bits(got["loss"], base["loss"]) and same_bits(got["logratio"], base["logratio"])
        real = idx >= 0
        assert same_bits(got["grad"][real.to(DEV)], base["grad"][idx[real].to(DEV)])
        assert not bool(got["grad"][~real.to(DEV)].any())
    assert rk.get_device_error() == 0


def test_one_cluster_and_the_whole_device_agree(rk):
    """Rows behind the last sequence take the call past what one cluster does."""
    c = pp.make_case([4000] * 40, 64, seed=9)
    small = run(rk, c)
    pad = (1 << 20) + 77 - c.logp.shape[0]
    big = pp.Case(torch.cat([c.logp, torch.full((pad,), float("nan"))]), torch.cat([c.ref, torch.ones(pad)]),
                  torch.cat([c.targets, torch.ones(pad, dtype=torch.int64)]), c.cu, c.chosen, c.rejected, None)
    got = run(rk, big)
    assert same_bits(got["loss"], small["loss"]) and same_bits(got["logratio"], small["logratio"])
    assert same_bits(got["grad"][:c.logp.shape[0]], small["grad"]) and not bool(got["grad"][c.logp.shape[0]:].any())
    want, bound = pp.plain(c, beta=float(np.float32(0.1)))
    check(small, want, bound)
    # addresses off 16 bytes
    args, named = c.to(DEV).args()

    def moved(t):
        m = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return m.copy_(t)
    shifted = rk.preference_loss(moved(args[0]), moved(args[1]), moved(args[2]), moved(args[3]), moved(args[4]),
                                 logp_ref=moved(named["logp_ref"]))
    assert all(same_bits(shifted[k], small[k]) for k in small)
    assert rk.get_device_error() == 0


def test_values_that_are_not_finite(rk):
    inf, nan = float("inf"), float("nan")
    logp = torch.tensor([-1.0, -2.0, -inf, -1.0, nan, -1.0, -1e30, -0.5, -inf, -2.0])
    targets = torch.zeros(10, dtype=torch.int64)
    cu = torch.tensor([0, 2, 4, 6, 8, 10], dtype=torch.int32)
    chosen = torch.tensor([0, 1, 2, 3, 1], dtype=torch.int32)
    rejected = torch.tensor([1, 0, 0, 0, 4], dtype=torch.int32)
    c = pp.Case(logp, None, targets, cu, chosen, rejected, None)
    got = run(rk, c, beta=0.5)
    ratio, loss = got["logratio"].cpu(), got["loss"].cpu()
    assert ratio[0] == -3 and ratio[1] == -inf and torch.isnan(ratio[2]) and ratio[3] == -inf and ratio[4] == -inf
    assert loss[0] == 0 and loss[1] == inf and torch.isnan(loss[2]) and loss[3] == inf and torch.isnan(loss[4])
    for kind, want in (("hinge", [0, inf]), ("ipo", [inf, inf])):
        loss = run(rk, c, beta=0.5, kind=kind)["loss"].cpu()
        assert loss[0] == want[0] and loss[1] == want[1] and torch.isnan(loss[2])
    # masked, none of it is seen
    targets = torch.where(torch.isfinite(logp) & (logp > -100), 0, -100)
    c = pp.Case(logp, None, targets, cu, chosen, rejected, None)
    clean = pp.Case(torch.where(targets >= 0, logp, torch.zeros(())), None, targets, cu, chosen, rejected, None)
    check(run(rk, c, beta=0.5), *pp.plain(clean, beta=0.5))
    # both parts of a ratio far away
    far = torch.tensor([-3e5, -1.0, -2e6, -1.0])
    c = pp.Case(far, torch.tensor([-3e5, -1.5, -2e6, -1.5]), torch.zeros(4, dtype=torch.int64),
                torch.tensor([0, 2, 4], dtype=torch.int32), torch.tensor([0], dtype=torch.int32),
                torch.tensor([1], dtype=torch.int32), None)
    got = run(rk, c)
    assert got["logratio"][0] == 0.5 and bool(torch.isnan(got["logratio"][1]))
    assert rk.get_device_error() == 0


def test_margins_far_from_the_middle(rk):
    """Losses from 0 to a thousand, with their slopes."""
    c = pp.make_case([50, 60], 9, seed=2)
    c.chosen[:], c.rejected[:] = 0, 1
    c.margin = torch.tensor([0.0, 20.0, -20.0, 90.0, -90.0, 120.0, -120.0, 1000.0, -1000.0])
    for smoothing in (0.0, 0.5):
        want, bound = pp.plain(c, beta=1.0, smoothing=smoothing)
        check(run(rk, c, beta=1.0, label_smoothing=smoothing), want, bound)


def test_bad_offsets_are_reported(rk):
    c = pp.make_case([5, 5, 5], 2, seed=1)
    for cu in ([0, 9, 5, 15], [-3, 5, 10, 15], [0, 5, 10, 16], [20, 21, 22, 23]):
        c.cu = torch.tensor(cu, dtype=torch.int32)
        run(rk, c)
        assert rk.get_device_error() == rk.DEVERR_RULES


def test_gradient_against_differences(rk):
    """The gradient is the derivative of the sum of the 64-bit losses."""
    for kind in ("sigmoid", "hinge", "ipo"):
        c = pp.make_case([9, 14, 6], 4, seed=8)
        kw = dict(kind=kind, beta=0.5, average=True, scale=0.7)
        grad = run(rk, c, **kw)["grad"].double().cpu().numpy()
        for t in (0, 3, 10, 20, 28):
            ends = []
            for h in (2.0 ** -12, -2.0 ** -12):  # both sums are exact in fp32
                logp = c.logp.double()
                logp[t] += h
                moved = pp.Case(logp, c.ref, c.targets, c.cu, c.chosen, c.rejected, None)
                ends.append(pp.plain(moved, **kw)[0][0].sum())
            # the difference leaves h^2 / 6 times a third derivative of at most 0.7 * 4 pairs * beta^3
            assert abs((ends[0] - ends[1]) * 2.0 ** 11 - grad[t]) <= 2e-7 + 1e-6 * abs(grad[t])


def test_streams_and_graphs(rk):
    c = pp.make_case([700, 800, 900, 1000] * 8, 40, seed=4).to(DEV)
    args, named = c.args()
    want = rk.preference_loss(*args, **named)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [rk.preference_loss(*args, **named, stream=s) for s in side]
        torch.cuda.synchronize()
        assert all(same_bits(one[k], want[k]) for one in got for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rk.preference_loss(*args, **named)
    c.logp.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    again = rk.preference_loss(*args, **named)
    assert all(same_bits(got[k], again[k]) for k in want)
    assert rk.get_device_error() == 0


def test_sums_and_margins_past_fixed_point(rk):
    """Ratios, margins and 1 / (2 beta) on both sides of where 64-bit floating point takes over."""
    n = 600
    logp = torch.cat([torch.full((n,), -400.0), torch.full((n,), -440.0), torch.full((n,), -0.25), torch.full((n,), -900.0)])
    cu = torch.arange(5, dtype=torch.int32) * n
    chosen, rejected = torch.tensor([0, 1, 2, 3, 0, 2, 1], dtype=torch.int32), torch.tensor([1, 0, 3, 1, 2, 0, 2], dtype=torch.int32)
    for margin in (None, torch.tensor([2.0 ** 18, -(2.0 ** 18), 1.0, 3e5, 1e9, -1e5, 24000.0])):
        c = pp.Case(logp, None, torch.zeros(4 * n, dtype=torch.int64), cu, chosen, rejected, margin)
        for kind, beta in (("sigmoid", 2.0 ** -14), ("hinge", 2.0 ** -10), ("ipo", 0.5), ("ipo", 2.0 ** -20), ("ipo", 2.0 ** -18)):
            want, bound = pp.plain(c, kind=kind, beta=beta)
            check(run(rk, c, kind=kind, beta=beta), want, bound)
    assert rk.get_device_error() == 0
