"""The preference loss on both sides of the border between one cluster and the whole device, where
neither may change a bit, and past what the whole device takes at once."""
import pytest
import torch

import preference_plain as pp
from helpers import same_bits
from test_gpu_preference import check, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BORDER = 16 * 1024 * 8  # tokens of the largest cluster
ROUND = 152 * 4 * 256 * 8  # tokens of the device's blocks at once

KINDS = [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)]


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def longer(c, tokens):
    """The same sequences with rows behind the last one, which belong to none."""
    pad = tokens - c.logp.shape[0]
    assert pad >= 0
    return pp.Case(torch.cat([c.logp, torch.full((pad,), float("nan"))]),
                   None if c.ref is None else torch.cat([c.ref, torch.ones(pad)]),
                   torch.cat([c.targets, torch.ones(pad, dtype=torch.int64)]), c.cu, c.chosen, c.rejected, c.margin)


def agree(got, want, tokens):
    assert same_bits(got["loss"], want["loss"]) and same_bits(got["logratio"], want["logratio"])
    assert same_bits(got["grad"][:tokens], want["grad"]) and not bool(got["grad"][tokens:].any())


@pytest.mark.parametrize("kind,smoothing", KINDS)
@pytest.mark.parametrize("ref,margin", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("average", [False, True])
def test_the_border_changes_no_bit(rk, average, ref, margin, kind, smoothing):
    """One cluster of 1, 13 and 16 blocks, and the same sequences in calls one token and much longer."""
    for lengths, P in (([300, 20, 1, 0, 77] * 5, 400), ([3000] * 35, 1000), ([1024] * 128, 16384)):
        c = pp.make_case(lengths, P, ref=ref, margin=margin, seed=len(lengths))
        if margin:
            c.margin = c.margin * 40 - 20
        tokens = c.logp.shape[0]
        assert tokens <= BORDER
        kw = dict(kind=kind, label_smoothing=smoothing, average=average, beta=0.25 if not average else 4.0, scale=0.37)
        small = run(rk, c, **kw)
        agree(run(rk, longer(c, BORDER), **kw), small, tokens)
        agree(run(rk, longer(c, BORDER + 1), **kw), small, tokens)
        agree(run(rk, longer(c, ROUND + 8 * 256 + 5), **kw), small, tokens)
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("many", ["pairs", "sequences"])
def test_the_border_of_pairs_and_sequences(rk, many):
    """One pair, or one sequence, more than the cluster takes: the others have the same bits."""
    c = pp.make_case([40] * 1000, 16 * 1024, seed=6, margin=True)
    small = run(rk, c, beta=0.25)
    if many == "pairs":
        none = torch.full((1,), -1, dtype=torch.int32)
        c.chosen, c.rejected, c.margin = (torch.cat([t, n]) for t, n in ((c.chosen, none), (c.rejected, none), (c.margin, torch.zeros(1))))
        got = run(rk, c, beta=0.25)
        assert same_bits(got["loss"][:-1], small["loss"]) and got["loss"][-1] == 0
        assert same_bits(got["logratio"], small["logratio"])
    else:
        c.cu = torch.cat([c.cu, c.cu[-1:].expand(7193)])  # empty ones: 8193 in all
        got = run(rk, c, beta=0.25)
        assert same_bits(got["loss"], small["loss"]) and same_bits(got["logratio"][:1000], small["logratio"])
        assert not bool(got["logratio"][1000:].any())
    assert same_bits(got["grad"], small["grad"])
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("average,kind,smoothing", [(False, "sigmoid", 0.2), (True, "hinge", 0.0), (True, "ipo", 0.0)])
def test_more_tokens_than_the_device_takes_at_once(rk, average, kind, smoothing):
    """A second pass of the blocks over tokens that count, against 64 bits."""
    c = pp.make_case([(7919 * i) % 4001 for i in range(700)], 300, margin=True, lead=3, trail=9, seed=12)
    assert c.logp.shape[0] > ROUND + 8 * 256
    kw = dict(kind=kind, beta=0.125 if not average else 2.0, average=average, scale=0.5)
    want, bound = pp.plain(c, smoothing=smoothing, **kw)
    check(run(rk, c, label_smoothing=smoothing, **kw), want, bound)
    assert rk.get_device_error() == 0
