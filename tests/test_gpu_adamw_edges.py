"""The AdamW step where its definition leaves little room: 8-bit states of very small values and of blocks with
values that are not finite, gradients that a graph holds, the first step on another stream, rates from the host
and from the device."""
import gc
import weakref

import pytest
import torch

from helpers import same_bits
from test_gpu_adamw import BF16, DEV, E4M3, FP32, HYPER, SIZES, make, snapshot, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


@pytest.mark.parametrize("offset", [0, 1])
def test_8_bit_states_of_blocks_that_are_not_finite(rk, offset):
    """An infinite gradient makes the scales of its block infinite: the codes are those of the quotients, 0 (the root's
    smallest) for the others and NaN for itself, and the block's states are NaN from then on.  A NaN stays in its element.
    Neighbouring blocks, and every weight but that one in this step, know nothing of it."""
    n = 256 * 4 + 40
    opt, other = (make(rk, [n], BF16, FP32, 8, offset=offset) for _ in range(2))
    g = opt.grads[0]
    g[256 + 7] = float("inf")
    g[512 + 9] = float("nan")
    g[256 * 4 + 39] = -float("inf")
    hit = torch.zeros(n, dtype=torch.bool)
    hit[[256 + 7, 512 + 9, 256 * 4 + 39]] = True
    blocks = torch.arange(n) // 256
    wide = (blocks == 1) | (blocks == 4)
    rk.adamw_step(opt, **HYPER)
    rk.adamw_step(other, **HYPER)
    a, b = snapshot(opt), snapshot(other)
    assert same_bits(a["master"][0][~hit], b["master"][0][~hit]) and same_bits(a["params"][0][~hit], b["params"][0][~hit])
    assert bool(torch.isnan(a["master"][0][hit]).all())
    for k, rest in (("m", 0.0), ("v", 2.0 ** -9)):
        code, clean, scale = a[k][0].float(), b[k][0].float(), a[k + "_scale"][0]
        assert torch.equal(torch.isinf(scale), torch.tensor([False, True, False, False, True]))
        assert bool((scale[[0, 2, 3]] > 0).all())
        assert bool(torch.isnan(code[hit]).all()) and not bool(torch.isnan(code[~hit]).any())
        nonzero = clean[wide & ~hit] != 0
        assert torch.equal(code[wide & ~hit].abs(), torch.where(nonzero, rest, 0.0))
        far = ~wide & (blocks != 2)
        assert torch.equal(code[far], clean[far])
    # the next step: the two blocks are lost, the third but for its element is not
    g.fill_(1e-3)
    rk.adamw_step(opt, **{**HYPER, "step": 8})
    w = opt.master[0].cpu()
    assert torch.equal(torch.isnan(w), wide | hit)


def test_codes_of_very_small_states(rk):
    """Scales down to 2^-120: codes are those of the quotients in fp32, as everywhere."""
    g = torch.Generator().manual_seed(1)
    for power in (-130, -118, -100, -90, -70, -62, -58, -30):
        n = 256 * 40
        p, grad = torch.zeros(n, device=DEV), (torch.randn(n, generator=g) * 2.0 ** power).to(DEV)
        opt = rk.AdamW([p], [grad], bits=8)
        rk.adamw_step(opt, lr=1e-3, step=1, beta1=0.5, beta2=0.75)
        m = grad.cpu() * 0.5
        v = grad.cpu().square() * 0.25
        for name, x in (("m", m), ("v", v.sqrt())):
            x = x.view(-1, 256)
            top = x.abs().amax(1, keepdim=True)
            s = torch.where(top > 0, (top * (torch.tensor(1.0) / 448.0)).clamp(min=2.0 ** -120), 0.0)
            q = torch.where(s > 0, x / s, 0.0)
            if name == "v":
                q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
            assert torch.equal(getattr(opt, name + "_scale")[0].cpu(), s[:, 0]), (name, power)
            assert torch.equal(getattr(opt, name)[0].cpu().float(), q.clamp(-448, 448).to(E4M3).float().view(-1)), (name, power)
    assert rk.get_device_error() == 0


def test_a_graph_keeps_the_gradients_that_it_was_captured_with(rk):
    """use_grads is for steps to come: what a captured step reads stays alive with the object."""
    opt, other = (make(rk, [5000, 300], BF16, FP32, 32) for _ in range(2))
    old = [g.clone() for g in opt.grads]
    opt.use_grads(old)
    alive = [weakref.ref(g) for g in old]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rk.adamw_step(opt, **HYPER)
    new = [torch.full_like(g, 3.0) for g in old]
    opt.use_grads(new)
    del old
    gc.collect()
    assert all(ref() is not None for ref in alive)
    graph.replay()
    rk.adamw_step(other, **HYPER)
    assert all(same_bits(a, b) for a, b in zip(opt.master, other.master))
    # eager steps hold on to nothing
    last = weakref.ref(new[0])
    rk.adamw_step(opt, **HYPER)
    opt.use_grads([torch.zeros_like(g) for g in new])
    torch.cuda.synchronize()
    del new
    gc.collect()
    assert last() is None
    # captured on a stream that is passed
    held = [torch.zeros_like(g) for g in opt.grads]
    opt.use_grads(held)
    ref, side, beside = weakref.ref(held[0]), torch.cuda.Stream(), torch.cuda.Stream()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2, stream=side):
        with torch.cuda.stream(beside):
            rk.adamw_step(opt, stream=side, **HYPER)
    del held
    opt.use_grads(other.grads)
    gc.collect()
    assert ref() is not None


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_step_may_be_on_another_stream(rk, bits):
    """States and masters that are made with the object are there when it is, while the stream that
    made them is still busy with something else."""
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device=DEV)
    for turn in range(4):
        p, g = tensors([70001, 300], BF16, 0.1, turn), tensors([70001, 300], FP32, 0.1, turn + 1)
        want = rk.AdamW([t.clone() for t in p], g, bits=bits, master=True)
        rk.adamw_step(want, **HYPER)
        # memory of the states' sizes that is not zero, for the allocator to hand out again
        junk = [torch.full((t.numel(),), 7.0, device=DEV) for t in p for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for _ in range(20):
            busy.add_(1.0)
        opt = rk.AdamW(p, g, bits=bits, master=True)
        rk.adamw_step(opt, **HYPER, stream=side)
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(opt.master, want.master))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.95), (0.0, 0.5), (0.99, 0.9999)])
def test_a_step_has_the_same_bits_from_the_host_and_from_the_device(rk, bits, betas):
    """... so an eager step and a captured one that follows a counter agree."""
    for step in (1, 2, 3, 7, 10, 33, 100, 1000, 12345, 10 ** 6, 10 ** 9, 2 ** 40):
        hyper = dict(step=step, beta1=betas[0], beta2=betas[1], eps=1e-8)
        a, b = (make(rk, SIZES, BF16, FP32, bits, seed=step % 1000) for _ in range(2))
        rk.adamw_step(a, lr=1e-3, **hyper)
        rk.adamw_step(b, lr=torch.tensor([1e-3], device=DEV), **{**hyper, "step": torch.tensor([step], device=DEV)})
        x, y = snapshot(a), snapshot(b)
        for k in x:
            for s, t in zip(x[k] or [], y[k] or []):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8)), (k, step)
    assert rk.get_device_error() == 0
