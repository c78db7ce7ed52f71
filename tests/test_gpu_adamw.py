"""The AdamW step on the GPU against its 64-bit form, over many tensors, with both kinds of
states, off alignment, on other streams and in graphs."""
import pytest
import torch

import adamw_plain as ap
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, step=7, beta1=0.9, beta2=0.95, eps=1e-8)
SIZES = [1, 7, 8, 255, 256, 257, 1000, 4096, 4097, 0, 8191, 100003]


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def tensors(sizes, dtype, scale, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        buf = torch.zeros(n + offset, dtype=dtype, device=DEV)
        buf[offset:] = (torch.randn(n, generator=g) * scale).to(dtype).to(DEV)
        out.append(buf[offset:])
    return out


def make(rk, sizes, param, grad, bits, *, master=True, decay=0.1, seed=0, offset=0, fresh=False):
    """An AdamW with states that are not zero (unless fresh), all tensors `offset` elements into their buffers."""
    p = tensors(sizes, param, 0.05, seed, offset)
    gr = tensors(sizes, grad, 1e-2, seed + 1, offset)
    for t in gr:  # rows without a gradient
        t[::5] = 0
    opt = rk.AdamW(p, gr, bits=bits, master=master or None, weight_decay=decay)
    if offset:  # the states off alignment too
        odd = lambda t: torch.empty(t.numel() + offset, dtype=t.dtype, device=DEV)[offset:].copy_(t)  # noqa: E731
        copy = lambda ts: None if ts is None else [None if t is None else odd(t) for t in ts]  # noqa: E731
        opt = rk.AdamW(p, gr, copy(opt.m), copy(opt.v), m_scale=copy(opt.m_scale), v_scale=copy(opt.v_scale),
                       master=copy(opt.master), weight_decay=decay)
    if not fresh:
        for s in (1, 2):
            rk.adamw_step(opt, **{**HYPER, "step": s})
            for t in gr:
                t.mul_(-0.7)
    return opt


def snapshot(opt):
    copy = lambda ts: None if ts is None else [None if t is None else t.clone().cpu() for t in ts]  # noqa: E731
    return {k: copy(getattr(opt, k)) for k in ("params", "grads", "m", "v", "m_scale", "v_scale", "master")}


def check(before, opt, grad_scale=1.0, decay=0.1, hyper=HYPER):
    after = snapshot(opt)
    for i, p in enumerate(before["params"]):
        n = p.numel()
        if n == 0:
            continue
        eight = before["m_scale"] is not None
        if eight:
            m = ap.decode(before["m"][i], before["m_scale"][i], False)
            v = ap.decode(before["v"][i], before["v_scale"][i], True)
        else:
            m, v = before["m"][i].double(), before["v"][i].double()
        has_master = before["master"] is not None and before["master"][i] is not None
        w = (before["master"][i] if has_master else p).double()
        (w1, m1, v1), (dw, dm, dv) = ap.step(w, before["grads"][i], m, v, decay=decay, grad_scale=grad_scale, **hyper)
        if has_master:
            assert bool(((after["master"][i].double() - w1).abs() <= dw).all())
            assert same_bits(after["params"][i], after["master"][i].to(p.dtype))
        else:
            half = 0.0 if p.dtype is FP32 else 2.0 ** -8
            assert bool(((after["params"][i].double() - w1).abs() <= dw + half * 1.01 * (w1.abs() + dw)).all())
        if eight:
            # the decoded states carry two roundings of their own (code * scale, the square)
            ap.check_state(after["m"][i], after["m_scale"][i], m1, dm + 2 * ap.U * m.abs(), False)
            ap.check_state(after["v"][i], after["v_scale"][i], v1, dv + 6 * ap.U * v, True)
        else:
            assert bool(((after["m"][i].double() - m1).abs() <= dm).all())
            assert bool(((after["v"][i].double() - v1).abs() <= dv).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(FP32, FP32, False), (FP32, BF16, False), (BF16, FP32, True),
                                               (BF16, BF16, True), (BF16, BF16, False)])
def test_against_64_bits(rk, param, grad, master, bits):
    for fresh in (True, False):
        opt = make(rk, SIZES, param, grad, bits, master=master, fresh=fresh)
        before = snapshot(opt)
        rk.adamw_step(opt, **HYPER)
        check(before, opt)
    before = snapshot(opt)
    scale = torch.tensor([0.37], device=DEV)
    rk.adamw_step(opt, grad_scale=scale, **HYPER)
    check(before, opt, grad_scale=float(scale))
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("grad", [FP32, BF16])
@pytest.mark.parametrize("bits", [32, 8])
def test_states_have_the_bits_of_elementary_operations(rk, bits, grad):
    """Products, sums, roots and quotients in fp32, each rounded by itself; only zeros may differ in sign."""
    opt = make(rk, [70001], BF16, grad, bits)
    before = snapshot(opt)
    scale = torch.tensor([0.37], device=DEV)
    rk.adamw_step(opt, grad_scale=scale, **HYPER)
    after = snapshot(opt)
    g = before["grads"][0].float() * scale.cpu()
    m, v = before["m"][0], before["v"][0]
    if bits == 8:
        m = m.float() * before["m_scale"][0].repeat_interleave(256)[:70001]
        v = (v.float() * before["v_scale"][0].repeat_interleave(256)[:70001]).square()
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + g * g * f(1 - b2)
    if bits == 32:
        assert torch.equal(after["m"][0], m) and torch.equal(after["v"][0], v)
        return
    for name, x in (("m", m), ("v", v.sqrt())):
        x = torch.nn.functional.pad(x, (0, -70001 % 256)).view(-1, 256)
        s = x.abs().amax(1, keepdim=True) * (f(1.0) / f(448.0))
        q = torch.where(s > 0, x / s, 0.0)
        if name == "v":
            q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
        code = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(-1)[:70001]
        assert torch.equal(after[name + "_scale"][0], s[:, 0])
        assert torch.equal(after[name][0].float(), code.float())


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", [BF16, FP32])
def test_alignment_has_the_same_bits(rk, param, bits, offset):
    a = make(rk, SIZES, param, FP32, bits, master=param is BF16)
    b = make(rk, SIZES, param, FP32, bits, master=param is BF16, offset=offset)
    rk.adamw_step(a, **HYPER)
    rk.adamw_step(b, **HYPER)
    x, y = snapshot(a), snapshot(b)
    for k in x:
        for s, t in zip(x[k] or [], y[k] or []):
            if s is not None:
                assert torch.equal(s.view(torch.uint8), t.contiguous().view(torch.uint8)), k


def test_more_tensors_than_a_launch_takes(rk):
    sizes = [1 + (37 * i) % 700 for i in range(600)]
    for bits in (32, 8):
        opt = make(rk, sizes, BF16, FP32, bits)
        before = snapshot(opt)
        rk.adamw_step(opt, **HYPER)
        check(before, opt)


def test_rates_of_each_tensor(rk):
    p, g = tensors([300, 300, 300], FP32, 0.1, 1), tensors([300, 300, 300], FP32, 0.1, 2)
    opt = rk.AdamW(p, g, weight_decay=[0.0, 0.5, 0.0], lr_scale=[1.0, 1.0, 0.0])
    before = [t.clone() for t in p]
    rk.adamw_step(opt, **HYPER)
    for i, (decay, rate) in enumerate(((0.0, 1.0), (0.5, 1.0), (0.0, 0.0))):
        z = torch.zeros(300, dtype=torch.float64)
        (w1, _, _), (dw, _, _) = ap.step(before[i].cpu().double(), g[i].cpu(), z, z, decay=decay,
                                         **{**HYPER, "lr": HYPER["lr"] * rate})
        assert bool(((p[i].cpu().double() - w1).abs() <= dw).all())
    assert same_bits(p[2], before[2])


@pytest.mark.parametrize("step", [1, 2, 10, 1000, 1000000, 10 ** 9])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.95), (0.0, 0.5), (0.99, 0.9999), (0.5, 0.0)])
def test_bias_corrections(rk, step, betas):
    """Step and rate from the host and from the device."""
    hyper = dict(lr=1e-3, step=step, beta1=betas[0], beta2=betas[1], eps=1e-8)
    for device in (False, True):
        opt = make(rk, [1000], FP32, FP32, 32, master=False)
        before = snapshot(opt)
        given = dict(hyper)
        if device:
            given.update(lr=torch.tensor(1e-3, device=DEV), step=torch.tensor([step], device=DEV))
        rk.adamw_step(opt, **given)
        check(before, opt, hyper=hyper)
    assert rk.get_device_error() == 0


def test_a_step_below_one_changes_nothing(rk):
    opt = make(rk, [1000, 5], BF16, FP32, 8)
    before = snapshot(opt)
    rk.adamw_step(opt, **{**HYPER, "step": torch.zeros(1, dtype=torch.int64, device=DEV)})
    assert rk.get_device_error() == rk.DEVERR_RULES
    after = snapshot(opt)
    for k in ("params", "master", "m", "v"):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before[k], after[k]))


def test_8_bit_states_of_extreme_blocks(rk):
    """Blocks of zeros, of one value, of values 2^40 apart; and a gradient that stops coming."""
    n = 256 * 6 + 9
    g = torch.zeros(n, device=DEV)
    g[256:512] = 1e-3
    g[512:768] = torch.logspace(-14, -2, 256)
    g[768] = 1e4
    g[769:1024] = 1e-6
    g[1024:1280] = 1e-30
    p = torch.zeros(n, device=DEV)
    opt = rk.AdamW([p], [g], bits=8, weight_decay=0.0)
    for s in range(1, 6):
        before = snapshot(opt)
        hyper = {**HYPER, "step": s}
        rk.adamw_step(opt, **hyper)
        check(before, opt, decay=0.0, hyper=hyper)
        if s == 3:
            g.zero_()
    assert not bool(p[:256].any()) and not bool(p[1280:].any())
    # no step is larger than a few times the rate
    assert float(p.abs().max()) <= 5 * HYPER["lr"] * 10
    assert rk.get_device_error() == 0


def test_gradients_that_are_not_finite_stay_in_their_element(rk):
    p, g = tensors([2000], FP32, 1.0, 1), tensors([2000], FP32, 1.0, 2)
    opt = rk.AdamW(p, g)
    other = rk.AdamW([p[0].clone()], [g[0].clone()])
    g[0][5], g[0][700] = float("nan"), float("inf")
    rk.adamw_step(opt, **HYPER)
    rk.adamw_step(other, **HYPER)
    keep = torch.ones(2000, dtype=torch.bool, device=DEV)
    keep[5] = keep[700] = False
    assert same_bits(p[0][keep], other.params[0][keep]) and bool(torch.isnan(p[0][~keep]).all())


def test_other_gradients(rk):
    p, g = tensors([100, 9], BF16, 1.0, 1), tensors([100, 9], FP32, 1.0, 2)
    a = rk.AdamW(p, g, master=True)
    b = rk.AdamW([t.clone() for t in p], tensors([100, 9], BF16, 1.0, 3), master=True)
    b.use_grads(g)
    rk.adamw_step(a, **HYPER)
    rk.adamw_step(b, **HYPER)
    assert all(same_bits(x, y) for x, y in zip(a.params, b.params))


def test_streams_and_graphs(rk):
    """A captured step follows the step number, the rate and the gradients; two objects on two streams."""
    for bits in (32, 8):
        live, eager = (make(rk, [5000, 300, 70001], BF16, FP32, bits) for _ in range(2))
        step = torch.tensor([7], device=DEV)
        lr = torch.tensor([1e-3], device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rk.adamw_step(live, **{**HYPER, "lr": lr, "step": step})
            step += 1
        for i in range(3):
            for t in live.grads:
                t.mul_(0.9)
            lr.mul_(0.5)
            graph.replay()
        for i in range(3):
            for t in eager.grads:
                t.mul_(0.9)
            rk.adamw_step(eager, **{**HYPER, "lr": torch.tensor([1e-3 * 0.5 ** (i + 1)], device=DEV),
                                    "step": torch.tensor([7 + i], device=DEV)}, stream=None)
        torch.cuda.synchronize()
        assert int(step) == 10
        for k in ("params", "master", "m", "v"):
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(getattr(live, k), getattr(eager, k))), k
        a, b = (make(rk, [70001], BF16, FP32, bits) for _ in range(2))
        torch.cuda.synchronize()
        for _ in range(4):
            rk.adamw_step(a, **HYPER, stream=side)
            rk.adamw_step(b, **HYPER)
        torch.cuda.synchronize()
        assert same_bits(a.params[0], b.params[0])
    assert rk.get_device_error() == 0


def test_no_tensors(rk):
    rk.adamw_step(rk.AdamW([], []), **HYPER)
    empty = torch.empty(0, device=DEV)
    rk.adamw_step(rk.AdamW([empty], [empty.clone()], bits=8), **HYPER)


def test_a_tensor_past_32_bits(rk):
    """More than 2^31 elements: the first and the last have the bits that they have alone."""
    n = 2 ** 31 + 256 * 5 + 77
    p, g = (torch.empty(n, dtype=BF16, device=DEV) for _ in range(2))
    for t, seed in ((p, 1), (g, 2)):
        gen = torch.Generator(DEV).manual_seed(seed)
        for a in range(0, n, 2 ** 28):
            b = min(n, a + 2 ** 28)
            t[a:b] = torch.randn(b - a, generator=gen, device=DEV)
    ends = [slice(0, 1000), slice(n - (n % 256) - 256 * 3, n)]
    small = rk.AdamW([p[e].clone() for e in ends], [g[e].clone() for e in ends], bits=8)
    big = rk.AdamW([p], [g], bits=8)
    for step in (1, 2):
        rk.adamw_step(big, **{**HYPER, "step": step})
        rk.adamw_step(small, **{**HYPER, "step": step})
    for i, e in enumerate(ends):
        keep = 768 if i == 0 else small.params[1].numel()  # whole blocks of 256
        assert same_bits(p[e][:keep], small.params[i][:keep])
        for k in ("m", "v"):
            a, b = getattr(big, k)[0][e][:keep], getattr(small, k)[i][:keep]
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_overlaps_are_refused(rk):
    p, g = torch.zeros(600, device=DEV), torch.zeros(600, device=DEV)
    rk.AdamW([p[:300], p[300:]], [g[:300], g[:300]])  # side by side; gradients may be shared
    for params, grads in (([p, p], [g, g]), ([p[:300], p[299:]], [g[:300], g[299:]]), ([p], [p]),
                          ([p[:300]], [p[299:599]]), ([p[300:]], [p[1:301]])):
        with pytest.raises(ValueError, match="overlap"):
            rk.AdamW(params, grads)
    with pytest.raises(ValueError, match="overlap"):
        rk.AdamW([p], [g], [g.clone()], [p])
    opt = rk.AdamW([p], [g])
    with pytest.raises(ValueError, match="overlap"):
        opt.use_grads([opt.m[0]])
    assert opt.grads[0] is g
