"""The root-mean-square norm and its gradient on the GPU against their 64-bit forms, in
other layouts, on other streams and in graphs."""
import pytest
import torch

import norm_plain as npl
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# widths on both sides of every change of team, odd ones, one column; several rows a unit and a
# last unit that is not full
SHAPES = [(1, 1), (3, 7), (37, 8), (2, 100), (640, 64), (17, 256), (9, 264), (33, 513), (40, 512), (300, 1000),
          (7, 1023), (65, 1024), (11, 2047), (12, 2048), (1300, 2056), (13, 4096), (5, 4097), (700, 5000),
          (6, 8192), (3, 8193), (3, 16384), (2, 16383), (1000, 65), (999, 128), (301, 129)]


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weight_of(g, H, dtype):
    return (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)


def close(got, want, bound):
    d = got.double().cpu()
    ok = (d - want).abs() <= bound
    return bool(ok.all()), float(((d - want).abs() - bound).max())


@pytest.mark.parametrize("residual", [None, BF16, FP32])
@pytest.mark.parametrize("x_type", [BF16, FP32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(rk, T, H, x_type, residual):
    g = gen(T * H)
    x = npl.matrix(g, T, H, x_type, scale=2.0)
    res = None if residual is None else npl.matrix(g, T, H, residual, scale=3.0)
    w = weight_of(g, H, BF16 if H % 2 else FP32)
    r = npl.stream(x, res)
    want = npl.forward(r, w, npl.active(T, None, None))
    for out_type in (BF16, FP32):
        y, kept = rk.rms_norm(npl.to(x, DEV), w.to(DEV), residual=npl.to(res, DEV), eps=npl.EPS, out_dtype=out_type)
        assert y.dtype == out_type and same_bits(kept, r)
        half = npl.HALF_STEP[out_type]
        assert close(y, want, want.abs() * (npl.FORWARD + half * 1.01))[0]
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_in_8_bits(rk, T, H, group):
    g = gen(T + H)
    x = npl.matrix(g, T, H, BF16)
    x[0, : H // 2] = 0
    if T > 1:
        x[1] = 0
    res = None if H % 3 else npl.matrix(g, T, H, FP32)
    w = weight_of(g, H, BF16)
    r = npl.stream(x, res)
    y = npl.forward(r, w, npl.active(T, None, None))
    q, s, kept = rk.rms_norm_e4m3(npl.to(x, DEV), w.to(DEV), residual=npl.to(res, DEV), eps=npl.EPS, group=group)
    assert q.dtype == E4M3 and same_bits(kept, r)
    width = group or H
    n = -(-H // width)
    assert s.shape == (T, n)
    top = torch.nn.functional.pad(y, (0, n * width - H)).view(T, n, width).abs().amax(2) / 448
    # y, its product with 1 / 448, and that number's own rounding
    assert close(s, top, top * (npl.FORWARD + 2 * npl.U) * 1.01)[0]
    s = s.double().cpu()
    z = y / torch.where(s > 0, s, 1.0).repeat_interleave(width, 1)[:, :H]
    assert close(q.float(), z, npl.e4m3_bound(z))[0]
    assert bool((s[top == 0] == 0).all())
    assert rk.get_device_error() == 0


def bwd_case(g, T, H, r_type, d_type, dr_type, ld=0, offset=0):
    r = npl.matrix(g, T, H, r_type, ld, offset, 2.0)
    dout = npl.matrix(g, T, H, d_type, ld, offset)
    dr = None if dr_type is None else npl.matrix(g, T, H, dr_type, ld, offset)
    return r, dout, dr, weight_of(g, H, FP32 if H % 2 else BF16)


def check_bwd(got, dw, r, dout, dr, w, live, old=None, times=None):
    dx, terms, bound = npl.backward(dout, r, w, dr, live)
    half = npl.HALF_STEP[got.dtype] if got.dtype is not FP32 else 0.0
    ok, over = close(got, dx, bound + half * 1.01 * (dx.abs() + bound))
    assert ok, over
    if times is not None:
        terms = terms * times[:, None]
    want, mag = terms.sum(0), terms.abs().sum(0)
    # a term: n 17; sums: a run of rows, 8 teams of a block, 40 blocks of a lane, 32 lanes
    adds = 17 + min(int(live.sum()) if times is None else int(times.sum()), 2000) + 80
    if old is not None:
        want, mag, adds = want + old.double(), mag + old.double().abs(), adds + 1
    ok, over = close(dw, want, adds * npl.U * 1.01 * mag)
    assert ok, over


@pytest.mark.parametrize("r_type,d_type,dr_type,out", [(BF16, FP32, None, FP32), (BF16, BF16, BF16, BF16),
                                                        (FP32, FP32, FP32, FP32), (FP32, BF16, BF16, BF16)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(rk, T, H, r_type, d_type, dr_type, out):
    g = gen(T * 3 + H)
    r, dout, dr, w = bwd_case(g, T, H, r_type, d_type, dr_type)
    dx, dw = rk.rms_norm_bwd(npl.to(dout, DEV), npl.to(r, DEV), w.to(DEV), grad_residual=npl.to(dr, DEV),
                             eps=npl.EPS, out_dtype=out)
    check_bwd(dx, dw, r, dout, dr, w, npl.active(T, None, None))
    assert rk.get_device_error() == 0


# rows that start on every element, gaps between them, results inside wider rows
@pytest.mark.parametrize("H", [40, 264, 1001, 2048, 4104])
@pytest.mark.parametrize("ld,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (2, 4), (1, 7)])
def test_strides_and_offsets_give_the_same_bits(rk, H, ld, offset):
    T = 21
    for x_type, res_type in ((BF16, FP32), (FP32, BF16), (BF16, BF16)):
        g = gen(H)
        x, res = npl.matrix(g, T, H, x_type), npl.matrix(g, T, H, res_type)
        d = npl.matrix(g, T, H, BF16)
        w = weight_of(g, H, BF16)

        def moved(t):
            m = npl.matrix(gen(0), T, H, t.dtype, ld, offset)
            m.copy_(t)
            return npl.to(m, DEV)
        xs, rs, ds = npl.to(x, DEV), npl.to(res, DEV), npl.to(d, DEV)
        y0, r0 = rk.rms_norm(xs, w.to(DEV), residual=rs, out_dtype=FP32)
        w1 = torch.empty(H + 1, dtype=BF16, device=DEV)[1:]
        w1.copy_(w)
        out = moved(y0.cpu())
        ro = moved(r0.cpu())
        frame = torch.empty(0, dtype=FP32, device=DEV).set_(out.untyped_storage())
        before = frame.clone()
        y1, r1 = rk.rms_norm(moved(x), w1, residual=moved(res), out=out.zero_(), residual_out=ro.zero_())
        assert y1 is out and same_bits(y1.contiguous(), y0) and same_bits(r1.contiguous(), r0)
        assert same_bits(frame, before)  # nothing beside the rows is written
        for group in (0, 128):
            q0, s0, _ = rk.rms_norm_e4m3(xs, w.to(DEV), residual=rs, group=group)
            buf = torch.empty(T * (H + ld) + offset, dtype=E4M3, device=DEV)
            q1 = buf[offset:].view(T, H + ld)[:, :H]
            _, s1, _ = rk.rms_norm_e4m3(moved(x), w1, residual=moved(res), group=group, out=q1)
            assert torch.equal(q1.contiguous().view(torch.uint8), q0.view(torch.uint8)) and same_bits(s1, s0)
        dx0, dw0 = rk.rms_norm_bwd(ds, r0, w.to(DEV), grad_residual=xs, out_dtype=FP32)
        dx1, dw1 = rk.rms_norm_bwd(moved(d), moved(r0.cpu()), w1, grad_residual=moved(x), out=moved(y0.cpu()))
        assert same_bits(dx1.contiguous(), dx0) and same_bits(dw1, dw0)
    assert rk.get_device_error() == 0


def padded_like(g, T, share=0.4):
    tg = torch.randint(0, 100, (T,), generator=g)
    tg[torch.rand(T, generator=g) < share] = -100
    return tg


@pytest.mark.parametrize("T,H", [(9, 24), (50, 264), (333, 1000), (90, 4096), (70, 2047), (5, 16384)])
def test_inactive_rows(rk, T, H):
    g = gen(T)
    x, res, d = npl.matrix(g, T, H, BF16), npl.matrix(g, T, H, BF16), npl.matrix(g, T, H, FP32)
    w = weight_of(g, H, FP32)
    for targets, cu in ((padded_like(g, T), None), (None, [2, T - 3]), (padded_like(g, T), [1, 4, T - 1]),
                        (torch.full((T,), -100), None), (None, [3, 3]), (None, [-5, T + 9])):
        live = npl.active(T, targets, cu)
        xp, rp, dp = x.clone(), res.clone(), d.clone()
        for m in (xp, rp, dp):
            m[~live] = float("nan")
        tg = None if targets is None else targets.to(DEV)
        cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
        full = torch.full((T, H), float("nan"), device=DEV)
        y, r = rk.rms_norm(xp.to(DEV), w.to(DEV), tg, cut, residual=rp.to(DEV), out=full)
        want, stream = npl.forward(npl.stream(x, res), w, live), npl.stream(x, res)
        stream[~live] = 0
        assert same_bits(r, stream) and close(y, want, want.abs() * 19 * npl.U)[0]
        q, s, _ = rk.rms_norm_e4m3(xp.to(DEV), w.to(DEV), tg, cut, residual=rp.to(DEV), group=128)
        assert not bool(q.float()[~live].any()) and not bool(s[~live].any())
        full.fill_(float("nan"))
        dx, dw = rk.rms_norm_bwd(dp.to(DEV), xp.to(DEV), w.to(DEV), tg, cut, out=full)
        assert not bool(dx[~live].any())
        check_bwd(dx, dw, x, d, None, w, live)
    assert rk.get_device_error() == 0


def test_canonical_order(rk):
    """The same rows in the same order have the same dweight in every layout, and a row the same
    results wherever it sits."""
    for H in (40, 512, 1000, 4096, 8195):
        g = gen(H)
        T = 700
        r, d = npl.matrix(g, T, H, BF16), npl.matrix(g, T, H, FP32)
        w = weight_of(g, H, BF16).to(DEV)
        dx0, dw0 = rk.rms_norm_bwd(d.to(DEV), r.to(DEV), w)
        y0, _ = rk.rms_norm(r.to(DEV), w)
        # padded: the rows in order at random places
        P = 1500
        at = torch.randperm(P, generator=g)[:T].sort().values
        rp, dp = torch.full((P, H), float("nan"), dtype=BF16), torch.full((P, H), float("nan"))
        rp[at], dp[at] = r, d
        tg = torch.full((P,), -100)
        tg[at] = 1
        dx, dw = rk.rms_norm_bwd(dp.to(DEV), rp.to(DEV), w, tg.to(DEV))
        assert same_bits(dw, dw0) and same_bits(dx[at.to(DEV)], dx0)
        y, _ = rk.rms_norm(rp.to(DEV), w, tg.to(DEV))
        assert same_bits(y[at.to(DEV)], y0)
        # shuffled, with the order given; entries out of range are passed over
        perm = torch.randperm(P, generator=g)
        back = torch.empty(P, dtype=torch.int64)
        back[perm] = torch.arange(P)
        order = torch.cat([torch.tensor([-1, P, 1 << 40]), back[torch.arange(P)]])
        dx, dw = rk.rms_norm_bwd(dp[perm].to(DEV), rp[perm].to(DEV), w, tg[perm].to(DEV),
                                 row_order=order.to(DEV))
        assert same_bits(dw, dw0) and same_bits(dx[back[at].to(DEV)], dx0)
        # inside a cu_seqlens range
        rq, dq = torch.cat([rp[:5] * float("nan"), r, r[:9]]), torch.cat([d[:5], d, d[:9]])
        cu = torch.tensor([5, 100, 5 + T], dtype=torch.int32, device=DEV)
        dx, dw = rk.rms_norm_bwd(dq.to(DEV), rq.to(DEV), w, cu_seqlens=cu)
        assert same_bits(dw, dw0) and same_bits(dx[5:5 + T], dx0)
        # alone
        for t in (0, 699):
            assert same_bits(rk.rms_norm(r[t:t + 1].to(DEV), w)[0], y0[t:t + 1])
            assert same_bits(rk.rms_norm_bwd(d[t:t + 1].to(DEV), r[t:t + 1].to(DEV), w)[0], dx0[t:t + 1])
        # some rows twice, some not at all
        order = torch.randint(0, T, (900,), generator=g)
        times = torch.bincount(order, minlength=T)
        dx, dw = rk.rms_norm_bwd(d.to(DEV), r.to(DEV), w, row_order=order.to(DEV))
        check_bwd(dx, dw, r, d, None, w.cpu(), times > 0, times=times)
        # nothing at all
        dx, dw = rk.rms_norm_bwd(d.to(DEV), r.to(DEV), w, row_order=order[:0].to(DEV))
        assert not bool(dx.any()) and not bool(dw.any())
    assert rk.get_device_error() == 0


def test_long_candidate_lists(rk):
    """More candidates than one block lists."""
    T, H = 40001, 16
    g = gen(1)
    r, d = npl.matrix(g, T, H, BF16), npl.matrix(g, T, H, BF16)
    w = weight_of(g, H, BF16)
    tg = padded_like(g, T)
    live = tg >= 0
    dx, dw = rk.rms_norm_bwd(d.to(DEV), r.to(DEV), w.to(DEV), tg.to(DEV))
    dx0, dw0 = rk.rms_norm_bwd(d[live].to(DEV), r[live].to(DEV), w.to(DEV))
    assert same_bits(dw, dw0) and same_bits(dx[live.to(DEV)], dx0) and not bool(dx[~live.to(DEV)].any())
    check_bwd(dx, dw, r, d, None, w, live)


@pytest.mark.parametrize("H", [40, 264, 1000, 2047, 2048, 4096, 5000])
@pytest.mark.parametrize("n", [0, 1, 300, 1023, 1024, 1025])
def test_short_and_long_candidate_lists(rk, n, H):
    """Inactive candidates in between change neither bits nor which rows are 0, however the list is
    made of them; more rows than candidates and fewer."""
    g = gen(n + H)
    T = 1024
    r, d = npl.matrix(g, T, H, BF16).to(DEV), npl.matrix(g, T, H, FP32).to(DEV)
    w = weight_of(g, H, BF16).to(DEV)
    targets = torch.ones(T, dtype=torch.int64)
    targets[::5] = -1
    alive, dead = torch.arange(T)[targets >= 0], torch.arange(T)[targets < 0]
    order = torch.cat([alive, dead, alive, dead])[torch.randperm(2 * T, generator=g)[:n]]
    gaps = torch.randint(0, 4, (n,), generator=g) + (2048 if n == 1 else 0)
    mixed = torch.cat([torch.cat([o[None], dead[torch.randint(0, len(dead), (int(k),), generator=g)]])
                       for o, k in zip(order, gaps)] + [dead, dead[:7]]) if n else dead.repeat(10)
    call = lambda o, t: rk.rms_norm_bwd(d[:t], r[:t], w, targets[:t].to(DEV), eps=npl.EPS, row_order=o.to(DEV))  # noqa: E731
    dx, dw = call(order, T)
    mx, mw = call(mixed, T)
    assert same_bits(dx, mx) and same_bits(dw, mw)
    named = torch.zeros(T, dtype=torch.bool)
    named[order] = True
    assert not dx[~(named & (targets >= 0)).to(DEV)].any()
    # the same rows of a matrix that is too long for the short list
    long = lambda x: torch.cat([x, torch.full_like(x, float("nan"))])  # noqa: E731
    lx, lw = rk.rms_norm_bwd(long(d), long(r), w, torch.cat([targets, -targets.abs()]).to(DEV), eps=npl.EPS,
                             row_order=order.to(DEV))
    assert same_bits(lx[:T], dx) and same_bits(lw, dw) and not lx[T:].any()


def test_fused_addition_has_the_bits_of_two_calls(rk):
    g = gen(2)
    for H in (100, 1000, 4096):
        x, res = npl.matrix(g, 77, H, BF16).to(DEV), npl.matrix(g, 77, H, BF16).to(DEV)
        w = weight_of(g, H, BF16).to(DEV)
        y, r = rk.rms_norm(x, w, residual=res)
        y2, r2 = rk.rms_norm((x.float() + res.float()).bfloat16(), w)
        assert same_bits(y, y2) and same_bits(r, r2)


def test_in_place(rk):
    g = gen(3)
    for H in (24, 777, 2048, 4096):
        x, res = npl.matrix(g, 301, H, BF16).to(DEV), npl.matrix(g, 301, H, BF16).to(DEV)
        w = weight_of(g, H, BF16).to(DEV)
        y0, r0 = rk.rms_norm(x, w, residual=res)
        x1, res1 = x.clone(), res.clone()
        y, r = rk.rms_norm(x1, w, residual=res1, out=x1, residual_out=res1)
        assert y is x1 and r is res1 and same_bits(y, y0) and same_bits(r, r0)
        d = npl.matrix(g, 301, H, BF16).to(DEV)
        dx0, dw0 = rk.rms_norm_bwd(d, r0, w, grad_residual=x)
        for place in range(3):
            ops = [d.clone(), r0.clone(), x.clone()]
            dx, dw = rk.rms_norm_bwd(ops[0], ops[1], w, grad_residual=ops[2], out=ops[place])
            assert same_bits(dx, dx0) and same_bits(dw, dw0)
    # dweight added to what is there
    old = torch.randn(4096, generator=g)
    dw = old.to(DEV)
    rk.rms_norm_bwd(d, r0, w, dweight=dw, accumulate=True)
    check_bwd(*rk.rms_norm_bwd(d, r0, w, dweight=old.to(DEV), accumulate=True)[:2], r0.cpu(), d.cpu(), None, w.cpu(),
              torch.ones(301, dtype=torch.bool), old=old)
    assert rk.get_device_error() == 0


def test_large_and_small_values(rk):
    """Sums of squares past fp32, rows of tiny values, and what is not finite stays in its row."""
    for H in (64, 1000, 4096):
        g = gen(H)
        x = npl.matrix(g, 6, H, FP32)
        x[0] *= 1e25
        x[1] *= 1e37
        x[2] *= 1e-30
        d = npl.matrix(g, 6, H, FP32)
        w = weight_of(g, H, BF16)
        live = torch.ones(6, dtype=torch.bool)
        want = npl.forward(x, w, live)
        y, _ = rk.rms_norm(x.to(DEV), w.to(DEV))
        assert close(y, want, want.abs() * (npl.FORWARD + npl.U))[0]
        dx, dw = rk.rms_norm_bwd(d.to(DEV), x.to(DEV), w.to(DEV))
        want_dx, _, bound = npl.backward(d, x, w, None, live)
        # quotients of 1e37 leave the normal numbers
        assert close(dx, want_dx, bound + 2.0 ** -126)[0] and bool(torch.isfinite(dw).all())
        x[3, H // 2] = float("inf")
        x[4, 0] = float("nan")
        y2, _ = rk.rms_norm(x.to(DEV), w.to(DEV))
        keep = torch.tensor([0, 1, 2, 5], device=DEV)
        assert same_bits(y2[keep], y[keep]) and bool(torch.isnan(y2[4]).all()) and bool(torch.isnan(y2[3, H // 2]))
    assert rk.get_device_error() == 0


def test_no_rows(rk):
    w = torch.ones(64, device=DEV)
    none = torch.empty(0, 64, device=DEV)
    y, r = rk.rms_norm(none, w)
    assert y.shape == (0, 64) and r is none
    q, s, _ = rk.rms_norm_e4m3(none, w, group=128)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    dw = torch.ones(64, device=DEV)
    dx, got = rk.rms_norm_bwd(none, none, w, dweight=dw, accumulate=True)
    assert dx.shape == (0, 64) and bool((got == 1).all())
    assert not bool(rk.rms_norm_bwd(none, none, w, dweight=dw)[1].any())


def test_streams_and_graphs(rk):
    g = gen(5)
    T, H = 600, 4096
    x, res, d = (npl.matrix(g, T, H, BF16).to(DEV) for _ in range(3))
    tg = padded_like(g, T).to(DEV)
    w = weight_of(g, H, BF16).to(DEV)

    def step(stream=None):
        y, r = rk.rms_norm(x, w, tg, residual=res, stream=stream)
        q, s, _ = rk.rms_norm_e4m3(x, w, tg, residual=res, group=128, stream=stream)
        dx, dw = rk.rms_norm_bwd(d, r, w, tg, grad_residual=y, stream=stream)
        return y, r, q.view(torch.uint8), s, dx, dw
    want = step()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):  # two at once
        got = [step(s) for s in side]
        torch.cuda.synchronize()
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(one, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(torch.randn(T, H, generator=g).to(BF16))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert rk.get_device_error() == 0


def test_gradients_are_the_forward_s_differences(rk):
    """A directional difference of a 64-bit sum over the fp32 forward's 64-bit form, and autograd."""
    g = gen(6)
    T, H = 5, 72
    x, w, d = npl.matrix(g, T, H, FP32), weight_of(g, H, FP32), npl.matrix(g, T, H, FP32)
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    y = xd * (xd.square().mean(1, keepdim=True) + npl.EPS).rsqrt() * wd
    (y * d.double()).sum().backward()
    live = torch.ones(T, dtype=torch.bool)
    dx, terms, bound = npl.backward(d, x, w, None, live)
    assert torch.allclose(dx, xd.grad, rtol=1e-12, atol=1e-14) and torch.allclose(terms.sum(0), wd.grad, rtol=1e-12, atol=1e-14)
    v = torch.randn(T, H, generator=g).double()
    h = 1e-5
    up = (npl.forward(x.double() + h * v, w, live) * d.double()).sum()
    down = (npl.forward(x.double() - h * v, w, live) * d.double()).sum()
    got, _ = rk.rms_norm_bwd(d.to(DEV), x.to(DEV), w.to(DEV))
    # the difference's own error: h^2 times a third derivative of order one, and 2^-53 / h
    assert abs(float((got.double().cpu() * v).sum() - (up - down) / (2 * h))) <= float((bound * v.abs()).sum()) + 1e-7


def test_sums_of_bf16_are_rounded_once(rk):
    """Every kind of pair, subnormal numbers and infinities among them, as fp32 and then bf16 rounds them."""
    g = gen(7)
    bits = torch.randint(-2 ** 15, 2 ** 15, (2, 40000, 64), generator=g, dtype=torch.int16)
    bits[:, :8000] &= 0x80FF - 0x10000  # subnormal and smallest
    near = torch.randint(-3, 4, (16000, 64), generator=g) * 128
    bits[1, 8000:24000] = ((bits[0, 8000:24000].int() & 0x7FFF) + near).clamp(0, 0x7F80).short() ^ -0x8000
    x, r = (b.view(BF16).clone() for b in bits)
    x[torch.isnan(x)], r[torch.isnan(r)] = 1.0, -2.0
    want = npl.stream(x, r)
    _, got = rk.rms_norm(x.to(DEV), torch.ones(64, dtype=BF16, device=DEV), residual=r.to(DEV))
    got = got.cpu()
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all()) and same_bits(got[~nan], want[~nan])


def test_weights_that_are_not_finite(rk):
    """They reach the active rows alone."""
    g = gen(8)
    for H in (40, 1001, 4096):
        w = weight_of(g, H, BF16)
        w[3], w[4] = float("nan"), float("inf")
        x = npl.matrix(g, 6, H, BF16).to(DEV)
        tg = torch.tensor([1, -1, 1, -100, 1, -1], device=DEV)
        y, _ = rk.rms_norm(x, w.to(DEV), tg)
        q, s, _ = rk.rms_norm_e4m3(x, w.to(DEV), tg)
        off = tg < 0
        assert not bool(y[off].any()) and not bool(q.float()[off].any()) and not bool(s[off].any())
        assert bool(torch.isnan(y[~off][:, 3]).all())


def test_without_dweight(rk):
    g = gen(9)
    r, d = npl.matrix(g, 50, 264, BF16).to(DEV), npl.matrix(g, 50, 264, BF16).to(DEV)
    w = weight_of(g, 264, BF16).to(DEV)
    dx, none = rk.rms_norm_bwd(d, r, w, need_dweight=False)
    assert none is None and same_bits(dx, rk.rms_norm_bwd(d, r, w)[0])
    with pytest.raises(ValueError, match="need_dweight"):
        rk.rms_norm_bwd(d, r, w, need_dweight=False, dweight=torch.zeros(264, device=DEV))


def test_rows_past_32_bits(rk):
    """More than 2^32 bytes, and more than 2^31 elements: the last rows have the bits that they have alone."""
    T, H = 140000, 16384
    x = torch.empty(T, H, dtype=BF16, device=DEV)
    g = torch.Generator(DEV).manual_seed(1)
    for a in range(0, T, 20000):
        x[a:a + 20000] = torch.randn(20000, H, generator=g, device=DEV)
    w = torch.ones(H, dtype=BF16, device=DEV)
    tail = x[-3:].clone()
    tg = torch.full((T,), -1, device=DEV)
    tg[-3:] = 1
    tg[::7000] = 1
    y, _ = rk.rms_norm(x, w, tg)
    assert same_bits(y[-3:], rk.rms_norm(tail, w)[0]) and not bool(y[-10:-3].any())
    q, s, _ = rk.rms_norm_e4m3(x, w, tg, group=128)
    q0, s0, _ = rk.rms_norm_e4m3(tail, w, group=128)
    assert torch.equal(q[-3:].view(torch.uint8), q0.view(torch.uint8)) and same_bits(s[-3:], s0)
    del q, s
    dx, dw = rk.rms_norm_bwd(y, x, w, tg)
    assert same_bits(dx[-3:], rk.rms_norm_bwd(y[-3:], tail, w)[0]) and not bool(dx[-10:-3].any())
    live = tg >= 0
    _, dw0 = rk.rms_norm_bwd(y[live], x[live], w)
    assert same_bits(dw, dw0)
    assert rk.get_device_error() == 0
