"""The norm and its gradient at the edges: sums that leave fp32, a norm over its own input, what
the weight's gradient knows of the residual's, and the gradient in every combination of types at every width
where its shape changes, with masks and off alignment."""
import pytest
import torch

import norm_plain as npl
from helpers import same_bits
from test_gpu_norm import BF16, DEV, FP32, bwd_case, check_bwd, gen, padded_like, weight_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


@pytest.mark.parametrize("H", [1, 40, 264, 512, 1000, 1001, 2048, 3000, 4096, 5000, 8192, 16384])
def test_products_past_fp32(rk, H):
    """Gradients so large that the sum of g r, or of g n, leaves fp32 where the result does not; with and
    without a sum of squares that leaves it too."""
    g = gen(H)
    # (size of r, size of dout): sizes of g r, g n and of the result, rstd g
    sizes = [(1e17, 1e22), (1e17, 1e34), (1e30, 1e20), (1e37, 1e36), (1e3, 2e37), (1e-3, 1e-20), (1.0, 1.0)]
    kinds = ((FP32, FP32, None), (BF16, BF16, BF16), (BF16, FP32, FP32), (FP32, BF16, BF16))
    for r_type, d_type, dr_type, one_sign in [(*k, s) for k in kinds for s in (True, False)]:
        r = npl.matrix(g, len(sizes), H, FP32)
        d = npl.matrix(g, len(sizes), H, FP32)
        for i, (size, up) in enumerate(sizes):
            r[i] *= size
            d[i] = (d[i] * up).clamp(-5e37, 5e37)
        if one_sign:
            d = d.abs() * torch.where(r < 0, -1.0, 1.0)
        r, d = r.to(r_type), d.to(d_type)
        w = (1 + 0.2 * torch.rand(H, generator=g)).to(BF16)
        dr = None if dr_type is None else npl.matrix(g, len(sizes), H, dr_type)
        live = torch.ones(len(sizes), dtype=torch.bool)
        got, dw = rk.rms_norm_bwd(d.to(DEV), r.to(DEV), w.to(DEV), grad_residual=None if dr is None else dr.to(DEV),
                                  eps=npl.EPS, out_dtype=FP32)
        want, terms, bound = npl.backward(d, r, w, dr, live)
        ok = (got.double().cpu() - want).abs() <= bound + 2.0 ** -126
        assert bool(ok.all()), [(sizes[i], int((~ok[i]).sum())) for i in range(len(sizes))]
        ok = (dw.double().cpu() - terms.sum(0)).abs() <= (17 + 80) * 1.01 * npl.U * terms.abs().sum(0)
        assert bool(ok.all())
        # a row of its own has the same bits, beside whatever
        alone = [rk.rms_norm_bwd(d[i:i + 1].to(DEV), r[i:i + 1].to(DEV), w.to(DEV), eps=npl.EPS, out_dtype=FP32,
                                 grad_residual=None if dr is None else dr[i:i + 1].to(DEV))[0] for i in range(len(sizes))]
        assert same_bits(torch.cat(alone), got)
    assert rk.get_device_error() == 0


def test_in_place_without_a_residual(rk):
    """The norm over its own input keeps no r: none is returned, and the gradient refuses to work without."""
    g = gen(4)
    for H in (24, 777, 4096):
        x = npl.matrix(g, 9, H, BF16).to(DEV)
        w = weight_of(g, H, BF16).to(DEV)
        y0, r0 = rk.rms_norm(x, w)
        assert r0 is x
        over = x.clone()
        y, r = rk.rms_norm(over, w, out=over)
        assert y is over and r is None and same_bits(y, y0)
        over.copy_(x)
        y, r = rk.rms_norm(over, w, out=over.view(9, H))
        assert r is None and same_bits(y, y0)
        with pytest.raises(TypeError, match="r must be a torch.Tensor"):
            rk.rms_norm_bwd(y0, r, w)
        # with one, r is residual_out
        over.copy_(x)
        y, r = rk.rms_norm(over, w, residual=x, out=over)
        assert y is over and same_bits(r, (x.float() + x.float()).bfloat16())
    none = torch.empty(0, 8, device=DEV)
    assert rk.rms_norm(none, torch.ones(8, device=DEV), out=none)[1] is none


# every pair of a team and its vectors, whole and halved, on both sides of every limit
WIDTHS = [24, 264, 513, 1000, 1024, 1025, 1408, 1416, 1536, 1537, 1792, 1800, 2048, 2049, 2056, 3000, 3001, 4096, 4104,
          6144, 6145, 6152, 8190, 8192, 8200]
TYPES = [(r, d, z) for r in (BF16, FP32) for d in (BF16, FP32) for z in (None, BF16, FP32)]


def moved(t, ld, offset):
    m = npl.matrix(gen(0), *t.shape, t.dtype, ld, offset)
    m.copy_(t)
    return npl.to(m, DEV)


@pytest.mark.parametrize("r_type,d_type,dr_type", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_of_every_combination_of_types(rk, H, r_type, d_type, dr_type):
    """Against 64 bits with a mask, all at once and by short lists; NaN in rows that are not active; rows
    off 16 bytes have the same bits."""
    g = gen(H)
    T = 37
    r, dout, dr, w = bwd_case(g, T, H, r_type, d_type, dr_type)
    targets = padded_like(g, T)
    live = targets >= 0
    rp, dp, zp = r.clone(), dout.clone(), None if dr is None else dr.clone()
    for m in (rp, dp, zp):
        if m is not None:
            m[~live] = float("nan")
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    w_dev, tg = w.to(DEV), targets.to(DEV)
    full = torch.full((T, H), float("nan"), device=DEV)
    dx, dw = rk.rms_norm_bwd(to(dp), to(rp), w_dev, tg, grad_residual=to(zp), eps=npl.EPS, out=full)
    check_bwd(dx, dw, r, dout, dr, w, live)
    assert not bool(dx[~live.to(DEV)].any())
    # packed, without a mask
    px, pw = rk.rms_norm_bwd(to(dout[live]), to(r[live]), w_dev, grad_residual=to(None if dr is None else dr[live]),
                             eps=npl.EPS, out_dtype=FP32)
    assert same_bits(px, dx[live.to(DEV)]) and same_bits(pw, dw)
    # behind more rows than blocks list for themselves
    far = lambda t: None if t is None else torch.cat([torch.full((1100, H), float("nan"), dtype=t.dtype), t]).to(DEV)  # noqa: E731
    fx, fw = rk.rms_norm_bwd(far(dp), far(rp), w_dev, torch.cat([torch.full((1100,), -1), targets]).to(DEV),
                             grad_residual=far(zp), eps=npl.EPS, out_dtype=FP32)
    assert same_bits(fx[1100:], dx) and same_bits(fw, dw) and not bool(fx[:1100].any())
    # off 16 bytes
    for ld, offset in ((3, 1), (8, 4)):
        off = lambda t: None if t is None else moved(t, ld, offset)  # noqa: E731
        ox, ow = rk.rms_norm_bwd(off(dp), off(rp), w_dev, tg, grad_residual=off(zp), eps=npl.EPS, out=off(full.cpu()))
        assert same_bits(ox.contiguous(), dx) and same_bits(ow, dw)
    # some rows twice, with the mask
    order = torch.randint(0, T, (50,), generator=g)
    times = torch.bincount(order, minlength=T) * live
    dx, dw = rk.rms_norm_bwd(to(dp), to(rp), w_dev, tg, grad_residual=to(zp), eps=npl.EPS, out_dtype=FP32, row_order=to(order))
    check_bwd(dx, dw, r, dout, dr, w, times > 0, times=times)
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("r_type", [BF16, FP32])
@pytest.mark.parametrize("H", WIDTHS)
def test_a_residual_s_gradient_of_the_same_type_leaves_dweight_s_bits(rk, H, r_type):
    """dweight has no term of dr, and the order of its sum knows of dr by its type alone where r is bf16; where r is
    fp32 it knows whether there is one in some widths, and then of no type."""
    g = gen(H + 1)
    T = 3000 if H <= 2056 else 1300
    r, dout = npl.matrix(g, T, H, r_type).to(DEV), npl.matrix(g, T, H, BF16).to(DEV)
    w = weight_of(g, H, BF16).to(DEV)
    _, without = rk.rms_norm_bwd(dout, r, w)
    a, b = (rk.rms_norm_bwd(dout, r, w, grad_residual=npl.matrix(g, T, H, t).to(DEV))[1] for t in (BF16, FP32))
    if r_type is BF16:
        assert same_bits(a, without)
    else:
        assert same_bits(a, b)
    if H <= 1024 or 4096 < H <= 6144 or H > 8192:
        assert same_bits(a, without) and same_bits(b, without)
