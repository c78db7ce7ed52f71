"""Refusals of the root-mean-square norm and its gradient (no GPU needed: refused calls read
none of the addresses)."""
import pytest
import torch

FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BF16, FP32, E4M3 = 0, 1, 2
FAR = 1 << 30


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def forward(rk, T=4, H=64, x=FAKE, xt=BF16, ld=64, res=None, rt=BF16, ldr=64, w=2 * FAR, wt=BF16, eps=1e-6, tg=None,
            cu=None, ns=0, ro=None, ldro=64, out=FAR, ot=BF16, ldo=64, s=None, group=0):
    return rk.load_library().rk_rms_norm(x, xt, ld, res, rt, ldr, w, wt, eps, tg, cu, ns, T, H, ro, ldro, out, ot,
                                         ldo, s, group, None)


def backward(rk, T=4, H=64, d=FAKE, dt=BF16, ldd=64, r=FAR, rt=BF16, ldr=64, w=2 * FAR, wt=BF16, eps=1e-6, dr=None,
             drt=BF16, lddr=64, tg=None, cu=None, ns=0, order=None, n=0, dx=3 * FAR, xt=BF16, ldx=64, dw=4 * FAR,
             acc=0, ws=5 * FAR, wb=1 << 30):
    return rk.load_library().rk_rms_norm_bwd(d, dt, ldd, r, rt, ldr, w, wt, eps, dr, drt, lddr, tg, cu, ns, T, H,
                                             order, n, dx, xt, ldx, dw, acc, ws, wb, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(x=None), dict(w=None), dict(out=None), dict(xt=2), dict(xt=3), dict(wt=2), dict(ot=3),
    dict(ld=63), dict(ldo=63), dict(x=FAKE + 1), dict(xt=FP32, x=FAKE + 2), dict(out=FAR + 1), dict(w=FAR + 1),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(cu=FAKE, ns=-1),
    dict(res=3 * FAR), dict(ro=3 * FAR), dict(res=3 * FAR, ro=4 * FAR, rt=E4M3), dict(res=3 * FAR, ro=4 * FAR, ldr=60),
    dict(res=3 * FAR, ro=4 * FAR + 1), dict(group=128), dict(s=3 * FAR), dict(ot=E4M3), dict(ot=E4M3, s=3 * FAR, group=64),
    dict(ot=E4M3, s=3 * FAR + 2)])
def test_forward_refusals(rk, bad):
    assert forward(rk, **bad) == INVALID


def test_forward_limits(rk):
    assert forward(rk, T=0) == OK
    assert forward(rk, H=16385, ld=16385, ldo=16385) == UNSUPPORTED
    assert forward(rk, T=1 << 31) == UNSUPPORTED


# rows of 64 columns, 128 bytes in bf16
@pytest.mark.parametrize("bad", [
    dict(out=FAKE + 2), dict(out=FAKE - 2), dict(out=FAKE + 4 * 128 - 2), dict(out=FAKE, ot=FP32),
    dict(out=FAKE, ldo=72), dict(out=FAKE, ot=E4M3, s=3 * FAR), dict(w=FAR), dict(w=FAR + 511), dict(w=FAR - 126),
    dict(res=3 * FAR, ro=FAR), dict(res=3 * FAR, ro=FAR + 510), dict(res=3 * FAR, ro=3 * FAR + 4),
    dict(res=3 * FAR, ro=FAKE + 4), dict(res=3 * FAR, ro=FAKE, rt=FP32), dict(res=FAR + 2, ro=3 * FAR),
    dict(res=3 * FAR, ro=2 * FAR), dict(ot=E4M3, s=FAKE + 508), dict(ot=E4M3, s=FAR + 252),
    dict(ot=E4M3, s=2 * FAR + 124), dict(ot=E4M3, s=3 * FAR, res=3 * FAR, ro=4 * FAR),
    dict(ot=E4M3, s=4 * FAR + 508, res=3 * FAR, ro=4 * FAR)])
def test_forward_overlaps(rk, bad):
    assert forward(rk, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(d=None), dict(r=None), dict(w=None), dict(dx=None), dict(dt=2), dict(rt=2), dict(wt=7),
    dict(xt=2), dict(ldd=63), dict(ldr=63), dict(ldx=1), dict(d=FAKE + 1), dict(dw=4 * FAR + 2), dict(acc=2),
    dict(eps=0.0), dict(cu=FAKE, ns=-1), dict(order=FAKE, n=-1), dict(dr=6 * FAR, drt=E4M3), dict(dr=6 * FAR, lddr=2),
    dict(ws=5 * FAR + 8), dict(dx=FAKE + 2), dict(dx=FAR + 4), dict(dx=FAKE, xt=FP32), dict(dr=6 * FAR, dx=6 * FAR + 2),
    dict(dx=2 * FAR), dict(dw=FAKE), dict(dw=FAR + 508), dict(dw=3 * FAR), dict(dw=2 * FAR), dict(dr=6 * FAR, dw=6 * FAR),
    # in place, where the order may name a row twice
    dict(order=FAKE, n=4, dx=FAKE), dict(order=FAKE, n=4, dx=FAR), dict(order=FAKE, n=4, dr=6 * FAR, dx=6 * FAR)])
def test_backward_refusals(rk, bad):
    assert backward(rk, **bad) == INVALID


def test_backward_limits(rk):
    assert backward(rk, ws=None) == WORKSPACE and backward(rk, wb=64) == WORKSPACE
    assert backward(rk, H=16385, ldd=16385, ldr=16385, ldx=16385) == UNSUPPORTED
    assert backward(rk, T=1 << 31) == UNSUPPORTED and backward(rk, order=FAKE, n=1 << 31) == UNSUPPORTED
    f = rk.rms_norm_bwd_workspace_size
    assert f(0, 0, 64) == 0 and f(4, 4, 16385) == 0 and f(4, 4, 0) == 0
    assert f(100, 100, 4096) >= 152 * 4096 * 4 and f(1 << 30, 1 << 30, 64) > (1 << 32)


def test_binding_refuses(rk):
    x, w = torch.zeros(3, 8), torch.ones(8)
    for call in (lambda: rk.rms_norm(x, w), lambda: rk.rms_norm_e4m3(x, w), lambda: rk.rms_norm_bwd(x, x, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="Tensor"):
        rk.rms_norm([1.0], w)
