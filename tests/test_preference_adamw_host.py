"""Refusals of the preference loss and the AdamW step (no GPU needed: refused calls read none of
the addresses)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20
FAR = 1 << 30
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BF16, FP32, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def preference(rk, lp=FAKE, ref=None, tg=FAR, cu=2 * FAR, ns=4, T=100, c=3 * FAR, r=4 * FAR, P=8, margin=None, kind=0,
               beta=0.1, e=0.0, avg=0, scale=1.0, loss=5 * FAR, grad=6 * FAR, ratio=7 * FAR, ws=8 * FAR, wb=1 << 20):
    return rk.load_library().rk_preference_loss(lp, ref, tg, cu, ns, T, c, r, P, margin, kind, beta, e, avg, scale,
                                                loss, grad, ratio, ws, wb, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(P=-1), dict(ns=-1), dict(cu=None), dict(lp=None), dict(tg=None), dict(grad=None), dict(c=None),
    dict(r=None), dict(loss=None), dict(kind=3), dict(kind=-1), dict(beta=0.0), dict(beta=-1.0),
    dict(beta=float("nan")), dict(beta=float("inf")), dict(e=-0.1), dict(e=1.1), dict(e=0.1, kind=1),
    dict(e=0.1, kind=2), dict(avg=2), dict(lp=FAKE + 2), dict(tg=FAR + 4), dict(grad=6 * FAR + 1), dict(ws=8 * FAR + 8),
    # results over inputs, or over one another
    dict(grad=FAKE), dict(grad=FAKE + 396), dict(grad=FAR + 792), dict(grad=2 * FAR + 16), dict(loss=3 * FAR),
    dict(loss=4 * FAR + 28), dict(loss=6 * FAR), dict(ratio=6 * FAR + 396), dict(ratio=5 * FAR),
    dict(margin=9 * FAR, loss=9 * FAR), dict(ref=9 * FAR, ratio=9 * FAR + 12)])
def test_preference_refusals(rk, bad):
    assert preference(rk, **bad) == INVALID


def test_preference_limits(rk):
    assert preference(rk, T=0, P=0, ns=0) == OK
    assert preference(rk, T=1 << 31) == UNSUPPORTED and preference(rk, P=1 << 31) == UNSUPPORTED
    assert preference(rk, ws=None) == WORKSPACE and preference(rk, wb=200) == WORKSPACE
    f = rk.preference_loss_workspace_size
    assert f(-1, 4) == 0 and f(4, -1) == 0 and f(0, 0) == 0 and f(1000, 10) >= 1000 * 32 + 40


def tensor(rk, **kw):
    base = dict(param=FAKE, master=FAR, grad=2 * FAR, m=3 * FAR, v=4 * FAR, m_scale=None, v_scale=None, n=100,
                param_type=BF16, grad_type=FP32, lr_scale=1.0, weight_decay=0.1)
    return rk._AdamWTensor(**{**base, **kw})


def adamw(rk, tensors, options=None, **kw):
    o = rk._AdamWOptions(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1), **kw})
    array = (rk._AdamWTensor * max(1, len(tensors)))(*tensors)
    return rk.load_library().rk_adamw_step(ctypes.addressof(array), len(tensors), ctypes.addressof(o), None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param_type=E4M3),
    dict(grad_type=E4M3), dict(param_type=FP32), dict(m_scale=5 * FAR), dict(v_scale=5 * FAR), dict(param=FAKE + 1),
    dict(grad=2 * FAR + 2), dict(m=3 * FAR + 2), dict(v=4 * FAR + 1), dict(master=FAR + 2),
    dict(m_scale=5 * FAR + 2, v_scale=6 * FAR), dict(lr_scale=float("nan")), dict(weight_decay=float("inf"))])
def test_adamw_tensor_refusals(rk, bad):
    assert adamw(rk, [tensor(rk), tensor(rk, **bad)]) == INVALID


def test_adamw_refusals(rk):
    lib = rk.load_library()
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("inf")), dict(eps=1e-60), dict(lr=float("nan")), dict(lr=float("inf")),
                dict(step=0), dict(lr_device=FAKE + 2), dict(step_device=FAKE + 4), dict(grad_scale=FAKE + 1)):
        assert adamw(rk, [tensor(rk)], **bad) == INVALID, bad
    assert adamw(rk, [tensor(rk, n=1 << 40)]) == UNSUPPORTED
    assert adamw(rk, []) == OK
    o = rk._AdamWOptions(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1)
    assert lib.rk_adamw_step(None, 1, ctypes.addressof(o), None) == INVALID
    assert lib.rk_adamw_step(None, -1, ctypes.addressof(o), None) == INVALID
    assert lib.rk_adamw_step(None, 0, None, None) == INVALID


def test_structs_have_the_header_s_layout(rk):
    """Offsets of the last members: the C compiler's, and ctypes'."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ('#include <stddef.h>\n#include <stdio.h>\n#include "rk.h"\nint main(void) { printf("%zu %zu %zu %zu", '
            'sizeof(rk_adamw_tensor), offsetof(rk_adamw_tensor, weight_decay), sizeof(rk_adamw_options), '
            'offsetof(rk_adamw_options, grad_scale)); return 0; }\n')
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        with open(src, "w") as f:
            f.write(code)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    t, o = rk._AdamWTensor, rk._AdamWOptions
    assert got == [ctypes.sizeof(t), t.weight_decay.offset, ctypes.sizeof(o), o.grad_scale.offset]


def test_bindings_refuse(rk):
    x, i = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rk.preference_loss(x, i, s, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        rk.AdamW([x], [x])
    with pytest.raises(TypeError, match="AdamW"):
        rk.adamw_step([x], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="go together"):
        rk.AdamW([], [], m=[])
    with pytest.raises(ValueError, match="one entry"):
        rk.AdamW([], [x])
