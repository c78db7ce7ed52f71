"""The AdamW step written out in 64 bits, with bounds on what fp32 and the 8-bit states may add."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32, relative
BLOCK = 256


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def spread(scale, n):
    return scale.repeat_interleave(BLOCK)[:n]


def step(w, g, m, v, *, lr, step, beta1, beta2, eps, decay=0.0, grad_scale=1.0):
    """(w, m, v) in float64 after a step and bounds on their errors in fp32."""
    g = g.double() * grad_scale
    a, b = m * beta1, g * (1 - beta1)
    m1 = a + b
    v1 = v * beta2 + g * g * (1 - beta2)
    rate, den = lr / (1 - beta1 ** step), (v1 / (1 - beta2 ** step)).sqrt() + eps
    move = m1 * rate / den
    w1 = w - lr * decay * w - move
    # m: beta, 1 - beta, g * scale, its product and the sum; v: the same with two g and the square
    dm = 5 * U * (a.abs() + b.abs())
    dv = 7 * U * v1
    # rate 8 (a step on the device: log, product, expm1, quotient, lr, lr_scale, product), its product
    # 1, the root 3.5 + 1 + 7, sum and quotient 2
    dmove = 24 * U * move.abs() + dm * rate / den
    dw = U * (w.abs() * (1 + 4 * lr * decay) + 2 * (w1.abs() + dmove)) + dmove
    tiny = 2.0 ** -126
    return (w1, m1, v1), (1.01 * dw + tiny, 1.01 * dm + tiny, 1.01 * dv + tiny)


def decode(code, scale, root):
    x = code.float().double() * spread(scale.double(), code.numel())
    return x * x if root else x


def check_state(code, scale, want, bound, root):
    """An 8-bit state against a float64 one: its scales, and its codes under these."""
    n = want.numel()
    if root:
        bound, want = bound / (2 * want.sqrt()).clamp(min=1e-30), want.sqrt()
        bound = torch.minimum(bound, want) + U * want
    pad = lambda t: torch.nn.functional.pad(t, (0, blocks(n) * BLOCK - n)).view(-1, BLOCK)  # noqa: E731
    top = pad(want.abs()).amax(1) / 448
    slack = (pad(bound).amax(1)) / 448 + 2 * U * top
    assert bool(((scale.double() - top).abs() <= slack).all())
    s = spread(scale.double(), n)
    live = s > 0
    z = torch.where(live, want / torch.where(live, s, 1.0), 0.0)
    e = torch.where(live, bound / torch.where(live, s, 1.0), 0.0)
    if root:
        # a scale of 0 stands for a block whose v fp32 cannot hold (1e-30 squared is below 2^-149):
        # its codes are 0, which the check of the scale above has allowed within the bound
        z = torch.where((want > 0) & live, z.clamp(min=2.0 ** -9), z)
    half = torch.maximum(z.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    over = (code.float().double() - z).abs() - (half * (1 + 4 * U) + 2 * e)
    assert float(over.max()) <= 0, float(over.max())
    if root:
        assert bool((code.float()[(want > 0) & live] > 0).all())
