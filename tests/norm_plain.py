"""The root-mean-square norm and its gradient written out in 64 bits, row by row, with
bounds on what fp32 may add, and the cases the tests draw."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def matrix(g, T, H, dtype, ld=0, offset=0, scale=1.0):
    """[T, H] on the CPU inside a buffer: `ld` unused columns behind each row, `offset`
    elements in front."""
    buf = torch.full((T * (H + ld) + offset,), float("nan"), dtype=dtype)
    m = buf[offset:].view(T, H + ld)[:, :H]
    m.copy_(torch.randn(T, H, generator=g) * scale)
    return m


def to(t, device):
    """The same view on a device: strides and the offset from 16 bytes are kept."""
    if t is None:
        return None
    base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage())
    return torch.as_strided(base.to(device), t.shape, t.stride(), t.storage_offset())


def active(T, targets, cu):
    a = torch.ones(T, dtype=torch.bool) if targets is None else targets >= 0
    if cu is not None:
        t = torch.arange(T)
        a = a & (t >= int(cu[0])) & (t < int(cu[-1]))
    return a


def stream(x, residual):
    """r, in residual's type."""
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def forward(r, weight, live, eps=EPS):
    """y in float64, 0 in rows that are not live."""
    z = r.double()
    y = z / (z.square().mean(1, keepdim=True) + eps).sqrt() * weight.double()
    return torch.where(live[:, None], y, 0.0)


# rstd: at most 16 products and sums in a thread, 10 sums over the team, 1 / H and its product,
# eps and its addition: 30 roundings of which the root takes half, then its own; two
# products: 15 + 1 + 2 half steps of fp32
FORWARD = 18 * U


def e4m3_bound(z):
    """How far a rounded e4m3 value may be from z."""
    return torch.maximum(z.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) + 2 * FORWARD * z.abs()


def backward(dout, r, weight, dr, live, eps=EPS):
    """(dx, terms of dweight, bound on dx's error, sum of the magnitudes of dweight's terms)."""
    d, z, w = dout.double(), r.double(), weight.double()
    rstd = (z.square().mean(1, keepdim=True) + eps).rsqrt()
    n, g = z * rstd, d * w
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    # relative to rstd |g|: g 1, the fused difference 1, rstd 16 and its product 1.  Relative
    # to rstd |n| mean|g n|: n 17, the mean's sums 28, 1 / H, its product and the root 2 + 16 + 1, their
    # product and the difference 2, rstd 16 + 1
    bound = 20 * U * rstd * g.abs() + 84 * U * rstd * n.abs() * (g * n).abs().mean(1, keepdim=True)
    if dr is not None:
        dx = dx + dr.double()
    bound = 1.01 * (bound + U * dx.abs())
    zero = torch.zeros((), dtype=torch.float64)
    keep = live[:, None]
    return torch.where(keep, dx, zero), torch.where(keep, d * n, zero), torch.where(keep, bound, zero)
