"""The preference loss written out in 64 bits, pair by pair, with bounds on what the
fixed-point sums and fp32 may add, and the cases the tests draw."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32, relative


@dataclasses.dataclass
class Case:
    logp: torch.Tensor
    ref: torch.Tensor | None
    targets: torch.Tensor
    cu: torch.Tensor
    chosen: torch.Tensor
    rejected: torch.Tensor
    margin: torch.Tensor | None

    def to(self, device):
        move = lambda t: None if t is None else t.to(device)  # noqa: E731
        return Case(*(move(getattr(self, f.name)) for f in dataclasses.fields(self)))

    def args(self):
        return (self.logp, self.targets, self.cu, self.chosen, self.rejected), {"logp_ref": self.ref, "margin": self.margin}


def make_case(lengths, P, *, ref=True, margin=False, share=0.7, lead=0, trail=0, seed=0) -> Case:
    """Sequences of the given lengths behind `lead` rows and before `trail`, random pairs."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.tensor(lengths, dtype=torch.int64)
    Q, T = len(lengths), int(lengths.sum()) + lead + trail
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)]) + lead
    logp = torch.log(1 - torch.rand(T, generator=g)) * 1.3
    targets = torch.randint(0, 500, (T,), generator=g)
    targets[torch.rand(T, generator=g) > share] = -100
    chosen, rejected = (torch.randint(0, max(Q, 1), (P,), generator=g, dtype=torch.int32) for _ in range(2))
    return Case(logp, logp + 0.2 * torch.randn(T, generator=g) if ref else None, targets, cu.int(), chosen, rejected,
                torch.rand(P, generator=g) if margin else None)


def plain(c: Case, kind="sigmoid", beta=0.125, smoothing=0.0, average=False, scale=1.0):
    """(loss, grad, logratio) in float64 and bounds on each one's error."""
    cu = c.cu.tolist()
    Q, T, P = len(cu) - 1, c.logp.shape[0], c.chosen.shape[0]
    lp = c.logp.double().numpy()
    v = lp if c.ref is None else lp - c.ref.double().numpy()
    live = c.targets.numpy() >= 0
    s, n, ds = [0.0] * Q, [1] * Q, [0.0] * Q
    for q in range(Q):
        part = v[cu[q]:cu[q + 1]][live[cu[q]:cu[q + 1]]]
        n[q] = max(1, len(part)) if average else 1
        total = math.fsum(part)
        s[q] = total / n[q]
        # two roundings to 2^-42 a token and one of the quotient; 64 bits where fixed point ends
        ds[q] = (len(part) * 2.0 ** -42) / n[q] + 2.0 ** -43 + 4 * 2.0 ** -53 * abs(s[q])
    loss, dloss = np.zeros(P), np.zeros(P)
    coef, dcoef, terms = [0.0] * Q, [0.0] * Q, [0] * Q
    for p in range(P):
        i, j = int(c.chosen[p]), int(c.rejected[p])
        if i < 0 or j < 0:
            continue
        d = s[i] - s[j] - (0.0 if c.margin is None else float(c.margin[p]))
        # ... and of the margin and 1 / (2 beta)
        dd = ds[i] + ds[j] + 2.0 ** -42 + 4 * 2.0 ** -53 * (abs(s[i]) + abs(s[j]) + abs(d))
        x = beta * d
        if kind == "sigmoid":
            soft = lambda t: max(t, 0.0) + math.log1p(math.exp(-abs(t)))  # noqa: E731
            sig = lambda t: 1 / (1 + math.exp(-t)) if t > 0 else math.exp(t) / (1 + math.exp(t))  # noqa: E731
            f = (1 - smoothing) * soft(-x) + smoothing * soft(x)
            up, down = smoothing * sig(x), (1 - smoothing) * sig(-x)
            slope, size, curve = beta * (up - down), beta * (up + down), beta * beta / 4
        elif kind == "hinge":
            f, slope, curve = max(0.0, 1 - x), -beta if x < 1 else 0.0, 0.0
            size = abs(slope)
            assert abs(1 - x) > 1e-6  # on the border either side would do
        else:
            f, slope, curve = (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta), 2.0
            size = abs(slope)
        # the exponential 4 half steps, its compensation 3, log1p or the quotient 4, products and
        # sums 4, scale 1
        df = 16 * U * f + size * dd + curve * dd * dd
        if kind == "hinge":
            df += 4 * U  # 1 - x, from numbers of order one
        dslope = 16 * U * size + curve * dd
        loss[p], dloss[p] = scale * f, abs(scale) * df
        for q, sign in ((i, 1), (j, -1)):
            coef[q] += sign * scale * slope
            dcoef[q] += abs(scale) * (dslope + U * size)
            terms[q] += 1
    grad, dgrad = np.zeros(T), np.zeros(T)
    size_of = _sizes(c, s, kind, beta, smoothing, scale)
    for q in range(Q):
        here = slice(cu[q], cu[q + 1])
        grad[here] = np.where(live[here], coef[q] / n[q], 0)
        dgrad[here] = np.where(live[here], (dcoef[q] + terms[q] * U * size_of[q]) / n[q] + 2 * U * abs(coef[q]) / n[q], 0)
    s, ds = np.array(s), np.array(ds)
    tiny = 2.0 ** -126  # numbers below the normal ones of fp32
    return (loss, grad, s), (1.01 * dloss + tiny, 1.01 * dgrad + tiny, ds + 1.01 * U * np.abs(s) + tiny)


def _sizes(c, s, kind, beta, smoothing, scale):
    """Sum of the magnitudes of each sequence's slopes, an upper bound."""
    out = [0.0] * len(s)
    for p in range(c.chosen.shape[0]):
        i, j = int(c.chosen[p]), int(c.rejected[p])
        if i < 0 or j < 0:
            continue
        d = s[i] - s[j] - (0.0 if c.margin is None else float(c.margin[p]))
        top = beta if kind != "ipo" else 2 * abs(d - 0.5 / beta)
        out[i] += abs(scale) * top
        out[j] += abs(scale) * top
    return out
