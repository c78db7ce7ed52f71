"""Logits under sampling rules and the embedding gradient, written out in 64 bits
(numpy, row by row, token by token), and the cases the tests draw."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32, relative


@dataclasses.dataclass
class Case:
    """CPU tensors of one call; `kw` are LogitsRules' arguments."""
    logits: torch.Tensor
    targets: torch.Tensor
    kw: dict
    ld: int

    @property
    def T(self):
        return self.logits.shape[0]

    @property
    def V(self):
        return self.logits.shape[1]


def make_case(T, V, *, dtype=torch.bfloat16, requests=None, history=20, penalties=True, bias=0,
              mask=None, packed=False, ld=None, seed=0) -> Case:
    """Random rows.  packed: rows are prefixes of `requests` sequences, in order;
    otherwise row t has request t.  mask: None, "half", "few" or "mixed"."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.RandomState(seed)
    kw = {}
    if packed:
        R = requests or max(1, T // 7)
        cuts = np.sort(rng.randint(0, T + 1, R - 1)) if R > 1 else np.array([], dtype=int)
        rows_of = np.diff(np.concatenate([[0], cuts, [T]])).astype(int)
        prompts = rng.randint(0, history + 1, R)
        ntok = prompts + rows_of
        kw["row_request"] = torch.tensor(np.repeat(np.arange(R), rows_of), dtype=torch.int32)
        kw["row_length"] = torch.tensor(np.concatenate(
            [prompts[r] + np.arange(rows_of[r]) for r in range(R)]), dtype=torch.int32)
    else:
        R = T
        ntok = rng.randint(0, max(history, 0) + 1, R)
        prompts = np.array([rng.randint(0, n + 1) for n in ntok])
    offs = np.concatenate([[0], np.cumsum(ntok)])
    if history >= 0:
        # few distinct ids, so that tokens repeat
        hot = torch.randint(0, V, (max(1, min(V, history)),), generator=g)
        kw["tokens"] = hot[torch.randint(0, hot.numel(), (int(offs[-1]),), generator=g)]
        kw["token_offsets"] = torch.tensor(offs, dtype=torch.int64)
        kw["prompt_lengths"] = torch.tensor(prompts, dtype=torch.int32)
    if penalties:
        u = lambda lo, hi: torch.rand(R, generator=g) * (hi - lo) + lo  # noqa: E731
        kw.update(temperature=u(0.5, 1.5), repetition=u(0.8, 1.4), frequency=u(-0.3, 0.7),
                  presence=u(-0.3, 0.7))
    if bias:
        kw["bias_ids"] = torch.randint(0, V, (R * bias,), generator=g)
        kw["bias_values"] = torch.randn(R * bias, generator=g) * 3
        kw["bias_offsets"] = torch.arange(R + 1) * bias
    targets = torch.randint(0, V, (T,), generator=g)
    if mask:
        words = (V + 31) // 32
        w = lambda: torch.randint(-(1 << 31), 1 << 31, (T, words), generator=g).to(torch.int32)  # noqa: E731
        m = w()
        if mask == "few":
            m &= w() & w() & w() & w()
        kw["mask"] = m
        if mask == "mixed":
            kw["row_mask"] = torch.tensor([t if t % 3 else -1 for t in range(T)], dtype=torch.int32)
    ld = ld or V
    z = (torch.randn(T, ld, generator=g) * 2)
    z[:, V:] = float("nan")  # columns behind the row must not be read
    return Case(z.to(dtype)[:, :V], targets, kw, ld)


def to_cuda(t: torch.Tensor) -> torch.Tensor:
    return t.to("cuda:0")


def cuda_case(rk, c: Case, shift=0):
    """(logits, targets, rules) on the GPU; `shift`: elements the matrix starts off an
    aligned address."""
    buf = torch.full((c.T * c.ld + 64 + shift,), float("nan"), dtype=c.logits.dtype, device="cuda:0")
    z = buf[shift:].as_strided((c.T, c.V), (c.ld, 1), storage_offset=shift)
    z.copy_(c.logits)
    return z, c.targets.to("cuda:0"), rk.LogitsRules(**{k: v.to("cuda:0") for k, v in c.kw.items()})


def plain_row(c: Case, t: int):
    """(x, dx/dz, a) of row t in float64: the logits under the rules, the slope, and the
    size of what was added up (for error bounds); masked: x = -inf, slope = 0."""
    kw, V = c.kw, c.V
    z = c.logits[t].double().numpy()
    r = int(kw["row_request"][t]) if "row_request" in kw else t
    par = lambda n, d: float(kw[n][r]) if n in kw else d  # noqa: E731
    tau, rep = par("temperature", 1.0), par("repetition", 1.0)
    freq, pres = par("frequency", 0.0), par("presence", 0.0)
    seen, n = np.zeros(V, dtype=bool), np.zeros(V)
    if "tokens" in kw:
        a, b = int(kw["token_offsets"][r]), int(kw["token_offsets"][r + 1])
        toks = kw["tokens"][a:b].numpy()
        L = min(max(int(kw["row_length"][t]), 0), len(toks)) if "row_length" in kw else len(toks)
        prompt = int(kw["prompt_lengths"][r]) if "prompt_lengths" in kw else 0
        for i in range(L):
            v = int(toks[i])
            if 0 <= v < V:
                seen[v] = True
                if i >= prompt:
                    n[v] += 1
    gain = np.where(seen, np.where(z > 0, 1.0 / rep, rep), 1.0)
    bias = np.zeros(V)
    if "bias_ids" in kw:
        for i in range(int(kw["bias_offsets"][r]), int(kw["bias_offsets"][r + 1])):
            v = int(kw["bias_ids"][i])
            if 0 <= v < V:
                bias[v] = float(kw["bias_values"][i])  # the last one counts
    y = z * gain - freq * n - pres * (n > 0) + bias
    with np.errstate(invalid="ignore"):
        size = (np.abs(z * gain) + abs(freq) * n + abs(pres) * (n > 0) + np.abs(bias)) / tau
    x, slope = y / tau, gain / tau
    mrow = -1
    if "mask" in kw:
        mrow = int(kw["row_mask"][t]) if "row_mask" in kw else t
    if mrow >= 0:
        bits = np.unpackbits(kw["mask"][mrow].numpy().view(np.uint8), bitorder="little")[:V]
        x = np.where(bits == 1, x, -np.inf)
        slope = np.where(bits == 1, slope, 0.0)
        size = np.where(bits == 1, size, 0.0)
    return x, slope, size


def plain_lse(x):
    m = x.max()
    if m == -np.inf:
        return -np.inf
    return float(m + np.log(np.exp(x - m).sum()))


# Roundings between z and x: 1/rep, the product with it, freq n + pres, its
# subtraction, the bias, 1/temperature and the product with it -- seven at most,
# each half an fp32 step of at most `size`; 8 covers their products.
def x_bound(size):
    return 8 * U * size


# lse = m / tau + log(sum): the error of every x enters with its weight p (at most
# the largest of them); the exponent's rounding, u |x - m| log2e, enters with weight
# p too, and sum p |x - m| <= ln V < 20 for any distribution over V < 2^28 columns;
# ex2 is good to 2^-22 = 4u; the tree of sums rounds at most 8 + 4 + 5 + 6 + 5 times
# between a term and the total; log and the last operations half a step each.
def lse_bound(size, lse):
    return x_bound(size.max()) + (20 * 1.45 + 4 + 28 + 4) * U + 3 * U * abs(lse)


def logp_bound(size, tgt, logp, lse):
    return lse_bound(size, 0.0) + x_bound(size[tgt]) + 3 * U * abs(logp) + 2 * U


# dlogits = g slope (onehot - p): p carries the error of x, the exponent's rounding
# (u |x - lse| log2e, where p |x - lse| < 1), ex2's 4u and a few products.
def grad_bound(g, slope, size, p):
    return abs(g) * slope * (p * (x_bound(size) + 12 * U) + 1.5 * U + 8 * U * 1.0) + 1e-36


def half_step(dtype, v):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2 * np.abs(v)


def plain_embedding_bwd(dout, ids, V, scale, order=None, active=None):
    """(dE, sum of magnitudes, count per id) in float64, token by token."""
    H = dout.shape[1]
    d = dout.double().numpy()
    dE, mag, count = np.zeros((V, H)), np.zeros((V, H)), np.zeros(V, dtype=int)
    T = len(ids)
    for r in (range(T) if order is None else order):
        if not 0 <= r < T or (active is not None and not active[r]):
            continue
        v = int(ids[r])
        if 0 <= v < V:
            dE[v] += scale * d[r]
            mag[v] += abs(scale) * np.abs(d[r])
            count[v] += 1
    return dE, mag, count
