"""Cases for the operators at the two ends of the vocabulary.

Logits under sampling rules (penalties for repeated tokens, biases, grammar
masks, temperature), per row t with request r and the tokens before it:

    y = z                                  or, for a token seen before,  z / rep (z > 0),  z * rep (z <= 0)
    y = y - freq * n - pres * [n > 0] + bias,   n: how often the request has produced the token (prompt not counted)
    x = y / temperature,                        -inf where the grammar mask has a 0 bit

    apply:  x itself
    logp:   lse = log sum_v exp(x[v]),  logp = x[target] - lse
    bwd:    dz[v] = g * ([v == target] - exp(x[v] - lse)) * dx/dz,  0 where masked

and the embedding:

    embed:      out[t] = scale * E[id_t]   (0 where id_t < 0)
    embed_bwd:  dE[v] (+)= scale * sum over t with id_t = v of dout[t]
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one request decodes one token: the launch and the history count are all there is
        {"name": "apply_1", "op": "apply", "rows": 1, "V": 32000, "dtype": "bf16", "out": "fp32", "packed": False, "history": 512, "mask": False, "bias": 0, "padded": False},
        # a serving step with fp32 logits, histories of up to 4096 tokens, biases and grammar masks
        {"name": "apply_256", "op": "apply", "rows": 256, "V": 152064, "dtype": "fp32", "out": "fp32", "packed": False, "history": 4096, "mask": True, "bias": 16, "padded": False},
        # logprobs of 64 decoded tokens under the rules they were sampled with
        {"name": "logp_64", "op": "logp", "rows": 64, "V": 128256, "dtype": "bf16", "packed": False, "history": 2048, "mask": False, "bias": 0, "padded": False},
        # packed sequences scored at once, each row with its own prefix as its history
        {"name": "logp_2048", "op": "logp", "rows": 2048, "V": 32000, "dtype": "bf16", "packed": True, "history": 256, "mask": False, "bias": 0, "padded": False},
        # the same at full size with a grammar mask on two rows of three
        {"name": "logp_8192", "op": "logp", "rows": 8192, "V": 128256, "dtype": "bf16", "packed": True, "history": 512, "mask": True, "bias": 8, "padded": False},
        # the gradient with an odd vocabulary: rows start at every 2-byte alignment
        {"name": "bwd_300_odd", "op": "bwd", "rows": 300, "V": 50257, "dtype": "bf16", "out": "fp32", "packed": True, "history": 100, "mask": False, "bias": 4, "padded": False},
        # the gradient in bf16 for the products that follow, with masks
        {"name": "bwd_4096", "op": "bwd", "rows": 4096, "V": 128256, "dtype": "bf16", "out": "bf16", "packed": True, "history": 512, "mask": True, "bias": 0, "padded": False},
        # the embedding of a decode step
        {"name": "embed_64", "op": "embed", "rows": 64, "V": 32000, "H": 4096, "dtype": "bf16", "out": "bf16"},
        # and of a training batch
        {"name": "embed_65536", "op": "embed", "rows": 65536, "V": 128256, "H": 4096, "dtype": "bf16", "out": "bf16"},
        # its gradient for a handful of tokens of a small model
        {"name": "embed_bwd_100", "op": "embed_bwd", "rows": 100, "V": 4096, "H": 256, "dtype": "bf16", "accumulate": False},
        # into a fresh gradient, most of whose rows no token names
        {"name": "embed_bwd_8192", "op": "embed_bwd", "rows": 8192, "V": 152064, "H": 3584, "dtype": "bf16", "accumulate": False},
        # added to the gradient that the tied output weight already has
        {"name": "embed_bwd_65536", "op": "embed_bwd", "rows": 65536, "V": 128256, "H": 4096, "dtype": "bf16", "accumulate": True},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["apply", "logp", "bwd", "embed", "embed_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("embed", "embed_bwd"):
        H = rng.choice([_spread(rng, 16, 4096), 8 * _spread(rng, 2, 512), 64 * rng.randint(1, 64)])
        c = {"op": op, "rows": _spread(rng, 1, 32768), "V": _spread(rng, 500, 128256), "H": H, "dtype": dtype}
        if op == "embed":
            c["out"] = rng.choice(["bf16", "fp32"])
        else:
            c["accumulate"] = rng.random() < 0.5
        return c
    V = rng.choice([_spread(rng, 500, 152064), 8 * _spread(rng, 64, 19008)])
    rows = _spread(rng, 1, min(4096, (1 << 28) // V))
    packed = op == "bwd" or (op == "logp" and rng.random() < 0.6)
    history = _spread(rng, 1, 1024) if packed else _spread(rng, 1, min(32768, (1 << 22) // rows))
    c = {"op": op, "rows": rows, "V": V, "dtype": dtype, "packed": packed, "history": history, "mask": rng.random() < 0.5,
         "bias": rng.choice([0, 1, 32]), "padded": rng.random() < 0.4}
    if op != "logp":
        c["out"] = rng.choice(["bf16", "fp32"])
    return c


# ---------------------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------------------

def _zipf_ids(gen, n, V):
    """Ids with P(v) proportional to log((v + 2) / (v + 1)): a few tokens make up much of a text."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.pow(float(V + 1), u) - 1).long().clamp_(0, V - 1)


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _prepare_logits(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    T, V, hist = case["rows"], case["V"], case["history"]
    if case["packed"]:  # sequences of responses, packed; `history` is the longest prompt
        lengths, left = [], T
        while left:
            n = min(left, rng.randint(128, 2048))
            lengths.append(n)
            left -= n
        prompts = [rng.randint(1, hist) for _ in lengths]
    else:  # one row for each request, its history drawn over the logarithm up to `history`
        total = [_spread(rng, 1, hist) for _ in range(T)]
        prompts = [rng.randint(0, n) for n in total]
        lengths = [n - p for n, p in zip(total, prompts)]
    R = len(lengths)
    tokens_of = [p + n for p, n in zip(prompts, lengths)]
    offs = _offsets(tokens_of)
    tokens = _zipf_ids(gen, offs[-1], V)
    if case["packed"]:
        row_request = [r for r, n in enumerate(lengths) for _ in range(n)]
        row_length = [prompts[r] + i for r, n in enumerate(lengths) for i in range(n)]
        where = [offs[r] + prompts[r] + i for r, n in enumerate(lengths) for i in range(n)]
        targets = tokens[torch.tensor(where, device="cuda")]
    else:
        row_request, row_length = list(range(T)), tokens_of
        targets = _zipf_ids(gen, T, V)
    dev = dict(device="cuda")
    uniform = lambda lo, hi: torch.rand(R, generator=gen, **dev) * (hi - lo) + lo  # noqa: E731
    rules = {
        "temperature": uniform(0.6, 1.2), "repetition": uniform(1.0, 1.3), "frequency": uniform(0.0, 0.6), "presence": uniform(0.0, 0.6),
        "tokens": tokens, "token_offsets": torch.tensor(offs, dtype=torch.int64, **dev), "prompt_lengths": torch.tensor(prompts, dtype=torch.int32, **dev),
        "row_request": torch.tensor(row_request, dtype=torch.int32, **dev), "row_length": torch.tensor(row_length, dtype=torch.int32, **dev),
    }
    if case["bias"]:
        ids = torch.stack([torch.randperm(V, generator=gen, **dev)[: case["bias"]] for _ in range(R)])
        values = torch.randn(R, case["bias"], generator=gen, **dev) * 4
        values[:, 0] = -100.0  # a token that is as good as banned
        rules.update(bias_ids=ids.reshape(-1), bias_values=values.reshape(-1), bias_offsets=torch.arange(R + 1, **dev) * case["bias"])
    ld = (V + 7) // 8 * 8 if case["padded"] else V
    z = torch.empty(T, ld, dtype=DTYPES[case["dtype"]], **dev)
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        v = torch.randn(b - a, ld, generator=gen, **dev) * 2
        hot = torch.rand(b - a, generator=gen, **dev) < 0.01
        v[torch.arange(b - a, **dev), torch.randint(0, V, (b - a,), generator=gen, **dev)] += 20.0 * hot
        z[a:b] = v
    z = z[:, :V]
    if case["mask"]:  # of three rows one has no mask, one a mask that allows most tokens or half of them, one a mask that allows few
        words = (V + 31) // 32
        word = lambda: torch.randint(-(1 << 31), 1 << 31, (T, words), generator=gen, dtype=torch.int64, **dev).to(torch.int32)  # noqa: E731
        few, most = word(), word()
        for _ in range(4):
            few &= word()
            most |= word()
        kind = torch.randint(0, 6, (T,), generator=gen, **dev)
        mask = torch.where((kind < 2)[:, None], few, torch.where((kind < 3)[:, None], word(), most))
        rows = torch.arange(T, **dev)
        mask[rows, targets >> 5] |= torch.bitwise_left_shift(torch.ones_like(targets), targets & 31).to(torch.int32)
        rules.update(mask=mask, row_mask=torch.where(kind < 4, rows, -1).to(torch.int32))
    st = {"logits": z, "targets": targets, "rules": rules, "pairs": sum(row_length), "bias_rows": T * case["bias"]}
    if case["op"] == "bwd":
        st["grad"] = torch.randn(T, generator=gen, **dev)
        st["lse"] = _plain_lse(_plain_rules(st)[0])
    return st


def prepare(case, seed):
    if case["op"] in ("apply", "logp", "bwd"):
        return dict(_prepare_logits(case, seed), case=dict(case))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, V, H = case["rows"], case["V"], case["H"]
    ids = _zipf_ids(gen, T, V)
    ids[torch.rand(T, generator=gen, device="cuda") < 0.03] = -1  # padding
    st = {"case": dict(case), "ids": ids, "scale": float(H) ** 0.5}
    if case["op"] == "embed":
        st["table"] = (torch.randn(V, H, generator=gen, device="cuda") * 0.02).to(DTYPES[case["dtype"]])
    else:
        st["grad"] = torch.randn(T, H, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        if case["accumulate"]:
            st["dE"] = torch.randn(V, H, generator=gen, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------------------

def _ragged(begin, length, total):
    """(row, begin[row] + 0 .. length[row] - 1) of every row, one after the other."""
    rows = torch.repeat_interleave(torch.arange(length.shape[0], device="cuda"), length, output_size=total)
    first = torch.cumsum(length, 0) - length
    return rows, torch.arange(total, device="cuda") - first[rows], begin


def _plain_rules(st):
    """x [T, V] in fp32, and dx/dz."""
    z, p = st["logits"].float(), st["rules"]
    T, V = z.shape
    r = p["row_request"].long()
    per_row = lambda name: p[name][r][:, None]  # noqa: E731
    length = p["row_length"].long()
    rows, at, _ = _ragged(None, length, st["pairs"])
    flat = rows * V + p["tokens"][p["token_offsets"][r][rows] + at]
    produced = (at >= p["prompt_lengths"].long()[r][rows]).to(torch.int32)
    seen = torch.zeros(T * V, dtype=torch.int32, device="cuda").scatter_add_(0, flat, torch.ones_like(produced)).view(T, V) > 0
    n = torch.zeros(T * V, dtype=torch.int32, device="cuda").scatter_add_(0, flat, produced).view(T, V).float()
    rep = per_row("repetition")
    slope = torch.where(seen, torch.where(z > 0, 1.0 / rep, rep), 1.0)
    y = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    y = y - per_row("frequency") * n - per_row("presence") * (n > 0)
    if "bias_ids" in p:
        count = (p["bias_offsets"][1:] - p["bias_offsets"][:-1])[r]
        rows, at, _ = _ragged(None, count, st["bias_rows"])
        at = p["bias_offsets"][r][rows] + at
        y = y.contiguous().view(-1).index_add(0, rows * V + p["bias_ids"][at], p["bias_values"][at]).view(T, V)
    x = y / per_row("temperature")
    slope = slope / per_row("temperature")
    if "mask" in p:
        m = p["row_mask"].long()
        bits = p["mask"][m.clamp(min=0)]
        bits = (bits[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = (bits.view(T, -1)[:, :V] == 1) | (m < 0)[:, None]
        x = torch.where(allowed, x, -math.inf)
        slope = torch.where(allowed, slope, 0.0)
    return x, slope


def _plain_lse(x):
    m = x.amax(1)
    return m + torch.log(torch.exp(x - m[:, None]).sum(1))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "apply":
        return _plain_rules(st)[0].to(DTYPES[case["out"]])
    if op == "logp":
        x, _ = _plain_rules(st)
        lse = _plain_lse(x)
        return x.gather(1, st["targets"][:, None])[:, 0] - lse, lse
    if op == "bwd":
        x, slope = _plain_rules(st)
        at = torch.arange(x.shape[1], device="cuda")[None, :] == st["targets"][:, None]
        return (st["grad"][:, None] * (at.float() - torch.exp(x - st["lse"][:, None])) * slope).to(DTYPES[case["out"]])
    ids = st["ids"]
    live = (ids >= 0)[:, None]
    if op == "embed":
        return torch.where(live, st["table"][ids.clamp(min=0)].float() * st["scale"], 0.0).to(DTYPES[case["out"]])
    rows = torch.where(live, st["grad"].float() * st["scale"], 0.0)
    dE = st["dE"] if case["accumulate"] else torch.zeros(case["V"], case["H"], device="cuda")
    return dE.index_add_(0, ids.clamp(min=0), rows)


# ---------------------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------------------

def _run_own(st):
    import invariant_rl_logprob_gb300 as rk
    case = st["case"]
    op = case["op"]
    if op == "embed":
        return rk.embedding(st["ids"], st["table"], scale=st["scale"], out_dtype=DTYPES[case["out"]])
    if op == "embed_bwd":
        if case["accumulate"]:
            return rk.embedding_bwd(st["grad"], st["ids"], case["V"], scale=st["scale"], dE=st["dE"], accumulate=True)
        return rk.embedding_bwd(st["grad"], st["ids"], case["V"], scale=st["scale"])
    rules = rk.LogitsRules(**st["rules"])
    if op == "apply":
        return rk.logits_rules_apply(st["logits"], rules, out_dtype=DTYPES[case["out"]])
    if op == "logp":
        return rk.logp_from_logits_rules(st["logits"], st["targets"], rules)
    return rk.logp_from_logits_rules_bwd(st["logits"], st["targets"], rules, st["lse"], st["grad"], out_dtype=DTYPES[case["out"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------------------------------------------
# what each has to read, write and compute
# ---------------------------------------------------------------------------------------------------------------------------------

def _distinct(T, V):
    """How many different ids T draws of _zipf_ids give on average."""
    v = torch.arange(V, dtype=torch.float64)
    p = torch.log1p(1.0 / (v + 1.0)) / math.log(V + 1.0)
    return float((-torch.expm1(0.97 * T * torch.log1p(-p))).sum())


def work(case):
    size = {"bf16": 2, "fp32": 4}
    T, V, op = case["rows"], case["V"], case["op"]
    if op == "embed":
        u, H = _distinct(T, V), case["H"]
        return {"bytes": u * H * size[case["dtype"]] + T * H * size[case["out"]] + 8 * T, "flops": T * H}
    if op == "embed_bwd":
        u, H = _distinct(T, V), case["H"]
        return {"bytes": T * H * size[case["dtype"]] + 8 * T + (2 * u if case["accumulate"] else V) * H * 4, "flops": T * H}
    words = (V + 31) // 32
    b = T * V * size[case["dtype"]] + (T * words * 4 * 2 // 3 if case["mask"] else 0)
    # each request's tokens once: the packed rows of a sequence share theirs
    b += 8 * (T + T * case["history"] // 1088 // 2 if case["packed"] else T * case["history"] // max(1, round(math.log(case["history"] + 1))))
    if op == "apply":
        return {"bytes": b + T * V * size[case["out"]], "flops": 2 * T * V}
    if op == "logp":
        return {"bytes": b + 16 * T, "flops": 5 * T * V}
    return {"bytes": b + T * V * size[case["out"]] + 16 * T, "flops": 6 * T * V}


# ---------------------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------------------

def _exact_row(st, t, V):
    """(x, dx/dz) of row t in float64, token by token from the request's list."""
    p = st["host"]
    r = p["row_request"][t]
    b = p["token_offsets"][r]
    prompt, length = p["prompt_lengths"][r], p["row_length"][t]
    z = st["logits"][t].double()
    tau, rep = st["rules"]["temperature"][r].double(), st["rules"]["repetition"][r].double()
    history = st["rules"]["tokens"][b: b + length]
    times = torch.bincount(history[prompt:], minlength=V).double()
    gain = torch.ones_like(z)
    uniq = torch.unique(history)
    gain[uniq] = torch.where(z[uniq] > 0, rep.reciprocal(), rep)
    x = z * gain - st["rules"]["frequency"][r].double() * times - st["rules"]["presence"][r].double() * times.sign()
    if "bias_ids" in st["rules"]:
        c, d = p["bias_offsets"][r], p["bias_offsets"][r + 1]
        x[st["rules"]["bias_ids"][c:d]] += st["rules"]["bias_values"][c:d].double()
    x /= tau
    gain /= tau
    if "mask" in st["rules"] and p["row_mask"][t] >= 0:
        v = torch.arange(V, device="cuda")
        word = st["rules"]["mask"][p["row_mask"][t]].long() & 0xFFFFFFFF
        banned = (torch.bitwise_right_shift(word[v // 32], v % 32) % 2) == 0
        x[banned] = -math.inf
        gain[banned] = 0.0
    return x, gain


def exact(case, seed):
    st = prepare(case, seed)
    op, T, V = case["op"], case["rows"], case["V"]
    if op == "embed":
        out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        live = torch.nonzero(st["ids"] >= 0)[:, 0]
        out[live] = st["table"].double()[st["ids"][live]] * st["scale"]
        return out
    if op == "embed_bwd":
        live = torch.nonzero(st["ids"] >= 0)[:, 0]
        order = live[torch.argsort(st["ids"][live], stable=True)]
        names, counts = torch.unique_consecutive(st["ids"][order], return_counts=True)
        ends = torch.cumsum(counts, 0)
        out = torch.zeros(V, case["H"], dtype=torch.float64, device="cuda")
        for a in range(0, case["H"], 512):
            sums = torch.cumsum(st["grad"][order][:, a: a + 512].double(), 0)
            total = sums[ends - 1]
            total[1:] -= sums[ends[:-1] - 1]
            out[names, a: a + 512] = total * st["scale"]
        return out + st["dE"].double() if case["accumulate"] else out
    st["host"] = {k: st["rules"][k].tolist() for k in ("row_request", "token_offsets", "prompt_lengths", "row_length", "bias_offsets", "row_mask") if k in st["rules"]}
    if op == "logp":
        logp, lse = (torch.empty(T, dtype=torch.float64, device="cuda") for _ in range(2))
        for t in range(T):
            x, _ = _exact_row(st, t, V)
            lse[t] = torch.logsumexp(x, 0)
            logp[t] = x[st["targets"][t]] - lse[t]
        return logp, lse
    out = torch.empty(T, V, dtype=torch.float64, device="cuda")
    for t in range(T):
        x, gain = _exact_row(st, t, V)
        if op == "bwd":
            p = torch.softmax(x, 0)
            x = -p
            x[st["targets"][t]] = 1.0 - p[st["targets"][t]]
            x *= st["grad"][t].double() * gain
        out[t] = x
    return out
