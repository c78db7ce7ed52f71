"""Cases for the operators that close a training step around the logprob.

The root-mean-square norm in front of the head, with the residual's addition and an
output in 8 bits; over a row of H columns:

    r = x  or  round(x + residual), rounded to residual's type: what the layers after it read
    y = r / sqrt(mean(r^2) + eps) * weight                        0 in inactive rows
    in e4m3:  s = max |y| / 448 of a row, or of each 128 columns of it,  q = round(y / s)   (s = q = 0 where y = 0)

and its gradient, dweight summed over the active rows:

    n = r / sqrt(mean(r^2) + eps),  g = dout * weight
    dx = (g - n * mean(g * n)) / sqrt(mean(r^2) + eps) + dr        0 in inactive rows
    dweight = sum_t dout * n

The preference loss on selected logprobs; sequence q, pair p:

    s_q = sum over its active tokens of (logp - logp_ref)          divided by their number with `average`
    d = s_chosen - s_rejected - margin
    sigmoid:  loss = (1 - e) * log(1 + exp(-beta d)) + e * log(1 + exp(beta d))       e: label smoothing
    hinge:    loss = max(0, 1 - beta d)
    ipo:      loss = (d - 1 / (2 beta))^2
    all three times scale;  grad_logp[t] = d (sum of the losses) / d logp[t]

The AdamW step, over many tensors at once:

    g = grad * grad_scale
    m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
    w = w - lr * weight_decay * w - lr * (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
    w: the parameter, or its fp32 master, of which the parameter is the rounded copy
    in 8 bits m is held as e4m3 * scale and v as (e4m3 * scale)^2, a scale for 256 elements: max |.| / 448
    of the new values (a positive v never becomes 0: its code is 2^-9 at least)
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
BETA1, BETA2, ADAM_EPS, LR, STEP = 0.9, 0.95, 1e-8, 3e-4, 100
BLOCK = 256  # elements that share a scale of an 8-bit state


def listed():
    return [
        # one token in front of the head of a decode step: latency alone
        {"name": "norm_1", "op": "norm", "rows": 1, "H": 4096, "x": "bf16", "residual": "bf16", "out": "bf16", "group": 0, "padding": 0.0, "ld": 0},
        # 64 tokens of a decode step, in 8 bits with a scale for each token
        {"name": "norm_64_e4m3", "op": "norm", "rows": 64, "H": 3584, "x": "bf16", "residual": "bf16", "out": "e4m3", "group": 0, "padding": 0.0, "ld": 0},
        # an odd width in fp32: rows at every 4-byte alignment, padding in between
        {"name": "norm_5000_odd", "op": "norm", "rows": 5000, "H": 2047, "x": "fp32", "residual": "", "out": "fp32", "group": 0, "padding": 0.2, "ld": 0},
        # a training batch: the residual stream goes on, the norm leaves in 8 bits with a scale for each 128 columns
        {"name": "norm_65536", "op": "norm", "rows": 65536, "H": 4096, "x": "bf16", "residual": "bf16", "out": "e4m3", "group": 128, "padding": 0.0, "ld": 0},
        # the gradient of a few packed rows, dout in fp32 as the head's backward leaves it
        {"name": "norm_bwd_300", "op": "norm_bwd", "rows": 300, "H": 3584, "r": "bf16", "dout": "fp32", "dr": "", "dx": "fp32", "padding": 0.3, "ld": 0},
        # and of a training batch, with the gradient of the residual stream that it joins
        {"name": "norm_bwd_65536", "op": "norm_bwd", "rows": 65536, "H": 4096, "r": "bf16", "dout": "bf16", "dr": "bf16", "dx": "bf16", "padding": 0.0, "ld": 0},
        # four pairs of answers, their prompts masked
        {"name": "preference_4", "op": "preference", "prompts": 4, "answers": 2, "length": 1024, "kind": "sigmoid", "reference": True, "average": False, "smoothing": 0.0},
        # eight answers to each of 64 prompts, every pair of them compared, without a reference and by mean logprobs
        {"name": "preference_64x8", "op": "preference", "prompts": 64, "answers": 8, "length": 2048, "kind": "sigmoid", "reference": False, "average": True, "smoothing": 0.1},
        # a small model of many small tensors, all in fp32
        {"name": "adamw_small", "op": "adamw", "tensors": 36, "elements": 2400000, "spread": True, "param": "fp32", "grad": "fp32", "bits": 32, "align": 16},
        # the head's weight with its fp32 master, 32-bit states and the fp32 gradient of the head's backward
        {"name": "adamw_head", "op": "adamw", "tensors": 1, "elements": 128256 * 4096, "spread": False, "param": "bf16", "grad": "fp32", "bits": 32, "align": 16},
        # many tensors of odd sizes with 8-bit states
        {"name": "adamw8_ragged", "op": "adamw", "tensors": 200, "elements": 30000001, "spread": True, "param": "bf16", "grad": "bf16", "bits": 8, "align": 16},
        # the largest head with 8-bit states
        {"name": "adamw8_head", "op": "adamw", "tensors": 1, "elements": 152064 * 3584, "spread": False, "param": "bf16", "grad": "bf16", "bits": 8, "align": 16},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "preference", "adamw", "adamw"])
    some = lambda *v: rng.choice(v)  # noqa: E731
    if op in ("norm", "norm_bwd"):
        H = some(_spread(rng, 1, 16384), 8 * _spread(rng, 2, 2048), 128 * rng.randint(1, 64))
        rows = _spread(rng, 1, min(65536, (1 << 27) // H))
        c = {"op": op, "rows": rows, "H": H, "padding": some(0.0, 0.0, 0.25), "ld": some(0, 0, 8, 3)}
        if op == "norm":
            c.update(x=some("bf16", "bf16", "fp32"), residual=some("", "bf16", "fp32"), out=some("bf16", "fp32", "e4m3"), group=some(0, 128))
        else:
            c.update(r=some("bf16", "bf16", "fp32"), dout=some("bf16", "fp32"), dr=some("", "bf16", "fp32"), dx=some("bf16", "fp32"))
        return c
    if op == "preference":
        answers = some(2, 2, 4, 8)
        length = _spread(rng, 1, 2048)
        prompts = _spread(rng, 1, min(512, max(1, (1 << 19) // (answers * length))))
        return {"op": op, "prompts": prompts, "answers": answers, "length": length, "kind": some("sigmoid", "sigmoid", "hinge", "ipo"),
                "reference": rng.random() < 0.7, "average": rng.random() < 0.3, "smoothing": some(0.0, 0.1)}
    tensors = _spread(rng, 1, 300)
    return {"op": op, "tensors": tensors, "elements": _spread(rng, tensors, 1 << 27), "spread": rng.random() < 0.7, "param": some("bf16", "bf16", "fp32"),
            "grad": some("bf16", "fp32"), "bits": some(8, 32), "align": some(16, 16, 1)}


# ---------------------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------------------

def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _matrix(gen, T, H, dtype, ld, scale=1.0):
    """Normal values, [T, H] with `ld` unused columns behind each row."""
    a = torch.empty(T, H + ld, dtype=DTYPES[dtype], device="cuda")
    for i in range(0, T, 8192):
        a[i: i + 8192] = torch.randn(min(T - i, 8192), H + ld, generator=gen, device="cuda") * scale
    return a[:, :H]


def _targets(gen, T, padding):
    """Tokens, -100 where a row is padding; None where none is."""
    if not padding:
        return None
    tg = torch.randint(0, 32000, (T,), generator=gen, device="cuda")
    tg[torch.rand(T, generator=gen, device="cuda") < padding] = -100
    return tg


def _prepare_norm(case, seed):
    gen = _generator(seed)
    T, H, ld = case["rows"], case["H"], case["ld"]
    st = {"targets": _targets(gen, T, case["padding"]), "weight": (1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()}
    # a few columns are far larger than the others, as in a deep model's residual stream
    big = torch.where(torch.rand(H, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    if case["op"] == "norm":
        st["x"] = _matrix(gen, T, H, case["x"], ld)
        if case["residual"]:
            st["residual"] = _matrix(gen, T, H, case["residual"], ld, 3.0).mul_(big)
        else:
            st["x"].mul_(big)
        main = st["x"]
    else:
        st["r"] = main = _matrix(gen, T, H, case["r"], ld, 3.0).mul_(big)
        st["dout"] = _matrix(gen, T, H, case["dout"], ld, 1e-3)
        if case["dr"]:
            st["dr"] = _matrix(gen, T, H, case["dr"], ld, 1e-3)
    if st["targets"] is not None:
        main[st["targets"] < 0] = math.nan  # whatever padding holds
    return st


def _prepare_preference(case, seed):
    gen = _generator(seed)
    answers = case["answers"]
    rng = random.Random(case["prompts"] * 4096 + case["length"])  # the lengths are the case's, the values the seed's
    lengths, prompt, chosen, rejected = [], [], [], []
    for i in range(case["prompts"]):
        first = _spread(rng, 1, max(1, case["length"] // 2))  # the prompt, in front of each of its answers
        for _ in range(answers):
            n = rng.randint(max(1, case["length"] // 8), case["length"])
            lengths.append(n)
            prompt.append(min(first, n))
        order = rng.sample(range(answers), answers)
        for a in range(answers):
            for b in range(a + 1, answers):
                chosen.append(i * answers + order[a])
                rejected.append(i * answers + order[b])
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    T = cu[-1]
    dev = dict(device="cuda")
    cu_t = torch.tensor(cu, dtype=torch.int32, **dev)
    which = torch.repeat_interleave(torch.arange(len(lengths), **dev), torch.tensor(lengths, **dev), output_size=T)
    at = torch.arange(T, **dev) - cu_t[which]
    targets = torch.randint(0, 32000, (T,), generator=gen, **dev)
    targets[at < torch.tensor(prompt, **dev)[which]] = -100
    logp = torch.log(1.0 - torch.rand(T, generator=gen, **dev)) * 1.2
    st = {"logp": logp, "targets": targets, "cu": cu_t, "T": T, "chosen": torch.tensor(chosen, dtype=torch.int32, **dev),
          "rejected": torch.tensor(rejected, dtype=torch.int32, **dev), "ref": None, "margin": None, "beta": 2.0 if case["average"] else 0.1,
          "smoothing": case["smoothing"] if case["kind"] == "sigmoid" else 0.0, "scale": 1.0 / len(chosen)}
    if case["reference"]:
        st["ref"] = logp + torch.randn(T, generator=gen, **dev) * 0.1
    else:
        st["margin"] = torch.rand(len(chosen), generator=gen, **dev)
    return st


def _sizes(case):
    """The number of elements of each tensor."""
    n, total = case["tensors"], case["elements"]
    if not case["spread"] or n == 1:
        return [total // n + (i < total % n) for i in range(n)]
    rng = random.Random(total)
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(n)]
    at = [0]
    for s in share:
        at.append(at[-1] + s)
    cut = [int((total - n) * a / at[-1]) for a in at]
    cut[-1] = total - n
    return [cut[i + 1] - cut[i] + 1 for i in range(n)]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _encode(values, floor):
    """(e4m3 codes, a scale for each BLOCK elements); `floor`: positive values keep a positive code."""
    n = values.numel()
    padded = torch.nn.functional.pad(values, (0, _blocks(n) * BLOCK - n)).view(-1, BLOCK)
    scale = padded.abs().amax(1) / 448.0
    q = torch.where(scale[:, None] > 0, padded / scale[:, None], 0.0)
    if floor:
        q = torch.where(padded > 0, q.clamp(min=2.0 ** -9), q)
    return q.clamp_(-448.0, 448.0).view(-1)[:n].to(torch.float8_e4m3fn), scale


def _decode(codes, scale):
    n = codes.numel()
    return codes.float() * torch.repeat_interleave(scale, BLOCK)[:n]


def _flat(sizes, align, dtype):
    """One buffer for all tensors, and each tensor's view of it."""
    at, views = 0, []
    for n in sizes:
        views.append((at, n))
        at += -(-n // align) * align
    buffer = torch.zeros(at, dtype=dtype, device="cuda")
    return buffer, [buffer[a: a + n] for a, n in views]


def _prepare_adamw(case, seed):
    gen = _generator(seed)
    sizes, align = _sizes(case), case["align"]
    normal = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    eight = case["bits"] == 8
    state = torch.float8_e4m3fn if eight else torch.float32
    types = {"param": (sizes, DTYPES[case["param"]]), "grad": (sizes, DTYPES[case["grad"]]), "m": (sizes, state), "v": (sizes, state)}
    if case["param"] == "bf16":
        types["master"] = (sizes, torch.float32)
    if eight:
        types["m_scale"] = types["v_scale"] = ([_blocks(n) for n in sizes], torch.float32)
    st = {"master": None, "m_scale": None, "v_scale": None, "buffers": {}}
    for k, (lengths, dtype) in types.items():
        st["buffers"][k], st[k] = _flat(lengths, align, dtype)
    for i, n in enumerate(sizes):
        w = normal(n).mul_(0.02)
        st["param"][i].copy_(w)
        if st["master"] is not None:
            st["master"][i].copy_(w)
        del w
        # gradients of rows differ in size; a row in four belongs to tokens that the batch has not named
        rows = (n + 1023) // 1024
        size = torch.exp(normal(rows)) * 1e-3 * (torch.rand(rows, generator=gen, device="cuda") < 0.75)
        size = torch.repeat_interleave(size, 1024)[:n]
        st["grad"][i].copy_(normal(n).mul_(size))
        typical = size.add_(1e-5)
        m, v = normal(n).mul_(typical).mul_(0.3), normal(n).mul_(typical).mul_(0.3).square_().add_(typical.square_())
        for k, values in (("m", m), ("v", v.sqrt_() if eight else v)):
            if eight:
                values, scale = _encode(values, k == "v")
                st[k + "_scale"][i].copy_(scale)
            st[k][i].copy_(values)
    # weight decay for the matrices, none for the smallest tensors (norms, biases)
    st["weight_decay"] = [0.1 if n > 8192 else 0.0 for n in sizes]
    st["grad_scale"] = torch.rand(1, generator=gen, device="cuda") * 0.5 + 0.5  # of a clipped gradient norm
    return st


def prepare(case, seed):
    st = {"norm": _prepare_norm, "norm_bwd": _prepare_norm, "preference": _prepare_preference, "adamw": _prepare_adamw}[case["op"]](case, seed)
    st["case"] = dict(case)
    if own and case["op"] == "adamw":
        import invariant_rl_logprob_gb300 as rk
        st["plan"] = rk.AdamW(st["param"], st["grad"], st["m"], st["v"], m_scale=st["m_scale"], v_scale=st["v_scale"], master=st["master"],
                              weight_decay=st["weight_decay"])
    return st


# ---------------------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------------------

def _plain_norm(st):
    case = st["case"]
    r = st["x"].float()
    stream = None
    if case["residual"]:
        stream = (r + st["residual"].float()).to(DTYPES[case["residual"]])
        r = stream.float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * st["weight"].float()
    if st["targets"] is not None:
        live = (st["targets"] >= 0)[:, None]
        y = torch.where(live, y, 0.0)
        if stream is not None:
            stream = torch.where(live, stream, torch.zeros_like(stream))
    if case["out"] != "e4m3":
        out = (y.to(DTYPES[case["out"]]),)
    else:
        T, H = y.shape
        group = case["group"] or H
        n = (H + group - 1) // group
        y = torch.nn.functional.pad(y, (0, n * group - H)).view(T, n, group)
        s = y.abs().amax(2) / 448.0
        q = torch.where(s[:, :, None] > 0, y / s[:, :, None], 0.0).clamp_(-448.0, 448.0)
        out = (q.view(T, n * group)[:, :H].to(torch.float8_e4m3fn), s)
    return out if stream is None else (*out, stream)


def _plain_norm_bwd(st):
    r, dout, w = st["r"].float(), st["dout"].float(), st["weight"].float()
    dr = st["dr"].float() if st["case"]["dr"] else 0.0
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r * rstd
    g = dout * w
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True)) + dr
    dw = dout * n
    if st["targets"] is not None:
        live = (st["targets"] >= 0)[:, None]
        dx, dw = torch.where(live, dx, 0.0), torch.where(live, dw, 0.0)
    return dx.to(DTYPES[st["case"]["dx"]]), dw.sum(0)


def _plain_preference(st):
    cu, T = st["cu"].long(), st["T"]
    Q = cu.shape[0] - 1
    which = torch.repeat_interleave(torch.arange(Q, device="cuda"), cu[1:] - cu[:-1], output_size=T)
    live = st["targets"] >= 0
    ratio = st["logp"].double() if st["ref"] is None else st["logp"].double() - st["ref"].double()
    s = torch.zeros(Q, dtype=torch.float64, device="cuda").index_add_(0, which, torch.where(live, ratio, 0.0))
    share = torch.ones(Q, dtype=torch.float64, device="cuda")
    if st["case"]["average"]:
        count = torch.zeros(Q, dtype=torch.float64, device="cuda").index_add_(0, which, live.double())
        share = 1.0 / count.clamp(min=1.0)
    s = s * share
    chosen, rejected = st["chosen"].long(), st["rejected"].long()
    d = s[chosen] - s[rejected]
    if st["margin"] is not None:
        d = d - st["margin"].double()
    b, e = st["beta"], st["smoothing"]
    if st["case"]["kind"] == "sigmoid":
        up = 1.0 / (1.0 + torch.exp(-b * d))
        tail = torch.log1p(torch.exp(-(b * d).abs()))
        loss = (1.0 - e) * (tail + (-b * d).clamp(min=0.0)) + e * (tail + (b * d).clamp(min=0.0))
        slope = b * (e * up - (1.0 - e) * (1.0 - up))
    elif st["case"]["kind"] == "hinge":
        loss = (1.0 - b * d).clamp(min=0.0)
        slope = torch.where(b * d < 1.0, -b, 0.0).double()
    else:
        loss = (d - 0.5 / b) ** 2
        slope = 2.0 * (d - 0.5 / b)
    slope = slope * st["scale"]
    coef = torch.zeros(Q, dtype=torch.float64, device="cuda").index_add_(0, chosen, slope).index_add_(0, rejected, -slope) * share
    grad = torch.where(live, coef[which], 0.0)
    return (loss * st["scale"]).float(), grad.float(), s.float()


def _plain_adamw(st):
    c1, c2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    for i, p in enumerate(st["param"]):
        g = st["grad"][i].float() * st["grad_scale"]
        if st["m_scale"] is None:
            m, v = st["m"][i], st["v"][i]
        else:
            m, v = _decode(st["m"][i], st["m_scale"][i]), _decode(st["v"][i], st["v_scale"][i]).square_()
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g * g * (1.0 - BETA2)
        w = p if st["master"] is None else st["master"][i]
        new = w - w * (LR * st["weight_decay"][i]) - (m / c1) / (torch.sqrt(v / c2) + ADAM_EPS) * LR
        if st["m_scale"] is None:
            st["m"][i].copy_(m)
            st["v"][i].copy_(v)
        else:
            for key, values, floor in (("m", m, False), ("v", v.sqrt_(), True)):
                codes, scale = _encode(values, floor)
                st[key][i].copy_(codes)
                st[key + "_scale"][i].copy_(scale)
        if st["master"] is not None:
            st["master"][i].copy_(new)
        p.copy_(new)
    return _adamw_outputs(st)


def _adamw_outputs(st):
    return {k: v for k, v in st["buffers"].items() if k != "grad"}


def _run_plain(st):
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "preference": _plain_preference, "adamw": _plain_adamw}[st["case"]["op"]](st)


# ---------------------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------------------

def _run_own(st):
    import invariant_rl_logprob_gb300 as rk
    case = st["case"]
    op = case["op"]
    if op == "norm":
        residual = st.get("residual")
        if case["out"] == "e4m3":
            out, scales, r = rk.rms_norm_e4m3(st["x"], st["weight"], st["targets"], residual=residual, eps=EPS, group=case["group"])
            return (out, scales) if residual is None else (out, scales, r)
        out, r = rk.rms_norm(st["x"], st["weight"], st["targets"], residual=residual, eps=EPS, out_dtype=DTYPES[case["out"]])
        return (out,) if residual is None else (out, r)
    if op == "norm_bwd":
        return rk.rms_norm_bwd(st["dout"], st["r"], st["weight"], st["targets"], grad_residual=st.get("dr"), eps=EPS, out_dtype=DTYPES[case["dx"]])
    if op == "preference":
        got = rk.preference_loss(st["logp"], st["targets"], st["cu"], st["chosen"], st["rejected"], logp_ref=st["ref"], margin=st["margin"],
                                 kind=case["kind"], beta=st["beta"], label_smoothing=st["smoothing"], average=case["average"], scale=st["scale"])
        return got["loss"], got["grad"], got["logratio"]
    rk.adamw_step(st["plan"], lr=LR, step=STEP, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, grad_scale=st["grad_scale"])
    return _adamw_outputs(st)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------------------------------------------
# what each has to read, write and compute
# ---------------------------------------------------------------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp32": 4, "e4m3": 1, "": 0}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, H = case["rows"], case["H"]
        live = T * (1.0 - case["padding"])  # padding is not read
        mask = 8 * T if case["padding"] else 0
        if op == "norm":
            scales = 0 if case["out"] != "e4m3" else 4 * T * ((H + case["group"] - 1) // case["group"] if case["group"] else 1)
            b = live * H * (size[case["x"]] + size[case["residual"]]) + T * H * (size[case["out"]] + size[case["residual"]]) + scales
            return {"bytes": int(b) + mask + 2 * H, "flops": int(5 * live * H)}
        b = live * H * (size[case["r"]] + size[case["dout"]] + size[case["dr"]]) + T * H * size[case["dx"]]
        return {"bytes": int(b) + mask + 6 * H, "flops": int(10 * live * H)}
    if op == "preference":
        Q = case["prompts"] * case["answers"]
        P = Q * (case["answers"] - 1) // 2
        T = int(Q * case["length"] * 9 / 16)
        return {"bytes": T * (16 if case["reference"] else 12) + 8 * Q + 12 * P + (0 if case["reference"] else 4 * P), "flops": 4 * T + 40 * P}
    n = case["elements"]
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK  # both, read and written
    weight = 8 if case["param"] == "fp32" else 10
    return {"bytes": int(n * (size[case["grad"]] + state + weight)), "flops": 16 * n}


# ---------------------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------------------

def _rows_at_once(H):
    return max(1, (1 << 25) // H)


def _exact_norm(st):
    """Codes of 8 bits come unrounded: the values that they stand for."""
    case = st["case"]
    T, H = st["x"].shape
    e4m3 = case["out"] == "e4m3"
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    width = (case["group"] or H) if e4m3 else H
    scales = torch.zeros(T, -(-H // width), dtype=torch.float64, device="cuda")
    stream = torch.zeros(T, H, dtype=DTYPES[case["residual"]], device="cuda") if case["residual"] else None
    live = torch.arange(T, device="cuda") if st["targets"] is None else torch.nonzero(st["targets"] >= 0)[:, 0]
    for a in range(0, live.shape[0], _rows_at_once(H)):
        rows = live[a: a + _rows_at_once(H)]
        z = st["x"][rows].double()
        if stream is not None:
            stream[rows] = (z + st["residual"][rows].double()).to(stream.dtype)
            z = stream[rows].double()
        z /= torch.sqrt(torch.linalg.vecdot(z, z) / H + EPS)[:, None]
        z *= st["weight"].double()
        if e4m3:
            for j in range(scales.shape[1]):
                part = z[:, j * width: (j + 1) * width]
                s = part.abs().max(1).values / 448.0
                scales[rows, j] = s
                part /= torch.where(s > 0, s, 1.0)[:, None]
        out[rows] = z
    got = (out, scales) if e4m3 else (out,)
    return got if stream is None else (*got, stream.double())


def _exact_norm_bwd(st):
    T, H = st["r"].shape
    w = st["weight"].double()
    dx, dw = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    live = torch.arange(T, device="cuda") if st["targets"] is None else torch.nonzero(st["targets"] >= 0)[:, 0]
    for a in range(0, live.shape[0], _rows_at_once(H)):
        rows = live[a: a + _rows_at_once(H)]
        z, up = st["r"][rows].double(), st["dout"][rows].double()
        var = (torch.linalg.vecdot(z, z) / H + EPS)[:, None]
        # d/dz of sum(up * w * z / sqrt(var))
        along = torch.linalg.vecdot(up * w, z)[:, None] / H
        dx[rows] = up * w / var.sqrt() - z * along / (var * var.sqrt())
        if st["case"]["dr"]:
            dx[rows] += st["dr"][rows].double()
        dw += (up * z / var.sqrt()).sum(0)
    return dx, dw


def _exact_preference(st):
    case = st["case"]
    cu = st["cu"].tolist()
    Q, T, b = len(cu) - 1, st["T"], st["beta"]
    terms = st["logp"].double() if st["ref"] is None else st["logp"].double() - st["ref"].double()
    active = st["targets"] >= 0
    sums, counts = [], []
    for q in range(Q):
        part = terms[cu[q]: cu[q + 1]][active[cu[q]: cu[q + 1]]]
        counts.append(max(1, part.shape[0]) if case["average"] else 1)
        sums.append(float(part.sum()) / counts[-1])
    margin = [0.0] * len(st["chosen"]) if st["margin"] is None else st["margin"].tolist()
    coef = [0.0] * Q
    loss = []
    for i, j, gap in zip(st["chosen"].tolist(), st["rejected"].tolist(), margin):
        d = sums[i] - sums[j] - gap
        x = b * d
        if case["kind"] == "sigmoid":
            soft = lambda t: max(t, 0.0) + math.log1p(math.exp(-abs(t)))  # noqa: E731
            half = 0.5 * (1.0 + math.tanh(0.5 * x))
            value = (1 - st["smoothing"]) * soft(-x) + st["smoothing"] * soft(x)
            slope = b * (half - (1 - st["smoothing"]))
        elif case["kind"] == "hinge":
            value, slope = max(0.0, 1.0 - x), -b if x < 1.0 else 0.0
        else:
            value, slope = (d - 0.5 / b) ** 2, 2 * d - 1.0 / b
        loss.append(st["scale"] * value)
        coef[i] += st["scale"] * slope
        coef[j] -= st["scale"] * slope
    grad = torch.zeros(T, dtype=torch.float64, device="cuda")
    for q in range(Q):
        grad[cu[q]: cu[q + 1]][active[cu[q]: cu[q + 1]]] = coef[q] / counts[q]
    as_double = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")  # noqa: E731
    return as_double(loss), grad, as_double(sums)


def _exact_adamw(st):
    """Codes of 8 bits come unrounded, as above."""
    eight = st["m_scale"] is not None
    lengths = [p.numel() for p in st["param"]]
    out, parts = {}, {}
    for k, buffer in _adamw_outputs(st).items():
        scales = k.endswith("_scale")
        out[k], parts[k] = _flat([_blocks(n) if scales else n for n in lengths], st["case"]["align"], torch.float64)
    wide = lambda codes, scale: codes.double() * scale.double()[torch.arange(codes.numel(), device="cuda") // BLOCK]  # noqa: E731
    for i, n in enumerate(lengths):
        g = st["grad"][i].double() * st["grad_scale"].double()
        m = wide(st["m"][i], st["m_scale"][i]) if eight else st["m"][i].double()
        v = wide(st["v"][i], st["v_scale"][i]) ** 2 if eight else st["v"][i].double()
        m += (g - m) * (1 - BETA1)
        v += (g * g - v) * (1 - BETA2)
        del g
        w = (st["param"] if st["master"] is None else st["master"])[i].double()
        w = w * (1 - LR * st["weight_decay"][i]) - LR * m / (1 - BETA1 ** STEP) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + ADAM_EPS)
        parts["param"][i].copy_(w)
        if st["master"] is not None:
            parts["master"][i].copy_(w)
        del w
        for key, values in (("m", m), ("v", v ** 0.5 if eight else v)):
            if eight:
                whole = n // BLOCK * BLOCK
                scale = parts[key + "_scale"][i]
                scale[: n // BLOCK] = values[:whole].view(-1, BLOCK).abs().amax(1)
                if whole < n:
                    scale[-1] = values[whole:].abs().max()
                scale /= 448.0
                code = values / torch.where(scale > 0, scale, 1.0)[torch.arange(n, device="cuda") // BLOCK]
                values = torch.where(values > 0, code.clamp(min=2.0 ** -9), code) if key == "v" else code
            parts[key][i].copy_(values)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "preference": _exact_preference, "adamw": _exact_adamw}[case["op"]](st)
