"""A whole step of the operators around the logprob: embedding, norm, logprob, preference loss,
all their gradients and the optimizer, each against its 64-bit form on what the one before it
left, end to end against autograd in 64 bits, and captured in a graph."""
import pytest
import torch

import adamw_plain as ap
import norm_plain as npl
import preference_plain as pp
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, H = 700, 128
LENGTHS = [40, 33, 64, 5, 21, 90]
HYPER = dict(lr=1e-3, step=1, beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


class Model:
    def __init__(self, rk, bits):
        g = torch.Generator().manual_seed(0)
        E, W = (torch.randn(V, H, generator=g) * s for s in (1.0, 0.05))
        self.w = {"E": E.bfloat16().to(DEV), "W": W.bfloat16().to(DEV),
                  "norm": (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().to(DEV)}
        self.grads = {k: torch.zeros(v.shape, device=DEV) for k, v in self.w.items()}
        self.opt = rk.AdamW(list(self.w.values()), list(self.grads.values()), bits=bits, master=True,
                            weight_decay=[0.0, 0.1, 0.0])
        T = sum(LENGTHS)
        self.ids = torch.randint(0, V, (T,), generator=g).to(DEV)
        self.residual = torch.randn(T, H, generator=g).to(DEV)
        c = pp.make_case(LENGTHS, 3, seed=1)
        self.targets = torch.randint(0, V, (T,), generator=g)
        self.targets[c.targets < 0] = -100
        self.targets = self.targets.to(DEV)
        self.cu = c.cu.to(DEV)
        self.chosen = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
        self.rejected = torch.tensor([1, 3, 2], dtype=torch.int32, device=DEV)
        self.ref = -6 + 0.3 * torch.randn(T, generator=g).to(DEV)

    def gradients(self, rk):
        """Everything between the weights and their gradients."""
        w, s = self.w, {}
        s["x"] = rk.embedding(self.ids, w["E"], self.cu, scale=2.0, out_dtype=torch.float32)
        s["h"], s["r"] = rk.rms_norm(s["x"], w["norm"], None, self.cu, residual=self.residual, out_dtype=torch.bfloat16)
        s["logp"], s["lse"], saved = rk.linear_logp_fwd_saved(s["h"], w["W"], self.targets, self.cu)
        s["loss"] = rk.preference_loss(s["logp"], self.targets, self.cu, self.chosen, self.rejected,
                                       logp_ref=self.ref, scale=1 / 3)
        s["dh"], _ = rk.linear_logp_bwd_full_saved(s["h"], w["W"], self.targets, s["lse"], s["loss"]["grad"], saved,
                                                   self.cu, dW=self.grads["W"])
        s["dx"], _ = rk.rms_norm_bwd(s["dh"], s["r"], w["norm"], None, self.cu, out_dtype=torch.float32,
                                     dweight=self.grads["norm"])
        rk.embedding_bwd(s["dx"], self.ids, V, self.cu, scale=2.0, dE=self.grads["E"])
        return s


def test_each_operator_on_what_the_one_before_left(rk):
    m = Model(rk, 32)
    s = {k: (v.cpu() if isinstance(v, torch.Tensor) else {n: t.cpu() for n, t in v.items()}) for k, v in m.gradients(rk).items()}
    live = torch.ones(len(m.ids), dtype=torch.bool)
    x = m.w["E"].cpu().double()[m.ids.cpu()] * 2
    assert torch.equal(s["x"].double(), x)
    r = npl.stream(s["x"], m.residual.cpu())
    assert same_bits(s["r"], r)
    y = npl.forward(r, m.w["norm"].cpu(), live)
    assert bool(((s["h"].double() - y).abs() <= y.abs() * (npl.FORWARD + 2.0 ** -8 * 1.01)).all())
    c = pp.Case(s["logp"], m.ref.cpu(), m.targets.cpu(), m.cu.cpu(), m.chosen.cpu(), m.rejected.cpu(), None)
    want, bound = pp.plain(c, beta=float(torch.tensor(0.1)), scale=float(torch.tensor(1 / 3)))
    for k, a, b in zip(("loss", "grad", "logratio"), want, bound):
        assert bool(((s["loss"][k].double() - torch.tensor(a)).abs() <= torch.tensor(b)).all()), k
    dx, terms, bound = npl.backward(s["dh"], r, m.w["norm"].cpu(), None, live)
    assert bool(((s["dx"].double() - dx).abs() <= bound).all())
    dn = m.grads["norm"].cpu().double()
    assert bool(((dn - terms.sum(0)).abs() <= 400 * npl.U * terms.abs().sum(0)).all())
    dE, mag = torch.zeros(V, H, dtype=torch.float64), torch.zeros(V, H, dtype=torch.float64)
    dE.index_add_(0, m.ids.cpu(), 2 * s["dx"].double())
    mag.index_add_(0, m.ids.cpu(), 2 * s["dx"].double().abs())
    assert bool(((m.grads["E"].cpu().double() - dE).abs() <= 40 * npl.U * mag).all())
    masters = [t.clone().cpu().double() for t in m.opt.master]
    rk.adamw_step(m.opt, **HYPER)
    for w0, g, after, p, decay in zip(masters, m.opt.grads, m.opt.master, m.opt.params, (0.0, 0.1, 0.0)):
        zero = torch.zeros_like(w0)
        (w1, _, _), (dw, _, _) = ap.step(w0, g.cpu(), zero, zero, decay=decay, **HYPER)
        assert bool(((after.cpu().double() - w1).abs() <= dw).all()) and same_bits(p, after.bfloat16())
    assert rk.get_device_error() == 0


def test_end_to_end_against_autograd(rk):
    m = Model(rk, 32)
    s = m.gradients(rk)
    E, W, n = (m.w[k].cpu().double().requires_grad_() for k in ("E", "W", "norm"))
    r = 2 * E[m.ids.cpu()] + m.residual.cpu().double()
    y = r * (r.square().mean(1, keepdim=True) + 1e-6).rsqrt() * n
    h = y + (s["h"].cpu().double() - y).detach()  # what the head has seen
    logp = (h @ W.T).log_softmax(1).gather(1, m.targets.cpu().clamp(min=0)[:, None])[:, 0]
    live = m.targets.cpu() >= 0
    ratio = torch.where(live, logp - m.ref.cpu().double(), 0.0)
    cu = m.cu.tolist()
    sums = torch.stack([ratio[a:b].sum() for a, b in zip(cu, cu[1:])])
    d = sums[m.chosen.cpu().long()] - sums[m.rejected.cpu().long()]
    loss = torch.nn.functional.softplus(-0.1 * d).sum() / 3
    h.retain_grad()
    loss.backward()
    assert abs(float(s["loss"]["loss"].double().sum()) - float(loss.detach())) <= 1e-3 * (1 + float(loss.detach()))
    # the head's gradients are good to 1e-3 + 1e-3 of the largest; the norm's Jacobian has a norm of
    # at most 2 rstd max|weight|, and an id takes the rows that have it, with the scale of 2
    slack = lambda g: 1e-3 + 1e-3 * float(g.abs().max())  # noqa: E731
    dh_off = slack(h.grad)
    assert float((s["dh"].cpu().double() - h.grad).abs().max()) <= dh_off
    assert float((m.grads["W"].cpu().double() - W.grad).abs().max()) <= slack(W.grad)
    rstd = float((r.detach().square().mean(1) + 1e-6).rsqrt().max())
    times = torch.bincount(m.ids.cpu(), minlength=V).max()
    off = dh_off * 2 * rstd * float(n.detach().abs().max()) * H ** 0.5 * 2 * int(times)
    got = m.grads["E"].cpu().double()
    assert float((got - E.grad).abs().max()) <= off
    # and they point the same way, by far
    for a, b in ((got, E.grad), (m.grads["W"].cpu().double(), W.grad), (m.grads["norm"].cpu().double(), n.grad)):
        cos = float((a * b).sum() / (a.norm() * b.norm()))
        # bf16 probabilities are within 2^-8: a relative difference of that size turns by its square
        assert cos > 1 - 1e-4


@pytest.mark.parametrize("bits", [32, 8])
def test_captured(rk, bits):
    eager, live = Model(rk, bits), Model(rk, bits)
    step = torch.ones(1, dtype=torch.int64, device=DEV)
    eager_step = step.clone()

    def one(m, count):
        s = m.gradients(rk)
        rk.adamw_step(m.opt, **{**HYPER, "step": count})
        count += 1
        return s["loss"]["loss"]
    first = one(live, step)  # outside the capture: lazily set attributes
    assert same_bits(first, one(eager, eager_step))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = one(live, step)
    for _ in range(3):
        graph.replay()
        want = one(eager, eager_step)
        torch.cuda.synchronize()
        assert same_bits(loss, want)
    for a, b in zip(live.opt.master, eager.opt.master):
        assert same_bits(a, b)
    assert rk.get_device_error() == 0
