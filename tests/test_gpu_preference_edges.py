"""The preference loss where beta times a difference leaves fp32."""
import math

import numpy as np
import pytest
import torch

import preference_plain as pp
from test_gpu_preference import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


@pytest.mark.parametrize("tokens", [40, 200000])
def test_steep_losses(rk, tokens):
    """Losses are 0 or infinite, or what fp32 holds, and slopes 0 or scale * beta: never NaN."""
    logp = torch.zeros(tokens)
    logp[0], logp[1], logp[2], logp[3] = -1.0, -11.0, -1.0, -1.0 - 2.0 ** -23
    c = pp.Case(logp, None, torch.zeros(tokens, dtype=torch.int64), torch.arange(5, dtype=torch.int32),
                torch.tensor([0, 1, 0, 2, 3], dtype=torch.int32), torch.tensor([1, 0, 2, 3, 2], dtype=torch.int32), None)
    d = [10.0, -10.0, 0.0, 2.0 ** -23, -2.0 ** -23]
    for beta in (1e30, 1e37, 5e37, 3e38):
        beta = float(np.float32(beta))
        for kind in ("sigmoid", "hinge"):
            got = run(rk, c, kind=kind, beta=beta)
            for p, x in enumerate(d):
                flat = math.log(2) if kind == "sigmoid" else 1.0
                want = flat if x == 0 else 0.0 if x > 0 else -beta * x
                loss = float(got["loss"][p])
                if want > 3.5e38:
                    assert loss == math.inf, (beta, kind, p, loss)
                else:
                    assert abs(loss - want) <= 16 * pp.U * want, (beta, kind, p, loss)
            # token 1: its sequence is rejected by 10 and chosen by -10, of which the second has a slope
            grad = float(got["grad"][1])
            assert abs(grad + beta) <= 16 * pp.U * beta, (beta, kind, grad)
    # a margin past fixed point: in 64-bit floats
    c.margin = torch.tensor([-3e5, 3e5, 0.0, 0.0, 0.0])
    got = run(rk, c, beta=3e38)
    assert got["loss"][0] == 0 and got["loss"][1] == math.inf and not bool(torch.isnan(got["grad"]).any())
    assert rk.get_device_error() == 0
