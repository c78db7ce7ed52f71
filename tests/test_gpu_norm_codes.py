"""Codes and scales of the norm in 8 bits: those of the rounded quotient of the values that the
same call leaves in fp32."""
import pytest
import torch

import norm_plain as npl
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def groups(y, width):
    T, H = y.shape
    n = -(-H // width)
    return torch.nn.functional.pad(y, (0, n * width - H)).view(T, n, width)


def check(rk, x, w, residual, group):
    """Every operation of the definition in fp32, rounded by itself: the codes and scales have its bits."""
    move = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    y, _ = rk.rms_norm(move(x), move(w), residual=move(residual), out_dtype=FP32)
    q, s, _ = rk.rms_norm_e4m3(move(x), move(w), residual=move(residual), group=group)
    y, q, s = y.cpu(), q.cpu(), s.cpu()
    parts = groups(y, group or y.shape[1])
    top = torch.where(torch.isnan(parts), 0.0, parts.abs()).amax(2)
    want = torch.where(top > 0, (top * (torch.tensor(1.0) / 448.0)).clamp(min=2.0 ** -120), 0.0)
    assert same_bits(s, want)
    codes = torch.where(want[:, :, None] > 0, parts / want[:, :, None], parts)
    codes = codes.clamp(-448.0, 448.0).to(E4M3).float().flatten(1)[:, :y.shape[1]]
    q = q.float()
    nan = torch.isnan(codes)
    assert torch.equal(torch.isnan(q), nan)
    assert torch.equal(q[~nan], codes[~nan]), int((q != codes)[~nan].sum())


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,H", [(4000, 64), (3000, 100), (2000, 128), (1000, 256), (700, 1000), (64, 3584), (1000, 2047),
                                 (1000, 4096), (90, 5000), (40, 16384)])
def test_codes_are_those_of_the_rounded_quotient(rk, T, H, group):
    g = torch.Generator().manual_seed(T + H + group)
    for x_type, res_type in ((BF16, BF16), (FP32, None), (BF16, FP32)):
        x = npl.matrix(g, T, H, x_type, scale=2.0)
        res = None if res_type is None else npl.matrix(g, T, H, res_type, scale=3.0)
        check(rk, x, (1 + 0.3 * torch.randn(H, generator=g)).to(BF16), res, group)
    assert rk.get_device_error() == 0


@pytest.mark.parametrize("group", [0, 128])
def test_small_and_infinite_scales(rk, group):
    """Blocks of very small values, whose remainders would leave the normal numbers, and of infinities."""
    g = torch.Generator().manual_seed(3)
    for H in (100, 264, 4096):
        x = npl.matrix(g, 400, H, FP32)
        x[:4] = 0
        for power in (-140, -126, -120, -110, -100, -95, -90, -70, -61, -60, -59, -20, 60, 100):
            check(rk, x, torch.randn(H, generator=g) * 2.0 ** power, None, group)
        w = torch.randn(H, generator=g)
        w[H // 3], w[H // 2] = float("inf"), float("nan")
        check(rk, x, w, None, group)
    assert rk.get_device_error() == 0
