"""Results of the norm and its gradient over the lists that say which rows are active (no GPU needed: refused
calls read none of the addresses)."""
import pytest

from test_norm_host import E4M3, FAKE, FAR, FP32, INVALID, backward, forward, rk  # noqa: F401

LIST = 7 * FAR
# T = 4 rows of H = 64 columns: 512 bytes of bf16, 1024 of fp32; targets 32 bytes, 3 offsets 12, an order of 5 rows 40


@pytest.mark.parametrize("at", [0, 8, 31 * 8, 504, -24])
@pytest.mark.parametrize("result", ["out", "ro"])
def test_forward_over_targets(rk, result, at):  # noqa: F811
    more = dict(out=8 * FAR, res=3 * FAR, ro=LIST) if result == "ro" else dict(out=LIST)
    assert forward(rk, tg=LIST + at, **more) == INVALID


@pytest.mark.parametrize("at", [0, 4, 508, -8])
def test_forward_over_offsets(rk, at):  # noqa: F811
    assert forward(rk, cu=LIST + at, ns=2, out=LIST) == INVALID
    assert forward(rk, cu=LIST + at, ns=2, out=8 * FAR, res=3 * FAR, ro=LIST) == INVALID


def test_scales_over_the_lists(rk):  # noqa: F811
    assert forward(rk, ot=E4M3, s=LIST, tg=LIST + 8) == INVALID
    assert forward(rk, ot=E4M3, s=LIST + 28, tg=LIST) == INVALID
    assert forward(rk, ot=E4M3, s=LIST, cu=LIST + 12, ns=2) == INVALID
    assert forward(rk, ot=E4M3, s=LIST, cu=LIST - 8, ns=2) == INVALID


@pytest.mark.parametrize("result,size", [("dx", 512), ("dw", 256)])
def test_backward_over_the_lists(rk, result, size):  # noqa: F811
    for at in (0, 8, size - 8, -24):
        assert backward(rk, tg=LIST + at, **{result: LIST}) == INVALID
    for at in (0, size - 4, -8):
        assert backward(rk, cu=LIST + at, ns=2, **{result: LIST}) == INVALID
    for at in (0, 8, size - 8, -32):
        assert backward(rk, order=LIST + at, n=5, **{result: LIST}) == INVALID


def test_wider_results_reach_further(rk):  # noqa: F811
    assert forward(rk, tg=LIST + 1016, out=LIST, ot=FP32) == INVALID
    assert forward(rk, tg=LIST + 3 * 160 + 120, out=LIST, ldo=80) == INVALID
    assert backward(rk, order=LIST + 1016, n=1, dx=LIST, xt=FP32) == INVALID
    # an address that is not aligned is refused as well
    assert forward(rk, tg=LIST + 4) == INVALID and forward(rk, cu=LIST + 2, ns=2) == INVALID
    assert backward(rk, tg=LIST + 4) == INVALID and backward(rk, order=LIST + 4, n=2) == INVALID
