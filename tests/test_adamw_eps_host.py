"""Refusals of an AdamW step whose eps is out of range (no GPU needed: refused calls read none of the addresses)."""
import pytest

from test_preference_adamw_host import INVALID, OK, adamw, rk, tensor  # noqa: F401


@pytest.mark.parametrize("eps", [0.0, -1e-8, 1e-60, float("nan"), float("inf"), 2.0 ** 100, 1e38, 3.4e38, 1e39])
def test_eps_out_of_range(rk, eps):  # noqa: F811
    """From 2^126 on a quotient by sqrt(v) + eps would be 0."""
    assert adamw(rk, [tensor(rk)], eps=eps) == INVALID


def test_large_eps_is_taken(rk):  # noqa: F811
    assert adamw(rk, [], eps=2.0 ** 99) == OK and adamw(rk, [], eps=1e-30) == OK
