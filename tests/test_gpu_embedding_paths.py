"""Paths of the embedding gradient that differ by size: rows wider than a warp's columns, the sorts by
tiles with a canonical order and padding, and the zeros that are written beside the sort."""
import numpy as np
import pytest
import torch

import rules_plain as rp
from helpers import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rk():
    from invariant_rl_logprob_gb300 import build
    build.build()
    import invariant_rl_logprob_gb300 as rk
    rk.load_library()
    return rk


def some_ids(T, V, seed, hot=0.5):
    g = torch.Generator().manual_seed(seed)
    ids = torch.where(torch.rand(T, generator=g) < hot, torch.randint(0, min(V, 3), (T,), generator=g),
                      torch.randint(0, V, (T,), generator=g))
    ids[torch.rand(T, generator=g) < 0.1] = -1
    return ids


# vectors of 8 columns: a lane's second one from column 256 on, a warp's second 512 columns
@pytest.mark.parametrize("H", [256, 264, 520, 1024, 4096])
@pytest.mark.parametrize("T,hot", [(20, 0.0), (400, 0.6)])  # ids of one piece; of several
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_wide_rows(rk, dtype, T, hot, H):
    V = 37
    ids = some_ids(T, V, T + H, hot)
    g = torch.Generator().manual_seed(H)
    d = torch.randn(T, H, generator=g).to(dtype)
    old = torch.randn(V, H, generator=g)
    want, mag, count = rp.plain_embedding_bwd(d, ids.numpy(), V, 0.75)
    assert (count.max() > 64) == (hot > 0)
    # 32 additions in a piece, one for each piece, the product with the scale
    bound = (np.minimum(count, 32) + (count + 31) // 32 + 2)[:, None] * rp.U * 1.01 * mag
    got = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, scale=0.75)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    dE = old.to(DEV)
    rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, scale=0.75, dE=dE, accumulate=True)
    total = old.double().numpy() + want
    assert np.all(np.abs(dE.double().cpu().numpy() - total) <= bound + rp.U * 1.01 * (np.abs(total) + bound))
    # the same columns by single elements: off 16-byte boundaries
    buf = torch.empty(T * H + 1, dtype=dtype, device=DEV)[1:].view(T, H)
    buf.copy_(d)
    assert same_bits(rk.embedding_bwd(buf, ids.to(DEV), V, scale=0.75), got)
