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


# the one-block sorts reach to 1024 and 8192 tokens, tiles that scan the counts themselves to 131072
@pytest.mark.parametrize("n", [1024, 1025, 8192, 8193, 30000, 131072, 131073, 200000])
def test_the_sorts_agree(rk, n):
    """The same tokens in the same canonical order, and padding among them that takes n past the limits."""
    T, V, H = 1000, 700, 24
    ids = some_ids(T, V, 5)
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(6)).to(BF16)
    base = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V)
    want, mag, count = rp.plain_embedding_bwd(d, ids.numpy(), V, 1.0)
    bound = (np.minimum(count, 32) + (count + 31) // 32 + 2)[:, None] * rp.U * 1.01 * mag
    assert np.all(np.abs(base.double().cpu().numpy() - want) <= bound)
    g = torch.Generator().manual_seed(n)
    place = torch.randperm(n, generator=g)[:T].sort().values
    ids2 = torch.full((n,), -1)
    d2 = torch.full((n, H), float("nan"), dtype=BF16)
    ids2[place], d2[place] = ids, d
    assert same_bits(rk.embedding_bwd(d2.to(DEV), ids2.to(DEV), V), base)
    # as a canonical order of n entries into rows that lie elsewhere, most of them out of range
    where = torch.randperm(T, generator=g)
    order = torch.randint(-1000, 0, (n,), generator=g)
    order[::3] = torch.randint(T, 1 << 40, (len(order[::3]),), generator=g)
    order[place] = where
    d3, ids3 = torch.empty_like(d), torch.empty_like(ids)
    d3[where], ids3[where] = d, ids
    assert same_bits(rk.embedding_bwd(d3.to(DEV), ids3.to(DEV), V, row_order=order.to(DEV)), base)
    # between the rows that cu_seqlens leaves out
    lead = 13
    ids4 = torch.cat([torch.zeros(lead, dtype=torch.int64), ids2, torch.ones(5, dtype=torch.int64)])
    d4 = torch.full((n + lead + 5, H), float("nan"), dtype=BF16)
    d4[lead:lead + n] = d2
    cu = torch.tensor([lead, lead + 7, lead + n], dtype=torch.int32, device=DEV)
    assert same_bits(rk.embedding_bwd(d4.to(DEV), ids4.to(DEV), V, cu), base)
    assert rk.get_device_error() == 0


def test_a_row_named_twice_among_many(rk):
    T, V, H = 9000, 50, 8
    ids = some_ids(T, V, 8, 0.2)
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(9))
    order = torch.randint(0, T, (20000,), generator=torch.Generator().manual_seed(10))
    want, mag, count = rp.plain_embedding_bwd(d, ids.numpy(), V, 1.0, order=order.tolist())
    got = rk.embedding_bwd(d.to(DEV), ids.to(DEV), V, row_order=order.to(DEV)).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= (np.minimum(count, 32) + (count + 31) // 32 + 2)[:, None] * rp.U * 1.01 * mag)


# zeros in the grid of the smallest sort; beside the other one-block sort; in rows that no key names
@pytest.mark.parametrize("n,V,H", [(700, 8000, 64), (4000, 40000, 64), (8192, 65536, 9), (4000, 9000, 64), (20000, 200000, 16)])
def test_zeros_in_a_graph_and_between_readers(rk, n, V, H):
    """dE and the workspace used over and over on one stream, with readers of dE in between."""
    steps = 6
    ids = [some_ids(n, V, 20 + i, 0.3).to(DEV) for i in range(steps)]
    d = [torch.randn(n, H, device=DEV) for _ in range(steps)]
    want = [rk.embedding_bwd(d[i], ids[i], V) for i in range(steps)]
    for i in range(steps):  # the references: summed by index, zero elsewhere
        live = ids[i] >= 0
        ref = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[i][live], d[i][live].double())
        mag = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[i][live], d[i][live].double().abs())
        most = int(torch.bincount(ids[i][live]).max())
        assert bool(((want[i].double() - ref).abs() <= (32 + most // 32 + 3) * rp.U * 1.01 * mag).all())
    ws = torch.empty(rk.embedding_bwd_workspace_size(n, H, V), dtype=torch.uint8, device=DEV)
    dE = torch.full((V, H), float("nan"), device=DEV)
    seen = [torch.empty(V, H, device=DEV) for _ in range(2 * steps)]
    torch.cuda.synchronize()
    for k in range(2 * steps):
        rk.embedding_bwd(d[k % steps], ids[k % steps], V, dE=dE, workspace=ws)
        seen[k].copy_(dE)
    assert all(same_bits(seen[k], want[k % steps]) for k in range(2 * steps))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for k in range(steps):
            rk.embedding_bwd(d[k], ids[k], V, dE=dE, workspace=ws, stream=side)
            seen[k].copy_(dE)
    for _ in range(3):
        for s in seen:
            s.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(seen[k], want[k]) for k in range(steps))
