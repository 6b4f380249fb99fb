"""The paged cache and its attention on batches of many sequences, prompts of
many row tiles and mixed batches: the planning that single sequences never
reach, and which kernels an automatic call takes."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from oracle import attention as A
from test_gpu_attn import AUTO, FMTS, GENERIC, ROUTES, TILE, WARP, _run

pytestmark = pytest.mark.gpu

COUNTS = (8, 9, 10)  # generic, warp-level, tcgen05


def _batch(lq, fmt, n, d, dev, seed, heads=2, kv_heads=1, long=()):
    """n short sequences, a third of them without new tokens, and the `long`
    ones ((new, total)) spread among them."""
    rng = np.random.default_rng(seed)
    totals = rng.integers(1, 30, n)
    news = np.minimum(rng.integers(0, 3, n), totals)
    for i, (new, total) in enumerate(long):
        at = (2 * i + 1) * n // (2 * len(long))
        news[at], totals[at] = new, total
    return Paged(lq, fmt, news.tolist(), totals.tolist(), heads, kv_heads, d, 16, dev, seed=seed)


def _twice(lq, P, **kw):
    """Two calls on one work buffer give the same bits, and rows as expected."""
    cache, batch = P.cache(), P.batch()
    work = lq.attn_work(cache, batch, P.heads)
    P.cache = lambda: cache
    o, lse = _run(lq, P, work=work, **kw)
    o2, lse2 = _run(lq, P, work=work, **kw)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    want, tol, wl, ltol = P.expect(window=kw.get("window", 0), sinks=kw.get("sinks", 0))
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt,n,d,long", [("f16", 33, 128, [(3, 700)]), ("q8_0", 400, 64, [(40, 900), (1, 5000)]),
                                          ("f16", 400, 256, [(70, 90), (1, 2000)]), ("q4_0", 400, 128, [(1, 3000), (130, 200)]),
                                          ("q8_0", 70, 128, []), ("q4_0", 1000, 64, [])])
def test_many_sequences(lq, cuda_dev, route, fmt, n, d, long):
    _twice(lq, _batch(lq, fmt, n, d, cuda_dev, seed=n, long=long), route=route)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,d,longest", [(1, 128, 20000), (70, 128, 400), (400, 64, 60), (300, 256, 60), (33, 64, 2500)])
def test_single_tokens(lq, cuda_dev, fmt, n, d, longest):
    """A decoding step, the call told so: rows of eight only."""
    rng = np.random.default_rng(n)
    totals = rng.integers(1, longest + 1, n)
    totals[n // 2] = longest
    P = Paged(lq, fmt, [1] * n, totals.tolist(), 4, 1, d, 16, cuda_dev, seed=n)
    lq.reset_counts()
    _twice(lq, P, max_q=1)
    assert [lq.route_count(c) for c in COUNTS] == [0, 2, 0]
    if n > 1:
        _twice(lq, P, max_q=1, window=33, sinks=3)


@pytest.mark.parametrize("route", (AUTO, GENERIC, WARP, TILE))
def test_more_sequences_than_tiles_take(lq, cuda_dev, route):
    """Past 4096 sequences the warp-level kernel takes prompts too."""
    P = _batch(lq, "q8_0", 4100, 64, cuda_dev, seed=5, heads=1, long=[(120, 130)])
    lq.reset_counts()
    _twice(lq, P, route=route)
    if route == AUTO:
        assert [lq.route_count(c) for c in COUNTS] == [0, 2, 0]


@pytest.mark.parametrize("route", (AUTO, TILE))
@pytest.mark.parametrize("fmt,d,heads,news,totals,window", [
    ("f16", 64, 8, [1100], [1100], 0), ("q8_0", 128, 8, [5, 1050], [300, 1060], 300), ("f16", 256, 8, [1, 560, 40], [90, 560, 40], 0)])
def test_prompts_of_many_row_tiles(lq, cuda_dev, route, fmt, d, heads, news, totals, window):
    """More than 32 units of one head and sequence (256 rows, or 128 of 256 dims)."""
    P = Paged(lq, fmt, news, totals, heads, 1, d, 16, cuda_dev, seed=d)
    _twice(lq, P, route=route, window=window, sinks=4 if window else 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_mixed_batches_take_both_kernels(lq, cuda_dev, fmt, d):
    """Prompts and single tokens in one call, whatever it is told of its
    longest: the truth, nothing, too little or too much."""
    news = [1] * 20 + [150] + [1] * 15 + [97, 0, 33] + [2] * 5
    totals = [1 + 13 * i % 200 for i in range(20)] + [150] + [31 * i + 1 for i in range(15)] + [300, 7, 50] + [60] * 5
    P = Paged(lq, fmt, news, totals, 4, 1, d, 16, cuda_dev, seed=d)
    want, tol, wl, ltol = P.expect()
    for max_q, counts in ((150, [0, 1, 1]), (0, [0, 1, 1]), (1 << 20, [0, 1, 1]), (1, [0, 1, 0]), (3, [0, 1, 0])):
        lq.reset_counts()
        o, lse = _run(lq, P, max_q=max_q)
        assert [lq.route_count(c) for c in COUNTS] == counts, max_q
        compare(o, want, tol, f"output, max_q {max_q}")
        compare(lse, wl, ltol, f"lse, max_q {max_q}")


@pytest.mark.parametrize("news,totals,d,page,max_q,counts", [
    ([1], [100], 128, 16, 1, [0, 1, 0]), ([1], [100], 128, 16, 0, [0, 1, 0]), ([300], [300], 128, 16, 300, [0, 0, 1]),
    ([300], [300], 128, 16, 0, [0, 0, 1]), ([9], [9], 96, 16, 9, [1, 0, 0]), ([9], [9], 128, 7, 9, [1, 0, 0])])
def test_kernels_of_one_sequence(lq, cuda_dev, news, totals, d, page, max_q, counts):
    P = Paged(lq, "f16", news, totals, 4, 1, d, page, cuda_dev, seed=1)
    lq.reset_counts()
    _run(lq, P, max_q=max_q)
    assert [lq.route_count(c) for c in COUNTS] == counts


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [33, 400, 4100])
def test_cache_of_many_sequences(lq, cuda_dev, fmt, n):
    """Writing and reading back the new tokens of a large batch."""
    P = _batch(lq, fmt, n, 32, cuda_dev, seed=n, heads=1)
    k, v = (np.concatenate([x[i][t - m:] for i, (m, t) in enumerate(zip(P.news, P.totals))]) for x in (P.k, P.v))
    cache, batch = P.cache(), P.batch()
    lq.lq_kv_write(cache, batch, torch.from_numpy(v).to(cuda_dev), torch.from_numpy(k).to(cuda_dev))  # the other way round
    ko, vo = (torch.full((P.tokens, 1, 32), float("nan"), device=cuda_dev) for _ in range(2))
    lq.lq_kv_read(cache, batch, ko, vo)
    for got, x in ((ko, v), (vo, k)):
        assert np.array_equal(got.cpu().numpy(), A.cache_values(fmt, x.reshape(-1, 32)).reshape(x.shape))
    for w, x in ((0, P.v), (1, P.k)):  # the bytes of the whole pools: new tokens swapped, all else as it was
        for i, (m, t) in enumerate(zip(P.news, P.totals)):
            if m:
                P.store(w, i, x[i][t - m:], first=t - m)
    assert np.array_equal(cache.k.cpu().numpy(), P.pools[0]) and np.array_equal(cache.v.cpu().numpy(), P.pools[1])
    assert lq.last_device_error() == lq.LQ_OK


@pytest.mark.parametrize("fmt,d", [("f16", 256), ("q8_0", 128), ("q4_0", 64)])
def test_pools_beyond_32_bits(lq, cuda_dev, fmt, d):
    """Pools of more than 4 GiB a side, a sequence on their last pages and one
    that alternates between both ends: the same bits as from a small pool."""
    page, kv_heads, heads = 64, 2, 4
    P = Paged(lq, fmt, [3, 90], [200, 333], heads, kv_heads, d, page, cuda_dev, seed=d)
    small = P.cache()
    pages = (1 << 32) // (P.block * kv_heads) + 70
    big = lq.KVCache(fmt, pages, page, kv_heads, d, device=cuda_dev)
    used = P.table[P.table >= 0]
    moved = {int(p): pages - 1 - n if n % 3 else n for n, p in enumerate(used)}
    table = np.vectorize(lambda p: moved.get(int(p), -1))(P.table).astype(np.int32)
    assert (big.k.numel() > 1 << 32) and table.max() == pages - 2
    for a, b in ((small.k, big.k), (small.v, big.v)):
        for p, to in moved.items():
            b.view(pages, -1)[to] = a.view(P.pages, -1)[p]
    for route in ROUTES:
        P.cache = lambda: small
        o, lse = _run(lq, P, route=route)
        P.cache = lambda: big
        o2, lse2 = _run(lq, P, route=route, table=table)
        assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    out = [torch.empty(P.tokens, kv_heads, d, device=cuda_dev) for _ in range(4)]
    lq.lq_kv_read(small, P.batch(), *out[:2])
    lq.lq_kv_read(big, P.batch(table=table), *out[2:])
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
