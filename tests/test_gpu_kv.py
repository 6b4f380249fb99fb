"""The paged key/value cache: what lq_kv_write stores is what the oracle's
packer stores, byte for byte, and lq_kv_read gives back the values of those
bytes exactly (d * q is exact in float32), so nothing here has a tolerance."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged
from oracle import attention as A

pytestmark = pytest.mark.gpu

FMTS = ("f16", "q8_0", "q4_0")


def _up(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


def _new_rows(P):
    """The call's rows of K and V."""
    return tuple(np.concatenate([x[i][t - n:] if n else x[i][:0] for i, (n, t) in enumerate(zip(P.news, P.totals))])
                 for x in (P.k, P.v))


def _without_new(P):
    """The pools as they were before the call's tokens came: noise in their slots."""
    rng = np.random.default_rng(99)
    before = P.pools.copy()
    for i, (n, t) in enumerate(zip(P.news, P.totals)):
        for p in range(max(0, t - n), t):
            pg, slot = P.table[i, p // P.page], p % P.page
            before[:, pg, :, slot * P.row:(slot + 1) * P.row] = rng.integers(0, 256, size=(2, P.kv_heads, P.row), dtype=np.uint8)
    return before


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals,kv_heads,d,page", [
    ([1], [1], 1, 32, 16), ([1, 1, 1], [17, 1, 64], 2, 64, 16), ([40, 0, 3], [100, 5, 3], 3, 128, 16),
    ([7, 33], [33, 33], 2, 256, 64), ([5], [11], 2, 96, 7), ([130], [130], 8, 160, 1), ([9, 70], [9, 200], 1, 224, 32)])
def test_write_stores_the_packed_bytes_and_read_returns_their_values(lq, cuda_dev, fmt, news, totals, kv_heads, d, page):
    P = Paged(lq, fmt, news, totals, kv_heads, kv_heads, d, page, cuda_dev, seed=len(news) + d)
    after = P.pools.copy()
    P.pools = _without_new(P)
    cache, batch = P.cache(), P.batch()
    k, v = _new_rows(P)
    lq.lq_kv_write(cache, batch, _up(k, cuda_dev), _up(v, cuda_dev))
    got = [x.cpu().numpy() for x in (cache.k, cache.v)]
    for w in range(2):
        assert np.array_equal(got[w], after[w])
    ko, vo = (torch.full((P.tokens, kv_heads, d), float("nan"), device=cuda_dev) for _ in range(2))
    lq.lq_kv_read(cache, batch, ko, vo)
    for out, x in ((ko, k), (vo, v)):
        assert np.array_equal(out.cpu().numpy(), A.cache_values(fmt, x.reshape(-1, d)).reshape(x.shape))
    assert lq.last_device_error() == lq.LQ_OK


@pytest.mark.parametrize("fmt", FMTS)
def test_read_back_of_whole_sequences_and_of_one_side(lq, cuda_dev, fmt):
    P = Paged(lq, fmt, [50, 0, 33], [50, 0, 33], 2, 2, 64, 16, cuda_dev, seed=4)
    cache, batch = P.cache(), P.batch()
    for which in (0, 1):
        out = torch.full((P.tokens, 2, 64), float("nan"), device=cuda_dev)
        lq.lq_kv_read(cache, batch, *((out, None) if which == 0 else (None, out)))
        want = np.concatenate([P.values(which, i) for i in range(3)])
        assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_slices_of_a_fused_projection(lq, cuda_dev, fmt):
    """K and V as column ranges of one matrix, at offsets that are and are not
    multiples of 16 bytes; outputs as strided rows too."""
    P = Paged(lq, fmt, [5, 2], [20, 2], 2, 2, 64, 16, cuda_dev, seed=8)
    after = P.pools.copy()
    k, v = _new_rows(P)
    for pad in (0, 1, 4):
        P.pools = _without_new(P)
        cache, batch = P.cache(), P.batch()
        fused = torch.zeros(P.tokens, 3 * 128 + pad, device=cuda_dev)
        fused[:, pad:pad + 128] = _up(k, cuda_dev).flatten(1)
        fused[:, pad + 128:pad + 256] = _up(v, cuda_dev).flatten(1)
        lq.lq_kv_write(cache, batch, fused[:, pad:pad + 128], fused[:, pad + 128:pad + 256])
        assert np.array_equal(cache.k.cpu().numpy(), after[0]) and np.array_equal(cache.v.cpu().numpy(), after[1])
        out = torch.full((P.tokens, 3 * 128 + pad), -7.0, device=cuda_dev)
        lq.lq_kv_read(cache, batch, out[:, pad:pad + 128], out[:, pad + 128:pad + 256])
        o = out.cpu().numpy()
        assert np.array_equal(o[:, pad:pad + 128], A.cache_values(fmt, k.reshape(-1, 64)).reshape(-1, 128))
        assert np.array_equal(o[:, pad + 128:pad + 256], A.cache_values(fmt, v.reshape(-1, 64)).reshape(-1, 128))
        assert np.all(o[:, :pad] == -7.0) and np.all(o[:, pad + 256:] == -7.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_what_has_no_place_is_dropped(lq, cuda_dev, fmt):
    """Pages of -1 and beyond the pool, positions below 0 and rows of no
    sequence: nothing but the other tokens' slots changes, and reads of such
    places give zeros (rows of no sequence stay as they are)."""
    P = Paged(lq, fmt, [40, 6], [40, 4], 1, 1, 32, 16, cuda_dev, seed=5)
    table = P.table.copy()
    table[0, 1], table[1, 0] = -1, P.pages + 3
    before = _without_new(P)
    want = before.copy()
    for w in range(2):  # the tokens on the pages that are left
        for pg in (P.table[0, 0], P.table[0, 2]):
            want[w, pg] = P.pools[w, pg]
    P.pools = before
    P.tokens = 48  # rows 46 and 47 belong to no sequence
    cache, batch = P.cache(), P.batch(table=table)
    k, v = (np.concatenate([x[0], np.zeros((2, 1, 32), np.float32), x[1], np.ones((2, 1, 32), np.float32)]) for x in (P.k, P.v))
    lq.lq_kv_write(cache, batch, _up(k, cuda_dev), _up(v, cuda_dev))
    assert np.array_equal(cache.k.cpu().numpy(), want[0]) and np.array_equal(cache.v.cpu().numpy(), want[1])
    out = torch.full((48, 1, 32), -7.0, device=cuda_dev)
    lq.lq_kv_read(cache, batch, out, None)
    o = out.cpu().numpy()
    kept = A.cache_values(fmt, P.k[0][:, 0])
    kept[16:32] = 0
    assert np.array_equal(o[:40, 0], kept) and np.all(o[40:46] == 0) and np.all(o[46:] == -7.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_values_at_the_edges_of_the_formats(lq, cuda_dev, fmt):
    """Zero blocks, ties of magnitude, halves, subnormal scales; infinities
    and large values come back as +-65504 (within a code's step), a NaN as NaN
    over its element (f16) or block (quantised)."""
    d = 64
    x = np.zeros((12, 1, d), np.float32)
    x[1, 0, 3], x[1, 0, 7] = 1.0, -1.0
    x[2, 0, 5], x[2, 0, 9] = -1.0, 1.0
    x[3] = 0.37
    x[4, 0] = (np.arange(d) % 32 - 16) * 0.5
    x[5] = 1e-6
    x[6] = 3e-9
    x[7, 0, :32] = 1e7
    x[8, 0, 1], x[8, 0, 2] = np.inf, -np.inf
    x[9, 0, 40] = np.nan
    x[10, 0, 0] = 1e-41
    x[11] = -0.0
    P = Paged(lq, fmt, [12], [12], 1, 1, d, 16, cuda_dev)
    cache, batch = P.cache(), P.batch()
    lq.lq_kv_write(cache, batch, _up(x, cuda_dev), _up(x, cuda_dev))
    ko, vo = (torch.zeros(12, 1, d, device=cuda_dev) for _ in range(2))
    lq.lq_kv_read(cache, batch, ko, vo)
    got = ko.cpu().numpy()[:, 0]
    assert np.array_equal(got, vo.cpu().numpy()[:, 0], equal_nan=True)
    want = A.cache_values(fmt, np.nan_to_num(x[:, 0], nan=0.0, posinf=np.inf, neginf=-np.inf))
    if fmt == "f16":
        want[9, 40] = np.nan
    else:
        want[9, 32:] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


def test_on_another_stream_and_in_a_graph(lq, cuda_dev):
    P = Paged(lq, "q8_0", [4, 4], [30, 9], 2, 2, 64, 16, cuda_dev, seed=3)
    after = P.pools.copy()
    P.pools = _without_new(P)
    cache, batch = P.cache(), P.batch()
    k, v = (_up(x, cuda_dev) for x in _new_rows(P))
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lq.lq_kv_write(cache, batch, k, v, stream=side)
    lq.lq_kv_read(cache, batch, ko, vo, stream=side)
    side.synchronize()
    assert np.array_equal(cache.k.cpu().numpy(), after[0]) and np.array_equal(cache.v.cpu().numpy(), after[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lq.lq_kv_write(cache, batch, k, v)
        lq.lq_kv_read(cache, batch, ko, vo)
    k.mul_(2.0)  # new inputs of the same graph
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ko.cpu().numpy().reshape(-1, 64), A.cache_values("q8_0", k.cpu().numpy().reshape(-1, 64)))


def test_offsets_beyond_32_bits(lq, cuda_dev):
    """A pool of more than 4 GiB a side: the last page's tokens land there."""
    page, kv_heads, d = 64, 8, 256
    pages = (1 << 32) // (page * kv_heads * d * 2) + 3
    cache = lq.KVCache("f16", pages, page, kv_heads, d, device=cuda_dev)
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device=cuda_dev)
    batch = lq.KVBatch(table, torch.tensor([70], dtype=torch.int32, device=cuda_dev),
                       torch.tensor([0, 70], dtype=torch.int32, device=cuda_dev), 70)
    x = torch.randn(70, kv_heads, d, device=cuda_dev)
    lq.lq_kv_write(cache, batch, x, x)
    out = torch.zeros_like(x)
    lq.lq_kv_read(cache, batch, None, out)
    assert torch.equal(out, x.half().float())
    last = cache.v.view(torch.float16).view(pages, kv_heads, page, d)[pages - 1]
    assert torch.equal(last.float(), x[:64].half().float().transpose(0, 1))
