"""lq_attn_paged against the float64 formula (oracle/attention.py), on caches
whose bytes the oracle's packer made. Tolerances are the oracle's: derived
from the rounding of the kernels' steps, per element."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from oracle import attention as A

pytestmark = pytest.mark.gpu

FMTS = ("f16", "q8_0", "q4_0")
AUTO, GENERIC, WARP, TILE = range(4)
ROUTES = (AUTO, GENERIC, WARP, TILE)


def _run(lq, P, route=AUTO, window=0, sinks=0, scale=None, max_q=0, table=None, q=None, work=None):
    cache, batch = P.cache(), P.batch(max_q=max_q, table=table)
    Q = torch.from_numpy(P.q if q is None else q).to(P.dev)
    O = torch.full_like(Q, float("nan"))
    lse = torch.full((P.tokens, P.heads), float("nan"), device=P.dev)
    work = lq.attn_work(cache, batch, P.heads) if work is None else work
    lq.attn_route(route)
    try:
        lq.lq_attn_paged(cache, batch, Q, O, 1.0 / np.sqrt(P.d) if scale is None else scale, window=window, sinks=sinks,
                         lse=lse, work=work)
    except lq.LQError as e:
        if route in (WARP, TILE) and e.status == lq.LQ_ERR_UNSUPPORTED:
            pytest.skip("the forced kernel does not take this geometry")
        raise
    finally:
        lq.attn_route(AUTO)
    torch.cuda.synchronize()
    assert lq.last_device_error() == lq.LQ_OK
    return O.cpu().numpy(), lse.cpu().numpy()


def _check(lq, P, **kw):
    window, sinks, table, scale = (kw.get(n, z) for n, z in (("window", 0), ("sinks", 0), ("table", None), ("scale", None)))
    o, lse = _run(lq, P, **kw)
    want, tol, wl, ltol = P.expect(window=window, sinks=sinks, table=table, scale=scale)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")
    return o


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,heads,kv_heads,page", [(64, 4, 2, 16), (128, 8, 1, 16), (256, 8, 2, 64), (128, 3, 3, 32),
                                                   (96, 4, 2, 16), (32, 2, 1, 48), (128, 32, 2, 16), (64, 5, 1, 7)])
def test_lengths_from_one_token(lq, cuda_dev, route, fmt, d, heads, kv_heads, page):
    """One new token each, lengths around tile and page edges."""
    totals = [1, 2, 15, 16, 17, 31, 63, 65, 127, 128, 129, 300]
    P = Paged(lq, fmt, [1] * len(totals), totals, heads, kv_heads, d, page, cuda_dev, seed=d + heads)
    _check(lq, P, route=route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals,d,heads,kv_heads,page", [
    ([5, 1, 0, 9], [40, 1, 13, 9], 128, 4, 2, 16), ([70], [200], 64, 6, 3, 16), ([33, 2], [33, 150], 256, 2, 1, 16),
    ([140, 3], [300, 70], 128, 4, 4, 32), ([65], [129], 128, 8, 1, 64), ([300], [300], 64, 2, 1, 128)])
def test_chunks(lq, cuda_dev, route, fmt, news, totals, d, heads, kv_heads, page):
    """Ragged chunks over cached parts of odd lengths."""
    P = Paged(lq, fmt, news, totals, heads, kv_heads, d, page, cuda_dev, seed=sum(totals))
    _check(lq, P, route=route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (37, 1), (128, 33), (129, 150), (1000, 4), (64, 0)])
def test_window_and_sinks(lq, cuda_dev, route, fmt, window, sinks):
    P = Paged(lq, fmt, [1, 60, 200], [400, 400, 200], 4, 2, 128, 16, cuda_dev, seed=window)
    _check(lq, P, route=route, window=window, sinks=sinks)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 256])
def test_window_other_head_dims(lq, cuda_dev, route, fmt, d):
    P = Paged(lq, fmt, [3, 40], [290, 333], 8, 1, d, 32, cuda_dev, seed=d)
    _check(lq, P, route=route, window=100, sinks=5)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing(lq, cuda_dev, route, fmt):
    """More rows than positions (rows before position 0), empty sequences, and
    pages of -1 that leave a row without a key: zeros and -inf."""
    P = Paged(lq, fmt, [20, 2, 1, 40], [9, 0, 33, 100], 4, 2, 128, 16, cuda_dev, seed=2)
    table = P.table.copy()
    table[2, :] = -1
    table[3, 2:5] = P.pages  # beyond the pool
    table[3, 0] = -5
    o = _check(lq, P, route=route, table=table)
    assert np.all(o[:11] == 0) and np.all(o[20:23] == 0)
    _check(lq, P, route=route, table=table, window=17, sinks=3)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [0, 50])
def test_nothing_leaks_from_invisible_places(lq, cuda_dev, route, fmt, window):
    """Unused slots hold NaN; a NaN in the keys and values of a later token of
    the chunk reaches only the rows that see that token."""
    P = Paged(lq, fmt, [30, 1, 6], [100, 33, 6], 4, 2, 128, 16, cuda_dev, seed=6, fill="nan")
    _check(lq, P, route=route, window=window, sinks=2)
    k, v = [P.values(0, i) for i in range(3)], [P.values(1, i) for i in range(3)]
    cache = P.cache()

    def poison(pool, i, p, h, e):
        head = pool.view(P.pages, P.kv_heads, -1)[int(P.table[i, p // P.page]), h]
        slot = p % P.page
        if fmt == "f16":
            head[slot * 256 + 2 * e: slot * 256 + 2 * e + 2] = torch.tensor([0, 0x7E], dtype=torch.uint8, device=P.dev)
        else:
            at = P.page * P.row + slot * 8 + (e // 32) * 2
            head[at:at + 2] = torch.tensor([0, 0x7E], dtype=torch.uint8, device=P.dev)
    for which, i, p, h, e in ((1, 0, 90, 1, 70), (0, 2, 3, 0, 5), (1, 1, 20, 0, 0)):
        poison((cache.k, cache.v)[which], i, p, h, e)
        x = (k, v)[which][i]
        if fmt == "f16":
            x[p, h, e] = np.nan
        else:
            x[p, h, e // 32 * 32: e // 32 * 32 + 32] = np.nan
    P.cache = lambda: cache
    o, _ = _run(lq, P, route=route, window=window, sinks=2)
    with np.errstate(invalid="ignore"):
        want, tol, _, _ = P.expect(window=window, sinks=2, kv=(k, v))
    assert np.isnan(want).any() and not np.isnan(want).all()
    assert np.array_equal(np.isnan(o), np.isnan(want))
    compare(o, want, np.nan_to_num(tol), "output")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
def test_values_of_any_size(lq, cuda_dev, route, fmt):
    """Small and large keys, values and queries (the operands are split in two
    parts: no size may lose the second part), peaked and flat logits."""
    for sk, sv, sq in ((1e-3, 1e-4, 1e3), (30.0, 1e3, 0.02), (1.0, 1e-2, 6.0), (200.0, 1.0, 1e-4)):
        P = Paged(lq, fmt, [1, 20], [150, 70], 4, 2, 128, 16, cuda_dev, seed=11, scale_k=sk)
        P.v = [x * np.float32(sv) for x in P.v]
        for i in range(2):
            P.store(1, i, P.v[i])
        P.q = (P.q * np.float32(sq)).astype(np.float32)
        o = _check(lq, P, route=route)
        want = P.expect()[0]
        assert np.linalg.norm(o - want) <= 2e-5 * np.linalg.norm(want)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
def test_special_queries(lq, cuda_dev, route, fmt):
    """Zero queries average the values; a NaN or infinity in a query makes its
    own row NaN and no other."""
    P = Paged(lq, fmt, [3], [77], 2, 1, 128, 16, cuda_dev, seed=12)
    P.q[0, 0] = 0
    P.q[1, 1, 5] = np.nan
    o, _ = _run(lq, P, route=route)
    bad = np.zeros((3, 2), bool)
    bad[1, 1] = True
    assert np.array_equal(np.isnan(o).all(-1), bad) and np.array_equal(np.isnan(o).any(-1), bad)
    P.q[1, 1] = 0
    want, tol, _, _ = P.expect()
    o[1, 1] = want[1, 1]
    compare(o, want, tol, "rows beside a NaN query")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals", [([1], [5000]), ([1, 1, 1], [9000, 17, 2000]), ([40], [3000])])
def test_long_contexts_split_over_the_gpu(lq, cuda_dev, fmt, news, totals):
    P = Paged(lq, fmt, news, totals, 4, 2, 128, 16, cuda_dev, seed=9)
    _check(lq, P)
    _check(lq, P, window=2500, sinks=4)


def test_strided_rows_other_streams_graphs_and_repeats(lq, cuda_dev):
    """Q and O as column ranges of wider matrices, a call on a side stream, a
    captured call replayed; the result is the same bits every time."""
    for fmt, news, totals in (("q8_0", [1, 1], [900, 3000]), ("f16", [50, 7], [500, 7])):
        P = Paged(lq, fmt, news, totals, 8, 2, 128, 16, cuda_dev, seed=1)
        cache, batch = P.cache(), P.batch()
        work = lq.attn_work(cache, batch, 8)
        Q = torch.from_numpy(P.q).to(cuda_dev)
        O = torch.empty_like(Q)
        lq.lq_attn_paged(cache, batch, Q, O, 0.1, work=work)
        want, tol, _, _ = P.expect(scale=0.1)
        compare(O.cpu().numpy(), want, tol)
        for pad in (0, 1, 8):
            wide = torch.zeros(P.tokens, 8 * 128 + 300 + pad, device=cuda_dev)
            wide[:, pad:pad + 1024] = Q.flatten(1)
            out = torch.full((P.tokens, 8 * 128 + 5 + pad), -7.0, device=cuda_dev)
            lq.lq_attn_paged(cache, batch, wide[:, pad:pad + 1024], out[:, pad:pad + 1024], 0.1, work=work)
            assert torch.equal(out[:, pad:pad + 1024], O.flatten(1))
            assert bool((out[:, :pad] == -7).all()) and bool((out[:, pad + 1024:] == -7).all())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        O2 = torch.empty_like(Q)
        side.wait_stream(torch.cuda.current_stream())
        lq.lq_attn_paged(cache, batch, Q, O2, 0.1, work=work, stream=side)
        side.synchronize()
        assert torch.equal(O, O2)
        O3 = torch.empty_like(Q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lq.lq_attn_paged(cache, batch, Q, O3, 0.1, work=work)
        for _ in range(20):
            O3.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(O, O3)


def test_lse_joins_two_parts_of_a_context(lq, cuda_dev):
    """Attention over [0, n) from two caches that hold the two halves."""
    P = Paged(lq, "f16", [1, 1], [200, 200], 4, 2, 64, 16, cuda_dev, seed=21)
    whole, lw = _run(lq, P)
    left, right = P.table.copy(), P.table.copy()
    left[:, 6:] = -1
    right[:, :6] = -1
    (a, la), (b, lb) = _run(lq, P, table=left), _run(lq, P, table=right)
    la, lb = la.astype(np.float64), lb.astype(np.float64)
    lse = np.logaddexp(la, lb)
    joined = a * np.exp(la - lse)[..., None] + b * np.exp(lb - lse)[..., None]
    _, tol, _, ltol = P.expect()
    compare(joined, whole.astype(np.float64), 3 * tol)
    compare(lse, lw.astype(np.float64), 3 * ltol)


def test_layer_of_a_decoder(lq, cuda_dev):
    """The operators as a decoder uses them: fused QKV projection, cache
    write, attention, output projection with the residual added."""
    import oracle as O
    import synthetic
    E, heads, kv_heads, d, page = 512, 4, 2, 64, 16
    wide = (heads + 2 * kv_heads) * d
    Wqkv, X = synthetic.draw(23, wide, E, seed=1)
    Wo, _ = synthetic.draw(1, E, heads * d, seed=2)
    up = lambda W: torch.from_numpy(lq.pack("q8_0", W).reshape(-1)).to(cuda_dev)  # noqa: E731
    wqkv, wo = up(Wqkv.numpy()), up(Wo.numpy())
    cache = lq.KVCache("q8_0", 4, page, kv_heads, d, device=cuda_dev)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=cuda_dev)
    out, at = [], 0
    for n in (20, 1, 1, 1):  # a prompt, then three single tokens
        x = X[at:at + n].to(cuda_dev)
        at += n
        batch = lq.KVBatch(table, torch.tensor([at], dtype=torch.int32, device=cuda_dev),
                           torch.tensor([0, n], dtype=torch.int32, device=cuda_dev), n, max_q=n)
        qkv = lq.matmul("q8_0", x, wqkv, wide, E)
        q, k, v = qkv[:, :heads * d], qkv[:, heads * d:(heads + kv_heads) * d], qkv[:, (heads + kv_heads) * d:]
        lq.lq_kv_write(cache, batch, k, v)
        o = torch.empty(n, heads * d, device=cuda_dev)
        lq.lq_attn_paged(cache, batch, q, o, d ** -0.5, heads=heads)
        y = torch.empty_like(x)
        lq.lq_matmul_residual("q8_0", o, wo, x, y, n, E, heads * d)
        out.append((qkv.cpu().numpy(), o.cpu().numpy(), y.cpu().numpy()))
    # every stage against the oracle on the previous stage's own output
    qkv = np.concatenate([s[0] for s in out])
    o = np.concatenate([s[1] for s in out])
    k = A.cache_values("q8_0", qkv[:, heads * d:(heads + kv_heads) * d].reshape(-1, d)).reshape(-1, kv_heads, d)
    v = A.cache_values("q8_0", qkv[:, (heads + kv_heads) * d:].reshape(-1, d)).reshape(-1, kv_heads, d)
    for t in range(23):
        for h in range(heads):
            want, _, bound, logit = A.attend(qkv[t, h * d:(h + 1) * d], k[:, h // 2], v[:, h // 2], np.arange(23) <= t, d ** -0.5)
            compare(o[t, h * d:(h + 1) * d], want, A.tolerance(bound, logit, d))
    y = np.concatenate([s[2] for s in out])
    ref, tol = O.reference("q8_0", o, O.pack("q8_0", Wo.numpy()), E, heads * d, tensor_core=True)
    compare(y, ref + X.numpy()[:23], tol + 1e-6)


@pytest.mark.parametrize("route", (WARP, TILE))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals,heads,kv_heads,page,window,sinks", [
    ([300], [300], 2, 2, 16, 0, 0), ([129, 1, 64], [700, 50, 64], 4, 1, 32, 0, 0), ([128], [1000], 1, 1, 64, 0, 0),
    ([200, 3], [900, 33], 2, 1, 16, 150, 5), ([33], [2000], 8, 2, 128, 0, 0), ([100] * 5, [100, 163, 64, 99, 65], 3, 3, 16, 31, 33)])
def test_chunks_of_wide_heads(lq, cuda_dev, route, fmt, news, totals, heads, kv_heads, page, window, sinks):
    """Heads of 256: whole and partial units, units across CTAs, windows."""
    P = Paged(lq, fmt, news, totals, heads, kv_heads, 256, page, cuda_dev, seed=len(news) + page)
    _check(lq, P, route=route, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_heads_missing_keys_and_values_of_no_size(lq, cuda_dev, fmt):
    """Heads of 256 in tiles: pages that are not there, rows before position 0,
    and values that are not finite where only later rows see them."""
    P = Paged(lq, fmt, [20, 140, 90], [9, 400, 100], 2, 1, 256, 16, cuda_dev, seed=4)
    table = P.table.copy()
    table[1, 3] = -1
    table[2, :2] = -1
    _check(lq, P, route=TILE, table=table)
    pool, slot = P.pools[1, P.table[1, 390 // 16], 0], 390 % 16  # dim 200 of position 390, or its block's scale: NaN
    at = slot * P.row + 400 if fmt == "f16" else 16 * P.row + slot * 16 + 200 // 32 * 2
    pool[at:at + 2] = (0, 0x7E)
    o, _ = _run(lq, P, route=TILE)
    o = o[P.q_start[1]:P.q_start[2]]
    late = np.arange(140) + 260 >= 390
    block = np.zeros(256, dtype=bool)  # what the cache loses with it
    block[slice(200, 201) if fmt == "f16" else slice(192, 224)] = True
    assert np.isfinite(o[~late]).all() and np.isfinite(o[late][:, :, ~block]).all()
    assert np.isnan(o[late][:, :, block]).all()
    assert lq.last_device_error() == lq.LQ_OK


@pytest.mark.parametrize("args", [["--batch", "3", "--prompt", "90", "--steps", "4", "--embed", "512", "--heads", "8", "--kv-heads", "2"],
                                  ["--fmt", "q4_0", "--cache", "f16", "--batch", "1", "--prompt", "40", "--steps", "3", "--embed",
                                   "256", "--heads", "4", "--kv-heads", "4", "--head-dim", "64", "--window", "16", "--sinks", "2"]])
def test_example_of_an_attention_block(args):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "attention_block.py"), *args], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
