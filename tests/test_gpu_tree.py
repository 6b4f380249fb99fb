"""Trees of drafted tokens: lq_tree_plan, lq_attn_tree, lq_tree_accept and
lq_kv_keep against plain walks and the float64 formula. The attention's
tolerances are the oracle's (oracle/attention.py); all else is exact."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from tree_helpers import ancestor_bits, chain, expect_tree, random_parents, to_gpu, words_of

pytestmark = pytest.mark.gpu

FMTS = ("f16", "q8_0", "q4_0")
AUTO, GENERIC, WARP, TILE = range(4)
ROUTES = (AUTO, GENERIC, WARP, TILE)


def _attend(lq, P, mask, positions, route=AUTO, window=0, sinks=0, table=None, max_q=0, cache=None):
    cache, batch = cache or P.cache(), P.batch(max_q=max_q, table=table)
    Q = torch.from_numpy(P.q).to(P.dev)
    O = torch.full_like(Q, float("nan"))
    lse = torch.full((P.tokens, P.heads), float("nan"), device=P.dev)
    lq.attn_route(route)
    try:
        lq.lq_attn_tree(cache, batch, to_gpu(mask, P.dev), Q, O, 1.0 / np.sqrt(P.d),
                        positions=None if positions is None else to_gpu(positions, P.dev), window=window, sinks=sinks, lse=lse,
                        work=lq.attn_work(cache, batch, P.heads))
    except lq.LQError as e:
        if route in (WARP, TILE) and e.status == lq.LQ_ERR_UNSUPPORTED:
            pytest.skip("the forced kernel does not take this geometry")
        raise
    finally:
        lq.attn_route(AUTO)
    torch.cuda.synchronize()
    assert lq.last_device_error() == lq.LQ_OK
    return O.cpu().numpy(), lse.cpu().numpy()


def _trees(P, rng, roots=0.0):
    """(bits, positions) of a random tree in every sequence."""
    bits, positions = [], []
    for n, total in zip(P.news, P.totals):
        b, depth = ancestor_bits(random_parents(rng, n, roots))
        bits.append(b)
        positions.append(total - n + depth)
    return bits, np.concatenate(positions)


def _mask(P, bits, words=None):
    words = max(1, -(-max(P.news) // 32)) if words is None else words
    return np.concatenate([words_of(b, words) for b in bits])


GEOMETRIES = [
    ([5, 1, 0, 9], [40, 1, 13, 9], 128, 4, 2, 16),   # a sequence of nothing else, one without rows
    ([61], [200], 64, 6, 3, 16), ([33, 2], [33, 150], 256, 2, 1, 16),
    ([140, 3], [300, 70], 128, 4, 4, 32),            # five words a row
    ([64, 65, 1], [129, 300, 128], 128, 8, 1, 64),   # groups of eight
    ([100], [333], 256, 4, 2, 16),
    ([7, 12], [90, 41], 96, 4, 2, 16), ([9], [60], 128, 4, 2, 7), ([3], [40], 32, 2, 1, 48)]  # the generic kernel's


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals,d,heads,kv_heads,page", GEOMETRIES)
def test_trees(lq, cuda_dev, route, fmt, news, totals, d, heads, kv_heads, page):
    P = Paged(lq, fmt, news, totals, heads, kv_heads, d, page, cuda_dev, seed=sum(totals), fill="nan")
    bits, positions = _trees(P, np.random.default_rng(d + sum(news)), roots=0.1)
    o, lse = _attend(lq, P, _mask(P, bits), None, route=route)
    want, tol, wl, ltol = expect_tree(P, bits, positions)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (37, 1), (129, 150), (1000, 4), (64, 0)])
def test_window_and_sinks(lq, cuda_dev, route, fmt, window, sinks):
    """The cached part goes by the rows' positions, the new tokens by the bits."""
    P = Paged(lq, fmt, [1, 40, 70], [400, 400, 130], 4, 2, 128, 16, cuda_dev, seed=window)
    bits, positions = _trees(P, np.random.default_rng(window))
    o, lse = _attend(lq, P, _mask(P, bits), positions, route=route, window=window, sinks=sinks)
    want, tol, wl, ltol = expect_tree(P, bits, positions, window, sinks)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("words", [1, 2, 5])
def test_any_bits(lq, cuda_dev, route, fmt, words):
    """Bits of rows ahead, of none at all, of all; rows past the words' bits and
    bits past the rows; positions outside the sequence are taken as its ends."""
    P = Paged(lq, fmt, [40, 70, 1], [40, 300, 1], 4, 2, 128, 16, cuda_dev, seed=words)
    rng = np.random.default_rng(words)
    bits = [rng.random((n, n)) < 0.4 for n in P.news]
    for b in bits:
        b[len(b) // 2] = False
        b[-1] = len(b) > 1
    m = _mask(P, bits, words)
    if words * 32 > 70:
        m[:, -1] |= np.int32(-(1 << 31))  # a bit of no row
    for b in bits:
        b[:, words * 32:] = False
    positions = rng.integers(-1000, 1000, P.tokens)
    o, lse = _attend(lq, P, m, positions, route=route, window=50, sinks=3)
    want, tol, wl, ltol = expect_tree(P, bits, positions, 50, 3)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")
    assert (o[-1] == 0).all() and np.isneginf(lse[-1]).all()  # one row alone that does not see itself


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [1, 40])
def test_nan_in_rows_that_are_not_seen(lq, cuda_dev, route, fmt, rows):
    """A drafted token of NaN reaches the rows that see it and no others."""
    P = Paged(lq, fmt, [rows, 3], [rows + 61, 50], 4, 2, 128, 16, cuda_dev, seed=rows)
    rng = np.random.default_rng(rows)
    bits, positions = _trees(P, rng)
    if rows == 1:
        bits[0][0, 0] = False
    bad = rows // 2
    kv = [[P.values(w, i).copy() for i in range(2)] for w in (0, 1)]
    for w in (0, 1):
        kv[w][0][61 + bad] = np.nan
        for h in range(P.kv_heads):  # all ones: NaN as values and as scales
            at = P.pools[w, P.table[0, (61 + bad) // 16], h]
            slot = (61 + bad) % 16
            at[slot * P.row:(slot + 1) * P.row] = 0xFF
            if fmt != "f16":
                s = 16 * P.row + slot * (P.d // 16)
                at[s:s + P.d // 16] = 0xFF
    o, _ = _attend(lq, P, _mask(P, bits), None, route=route)
    want, tol, _, _ = expect_tree(P, bits, positions, kv=kv)
    assert np.isnan(want).any() == (rows > 1) and not np.isnan(want).all()
    compare(o, want, tol, "output")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
def test_a_chain_is_the_causal_call(lq, cuda_dev, route, fmt):
    """Rows that follow one another give lq_attn_paged's results."""
    P = Paged(lq, fmt, [50, 1, 12], [200, 77, 12], 8, 2, 128, 16, cuda_dev, seed=3)
    bits, positions = [], []
    for n, total in zip(P.news, P.totals):
        b, depth = ancestor_bits(np.arange(-1, n - 1), 20, 2, total - n)
        bits.append(b)
        positions.append(total - n + depth)
    o, lse = _attend(lq, P, _mask(P, bits), np.concatenate(positions), route=route, window=20, sinks=2)
    want, tol, wl, ltol = P.expect(window=20, sinks=2)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
def test_lengths_below_the_rows(lq, cuda_dev, route, fmt):
    """Caches shorter than the call's rows: the first rows have no slots."""
    P = Paged(lq, fmt, [40, 9, 5, 70], [30, 0, 5, 1], 4, 2, 128, 16, cuda_dev, seed=6)
    rng = np.random.default_rng(3)
    bits = [rng.random((n, n)) < 0.5 for n in P.news]
    positions = rng.integers(0, 40, P.tokens)
    for window, sinks in ((0, 0), (8, 2)):
        o, lse = _attend(lq, P, _mask(P, bits), positions, route=route, window=window, sinks=sinks)
        want, tol, wl, ltol = expect_tree(P, bits, positions, window, sinks)
        compare(o, want, tol, "output")
        compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
def test_pages_that_are_not_there(lq, cuda_dev, route):
    P = Paged(lq, "f16", [20, 30], [200, 130], 4, 2, 128, 16, cuda_dev, seed=8)
    table = P.table.copy()
    table[0, 3] = -1
    table[0, 12] = P.pages + 5  # of the new tokens' pages
    table[1, :] = -1
    bits, positions = _trees(P, np.random.default_rng(1))
    o, lse = _attend(lq, P, _mask(P, bits), None, route=route, table=table)
    want, tol, wl, ltol = expect_tree(P, bits, positions, table=table)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("news,max_q,kernels", [
    ([2, 90, 5], 90, (0, 1)), ([2, 90, 5], 0, (0, 1)), ([20, 5, 9], 20, (1, 0)), ([20, 5, 9], 1, (1, 0)), ([1], 1, (1, 0)),
    ([2] * 9 + [120], 120, (1, 1)), ([2] * 9 + [120], 0, (1, 1)), ([2] * 9 + [120], 7, (1, 0))])
def test_routes_by_the_rows(lq, cuda_dev, news, max_q, kernels):
    """Trees go to one kernel by their mean, unless some are far from it; max_q
    steers, results stay."""
    P = Paged(lq, "q8_0", news, [n + 37 * (i + 3) for i, n in enumerate(news)], 8, 2, 128, 16, cuda_dev, seed=5)
    bits, positions = _trees(P, np.random.default_rng(2))
    want, tol, _, _ = expect_tree(P, bits, positions)
    lq.reset_counts()
    o, _ = _attend(lq, P, _mask(P, bits), None, max_q=max_q)
    assert (lq.route_count(9), lq.route_count(10)) == kernels
    compare(o, want, tol, "output")


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("news,totals,page", [([40, 9], [300, 200], 16), ([17, 33, 1], [17, 900, 5], 64), ([130], [5000], 128)])
def test_wide_heads_of_quantised_caches(lq, cuda_dev, fmt, news, totals, page):
    """Heads of 256 with more than 32 rows: two row groups a tile of keys."""
    P = Paged(lq, fmt, news, totals, 4, 1, 256, page, cuda_dev, seed=sum(news), fill="nan")
    bits, positions = _trees(P, np.random.default_rng(4), roots=0.05)
    for window, sinks in ((0, 0), (50, 3)):
        o, lse = _attend(lq, P, _mask(P, bits), positions, route=WARP, window=window, sinks=sinks, max_q=max(news))
        want, tol, wl, ltol = expect_tree(P, bits, positions, window, sinks)
        compare(o, want, tol, "output")
        compare(lse, wl, ltol, "lse")


# ---- plan ---------------------------------------------------------------------
def _int_batch(lq, news, totals, dev, q_start=None, tokens=None):
    q_start = np.concatenate([[0], np.cumsum(news)]) if q_start is None else q_start
    return lq.KVBatch(torch.zeros(len(totals), 1, dtype=torch.int32, device=dev), to_gpu(totals, dev), to_gpu(q_start, dev),
                      int(q_start[-1]) if tokens is None else tokens)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 7), (1, 0), (3, 0), (5, 103), (40, 2)])
@pytest.mark.parametrize("news,words", [([1], 1), ([0, 5, 32, 0], 1), ([33, 64, 65, 7], 3), ([200, 31], 2), ([700, 300], 22)])
def test_plan(lq, cuda_dev, news, words, window, sinks):
    """Random forests, and parents that are none: ahead, itself, far below zero."""
    rng = np.random.default_rng(sum(news) + window)
    totals = [n + 100 for n in news]
    parents = [random_parents(rng, n, 0.05, reach=40) for n in news]
    for p in parents:
        if len(p) > 4:
            p[3], p[4] = 3, 2**31 - 1
            p[2] = -2**31
    batch = _int_batch(lq, news, totals, cuda_dev)
    t = sum(news)
    pos = torch.full((t,), -7, dtype=torch.int32, device=cuda_dev)
    mask = torch.full((t, words), -7, dtype=torch.int32, device=cuda_dev)
    parent = to_gpu(np.concatenate(parents), cuda_dev)
    lq.lq_tree_plan(batch, parent, pos, mask, window=window, sinks=sinks)
    want = [ancestor_bits(p, window, sinks, 100) for p in parents]
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([words_of(b, words) for b, _ in want]))
    assert np.array_equal(pos.cpu().numpy(), np.concatenate([100 + d for _, d in want]))
    alone = torch.full_like(pos, -7)
    lq.lq_tree_plan(batch, parent, alone, window=window)
    assert torch.equal(alone, pos)
    again = torch.full_like(mask, -7)
    lq.lq_tree_plan(batch, parent, None, again, window=window, sinks=sinks)
    assert torch.equal(again, mask)


def test_plan_leaves_rows_of_no_sequence(lq, cuda_dev):
    """Rows before the first and behind the last sequence."""
    batch = _int_batch(lq, None, [50, 60], cuda_dev, q_start=np.array([2, 5, 6]), tokens=9)
    pos, mask = (torch.full(s, -7, dtype=torch.int32, device=cuda_dev) for s in ((9,), (9, 1)))
    lq.lq_tree_plan(batch, to_gpu([-1, -1, -1, 0, 0, -1, -1, -1, -1], cuda_dev), pos, mask)
    assert pos.tolist() == [-7, -7, 47, 48, 48, 59, -7, -7, -7]
    assert mask[:, 0].tolist() == [-7, -7, 1, 3, 5, 1, -7, -7, -7]


# ---- accept -------------------------------------------------------------------
def _accept(parent, token, target, most):
    """The path by its definition."""
    if len(parent) == 0:
        return [], -1
    path = [0]
    while len(path) < most:
        after = [r for r in range(path[-1] + 1, len(parent)) if parent[r] == path[-1] and token[r] == target[path[-1]]]
        if not after:
            break
        path.append(after[0])
    return path, int(target[path[-1]])


@pytest.mark.parametrize("most", [1, 4, 40])
@pytest.mark.parametrize("news,choices", [([1], 3), ([0, 5, 32, 0, 33], 2), ([100, 64, 7], 2), ([700], 1), ([40] * 70, 3)])
def test_accept(lq, cuda_dev, news, choices, most):
    """Few different tokens, so that paths are long and siblings agree."""
    rng = np.random.default_rng(sum(news) + most)
    totals = [n + 10 * i for i, n in enumerate(news)]
    parents = [random_parents(rng, n, 0.05, reach=20) for n in news]
    t, b = sum(news), len(news)
    token, target = (rng.integers(0, choices, t).astype(np.int32) for _ in range(2))
    batch = _int_batch(lq, news, totals, cuda_dev)
    keep = torch.full((b, most), -7, dtype=torch.int32, device=cuda_dev)
    count, after, length = (torch.full((b,), -7, dtype=torch.int32, device=cuda_dev) for _ in range(3))
    lq.lq_tree_accept(batch, to_gpu(np.concatenate(parents), cuda_dev), to_gpu(token, cuda_dev), to_gpu(target, cuda_dev), keep, count, after,
                      length)
    at, longest = 0, 0
    for i, n in enumerate(news):
        path, last = _accept(parents[i], token[at:at + n], target[at:at + n], most)
        longest = max(longest, len(path))
        assert keep[i].tolist() == path + [-1] * (most - len(path))
        assert (count[i].item(), after[i].item(), length[i].item()) == (len(path), last, totals[i] - n + len(path))
        at += n
    assert longest > 1 or most == 1 or max(news) == 1


# ---- keep ---------------------------------------------------------------------
def _kept(P, keep, count):
    """The pools after the moves, token by token."""
    pools = P.pools.copy()
    for i, (n, total) in enumerate(zip(P.news, P.totals)):
        last = -1
        for k in range(min(count[i], keep.shape[1], n)):
            r = int(keep[i, k])
            if not last < r < n:
                break
            last = r
            p, q = total - n + r, total - n + k
            src, dst = P.table[i, p // P.page], P.table[i, q // P.page]
            if min(src, dst) < 0 or max(src, dst) >= P.pages or q < 0:
                continue
            s, e, w = p % P.page, q % P.page, P.d // 16
            pools[:, dst, :, e * P.row:(e + 1) * P.row] = pools[:, src, :, s * P.row:(s + 1) * P.row]
            if P.fmt != "f16":
                o = P.page * P.row
                pools[:, dst, :, o + e * w:o + (e + 1) * w] = pools[:, src, :, o + s * w:o + (s + 1) * w]
    return pools


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,totals,d,kv_heads,page", [
    ([9, 1, 0, 61], [40, 7, 13, 200], 128, 8, 16), ([300], [301], 64, 3, 16), ([33, 20], [33, 90], 256, 2, 64),
    ([50], [90], 96, 1, 5), ([40, 40], [77, 41], 32, 2, 1)])
def test_keep(lq, cuda_dev, fmt, news, totals, d, kv_heads, page):
    """Paths of all lengths, the identity and lists that stop ascending."""
    P = Paged(lq, fmt, news, totals, kv_heads, kv_heads, d, page, cuda_dev, seed=d)
    rng = np.random.default_rng(page)
    most = max(max(news), 16)
    for kind in ("path", "all", "torn", "none"):
        keep, count = np.full((len(news), most), -1, dtype=np.int32), np.zeros(len(news), dtype=np.int32)
        for i, n in enumerate(news):
            m = n if kind == "all" else int(rng.integers(0, n + 1)) if kind != "none" else 0
            keep[i, :m] = np.sort(rng.permutation(n)[:m])
            count[i] = m
            if kind == "torn" and m > 2:
                keep[i, m // 2] = [keep[i, 0], -1, n, 2**31 - 1][i % 4]
                count[i] = most + 5
        cache, batch = P.cache(), P.batch()
        lq.lq_kv_keep(cache, batch, to_gpu(keep, cuda_dev), to_gpu(count, cuda_dev))
        want = _kept(P, keep, count)
        assert np.array_equal(cache.k.cpu().numpy(), want[0]) and np.array_equal(cache.v.cpu().numpy(), want[1]), kind


def test_keep_without_pages_and_unaligned_pools(lq, cuda_dev):
    P = Paged(lq, "q8_0", [30, 30], [70, 64], 2, 2, 64, 16, cuda_dev, seed=1)
    P.table[0, 3] = -1
    P.table[1, 2] = P.pages
    keep = np.tile(np.arange(1, 26, dtype=np.int32), (2, 1))
    want = _kept(P, keep, np.array([25, 25]))
    flat = [torch.zeros(P.pools[w].size + 2, dtype=torch.uint8, device=cuda_dev) for w in (0, 1)]
    for w in (0, 1):
        flat[w][2:] = torch.from_numpy(P.pools[w].reshape(-1)).to(cuda_dev)
    cache = lq.KVCache("q8_0", P.pages, P.page, 2, 64, k=flat[0][2:], v=flat[1][2:])
    lq.lq_kv_keep(cache, P.batch(), to_gpu(keep, cuda_dev), to_gpu([25, 25], cuda_dev))
    for w in (0, 1):
        assert np.array_equal(flat[w][2:].cpu().numpy(), want[w].reshape(-1)) and not flat[w][:2].any()


# ---- a step as it is used -------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
def test_a_drafted_step_is_the_step_token_by_token(lq, cuda_dev, fmt):
    """Plan, positions, write, attention, acceptance and moving up, replayed as a
    graph, against the accepted tokens decoded alone into a cache of their own."""
    rng = np.random.default_rng(7)
    b, n, heads, kv_heads, d, page = 3, 13, 4, 2, 64, 16
    lens = np.array([37, 16, 5])
    rope = lq.Rope(d, base=1e4)
    parents = np.stack([random_parents(rng, n) for _ in range(b)])
    token, target = rng.integers(0, 2, (b, n)), rng.integers(0, 2, (b, n))
    q = rng.standard_normal((b * n, heads, d)).astype(np.float32)
    k, v = (rng.standard_normal((b * n, kv_heads, d)).astype(np.float32) for _ in range(2))
    pages = 6 * b
    table = to_gpu(rng.permutation(pages).reshape(b, 6), cuda_dev)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_dev)  # noqa: E731
    prompt = [up(rng.standard_normal((int(lens.sum()), kv_heads, d)).astype(np.float32)) for _ in range(2)]
    caches = []
    for _ in range(2):
        cache = lq.KVCache(fmt, pages, page, kv_heads, d)
        start = lq.KVBatch(table, to_gpu(lens, cuda_dev), to_gpu(np.concatenate([[0], np.cumsum(lens)]), cuda_dev), int(lens.sum()))
        lq.lq_kv_write(cache, start, *prompt)
        caches.append(cache)
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    kv_len = to_gpu(lens + n, cuda_dev)
    batch = lq.KVBatch(table, kv_len, to_gpu(np.arange(b + 1) * n, cuda_dev), b * n, max_q=n)
    parent, tok, tgt = (to_gpu(x.reshape(-1), cuda_dev) for x in (parents, token, target))
    pos, mask, keep, count, after, length = ints(b * n), ints(b * n, 1), ints(b, 8), ints(b), ints(b), ints(b)
    Q, K, V = up(q), up(k), up(v)
    qr, kr, O = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(Q)
    work = lq.attn_work(caches[0], batch, heads)

    def step():
        lq.lq_tree_plan(batch, parent, pos, mask)
        lq.lq_rope(rope, pos, Q, K, q_out=qr, k_out=kr)
        lq.lq_kv_write(caches[0], batch, kr, V)
        lq.lq_attn_tree(caches[0], batch, mask, qr, O, d**-0.5, work=work)
        lq.lq_tree_accept(batch, parent, tok, tgt, keep, count, after, length)
        lq.lq_kv_keep(caches[0], batch, keep, count)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    O.fill_(float("nan"))
    graph.replay()  # (writes the rows again before it moves them)
    torch.cuda.synchronize()
    got, paths = O.cpu().numpy(), keep.cpu().numpy()
    assert count.cpu().numpy().max() > 1
    # the accepted tokens one after another
    for i in range(b):
        for m in range(int(count[i])):
            r = i * n + int(paths[i, m])
            one = lq.KVBatch(table[i:i + 1].contiguous(), to_gpu([lens[i] + m + 1], cuda_dev), to_gpu([0, 1], cuda_dev), 1, max_q=1)
            at = to_gpu([lens[i] + m], cuda_dev)
            assert pos[r].item() == lens[i] + m
            q1, k1, o1 = Q[r:r + 1].clone(), K[r:r + 1].clone(), torch.empty_like(Q[:1])
            lq.lq_rope(rope, at, q1, k1)
            lq.lq_kv_write(caches[1], one, k1, V[r:r + 1])
            lq.lq_attn_paged(caches[1], one, q1, o1, d**-0.5)
            want = o1.cpu().numpy()[0].astype(np.float64)
            # (two results of the attention: twice its documented 2e-5 of a row)
            assert np.linalg.norm(got[r] - want) <= 4e-5 * np.linalg.norm(want)
        end = int(length[i])
        assert end == lens[i] + int(count[i])
        whole = lq.KVBatch(table[i:i + 1].contiguous(), to_gpu([end], cuda_dev), to_gpu([0, end], cuda_dev), end)
        kept = [torch.empty(end, kv_heads, d, device=cuda_dev) for _ in range(4)]
        lq.lq_kv_read(caches[0], whole, kept[0], kept[1])
        lq.lq_kv_read(caches[1], whole, kept[2], kept[3])
        assert torch.equal(kept[0], kept[2]) and torch.equal(kept[1], kept[3])
    assert chain(parents[0], 0) == [0]
