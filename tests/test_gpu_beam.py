"""Beam search: lq_beam_select, lq_beam_pages and lq_kv_copy against plain
computations in 64 bits, and a search as it is used.

Tolerance of a score: its rounding to float32, 2^-24 of itself; and the error of
log sum exp: each term 2^-22 (ex2) and 2^-22 of its exponent's size (two roundings
of at most 2^-24 of |y| <= 40, weighed by 2^-|y|: below 2^-23), a rescaling of 2^-22 a
round, and additions of 2^-24 each, 8 in a round, 20 in the tree: less than
2^-18 for vocabularies of up to 64 rounds a part."""
import numpy as np
import pytest
import torch

from tree_helpers import to_gpu

pytestmark = pytest.mark.gpu


def _scores(logits, scores, finished=None, pad=0):
    """Every continuation's score in float64 [rows, vocab]; -inf: never chosen."""
    x = logits.astype(np.float64)
    with np.errstate(all="ignore"):
        top = x.max(1, keepdims=True)  # (taken off first: 2.5e38 + log(30000) is 2.5e38 in 64 bits)
        s = scores.astype(np.float64)[:, None] + ((x - top) - np.log(np.exp(x - top).sum(1, keepdims=True)))
    s[np.isnan(s)] = -np.inf
    s[np.isneginf(scores) | np.isnan(scores)] = -np.inf
    if finished is not None:
        for r in np.nonzero(finished)[0]:
            s[r] = -np.inf
            s[r, pad] = scores[r] if not np.isnan(scores[r]) else -np.inf
    return s


def _best(s, beams, k):
    """(scores, parents, tokens) [groups, k] by a stable order of all candidates."""
    groups, v = s.shape[0] // beams, s.shape[1]
    flat = s.reshape(groups, beams * v)
    out = np.full((groups, k), -np.inf), np.full((groups, k), -1), np.full((groups, k), -1)
    for g in range(groups):
        at = np.argsort(-flat[g], kind="stable")[:k]
        at = at[flat[g][at] > -np.inf]
        out[0][g, :len(at)], out[1][g, :len(at)], out[2][g, :len(at)] = flat[g][at], at // v, at % v
    return out


def _select(lq, dev, logits, scores, beams, k, finished=None, pad=0, buffers=None, ld=None, offset=0):
    n, v = logits.shape
    ld = v if ld is None else ld
    room = torch.full((n * ld + offset,), float("nan"), device=dev)
    x = room[offset:].as_strided((n, v), (ld, 1))
    x.copy_(torch.from_numpy(logits))
    out_s, out_p, out_t, work = buffers or lq.beam_buffers(n // beams, beams, v, k)
    out_s.fill_(float("nan"))
    out_p.fill_(-9)
    out_t.fill_(-9)
    lq.lq_beam_select(x, torch.from_numpy(scores).to(dev), beams, k, out_s, out_p, out_t, work,
                      finished=None if finished is None else to_gpu(finished, dev), pad=pad)
    torch.cuda.synchronize()
    assert lq.last_device_error() == lq.LQ_OK
    return out_s.cpu().numpy(), out_p.cpu().numpy(), out_t.cpu().numpy()


def _check(got, want):
    s, p, t = got
    ws, wp, wt = want
    assert np.array_equal(p, wp) and np.array_equal(t, wt), f"differs at {np.argwhere((p != wp) | (t != wt))[0]}"
    fine = np.isfinite(ws)
    assert np.array_equal(fine, np.isfinite(s)) and np.array_equal(ws[~fine].astype(np.float32), s[~fine])
    assert (np.abs(s[fine] - ws[fine]) <= 2.0**-24 * np.abs(ws[fine]) + 2.0**-18).all()


@pytest.mark.parametrize("coarse", [False, True])
@pytest.mark.parametrize("groups,beams,vocab,k", [
    (1, 1, 1, 1), (3, 2, 5, 4), (1, 4, 151936, 8), (5, 3, 4095, 6), (2, 8, 4096, 16), (7, 1, 4097, 64), (1, 64, 1000, 64), (2, 16, 20001, 32),
    (40, 4, 33000, 8), (300, 3, 777, 5), (1, 2, 2**20 + 3, 4), (3, 5, 12289, 1)])
def test_against_64_bits(lq, cuda_dev, groups, beams, vocab, k, coarse):
    """Random logits; coarse ones are full of ties, which go to the lower token."""
    rng = np.random.default_rng(vocab + k)
    x = (2.5 * rng.standard_normal((groups * beams, vocab))).astype(np.float32)
    if coarse:
        x = np.round(x * 4) / 4
    scores = (-20 * rng.random(groups * beams)).astype(np.float32)
    got = _select(lq, cuda_dev, x, scores, beams, k)
    _check(got, _best(_scores(x, scores), beams, k))


@pytest.mark.parametrize("ld,offset", [(5000, 0), (5003, 0), (5004, 1), (5004, 4)])
def test_strides_and_alignment(lq, cuda_dev, ld, offset):
    rng = np.random.default_rng(ld + offset)
    x = rng.standard_normal((12, 4999)).astype(np.float32)
    scores = -rng.random(12).astype(np.float32)
    _check(_select(lq, cuda_dev, x, scores, 4, 9, ld=ld, offset=offset), _best(_scores(x, scores), 4, 9))


@pytest.mark.parametrize("k", [1, 7, 64])
def test_odd_rows(lq, cuda_dev, k):
    """Rows of one value, of nothing but -inf or the type's lowest, of few values
    among -inf, with NaN or +inf, rising and falling ones; beams that score -inf or
    NaN; a group of them alone."""
    rng = np.random.default_rng(k)
    v, low = 30000, np.finfo(np.float32).min
    x = rng.standard_normal((24, v)).astype(np.float32)
    x[0] = 1.5
    x[1] = -np.inf
    x[2] = low
    x[3] = -np.inf
    x[3, [5, 29999, 77]] = [1.0, 2.0, -1e30]
    x[4, 12345] = np.nan
    x[5, 23456] = np.inf
    x[6] = np.arange(v) / 1000.0
    x[7] = -np.arange(v) / 1000.0
    x[8] = low
    x[8, 4096] = 0.0
    x[9] = 2.5e38
    x[10] = np.where(np.arange(v) % 2, 0.0, -0.0)
    x[11] = -3e38
    x[12:16] = -np.inf
    x[20:24] = np.nan
    scores = -rng.random(24).astype(np.float32)
    scores[17], scores[18] = -np.inf, np.nan
    for beams in (4, 1, 24):
        _check(_select(lq, cuda_dev, x, scores, beams, k), _best(_scores(x, scores), beams, k))


def test_beams_that_are_alike(lq, cuda_dev):
    """Equal rows and scores: the lower beam, then the lower token."""
    rng = np.random.default_rng(5)
    x = np.tile(np.round(rng.standard_normal((1, 9000)) * 8).astype(np.float32) / 8, (8, 1))
    _check(_select(lq, cuda_dev, x, np.full(8, -3.25, np.float32), 8, 64), _best(_scores(x, np.full(8, -3.25, np.float32)), 8, 64))


def test_first_step_and_ended_beams(lq, cuda_dev):
    """One beam alive at first; ended ones stay with the padding token, and their
    logits are not read."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((16, 8000)).astype(np.float32)
    first = np.where(np.arange(16) % 4 == 0, 0.0, -np.inf).astype(np.float32)
    _check(_select(lq, cuda_dev, x, first, 4, 8), _best(_scores(x, first), 4, 8))
    ended = (np.arange(16) % 3 == 0).astype(np.int32) * 7
    ended[12:] = 1
    scores = (-12 * rng.random(16)).astype(np.float32)
    scores[15] = -np.inf
    x[ended != 0] = np.nan
    _check(_select(lq, cuda_dev, x, scores, 4, 8, finished=ended, pad=4321), _best(_scores(np.nan_to_num(x), scores, ended, 4321), 4, 8))


def test_work_is_ready_for_the_next_call(lq, cuda_dev):
    """One buffer, many calls, eager and captured."""
    rng = np.random.default_rng(8)
    buffers = lq.beam_buffers(5, 4, 20000, 8)
    for _ in range(4):
        x, scores = rng.standard_normal((20, 20000)).astype(np.float32), -rng.random(20).astype(np.float32)
        _check(_select(lq, cuda_dev, x, scores, 4, 8, buffers=buffers), _best(_scores(x, scores), 4, 8))
    X, S = torch.from_numpy(x).to(cuda_dev), torch.from_numpy(scores).to(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.lq_beam_select(X, S, 4, 8, *buffers)
    for _ in range(3):
        x, scores = rng.standard_normal((20, 20000)).astype(np.float32), -rng.random(20).astype(np.float32)
        X.copy_(torch.from_numpy(x))
        S.copy_(torch.from_numpy(scores))
        graph.replay()
        _check([b.cpu().numpy() for b in buffers[:3]], _best(_scores(x, scores), 4, 8))


@pytest.mark.parametrize("groups,beams,vocab,k", [(1100, 4, 301, 6), (70, 64, 64, 64), (5000, 1, 4100, 2)])
def test_more_rows_than_are_looked_over(lq, cuda_dev, groups, beams, vocab, k):
    """Beyond 4096 rows the rows that do not count are dealt like the others."""
    rng = np.random.default_rng(groups)
    n = groups * beams
    x = rng.standard_normal((n, vocab)).astype(np.float32)
    scores = (-9 * rng.random(n)).astype(np.float32)
    scores[rng.random(n) < 0.1] = -np.inf
    ended = (rng.random(n) < 0.3).astype(np.int32)
    ended[:3 * beams] = 1
    scores[3 * beams:5 * beams] = -np.inf
    x[ended != 0] = np.nan
    _check(_select(lq, cuda_dev, x, scores, beams, k, finished=ended, pad=vocab - 1),
           _best(_scores(np.nan_to_num(x), scores, ended, vocab - 1), beams, k))


def test_scores_that_are_not_finite(lq, cuda_dev):
    x = np.zeros((5, 100), np.float32)
    x[1, 7] = 2.0
    x[4, 3] = -np.finfo(np.float32).max
    x[4, 5] = np.finfo(np.float32).max
    scores = np.array([np.inf, -1.0, np.nan, np.inf, -2.0], np.float32)
    s, p, t = _select(lq, cuda_dev, x, scores, 5, 3, finished=np.array([0, 0, 1, 1, 0]), pad=0)
    # the last row's 5 has all of its weight: -2; of row 1, log(99 + e^2) = 4.667: 7 gives -3.667, 0 gives -5.667
    assert p.tolist() == [[4, 1, 1]] and t.tolist() == [[5, 7, 0]]


def test_scratch_of_any_content_two_streams(lq, cuda_dev):
    """Nothing is expected of the scratch memory; calls with their own run at once."""
    rng = np.random.default_rng(12)
    data, outs = [], []
    for i in range(2):
        x, scores = rng.standard_normal((32, 50000)).astype(np.float32), -rng.random(32).astype(np.float32)
        data.append((x, scores, torch.from_numpy(x).to(cuda_dev), torch.from_numpy(scores).to(cuda_dev)))
        buffers = lq.beam_buffers(8, 4, 50000, 8)
        buffers[3].fill_(255 - 85 * i)
        outs.append(buffers)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            lq.lq_beam_select(data[i][2], data[i][3], 4, 8, *outs[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        _check([b.cpu().numpy() for b in outs[i][:3]], _best(_scores(data[i][0], data[i][1]), 4, 8))


# ---- pages and copies ------------------------------------------------------------
def _pages(parent, beams, table, lens, page):
    """(tables, copies) by the definition."""
    out, copies = table.copy(), np.tile(np.array([-1, -1, 0], dtype=np.int32), (len(parent), 1))
    for g0 in range(0, len(parent), beams):
        par = [p if 0 <= p < beams else -1 for p in parent[g0:g0 + beams]]
        free = [b for b in range(beams) if b not in par]
        whole, rows = divmod(int(lens[g0]), page)
        for b, p in enumerate(par):
            own = p if p >= 0 and p not in par[:b] else free.pop(0)
            src = own if p < 0 else p
            out[g0 + b, :whole], out[g0 + b, whole:] = table[g0 + src, :whole], table[g0 + own, whole:]
            if src != own and rows and whole < table.shape[1]:
                copies[g0 + b] = table[g0 + src, whole], table[g0 + own, whole], rows
    return out, copies


@pytest.mark.parametrize("beams", [1, 2, 5, 32, 33, 64])
@pytest.mark.parametrize("page,max_pages,length", [(16, 7, 40), (16, 7, 48), (1, 300, 299), (64, 1, 63), (128, 2, 0), (16, 3, 100)])
def test_pages(lq, cuda_dev, beams, page, max_pages, length):
    rng = np.random.default_rng(beams + length)
    groups = 9
    n = groups * beams
    table = rng.permutation(n * max_pages).reshape(n, max_pages).astype(np.int32)
    parent = rng.integers(0, beams, n).astype(np.int32)
    parent[:beams] = 0
    parent[beams:2 * beams] = rng.permutation(beams)
    parent[2 * beams] = -1
    parent[3 * beams - 1] = beams
    parent[3 * beams:4 * beams] = -1
    lens = np.full(n, length, dtype=np.int32)
    lens[4 * beams + 1:5 * beams] = 3  # a group goes by its first beam's length
    out, copies = torch.full((n, max_pages), -7, dtype=torch.int32, device=cuda_dev), torch.full((n, 3), -7, dtype=torch.int32, device=cuda_dev)
    lq.lq_beam_pages(to_gpu(parent, cuda_dev), beams, to_gpu(table, cuda_dev), to_gpu(lens, cuda_dev), page, out, copies)
    want = _pages(parent, beams, table, lens, page)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(copies.cpu().numpy(), want[1])
    real = want[1][want[1][:, 2] > 0]
    assert len(set(real[:, 1])) == len(real) and not set(real[:, 1]) & set(real[:, 0])


@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("kv_heads,d,page,offset", [(8, 128, 16, 0), (1, 256, 128, 0), (3, 96, 5, 0), (2, 64, 16, 2), (2, 32, 1, 0)])
def test_copies(lq, cuda_dev, fmt, kv_heads, d, page, offset):
    """Every count of tokens, pages that are not there, nothing else touched."""
    rng = np.random.default_rng(d + page)
    row = {"f16": 2 * d, "q8_0": d, "q4_0": d // 2}[fmt]
    w = 0 if fmt == "f16" else d // 16
    pages, block = 64, page * (row + w)
    pools = rng.integers(0, 256, (2, pages, kv_heads, block), dtype=np.uint8)
    at = rng.permutation(pages)
    copies = np.stack([at[:24], at[24:48], rng.integers(1, page + 1, 24)], 1).astype(np.int32)
    copies[:6] = [[-1, at[50], 1], [at[50], -1, 1], [pages, at[50], 1], [at[50], 2**31 - 1, 1], [at[51], at[52], 0], [at[51], at[52], -5]]
    copies[6, 2] = page + 1000  # a page's worth
    copies[7] = [at[53], at[53], page]
    want = pools.copy()
    for src, dst, n in copies:
        if 0 <= src < pages and 0 <= dst < pages:
            n = max(0, min(int(n), page))
            want[:, dst, :, :n * row] = want[:, src, :, :n * row]
            want[:, dst, :, page * row:page * row + n * w] = want[:, src, :, page * row:page * row + n * w]
    flat = [torch.from_numpy(np.concatenate([np.zeros(offset, np.uint8), p.reshape(-1)])).to(cuda_dev) for p in pools]
    cache = lq.KVCache(fmt, pages, page, kv_heads, d, k=flat[0][offset:], v=flat[1][offset:])
    lq.lq_kv_copy(cache, to_gpu(copies, cuda_dev))
    torch.cuda.synchronize()
    assert lq.last_device_error() == lq.LQ_OK
    for i in (0, 1):
        assert np.array_equal(flat[i][offset:].cpu().numpy(), want[i].reshape(-1))


@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
def test_a_search_keeps_each_beams_own_past(lq, cuda_dev, fmt):
    """Steps of two searches of four beams: selection, pages, copies, the new
    tokens' write; at the end every beam's cache holds its own tokens' keys, in the
    order of its ancestry. The first beam's score is the sum of its steps'."""
    rng = np.random.default_rng(11)
    groups, beams, vocab, page, kv_heads, d, steps, prompt = 2, 4, 500, 4, 2, 32, 19, 6
    n = groups * beams
    width = -(-(prompt + steps) // page)
    whole = prompt // page
    pages = groups * whole + n * (width - whole)
    order = rng.permutation(pages)
    table = np.empty((n, width), dtype=np.int32)
    for g in range(groups):
        table[g * beams:(g + 1) * beams, :whole] = order[g * whole:(g + 1) * whole]
    table[:, whole:] = order[groups * whole:].reshape(n, width - whole)
    keys = rng.standard_normal((vocab, kv_heads, d)).astype(np.float32)  # a token's key and value
    cache = lq.KVCache(fmt, pages, page, kv_heads, d)
    tables = [to_gpu(table, cuda_dev), to_gpu(table, cuda_dev)]
    copies = torch.empty(n, 3, dtype=torch.int32, device=cuda_dev)
    past = [[int(x) for x in rng.integers(0, vocab, prompt)] for _ in range(groups) for _ in range(1)]
    past = [list(past[r // beams]) for r in range(n)]
    K = torch.from_numpy(keys).to(cuda_dev)

    def write(rows, lens, new):
        """The last `new` tokens of every beam in `past`."""
        x = K[torch.tensor([t for r in rows for t in past[r][lens - new:lens]], device=cuda_dev)]
        q_start = to_gpu(np.arange(len(rows) + 1) * new, cuda_dev)
        lq.lq_kv_write(cache, lq.KVBatch(tables[0][rows].contiguous(), to_gpu([lens] * len(rows), cuda_dev), q_start, len(rows) * new), x, x)

    write(list(range(n)), prompt, prompt)  # (full pages are shared: written with the same tokens)
    scores = torch.from_numpy(np.where(np.arange(n) % beams == 0, 0.0, -np.inf).astype(np.float32)).to(cuda_dev)
    out_s, out_p, out_t, work = lq.beam_buffers(groups, beams, vocab, beams)
    length, total = prompt, np.where(np.arange(n) % beams == 0, 0.0, -np.inf)
    copied = 0
    for _ in range(steps):
        x = (2.0 * rng.standard_normal((n, vocab))).astype(np.float32)
        lq.lq_beam_select(torch.from_numpy(x).to(cuda_dev), scores, beams, beams, out_s, out_p, out_t, work)
        lq.lq_beam_pages(out_p.view(-1), beams, tables[0], to_gpu([length] * n, cuda_dev), page, tables[1], copies)
        lq.lq_kv_copy(cache, copies)
        tables.reverse()
        scores.copy_(out_s.view(-1))
        copied += int((copies[:, 2] > 0).sum())
        parents, tokens = out_p.view(-1).tolist(), out_t.view(-1).tolist()
        logp = _scores(x, np.zeros(n, np.float32))
        total = np.array([total[r // beams * beams + p] + logp[r // beams * beams + p, t] for r, (p, t) in enumerate(zip(parents, tokens))])
        past = [past[r // beams * beams + p] + [t] for r, (p, t) in enumerate(zip(parents, tokens))]
        length += 1
        write(list(range(n)), length, 1)
    assert copied > 5
    np.testing.assert_allclose(scores.cpu().numpy(), total, atol=steps * (2.0**-18 + 2.0**-24 * 200), rtol=0)
    for r in range(n):
        one = lq.KVBatch(tables[0][r:r + 1].contiguous(), to_gpu([length], cuda_dev), to_gpu([0, length], cuda_dev), length)
        k, v = (torch.empty(length, kv_heads, d, device=cuda_dev) for _ in range(2))
        lq.lq_kv_read(cache, one, k, v)
        want = K[torch.tensor(past[r], device=cuda_dev)]
        fresh = lq.KVCache(fmt, width, page, kv_heads, d)
        alone = lq.KVBatch(torch.arange(width, dtype=torch.int32, device=cuda_dev)[None].contiguous(), to_gpu([length], cuda_dev), to_gpu([0, length], cuda_dev), length)
        lq.lq_kv_write(fresh, alone, want.contiguous(), want.contiguous())
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        lq.lq_kv_read(fresh, alone, k2, v2)
        assert torch.equal(k, k2) and torch.equal(v, v2), f"beam {r}"


@pytest.mark.parametrize("k", [3, 64])
def test_long_parts_whose_notes_run_full(lq, cuda_dev, k):
    """Rows enough that each is one part of many rounds: rows of one value, rising
    (every round's logits are noted), falling, of ties and plain ones."""
    rng = np.random.default_rng(k)
    n, v = 640, 40003
    x = rng.standard_normal((n, v)).astype(np.float32)
    x[0::5] = 0.25
    x[1::5] = np.arange(v, dtype=np.float32) / 1000
    x[2::5] = -np.arange(v, dtype=np.float32) / 1000
    x[3::5] = np.round(x[3::5] * 2) / 2
    scores = -rng.random(n).astype(np.float32)
    _check(_select(lq, cuda_dev, x, scores, 4, k), _best(_scores(x, scores), 4, k))
