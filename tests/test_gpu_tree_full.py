"""A drafted step that fills its cache to the last slot: what lq_tree_plan and
lq_tree_accept, which see no cache, give agrees with what the calls on the cache
do there. Attention's tolerances are the oracle's; all else is exact."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from test_gpu_tree import _accept, _kept
from tree_helpers import ancestor_bits, expect_tree, random_parents, to_gpu, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("news,page,pages", [([9, 1, 33], 16, 5), ([64, 7], 16, 4), ([20, 3], 7, 3)])
def test_a_step_that_fills_the_cache(lq, cuda_dev, fmt, news, page, pages):
    total, (window, sinks) = page * pages, (24, 2)
    P = Paged(lq, fmt, news, [total] * len(news), 4, 2, 64, page, cuda_dev, seed=sum(news))
    assert P.table.shape[1] * page == total
    rng = np.random.default_rng(page)
    parents = [random_parents(rng, n, reach=4) for n in news]
    flat = np.concatenate(parents)
    want = [ancestor_bits(p, window, sinks, total - n) for p, n in zip(parents, news)]
    words, t, b = max(1, -(-max(news) // 32)), sum(news), len(news)
    cache, batch = P.cache(), P.batch()
    ints = lambda *s: torch.full(s, -7, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    pos, mask, keep, count, after, length = ints(t), ints(t, words), ints(b, 16), ints(b), ints(b), ints(b)
    lq.lq_tree_plan(batch, to_gpu(flat, cuda_dev), pos, mask, window=window, sinks=sinks)
    positions = np.concatenate([total - n + depth for n, (_, depth) in zip(news, want)])
    assert np.array_equal(pos.cpu().numpy(), positions)
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([words_of(x, words) for x, _ in want]))
    Q = torch.from_numpy(P.q).to(cuda_dev)
    O = torch.full_like(Q, float("nan"))
    lq.lq_attn_tree(cache, batch, mask, Q, O, 64**-0.5, positions=pos, window=window, sinks=sinks, work=lq.attn_work(cache, batch, 4))
    o, tol, _, _ = expect_tree(P, [x for x, _ in want], positions, window, sinks)
    compare(O.cpu().numpy(), o, tol, "output")
    token, target = rng.integers(0, 2, t).astype(np.int32), rng.integers(0, 2, t).astype(np.int32)
    lq.lq_tree_accept(batch, to_gpu(flat, cuda_dev), to_gpu(token, cuda_dev), to_gpu(target, cuda_dev), keep, count, after, length)
    lq.lq_kv_keep(cache, batch, keep, count)
    paths, at = [], 0
    for i, n in enumerate(news):
        path, _ = _accept(parents[i], token[at:at + n], target[at:at + n], 16)
        assert keep[i].tolist() == path + [-1] * (16 - len(path)) and length[i].item() == total - n + len(path) <= total
        paths.append(path)
        at += n
    pools = _kept(P, keep.cpu().numpy(), count.cpu().numpy())
    assert np.array_equal(cache.k.cpu().numpy(), pools[0]) and np.array_equal(cache.v.cpu().numpy(), pools[1])
    # the path's rows are the last of the length that accept gives
    for i, path in enumerate(paths):
        m = len(path)
        one = lq.KVBatch(to_gpu(P.table[i:i + 1], cuda_dev), length[i:i + 1].contiguous(), to_gpu([0, m], cuda_dev), m)
        k, v = (torch.empty(m, 2, 64, device=cuda_dev) for _ in range(2))
        lq.lq_kv_read(cache, one, k, v)
        rows = total - news[i] + np.array(path)
        assert np.array_equal(k.cpu().numpy(), P.values(0, i)[rows].astype(np.float32))
        assert np.array_equal(v.cpu().numpy(), P.values(1, i)[rows].astype(np.float32))
    assert lq.last_device_error() == lq.LQ_OK
