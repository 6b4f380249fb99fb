"""Blocks with several values beyond the cache's range: they are clamped to
+-65504 first, and the first of the largest clamped magnitude gives a Q4_0
block's scale its sign. Stored bytes against the oracle's packer."""
import itertools

import numpy as np
import pytest
import torch

from attn_helpers import Paged
from oracle import attention as A

pytestmark = pytest.mark.gpu

BIG = (65504.0, 65505.0, 70000.0, 1e5, 3e38, np.inf)


@pytest.mark.parametrize("fmt", ("f16", "q8_0", "q4_0"))
@pytest.mark.parametrize("first,second", [(0, 1), (2, 3), (1, 6), (5, 27), (3, 4), (17, 31)])
def test_two_values_beyond_the_range(lq, cuda_dev, fmt, first, second):
    """Every pair of sizes and signs, in one lane's four elements, in
    neighbouring lanes and across the block; ordinary values around them."""
    rng = np.random.default_rng(first + second)
    pairs = [(a * s, b * t) for a, b in itertools.product(BIG, BIG) for s, t in ((1, 1), (1, -1), (-1, 1), (-1, -1))]
    d = 64
    x = rng.standard_normal((len(pairs), 1, d)).astype(np.float32) * 1000
    for i, (a, b) in enumerate(pairs):
        x[i, 0, first], x[i, 0, second] = a, b
        x[i, 0, 32 + first], x[i, 0, 32 + second] = b, 300.0  # the next block has one of them
    P = Paged(lq, fmt, [len(pairs)], [len(pairs)], 1, 1, d, 16, cuda_dev)
    before = P.pools.copy()
    P.store(0, 0, x)
    P.store(1, 0, x[::-1])
    want, P.pools = P.pools, before
    cache, batch = P.cache(), P.batch()
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)  # noqa: E731
    lq.lq_kv_write(cache, batch, up(x), up(x[::-1]))
    for got, w in zip((cache.k, cache.v), want):
        assert np.array_equal(got.cpu().numpy(), w)
    k, v = (torch.empty(len(pairs), 1, d, device=cuda_dev) for _ in range(2))
    lq.lq_kv_read(cache, batch, k, v)
    kept = A.cache_values(fmt, x[:, 0])
    assert np.array_equal(k.cpu().numpy()[:, 0], kept) and np.array_equal(v.cpu().numpy()[:, 0], kept[::-1])
    assert lq.last_device_error() == lq.LQ_OK
