"""A forced attention kernel runs wherever the geometry is its own: nothing is
skipped here. Tolerances are the oracle's."""
import numpy as np
import pytest

from attn_helpers import Paged, compare
from test_gpu_tree import FMTS, TILE, WARP, _trees
from test_gpu_tree_one import _run
from tree_helpers import expect_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("route,counter", [(WARP, 9), (TILE, 10)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("page", [7, 16, 48, 128])
def test_forced_kernels_run_where_they_can(lq, cuda_dev, route, counter, fmt, d, page):
    """Heads of 64, 128 and 256 with pages of whole 16s are both kernels'; all else
    is refused."""
    P = Paged(lq, fmt, [9, 3], [60, 20], 4, 2, d, page, cuda_dev, seed=d + page)
    bits, positions = _trees(P, np.random.default_rng(page))
    lq.reset_counts()
    if d in (64, 128, 256) and page % 16 == 0:
        o, lse = _run(lq, P, bits, positions, route=route)
        assert lq.route_count(counter) == 1 and sum(lq.route_count(c) for c in (8, 9, 10)) == 1
        want, tol, wl, ltol = expect_tree(P, bits, positions)
        compare(o, want, tol, "output")
        compare(lse, wl, ltol, "lse")
    else:
        with pytest.raises(lq.LQError) as e:
            _run(lq, P, bits, positions, route=route)
        assert e.value.status == lq.LQ_ERR_UNSUPPORTED
        assert sum(lq.route_count(c) for c in (8, 9, 10)) == 0
