"""One drafted tree over some thousand positions, where the warp-level kernel
widens its ranges so that a unit's parts are joined in one round, and lengths on
both sides of that rule. Tolerances are the oracle's."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from test_gpu_tree import FMTS, WARP, _mask, _trees
from tree_helpers import expect_tree, to_gpu

pytestmark = pytest.mark.gpu


def _run(lq, P, bits, positions, route=0, window=0, sinks=0):
    cache, batch = P.cache(), P.batch(max_q=max(P.news))
    Q = torch.from_numpy(P.q).to(P.dev)
    O = torch.full_like(Q, float("nan"))
    lse = torch.full((P.tokens, P.heads), float("nan"), device=P.dev)
    lq.attn_route(route)
    try:
        lq.lq_attn_tree(cache, batch, to_gpu(_mask(P, bits), P.dev), Q, O, P.d**-0.5, positions=to_gpu(positions, P.dev), window=window,
                        sinks=sinks, lse=lse, work=lq.attn_work(cache, batch, P.heads))
    finally:
        lq.attn_route(0)
    torch.cuda.synchronize()
    assert lq.last_device_error() == lq.LQ_OK
    return O.cpu().numpy(), lse.cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("new,total,heads,kv_heads,d,window", [
    (7, 1201, 32, 8, 128, 0), (7, 2000, 32, 8, 128, 0), (12, 3007, 16, 8, 64, 0), (7, 4500, 32, 8, 64, 0), (24, 4795, 16, 8, 64, 0),
    (7, 4801, 32, 8, 128, 0), (12, 4500, 32, 8, 128, 2100), (5, 2500, 32, 8, 256, 0)])
def test_one_tree(lq, cuda_dev, fmt, new, total, heads, kv_heads, d, window):
    P = Paged(lq, fmt, [new], [total], heads, kv_heads, d, 16, cuda_dev, seed=total + d, fill="nan")
    bits, positions = _trees(P, np.random.default_rng(new), roots=0.1)
    lq.reset_counts()
    o, lse = _run(lq, P, bits, positions, route=WARP, window=window, sinks=4)
    assert (lq.route_count(9), lq.route_count(10)) == (1, 0)
    want, tol, wl, ltol = expect_tree(P, bits, positions, window, 4)
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")
