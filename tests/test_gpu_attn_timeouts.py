"""Failure detection of the tile kernel of lq_attn_paged without a GPU fault:
with a wait limit of one poll (lq_debug_set_wait_limit_ns(1)) its bounded
waits give up at once; the kernel has to record LQ_ERR_DEVICE_TIMEOUT, let its
copies and MMAs finish, free its tensor memory and return, and the context
must compute correctly again with the default limit (and a work buffer that is
zero again)."""
import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,news,totals,d", [("f16", [300], [2000], 128), ("f16", [70, 5], [900, 300], 64),
                                               ("q8_0", [200], [1500], 128), ("q4_0", [90], [700], 64),
                                               ("f16", [150], [900], 256), ("q8_0", [140, 70], [900, 100], 256)])
def test_tile_kernel_timeout(lq, cuda_dev, fmt, news, totals, d):
    P = Paged(lq, fmt, news, totals, 4, 2, d, 16, cuda_dev, seed=3)
    cache, batch = P.cache(), P.batch()
    Q = torch.from_numpy(P.q).to(cuda_dev)
    O = torch.full_like(Q, float("nan"))
    lq.reset_counts()
    lq.attn_route(3)
    try:
        lq.set_wait_limit_ns(1)
        lq.last_device_error()
        lq.lq_attn_paged(cache, batch, Q, O, 1.0 / np.sqrt(d), work=lq.attn_work(cache, batch, 4))
        torch.cuda.synchronize()
        st = lq.last_device_error()
        assert lq.route_count(10) == 1
        assert st == lq.LQ_ERR_DEVICE_TIMEOUT
        lq.set_wait_limit_ns(0)
        O = torch.full_like(Q, float("nan"))
        lq.lq_attn_paged(cache, batch, Q, O, 1.0 / np.sqrt(d), work=lq.attn_work(cache, batch, 4))
        torch.cuda.synchronize()
    finally:
        lq.set_wait_limit_ns(0)
        lq.attn_route(0)
    assert lq.last_device_error() == lq.LQ_OK
    want, tol, _, _ = P.expect()
    compare(O.cpu().numpy(), want, tol)
