"""How many bits a weight keeps (include/lq.h): values whose sizes differ by
many binary orders between a head's blocks of 32 dims, and between keys."""
import numpy as np
import pytest

from attn_helpers import Paged, compare
from oracle import attention as A
from test_gpu_attn import FMTS, GENERIC, ROUTES, WARP, _run

pytestmark = pytest.mark.gpu


def _scales(fmt, v):
    """|d| of every block of the stored rows v [n, D] (f16 caches: none)."""
    if fmt == "f16":
        return np.ones((len(v), 1))
    _, bits = A.cache_rows(fmt, v)
    return np.abs(bits.view(np.float16).astype(np.float64))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("between", ["blocks", "keys"])
@pytest.mark.parametrize("orders", [0, 6, 12, 18, 24])
def test_values_of_many_sizes(lq, cuda_dev, route, fmt, between, orders):
    """Per element: the oracle's tolerance, and besides 2^-36 of the row's
    largest weight (few rows, quantised: weight times scale) for every key,
    times its value (code)."""
    d, totals = 128, [150, 70, 33]
    P = Paged(lq, fmt, [1, 20, 2], totals, 4, 2, d, 16, cuda_dev, seed=orders)
    for i, n in enumerate(totals):
        size = 2.0**-orders if between == "blocks" else 2.0 ** (-orders * (np.arange(n) % 4) / 3.0)[:, None, None]
        x = P.v[i] * 64.0
        if between == "blocks":
            x[:, :, 32:64] *= np.float32(size)
            x[:, :, 96:] *= np.float32(np.sqrt(size))
        else:
            x = x * size
        P.v[i] = x.astype(np.float32)
        P.store(1, i, P.v[i])
    P.q *= np.float32(2.0)
    o, _ = _run(lq, P, route=route)
    want, tol, _, _ = P.expect()
    for i, (new, n) in enumerate(zip(P.news, totals)):
        kall, vall = P.values(0, i).astype(np.float64), P.values(1, i).astype(np.float64)
        for r in range(new):
            t, last = P.q_start[i] + r, n - new + r + 1
            for h in range(P.heads):
                k, v = kall[:last, h // 2], vall[:last, h // 2]
                x = k @ P.q[t, h].astype(np.float64) / np.sqrt(d)
                p = np.exp(x - x.max())
                p /= p.sum()
                s = _scales(fmt, P.v[i][:last, h // 2])
                if fmt == "f16" or route not in (0, WARP):
                    step = 2.0**-36 * p.max() * np.abs(v).sum(0)
                else:
                    codes = np.abs(v) / np.maximum(np.repeat(s, 32, 1), 2.0**-30)
                    step = 2.0**-36 * (p[:, None] * s).max() * codes.sum(0)
                if route != GENERIC:
                    tol[t, h] += step
    compare(o, want, tol, f"values over {orders} binary orders")
