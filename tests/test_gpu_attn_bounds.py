"""The bounds-checking build (liblq_debug.so) on the paged cache and its
attention: small odd shapes through every kernel, each call with a clean
status word and the oracle's result."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import numpy as np, torch
import gemm_gemv_f16w_gb300 as lq
from attn_helpers import Paged, compare
assert lq.LIB_PATH.endswith("liblq_debug.so"), lq.LIB_PATH
dev = torch.device("cuda:0")
torch.cuda.set_device(dev)
runs = 0
for fmt in ("f16", "q8_0", "q4_0"):
    for route, d, heads, kv_heads, page, news, totals, window in [
            (1, 96, 4, 2, 7, [3, 1], [20, 9], 0), (2, 128, 8, 1, 16, [1, 1, 2], [300, 17, 40], 0), (2, 256, 2, 2, 32, [1, 5], [90, 5], 20),
            (2, 64, 6, 2, 16, [7], [200], 0), (3, 128, 4, 1, 16, [70, 3], [300, 40], 0), (3, 64, 4, 2, 32, [150], [150], 40), (3, 256, 4, 2, 16, [90, 3], [200, 30], 40)]:
        P = Paged(lq, fmt, news, totals, heads, kv_heads, d, page, dev, seed=d + route)
        cache, batch = P.cache(), P.batch()
        q = torch.from_numpy(P.q).to(dev)
        o = torch.full_like(q, float("nan"))
        lq.attn_route(route)
        lq.lq_attn_paged(cache, batch, q, o, 1.0 / np.sqrt(d), window=window, sinks=3, work=lq.attn_work(cache, batch, heads))
        lq.attn_route(0)
        torch.cuda.synchronize()
        st = lq.last_device_error()
        assert st == lq.LQ_OK, (fmt, route, d, lq.status_string(st))
        want, tol, _, _ = P.expect(window=window, sinks=3)
        compare(o.cpu().numpy(), want, tol, f"{fmt} route {route} head_dim {d}")
        k, v = (torch.randn(P.tokens, kv_heads, d, device=dev) for _ in range(2))
        lq.lq_kv_write(cache, batch, k, v)
        lq.lq_kv_read(cache, batch, torch.empty_like(k), torch.empty_like(v))
        torch.cuda.synchronize()
        assert lq.last_device_error() == lq.LQ_OK
        runs += 1
print("bounds ok", runs)
'''


def test_cache_and_attention_kernels_stay_in_bounds():
    from gemm_gemv_f16w_gb300 import build as b
    b.build(debug_bounds=True)
    env = dict(os.environ, LQ_LIBRARY="debug", PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       timeout=600)
    assert r.returncode == 0 and "bounds ok 21" in r.stdout, r.stdout[-3000:]
