"""The bounds-checking build (liblq_debug.so) on rotary positions, drafted trees
and beams, each call with a clean status word and the expected result; and the
tree instances of the tile kernel when their waits run out."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from attn_helpers import Paged, compare
from tree_helpers import ancestor_bits, expect_tree, random_parents, to_gpu, words_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import numpy as np, torch
import gemm_gemv_f16w_gb300 as lq
import test_gpu_beam as beam, test_gpu_rope as rope, test_gpu_tree as tree
assert lq.LIB_PATH.endswith("liblq_debug.so"), lq.LIB_PATH
dev = torch.device("cuda:0")
torch.cuda.set_device(dev)
runs = 0
def ran(f, *a):
    global runs
    f(lq, dev, *a)
    torch.cuda.synchronize()
    st = lq.last_device_error()
    assert st == lq.LQ_OK, (f.__name__, a, lq.status_string(st))
    runs += 1
for adjacent in (False, True):
    ran(rope.test_against_64_bits, 33, 4, 4, 256, 64, [12, 10, 10], True, adjacent)
    ran(rope.test_against_64_bits, 5, 3, 1, 34, 34, [17], True, adjacent)
for fmt in ("f16", "q8_0", "q4_0"):
    for route in (1, 2, 3):
        ran(tree.test_trees, route, fmt, [5, 1, 0, 9], [40, 1, 13, 9], 128, 4, 2, 16)
        ran(tree.test_window_and_sinks, route, fmt, 37, 1)
        ran(tree.test_any_bits, route, fmt, 5)
        ran(tree.test_lengths_below_the_rows, route, fmt)
    ran(tree.test_keep, fmt, [9, 1, 0, 61], [40, 7, 13, 200], 128, 8, 16)
    ran(tree.test_keep, fmt, [50], [90], 96, 1, 5)
    ran(beam.test_copies, fmt, 3, 96, 5, 0)
    if fmt != "f16":
        ran(tree.test_wide_heads_of_quantised_caches, fmt, [40, 9], [300, 200], 16)
ran(tree.test_plan, [200, 31], 2, 5, 103)
ran(tree.test_accept, [100, 64, 7], 2, 40)
for sizes in ((7, 1, 4097, 64), (2, 16, 20001, 32), (3, 2, 5, 4)):
    for coarse in (False, True):
        ran(beam.test_against_64_bits, *sizes, coarse)
ran(beam.test_odd_rows, 64)
ran(beam.test_long_parts_whose_notes_run_full, 64)
ran(beam.test_first_step_and_ended_beams)
ran(beam.test_pages, 33, 16, 7, 40)
print("bounds ok", runs)
'''


def test_kernels_stay_in_bounds():
    from gemm_gemv_f16w_gb300 import build as b
    b.build(debug_bounds=True)
    env = dict(os.environ, LQ_LIBRARY="debug", PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       timeout=900)
    assert r.returncode == 0 and "bounds ok 63" in r.stdout, r.stdout[-3000:]


@pytest.mark.parametrize("fmt,news,totals,d", [("f16", [70, 5], [900, 300], 128), ("q8_0", [90], [700], 64), ("q4_0", [140, 70], [900, 100], 256)])
def test_waits_that_run_out(lq, cuda_dev, fmt, news, totals, d):
    """With a wait limit of one poll the kernel reports a timeout and returns; the
    next call, with the default limit, is right."""
    P = Paged(lq, fmt, news, totals, 4, 2, d, 16, cuda_dev, seed=3)
    rng = np.random.default_rng(1)
    bits, positions = [], []
    for n, total in zip(news, totals):
        b, depth = ancestor_bits(random_parents(rng, n))
        bits.append(b)
        positions.append(total - n + depth)
    cache, batch = P.cache(), P.batch()
    mask = to_gpu(np.concatenate([words_of(b, 5) for b in bits]), cuda_dev)
    Q = torch.from_numpy(P.q).to(cuda_dev)
    O = torch.full_like(Q, float("nan"))
    lq.attn_route(3)
    try:
        lq.set_wait_limit_ns(1)
        lq.last_device_error()
        lq.lq_attn_tree(cache, batch, mask, Q, O, d**-0.5, work=lq.attn_work(cache, batch, 4))
        torch.cuda.synchronize()
        assert lq.last_device_error() == lq.LQ_ERR_DEVICE_TIMEOUT
        lq.set_wait_limit_ns(0)
        lq.lq_attn_tree(cache, batch, mask, Q, O, d**-0.5, work=lq.attn_work(cache, batch, 4))
        torch.cuda.synchronize()
    finally:
        lq.set_wait_limit_ns(0)
        lq.attn_route(0)
    assert lq.last_device_error() == lq.LQ_OK
    want, tol, _, _ = expect_tree(P, bits, np.concatenate(positions))
    compare(O.cpu().numpy(), want, tol)
