"""The angle of a rotary turn by itself: cosine and sine of positions near and far.

A pair of (1, 0) becomes (cos t, sin t). The table's turns times the position,
modulo 2^64, is the angle in integers. The kernel rounds it to 32 bits (2^-33 of
a turn) and what is left beside the nearest quarter of a turn to 24 bits (2^-28
of a turn); cosine and sine come within one last place, 2^-23 of themselves."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 64), (6, 6), (128, 32)])
@pytest.mark.parametrize("far", [100, 131071, 2**24, 2**31 - 1])
def test_cosine_and_sine(lq, cuda_dev, d, rotary, far, adjacent):
    rng = np.random.default_rng(far % 1000 + d)
    half, n = rotary // 2, 4001
    freqs = np.concatenate([[1.0, math.pi / 4, 2 * math.pi * 0.249999], rng.random(max(0, half - 3))])[:half]
    rope = lq.Rope(d, rotary, freqs=freqs, adjacent=adjacent)
    pos = rng.integers(-far - 1, far + 1, n).astype(np.int32)
    pos[:5] = [0, 1, -1, far, -far - 1]
    x = np.zeros((n, 1, d), np.float32)
    at = np.arange(0, rotary, 2) if adjacent else np.arange(half)
    x[:, 0, at] = 1.0
    X = torch.from_numpy(x).to(cuda_dev)
    lq.lq_rope(rope, torch.from_numpy(pos).to(cuda_dev), X)
    y = X.cpu().numpy().astype(np.float64)[:, 0]
    # (64-bit integers wrap as the angle does)
    units = pos.astype(np.int64).astype(np.uint64)[:, None] * np.array([rope.struct.turns[j] for j in range(half)], dtype=np.uint64)
    quarter = (units + np.uint64(1 << 61)) >> np.uint64(62)
    rest = (units - (quarter << np.uint64(62))).astype(np.int64).astype(np.float64) * 2.0**-63 * math.pi  # (an eighth of a turn at most)
    c, s, q = np.cos(rest), np.sin(rest), quarter.astype(int)
    cos, sin = np.choose(q, [c, -s, -c, s]), np.choose(q, [s, c, -s, -c])
    for got, want in ((y[:, at], cos), (y[:, at + (1 if adjacent else half)], sin)):
        assert (np.abs(got - want) <= 2 * math.pi * (2.0**-28 + 2.0**-33) + 2.0**-23 * np.abs(want) + 1e-15).all()
    assert lq.last_device_error() == lq.LQ_OK


@pytest.mark.parametrize("tokens", [1, 2, 70])
@pytest.mark.parametrize("interleaved", [False, True])
def test_one_row_of_positions_for_all_axes(lq, cuda_dev, tokens, interleaved):
    """Text has one position on every axis: an expanded row gives the bits of a
    copied one, and of a table with one axis."""
    rng = np.random.default_rng(tokens)
    rope = lq.Rope(128, sections=[24, 20, 20], interleaved=interleaved)
    row = torch.from_numpy(rng.integers(0, 10**6, tokens).astype(np.int32)).to(cuda_dev)
    q = torch.from_numpy(rng.standard_normal((tokens, 5, 128)).astype(np.float32)).to(cuda_dev)
    k = torch.from_numpy(rng.standard_normal((tokens, 2, 128)).astype(np.float32)).to(cuda_dev)
    results = []
    for table, positions in ((rope, row.expand(3, tokens)), (rope, row.expand(3, tokens).contiguous()), (lq.Rope(128), row)):
        out = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        lq.lq_rope(table, positions, q, k, q_out=out[0], k_out=out[1])
        results.append(out)
    for out in results[1:]:
        assert torch.equal(out[0], results[0][0]) and torch.equal(out[1], results[0][1])
    assert torch.isfinite(results[0][0]).all() and lq.last_device_error() == lq.LQ_OK
