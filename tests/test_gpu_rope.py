"""lq_rope against the rotation in 64 bits.

Tolerance: the angle reaches sincospif as a 24-bit fraction of half a turn, so it
is off by at most pi 2^-25 < 1.6 2^-24; sincospif by one last place (2^-24 below
1); the factor, the product and the fused sum round once each: together less than
6 2^-24 of factor (|x_a| + |x_b|). The reference's own angle, a product of doubles,
is off by 2^-52 of itself: 2^-28 at the farthest position here."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _axes(half, sections, interleaved):
    if sections is None:
        return np.zeros(half, dtype=int)
    n = len(sections)
    if not interleaved:
        return np.repeat(np.arange(n), sections)
    return np.array([j % n if j < n * sections[j % n] else 0 for j in range(half)])


def _expect(x, pos, rotary, freqs, axes, adjacent, factor=1.0, inverse=False):
    """(y, tolerance) of x [tokens, heads, D] in float64; pos [axes, tokens]."""
    half, x = rotary // 2, x.astype(np.float64)
    angle = pos.astype(np.float64)[axes].T * freqs
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor * (-1 if inverse else 1)
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if adjacent else (slice(0, half), slice(half, rotary))
    y, tol = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    tol[..., a] = tol[..., b] = 6 * 2.0**-24 * abs(factor) * (abs(x[..., a]) + abs(x[..., b])) + 1e-40
    return y, tol


def _check(got, want, tol):
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= tol).all(), f"largest error over tolerance {np.nanmax(err / np.where(tol > 0, tol, 1e-40))}"


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rotary,sections,interleaved", [
    (128, 128, None, False), (256, 64, [12, 10, 10], True), (64, 64, [8, 12, 12], False), (128, 128, [24, 20, 20], True),
    (96, 48, [3, 0, 21], False), (80, 80, None, False), (72, 20, [6, 4], True), (6, 2, None, False), (256, 256, [32, 32, 32, 32], True),
    (512, 256, [0, 128], False), (34, 34, [17], True)])
@pytest.mark.parametrize("tokens,heads,kv_heads", [(1, 32, 8), (5, 3, 1), (33, 4, 4), (2500, 2, 1)])
def test_against_64_bits(lq, cuda_dev, tokens, heads, kv_heads, d, rotary, sections, interleaved, adjacent):
    """Slices of fused rows, positions of both signs and far away, in place and not."""
    rng = np.random.default_rng(tokens + d)
    half, n_axes = rotary // 2, 1 if sections is None else len(sections)
    rope = lq.Rope(d, rotary, base=1e4, adjacent=adjacent, sections=sections, interleaved=interleaved)
    axes = _axes(half, sections, interleaved)
    freqs = 1e4 ** (-2.0 * np.arange(half) / rotary)
    pos = rng.integers(-2**24, 2**24, (n_axes, tokens)).astype(np.int32)
    pos[:, 0] = 0
    rows = rng.standard_normal((tokens, (heads + 2 * kv_heads) * d)).astype(np.float32)
    q, k = rows[:, : heads * d].reshape(tokens, heads, d), rows[:, heads * d: (heads + kv_heads) * d].reshape(tokens, kv_heads, d)
    R = torch.from_numpy(rows).to(cuda_dev)
    Q, K = R[:, : heads * d], R[:, heads * d: (heads + kv_heads) * d].unflatten(1, (kv_heads, d))
    P = torch.from_numpy(pos).to(cuda_dev)
    qo, ko = torch.full((tokens, heads, d), float("nan"), device=cuda_dev), torch.full((tokens, kv_heads, d), float("nan"), device=cuda_dev)
    lq.lq_rope(rope, P[0] if n_axes == 1 and tokens % 2 else P, Q, K, q_out=qo, k_out=ko)
    wq, wk = _expect(q, pos, rotary, freqs, axes, adjacent), _expect(k, pos, rotary, freqs, axes, adjacent)
    _check(qo.cpu().numpy(), *wq)
    _check(ko.cpu().numpy(), *wk)
    assert torch.equal(R, torch.from_numpy(rows).to(cuda_dev))
    lq.lq_rope(rope, P, Q, K)  # in place: the same bits, and V's columns stay
    assert torch.equal(Q.unflatten(1, (heads, d)), qo) and torch.equal(K, ko)
    assert torch.equal(R[:, (heads + kv_heads) * d:].cpu(), torch.from_numpy(rows[:, (heads + kv_heads) * d:]))
    assert lq.last_device_error() == lq.LQ_OK


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 1), (4, 4)])
def test_alignment(lq, cuda_dev, offset, pad):
    """Rows that 16-byte loads cannot take, out of place from and to them."""
    rng = np.random.default_rng(1)
    t, h, d = 37, 3, 64
    rope = lq.Rope(d, 32, base=500.0)
    x = rng.standard_normal((t, h, d)).astype(np.float32)
    pos = rng.integers(0, 1000, (1, t)).astype(np.int32)
    src = torch.zeros(t * (h * d + pad) + offset, device=cuda_dev)[offset:].as_strided((t, h, d), (h * d + pad, d, 1))
    src.copy_(torch.from_numpy(x))
    dst = torch.full((t * (h * d + pad) + offset,), -7.0, device=cuda_dev)
    out = dst[offset:].as_strided((t, h, d), (h * d + pad, d, 1))
    lq.lq_rope(rope, torch.from_numpy(pos).to(cuda_dev), src, q_out=out)
    _check(out.cpu().numpy(), *_expect(x, pos, 32, 500.0 ** (-np.arange(16) / 16.0), np.zeros(16, dtype=int), False))
    between = dst[offset:].as_strided((t, h * d + pad), (h * d + pad, 1))[:, h * d:]
    assert (between == -7.0).all() and (dst[:offset] == -7.0).all()


def test_frequencies_factor_and_back(lq, cuda_dev):
    """Given frequencies of any sign and size; turning back undoes the turn."""
    rng = np.random.default_rng(2)
    t, h, d = 70, 5, 128
    freqs = np.concatenate([rng.standard_normal(60) * 3, [0.0, 100.0, -1e-9, np.pi]])
    rope = lq.Rope(d, freqs=freqs, factor=1.25)
    x = rng.standard_normal((t, h, d)).astype(np.float32)
    pos = rng.integers(-5000, 5000, (1, t)).astype(np.int32)
    X, P = torch.from_numpy(x).to(cuda_dev), torch.from_numpy(pos).to(cuda_dev)
    y = torch.empty_like(X)
    lq.lq_rope(rope, P, X, q_out=y)
    _check(y.cpu().numpy(), *_expect(x, pos, d, freqs, np.zeros(64, dtype=int), False, 1.25))
    lq.lq_rope(rope, P, X, q_out=y, inverse=True)
    _check(y.cpu().numpy(), *_expect(x, pos, d, freqs, np.zeros(64, dtype=int), False, 1.25, True))
    plain = lq.Rope(d, freqs=freqs)
    lq.lq_rope(plain, P, X, q_out=y)
    lq.lq_rope(plain, P, y, inverse=True)
    size = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    # two turns: each within 6 2^-24 of its input's |x_a| + |x_b|, at most 2^0.5 of the first's
    assert (np.abs(y.cpu().numpy() - x) <= 15 * 2.0**-24 * np.concatenate([size, size], -1) + 1e-40).all()


def test_values_that_are_not_finite_stay_in_their_pairs(lq, cuda_dev):
    t, h, d = 3, 2, 64
    x = torch.ones(t, h, d, device=cuda_dev)
    x[1, 0, 5], x[2, 1, 40] = float("nan"), float("inf")
    lq.lq_rope(lq.Rope(d, 32), torch.arange(t, dtype=torch.int32, device=cuda_dev), x)
    bad = (~torch.isfinite(x)).nonzero().tolist()
    assert bad == [[1, 0, 5], [1, 0, 21], [2, 1, 40]]


def test_captured_and_on_a_stream_of_its_own(lq, cuda_dev):
    rng = np.random.default_rng(3)
    t, h, d = 9, 4, 128
    rope = lq.Rope(d, sections=[24, 20, 20])
    x = torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)).to(cuda_dev)
    pos = torch.zeros(3, t, dtype=torch.int32, device=cuda_dev)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lq.lq_rope(rope, pos, x, q_out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.lq_rope(rope, pos, x, q_out=y)
    for step in range(3):
        new = rng.integers(0, 10**6, (3, t)).astype(np.int32)
        pos.copy_(torch.from_numpy(new))
        graph.replay()
        _check(y.cpu().numpy(), *_expect(x.cpu().numpy(), new, d, 1e4 ** (-np.arange(64) / 64.0), np.repeat(np.arange(3), [24, 20, 20]), False))


def test_many_rows(lq, cuda_dev):
    """More values than 32 bits count: 2^31 + some, rows checked at the ends."""
    d, h = 256, 64
    t = 2**31 // (d * h) + 3
    x = torch.empty(t, h, d, device=cuda_dev)
    x.fill_(1.0)
    pos = torch.arange(t, dtype=torch.int32, device=cuda_dev)
    lq.lq_rope(lq.Rope(d, 64), pos, x)
    freqs, at = 1e4 ** (-np.arange(32) / 32.0), [0, 1, t // 2, t - 2, t - 1]
    want, tol = _expect(np.ones((len(at), 1, d), dtype=np.float32), np.array([at]), 64, freqs, np.zeros(32, dtype=int), False)
    for i, r in enumerate(at):
        got = x[r].cpu().numpy()
        _check(got[[0, h - 1]][:, None][:, 0], np.repeat(want[i], 2, 0), np.repeat(tol[i], 2, 0))
