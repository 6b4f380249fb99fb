"""lq_beam_select where the log of a row's sum decides: beams that are alike, and
one group among others. A row's sum depends on the row alone, so equal rows with
equal scores tie, and a group's results are the same bits wherever it stands in a
call, whatever else the call has, and however its rows are aligned."""
import numpy as np
import pytest
import torch

from test_gpu_beam import _best, _check, _scores, _select

pytestmark = pytest.mark.gpu


def _coarse(rng, shape):
    return (np.round(2.5 * rng.standard_normal(shape) * 8) / 8).astype(np.float32)


@pytest.mark.parametrize("groups,beams,vocab,k", [
    (32, 8, 151936, 16), (32, 8, 32000, 16), (3, 5, 20001, 7), (90, 16, 40003, 33), (1, 64, 65536, 64), (700, 8, 9000, 8), (57, 3, 131071, 64)])
def test_alike_beams_among_many(lq, cuda_dev, groups, beams, vocab, k):
    """Every group has one row and one score over and over: the lower beam comes
    first, then the lower token. Ranges of rounds begin and end anywhere in the rows
    (rounds of 4096 logits; 456 ranges)."""
    rng = np.random.default_rng(vocab + groups)
    x = np.repeat(_coarse(rng, (groups, vocab)), beams, 0)
    scores = np.repeat((-20 * rng.random(groups)).astype(np.float32), beams)
    # (one row's scores stand for the group's)
    one = _scores(x[::beams], scores[::beams])
    want = [np.empty((groups, k)), np.empty((groups, k), dtype=int), np.empty((groups, k), dtype=int)]
    for g in range(groups):
        s, _, t = _best(one[g:g + 1], 1, min(k, vocab))
        order = [(v, b, j) for v in sorted(set(s[0]), reverse=True) for b in range(beams) for j in t[0][s[0] == v]]
        # (equal logits: all of a beam's, by token, then the next beam's)
        last = s[0][-1]
        if (one[g] == last).sum() > (s[0] == last).sum():
            order = [c for c in order if c[0] > last]
            order += [(last, b, j) for b in range(beams) for j in np.nonzero(one[g] == last)[0]]
        for i, (v, b, j) in enumerate(order[:k]):
            want[0][g, i], want[1][g, i], want[2][g, i] = v, b, j
    _check(_select(lq, cuda_dev, x, scores, beams, k), want)


@pytest.mark.parametrize("vocab,beams,k", [(151936, 8, 16), (20001, 4, 9), (4096, 3, 5), (50000, 16, 64)])
def test_a_group_among_others(lq, cuda_dev, vocab, beams, k):
    """The same bits alone, at every place of batches of several sizes, with any
    beams of the other groups ended or out of the running, and from rows that
    16-byte loads cannot take."""
    rng = np.random.default_rng(vocab + beams)
    mine, mine_s = (2.5 * rng.standard_normal((beams, vocab))).astype(np.float32), (-20 * rng.random(beams)).astype(np.float32)
    alone = [o.view(np.int32) for o in _select(lq, cuda_dev, mine, mine_s, beams, k)]
    for extra in (dict(ld=vocab + 4 - vocab % 4 + 1), dict(ld=vocab + 4 - vocab % 4, offset=3), dict(ld=vocab + 4 - vocab % 4)):
        assert all(np.array_equal(a.view(np.int32), b) for a, b in zip(_select(lq, cuda_dev, mine, mine_s, beams, k, **extra), alone)), extra
    for groups in (2, 7, 33):
        x = (2.5 * rng.standard_normal((groups * beams, vocab))).astype(np.float32)
        scores = (-20 * rng.random(groups * beams)).astype(np.float32)
        for at in sorted({0, groups // 2, groups - 1}):
            y, s = x.copy(), scores.copy()
            y[at * beams:(at + 1) * beams], s[at * beams:(at + 1) * beams] = mine, mine_s
            ended = (rng.random(groups * beams) < 0.3).astype(np.int32)
            s[rng.random(groups * beams) < 0.1] = -np.inf
            ended[at * beams:(at + 1) * beams], s[at * beams:(at + 1) * beams] = 0, mine_s
            got = _select(lq, cuda_dev, y, s, beams, k, finished=ended, pad=1)
            assert all(np.array_equal(a[at].view(np.int32), b[0]) for a, b in zip(got, alone)), (groups, at)


@pytest.mark.parametrize("vocab", [1, 511, 4097, 151936, 2**20 + 3])
@pytest.mark.parametrize("value", [0.0, 1.5, -12.25])
def test_rows_of_one_value(lq, cuda_dev, vocab, value):
    """Every term is 2^0, which is exact, and so are sums of them up to 2^24. What is
    left is the logarithm: its own rounding is taken back by expf(-l), which is off
    by one last place (2^-23), and the square of that rounding (2^-20 at most where
    16 <= l < 32) is nothing. The score is rounded once (2^-24 of it)."""
    x = np.full((6, vocab), value, np.float32)
    scores = np.array([-1.0, -3.25, -0.5, -7.0, -100.0, 0.0], np.float32)
    s, p, t = _select(lq, cuda_dev, x, scores, 3, 2)
    two = vocab > 1
    order = np.array([[2, 2 if two else 0], [2, 2 if two else 0]])
    assert np.array_equal(p, order) and np.array_equal(t, [[0, 1 if two else 0]] * 2)
    want = scores.reshape(2, 3).astype(np.float64)[[[0], [1]], order] - np.log(float(vocab))
    assert (np.abs(s - want) <= 1.25 * 2.0**-23 + 2.0**-24 * np.abs(want)).all()


def test_scores_in_place(lq, cuda_dev):
    """As many results as beams may take the scores' place."""
    rng = np.random.default_rng(9)
    x, scores = rng.standard_normal((240, 5000)).astype(np.float32), (-9 * rng.random(240)).astype(np.float32)
    X, S = torch.from_numpy(x).to(cuda_dev), torch.from_numpy(scores).to(cuda_dev)
    _, out_p, out_t, work = lq.beam_buffers(60, 4, 5000, 4)
    lq.lq_beam_select(X, S, 4, 4, S.view(60, 4), out_p, out_t, work)
    _check([S.view(60, 4).cpu().numpy(), out_p.cpu().numpy(), out_t.cpu().numpy()], _best(_scores(x, scores), 4, 4))


@pytest.mark.parametrize("k", [4, 64])
def test_ranges_of_many_rounds(lq, cuda_dev, k):
    """Parts of more rounds than shared memory keeps sums of (64): a group among 32
    has the bits that it has alone, where its rows are cut into short parts; and
    the scores are those of the sums in 64 bits. One row grows, one has one value."""
    groups, beams, vocab = 32, 4, 2**20 + 5
    g = torch.Generator(device=cuda_dev).manual_seed(k)
    x = 2.5 * torch.randn(groups * beams, vocab, generator=g, device=cuda_dev)
    x[4 * 7 + 1] = torch.arange(vocab, device=cuda_dev) / 65536.0
    x[4 * 7 + 2] = 3.75
    scores = -9 * torch.rand(groups * beams, generator=g, device=cuda_dev)
    out = lq.beam_buffers(groups, beams, vocab, k)
    lq.lq_beam_select(x, scores, beams, k, *out)
    for at in (0, 7, 15, 31):
        one = lq.beam_buffers(1, beams, vocab, k)
        lq.lq_beam_select(x[at * beams:(at + 1) * beams], scores[at * beams:(at + 1) * beams].contiguous(), beams, k, *one)
        for a, b in zip(out[:3], one[:3]):
            assert torch.equal(a[at], b[0]), at
    lse = torch.stack([torch.logsumexp(r.double(), 0) for r in x])
    rows = out[1].long() + torch.arange(groups, device=cuda_dev)[:, None] * beams
    want = scores.double()[rows] + (x[rows, out[2].long()].double() - lse[rows])
    assert (out[1] >= 0).all() and ((out[0].double() - want).abs() <= 2.0**-24 * want.abs() + 2.0**-18).all()
    best = (scores.double()[:, None] - lse[:, None] + x.topk(k, 1).values.double()).view(groups, -1).sort(1, descending=True).values[:, :k]
    assert ((out[0].double() - best).abs() <= 2.0**-24 * best.abs() + 2.0**-18).all()
    assert lq.last_device_error() == lq.LQ_OK
