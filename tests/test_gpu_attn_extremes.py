"""lq_attn_paged far from ordinary logits: every kernel gives the formula's
result for any finite logit, and the stated one where there is none."""
import numpy as np
import pytest

from attn_helpers import Paged, compare
from oracle import attention as A
from test_gpu_attn import FMTS, ROUTES, _run

pytestmark = pytest.mark.gpu

# past 2^24 a step of float32 is more than one, past 2^27 (base 2) more than 15
SIZES = (0.0, 3.0, 1e5, 2.0**24, 3.1e7, 6.1e7, 9.9e7, 1.5e8, 1.8e8, 3e8, 1e12, 1e20, 8e29, 3e30, 1e35, 1e38)


def _rows(lq, fmt, d, dev, keys, seed, page=16):
    """A sequence of `keys` positions for each logit size and sign, its one
    query along its keys' common direction."""
    aims = [s * t for s in SIZES for t in (1, -1)]
    P = Paged(lq, fmt, [1] * len(aims), [keys] * len(aims), 2, 1, d, page, dev, seed=seed)
    return P, aims


def _aim(P, i, aim, k):
    """Query i so that scale q . k is `aim` (both query heads)."""
    k = k.astype(np.float64)
    P.q[i, :] = (aim * np.sqrt(P.d) / (k @ k) * k).astype(np.float32)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_key_of_any_logit(lq, cuda_dev, route, fmt, d):
    """The first token of a sequence sees itself alone: its value, whatever
    the logit, and the logit as lse."""
    P, aims = _rows(lq, fmt, d, cuda_dev, 1, seed=31)
    for i, aim in enumerate(aims):
        _aim(P, i, aim, P.values(0, i)[0, 0])
    o, lse = _run(lq, P, route=route)
    _, _, wl, ltol = P.expect()
    for i in range(len(aims)):
        v = P.values(1, i)[0, 0].astype(np.float64)
        compare(o[i], np.broadcast_to(v, o[i].shape), np.broadcast_to(2.0**-17 * np.abs(v) + 1e-37, o[i].shape), f"logit {aims[i]:.3g}")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,keys", [(64, 150), (128, 40), (256, 70)])
def test_equal_logits_of_any_size(lq, cuda_dev, route, fmt, d, keys):
    """Equal keys have equal logits, bit for bit: the mean of the values."""
    P, aims = _rows(lq, fmt, d, cuda_dev, keys, seed=32)
    for i, aim in enumerate(aims):
        P.k[i][:] = P.k[i][:1]
        P.store(0, i, P.k[i])
        _aim(P, i, aim, P.values(0, i)[0, 0])
    o, lse = _run(lq, P, route=route)
    _, _, wl, ltol = P.expect()
    for i in range(len(aims)):
        v = P.values(1, i)[:, 0].astype(np.float64)
        compare(o[i], np.broadcast_to(v.mean(0), o[i].shape), np.broadcast_to(A.tolerance(np.abs(v).mean(0), 0.0, d), o[i].shape),
                f"logit {aims[i]:.3g}")
    compare(lse, wl, ltol, "lse")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,order", [(64, 1), (128, 1), (128, -1), (256, -1)])
def test_one_key_above_all_others(lq, cuda_dev, route, fmt, d, order):
    """Logits that grow (or fall) by a hundredth of their size from key to
    key, far more than they can be off: the largest takes all weight."""
    keys = 80
    P, aims = _rows(lq, fmt, d, cuda_dev, keys, seed=33)
    steps = (0.2 + np.arange(keys) / 100.0)[::order]
    for i, aim in enumerate(aims):
        P.k[i][:] = P.k[i][:1] * steps[:, None, None].astype(np.float32)
        P.store(0, i, P.k[i])
        _aim(P, i, aim, P.values(0, i)[int(np.argmax(steps)), 0])
    o, _ = _run(lq, P, route=route)
    checked = 0
    for i, aim in enumerate(aims):
        x = P.values(0, i)[:, 0].astype(np.float64) @ P.q[i, 0].astype(np.float64) / np.sqrt(d)
        a = np.argsort(x)
        gap, off = x[a[-1]] - x[a[-2]], 2.0 * (d / 8 + 8) * 2.0**-23 * np.abs(x).max()
        if gap < 4 * off + 60.0:  # (ordinary sizes; equal stored keys)
            continue
        v = P.values(1, i)[a[-1], 0].astype(np.float64)
        compare(o[i], np.broadcast_to(v, o[i].shape), np.broadcast_to(2.0**-17 * np.abs(v) + 1e-37, o[i].shape), f"logit {aim:.3g}")
        checked += 1
    assert checked >= len(aims) - 8


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_logits_beyond_float32(lq, cuda_dev, route, fmt, d):
    """A logit of +inf makes its row NaN, one of -inf has no weight; rows that
    see nothing but such logits get zeros and -inf, as if they saw nothing."""
    P = Paged(lq, fmt, [1] * 4, [40, 40, 40, 7], 2, 1, d, 16, cuda_dev, seed=34)
    for i in range(4):
        P.k[i][:] = P.k[i][:1]
        if i == 2:
            P.k[i][35] *= np.float32(1e-3)
        P.store(0, i, P.k[i])
        k = P.values(0, i)[0, 0].astype(np.float64)
        big = 4e38 * np.sqrt(d) / (k @ k) * k  # scale q . k is 4e38
        assert np.abs(big).max() < 3e38
        P.q[i] = (big if i == 0 else -big).astype(np.float32)
    o, lse = _run(lq, P, route=route)
    assert np.isnan(o[0]).all() and not np.isfinite(lse[0]).any()
    for i in (1, 3):
        assert (o[i] == 0).all() and (lse[i] == -np.inf).all()
    v = P.values(1, 2)[35, 0].astype(np.float64)
    compare(o[2], np.broadcast_to(v, o[2].shape), np.broadcast_to(2.0**-17 * np.abs(v), o[2].shape), "the finite logit")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_queries_that_are_not_finite(lq, cuda_dev, route, fmt, what):
    """Their own rows become NaN, no others; a row that sees nothing stays
    zero whatever its query."""
    P = Paged(lq, fmt, [3, 2, 1], [77, 2, 1], 2, 1, 128, 16, cuda_dev, seed=35)
    P.k[0][:, :, 9] = np.abs(P.k[0][:, :, 9]) + 0.5  # every logit of that dim alone has the query's sign
    P.store(0, 0, P.k[0])
    table = P.table.copy()
    table[2, 0] = -1
    P.q[1, 1, 9] = what
    P.q[2, 0, 100] = what
    P.q[5, 1, 3] = what
    Q = P.q.copy()
    P.q[[1, 2, 5], [1, 0, 1]] = 0
    want, tol, wl, ltol = P.expect(table=table)
    o, lse = _run(lq, P, route=route, table=table, q=Q)
    bad = np.zeros((6, 2), bool)
    bad[1, 1] = bad[2, 0] = True
    assert np.isnan(o[bad]).all() and np.isnan(lse[bad]).all()
    compare(o[~bad], want[~bad], tol[~bad], "the other rows")
    compare(lse[~bad], wl[~bad], ltol[~bad], "the other rows' lse")
    assert (o[5] == 0).all() and (lse[5] == -np.inf).all()


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_and_values_at_the_top_of_the_range(lq, cuda_dev, route, fmt, d):
    """Elements of up to +-65504 (and clamped ones), whose blocks have the
    largest scales that the cache holds, beside ordinary ones."""
    P = Paged(lq, fmt, [1, 30], [140, 75], 4, 2, d, 16, cuda_dev, seed=36)
    rng = np.random.default_rng(36)
    for which, x in ((0, P.k), (1, P.v)):
        for i in range(2):
            x[i] *= np.float32(200.0)
            at = rng.random(x[i].shape) < 0.02
            x[i][at] = rng.choice(np.float32([65504, -65504, 65503, -65490, 1e6, -1e6, 60000, -33000]), at.sum())
            P.store(which, i, x[i])
    P.q *= np.float32(1e-4)
    o, lse = _run(lq, P, route=route)
    want, tol, wl, ltol = P.expect()
    assert all(np.abs(P.values(w, i)).max() >= 65504 for w in (0, 1) for i in (0, 1))
    compare(o, want, tol, "output")
    compare(lse, wl, ltol, "lse")
