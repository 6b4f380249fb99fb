"""What the rotary, tree and beam entry points refuse, and their no-ops, all
before any launch (no GPU needed): the C calls on addresses that are never
read, and the Python binding on stand-ins for GPU tensors."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_attn_abi_cpu import BAD_BATCHES, BAD_CACHES, P, _batch, _cache  # noqa: E402
from test_attn_refusals_cpu import I32, OnGpu  # noqa: E402


def _table(lq, **kw):
    t = lq.Rope(64, 32).struct
    for n, v in kw.items():
        setattr(t, n, v)
    return ctypes.byref(t)


# ---- tables of angles -----------------------------------------------------------
@pytest.mark.parametrize("head_dim,rotary,kw", [
    (63, 32, {}), (64, 31, {}), (64, 66, {}), (64, 0, {}), (0, 0, {}), (64, 64, dict(base=0.0)), (64, 64, dict(base=-1.0)),
    (64, 64, dict(base=math.inf)), (64, 64, dict(base=math.nan)), (64, 64, dict(factor=math.inf)), (64, 64, dict(factor=1e300)),
    (64, 64, dict(sections=[16, 15])), (64, 64, dict(sections=[33, -1])), (64, 64, dict(sections=[])), (64, 64, dict(sections=[31])),
    (20, 20, dict(sections=[4, 6], interleaved=True)), (64, 64, dict(freqs=[1.0] * 31 + [math.nan])), (64, 64, dict(freqs=[1.0] * 31)),
    (64, 64, dict(freqs=[math.inf] * 32)), (64, 64, dict(freqs=[5e9] * 32)), (64, 64, dict(base=1e-300))])
def test_angles_that_are_refused(lq, head_dim, rotary, kw):
    with pytest.raises(lq.LQError) as e:
        lq.Rope(head_dim, rotary, **kw)
    assert e.value.status == lq.LQ_ERR_INVALID_ARG


@pytest.mark.parametrize("head_dim,rotary,kw", [(512, 258, {}), (65538, 64, {}), (64, 64, dict(sections=[8, 8, 8, 4, 4]))])
def test_angles_that_are_too_many(lq, head_dim, rotary, kw):
    with pytest.raises(lq.LQError) as e:
        lq.Rope(head_dim, rotary, **kw)
    assert e.value.status == lq.LQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("sections,interleaved,want", [
    (None, False, [0] * 8), ([3, 2, 3], False, [0, 0, 0, 1, 1, 2, 2, 2]), ([0, 0, 8], False, [2] * 8), ([8, 0], True, [0] * 8),
    ([4, 2, 2], True, [0, 1, 2, 0, 1, 2, 0, 0]), ([2, 3, 3], False, [0, 0, 1, 1, 1, 2, 2, 2]), ([4, 3, 1], True, [0, 1, 2, 0, 1, 0, 0, 1])])
def test_axes_of_the_pairs(lq, sections, interleaved, want):
    r = lq.Rope(32, 16, sections=sections, interleaved=interleaved)
    assert list(r.struct.axis)[:8] == want
    assert [sum(a == x for a in want) for x in range(r.axes)] == (sections or [8])


def test_turns_are_the_frequencies(lq):
    """In 2^-64 of a turn, modulo one: the nearest whole number, within the two
    roundings of the pair of doubles."""
    freqs = [1.0, 1e-3, 1e-9, 0.0, -0.25, 7.0, -100.0, 2 * math.pi]
    r = lq.Rope(16, freqs=freqs)
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10**50)
    for f, turns in zip(freqs, r.struct.turns):
        want = Fraction(f) / two_pi
        off = (Fraction(turns) - (want - math.floor(want)) * 2**64) % 2**64
        assert min(off, 2**64 - off) <= 2 + abs(want) * Fraction(1, 2**40) * 2**24


# ---- the C calls -----------------------------------------------------------------
def test_rope_refusals(lq):
    L = lq.lib()

    def f(t=None, n=4, pos=P, ldp=4, q=P, ldq=128, qo=P, ldqo=128, h=2, k=P, ldk=64, ko=P, ldko=64, hk=1):
        return L.lq_rope(_table(lq) if t is None else t, n, pos, ldp, q, ldq, qo, ldqo, h, k, ldk, ko, ldko, hk, 0, 0)

    bad = lq.LQ_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(h=-1), dict(hk=-1), dict(pos=0), dict(pos=P + 2), dict(q=0), dict(qo=0), dict(k=0), dict(ko=0), dict(q=P + 1),
               dict(qo=P + 2), dict(k=P + 3), dict(ldq=127), dict(ldqo=127), dict(ldk=63), dict(ldko=63), dict(ldqo=132),
               dict(t=_table(lq, axes=0)), dict(t=_table(lq, axes=5)), dict(t=_table(lq, rotary_dim=33)), dict(t=_table(lq, rotary_dim=66)),
               dict(t=_table(lq, pairs=2)), dict(t=_table(lq, head_dim=0)), dict(t=_table(lq, factor=math.nan)),
               dict(t=_table(lq, axes=2), ldp=3)):
        assert f(**kw) == bad, kw
    t = lq.Rope(64, 32).struct
    t.axis[15] = 1
    assert f(t=ctypes.byref(t)) == bad
    assert L.lq_rope(None, 4, P, 4, P, 128, P, 128, 2, P, 64, P, 64, 1, 0, 0) == bad
    assert f(n=0) == lq.LQ_OK and f(h=0, hk=0, pos=0) == lq.LQ_OK
    assert f(h=65537, ldq=1 << 40, ldqo=1 << 40) == lq.LQ_ERR_UNSUPPORTED and f(n=1 << 31) == lq.LQ_ERR_UNSUPPORTED


def test_tree_refusals(lq):
    L = lq.lib()
    bad, big = lq.LQ_ERR_INVALID_ARG, lq.LQ_ERR_UNSUPPORTED
    b, c = _batch(lq), _cache(lq)

    def plan(b=b, parent=P, pos=P, mask=P, words=1, window=0, sinks=0):
        return L.lq_tree_plan(b, parent, pos, mask, words, window, sinks, 0)

    for kw in (dict(b=None), dict(parent=0), dict(parent=P + 1), dict(pos=P + 1), dict(mask=P + 2), dict(pos=0, mask=0), dict(words=0),
               dict(words=-1), dict(window=-1), dict(sinks=-1), dict(b=_batch(lq, batch=-1)), dict(b=_batch(lq, tokens=-1)),
               dict(b=_batch(lq, kv_len=None)), dict(b=_batch(lq, q_start=None)), dict(b=_batch(lq, q_start=P + 1))):
        assert plan(**kw) == bad, kw
    assert plan(words=65537) == big and plan(b=_batch(lq, tokens=1 << 31)) == big
    assert plan(b=_batch(lq, batch=0)) == plan(b=_batch(lq, tokens=0), parent=0) == lq.LQ_OK

    def tree(c=c, b=b, mask=P, words=1, pos=P, x=P, ld=256, y=P, ld2=256, heads=4, scale=0.1, window=0, sinks=0, lse=0, work=P):
        return L.lq_attn_tree(c, b, mask, words, pos, x, ld, y, ld2, lse, heads, scale, window, sinks, work, 0)

    for kw in ([dict(c=_cache(lq, **x)) for x in BAD_CACHES] + [dict(b=_batch(lq, **x)) for x in BAD_BATCHES] +
               [dict(c=None), dict(b=None), dict(mask=0), dict(mask=P + 1), dict(words=0), dict(words=-3), dict(pos=P + 2), dict(pos=0, window=9),
                dict(x=0), dict(y=0), dict(x=P + 1), dict(ld=255), dict(ld2=255), dict(heads=3), dict(heads=0), dict(scale=math.inf),
                dict(window=-1), dict(sinks=-1), dict(work=0), dict(work=P + 8), dict(lse=P + 1)]):
        assert tree(**kw) == bad, kw
    assert tree(words=65537) == big and tree(c=_cache(lq, head_dim=288), ld=4 * 288, ld2=4 * 288) == big
    assert tree(c=_cache(lq, fmt=3)) == big
    assert tree(b=_batch(lq, batch=0), mask=0, work=0) == lq.LQ_OK

    def accept(b=b, parent=P, token=P, target=P, keep=P, most=4, count=P, after=P, length=2 * P):
        return L.lq_tree_accept(b, parent, token, target, keep, most, count, after, length, 0)

    for kw in (dict(b=None), dict(parent=0), dict(token=0), dict(target=0), dict(keep=0), dict(count=0), dict(after=0), dict(length=0),
               dict(parent=P + 1), dict(keep=P + 1), dict(length=P + 2), dict(most=0), dict(length=P)):
        assert accept(**kw) == bad, kw
    assert accept(most=1 << 25) == big and accept(b=_batch(lq, batch=0), keep=0) == lq.LQ_OK

    def keep(c=c, b=b, k=P, most=4, count=P):
        return L.lq_kv_keep(c, b, k, most, count, 0)

    for kw in ([dict(c=_cache(lq, **x)) for x in BAD_CACHES] + [dict(b=_batch(lq, **x)) for x in BAD_BATCHES] +
               [dict(k=0), dict(k=P + 1), dict(count=0), dict(count=P + 3), dict(most=0), dict(most=-1)]):
        assert keep(**kw) == bad, kw
    assert keep(most=1 << 25) == big and keep(c=_cache(lq, fmt=3)) == big
    assert keep(b=_batch(lq, tokens=0), k=0) == lq.LQ_OK


def test_beam_refusals(lq):
    L = lq.lib()
    bad, big = lq.LQ_ERR_INVALID_ARG, lq.LQ_ERR_UNSUPPORTED

    def select(x=P, ld=100, s=P, groups=2, beams=4, vocab=100, k=4, done=0, pad=0, a=P, b=P, c=P, work=P):
        return L.lq_beam_select(x, ld, s, groups, beams, vocab, k, done, pad, a, b, c, work, 0)

    for kw in (dict(x=0), dict(s=0), dict(a=0), dict(b=0), dict(c=0), dict(work=0), dict(work=P + 8), dict(x=P + 1), dict(s=P + 2), dict(a=P + 1),
               dict(done=P + 1), dict(ld=99), dict(groups=-1), dict(beams=0), dict(vocab=0), dict(k=0), dict(done=P, pad=100), dict(done=P, pad=-1)):
        assert select(**kw) == bad, kw
    for kw in (dict(beams=65), dict(k=65), dict(vocab=(1 << 26) + 1, ld=1 << 27), dict(groups=(1 << 24) + 1), dict(groups=1 << 23)):
        assert select(**kw) == big, kw
    assert select(groups=0, x=0) == lq.LQ_OK
    work = L.lq_beam_work_bytes
    assert work(2, 4, 100, 4) > 0 and work(1, 64, 1 << 26, 64) > work(1, 4, 1 << 26, 4)
    for sizes in ((0, 4, 100, 4), (-1, 4, 100, 4), (2, 0, 100, 4), (2, 65, 100, 4), (2, 4, 0, 4), (2, 4, 100, 0), (2, 4, 100, 65),
                  (2, 4, (1 << 26) + 1, 4), (1 << 62, 4, 100, 4)):
        assert work(*sizes) == 0, sizes

    def pages(parent=P, groups=2, beams=4, table=P, most=3, lens=P, page=16, out=2 * P, copies=P):
        return L.lq_beam_pages(parent, groups, beams, table, most, lens, page, out, copies, 0)

    for kw in (dict(parent=0), dict(parent=P + 1), dict(table=0), dict(out=0), dict(lens=0), dict(copies=0), dict(out=P), dict(groups=-1),
               dict(beams=0), dict(most=-1), dict(page=0), dict(page=65537), dict(copies=P + 2)):
        assert pages(**kw) == bad, kw
    assert pages(beams=65) == big and pages(most=1 << 30) == big and pages(groups=1 << 29) == pages(beams=64, most=1 << 25, page=1) == big
    assert pages(groups=0, parent=0) == lq.LQ_OK

    for kw in BAD_CACHES:
        assert L.lq_kv_copy(_cache(lq, **kw), P, 3, 0) == bad, kw
    c = _cache(lq)
    assert L.lq_kv_copy(None, P, 3, 0) == L.lq_kv_copy(c, 0, 3, 0) == L.lq_kv_copy(c, P + 1, 3, 0) == L.lq_kv_copy(c, P, -1, 0) == bad
    assert L.lq_kv_copy(_cache(lq, fmt=3), P, 3, 0) == big
    assert L.lq_kv_copy(c, 0, 0, 0) == L.lq_kv_copy(_cache(lq, num_pages=0), P, 3, 0) == lq.LQ_OK


# ---- the Python calls --------------------------------------------------------------
@pytest.fixture
def calls(lq, monkeypatch):
    """The C calls that were reached, which do nothing here."""
    seen, real = [], lq.lib()
    fake = {"lq_rope", "lq_tree_plan", "lq_attn_tree", "lq_tree_accept", "lq_kv_keep", "lq_beam_select", "lq_beam_pages", "lq_kv_copy"}

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: seen.append(name) or 0) if name in fake else getattr(real, name)
    monkeypatch.setattr(lq, "_lib", Lib())
    return seen


def _refused(lq, call, *a, **kw):
    with pytest.raises(lq.LQError) as e:
        call(*a, **kw)
    assert e.value.status == lq.LQ_ERR_INVALID_ARG


def test_python_rope(lq, calls):
    r = lq.Rope(64, sections=[16, 16])
    q, k, pos = OnGpu(5, 4, 64), OnGpu(5, 2, 64), OnGpu(2, 5, dtype=I32)
    lq.lq_rope(r, pos, q, k, stream=0)
    lq.lq_rope(lq.Rope(64), OnGpu(5, dtype=I32), OnGpu(5, 256), stream=0)
    assert calls == ["lq_rope", "lq_rope"]
    for a, kw in (((OnGpu(5, dtype=I32), q), {}), ((OnGpu(3, 5, dtype=I32), q), {}), ((OnGpu(2, 4, dtype=I32), q), {}),
                  ((OnGpu(2, 5, dtype=torch.int64), q), {}), ((OnGpu(2, 5, dtype=I32, index=1), q), {}), ((pos, OnGpu(5, 4, 32)), {}),
                  ((pos, OnGpu(5, 100)), {}), ((pos, OnGpu(5, 4, 64, dtype=torch.float16)), {}), ((pos, OnGpu(5, 4, 64, dtype=I32)), {}),
                  ((pos, torch.zeros(5, 4, 64)), {}), ((pos, q, OnGpu(4, 2, 64)), {}), ((pos, q, OnGpu(5, 2, 64, index=1)), {}),
                  ((pos, q), dict(q_out=OnGpu(5, 3, 64))), ((pos, q, k), dict(k_out=OnGpu(5, 4, 64))), ((pos, q), dict(k_out=k))):
        _refused(lq, lq.lq_rope, r, *a, stream=0, **kw)
    x = OnGpu(5, 4, 64)
    x.x = torch.empty(5, 64, 4, device="meta").transpose(1, 2)
    _refused(lq, lq.lq_rope, r, pos, x, stream=0)
    assert len(calls) == 2


def _kv(lq, index=0):
    cache = lq.KVCache("f16", 4, 16, 2, 64, k=OnGpu(1 << 16, index=index), v=OnGpu(1 << 16, index=index))
    batch = lq.KVBatch(OnGpu(2, 3, dtype=I32, index=index), OnGpu(2, dtype=I32, index=index), OnGpu(3, dtype=I32, index=index), 6)
    return cache, batch


def test_python_tree(lq, calls):
    cache, batch = _kv(lq)
    t, m, ints = OnGpu(6, dtype=I32), OnGpu(6, 1, dtype=I32), OnGpu(2, dtype=I32)
    wrong = [OnGpu(5, dtype=I32), OnGpu(6, dtype=torch.int64), OnGpu(6, dtype=I32, index=1), torch.zeros(6, dtype=I32)]
    lq.lq_tree_plan(batch, t, t, m, stream=0)
    for x in wrong:
        _refused(lq, lq.lq_tree_plan, batch, x, t, m, stream=0)
        _refused(lq, lq.lq_tree_plan, batch, t, x, m, stream=0)
    _refused(lq, lq.lq_tree_plan, batch, t, t, OnGpu(5, 1, dtype=I32), stream=0)
    q, work = OnGpu(6, 4, 64), OnGpu(1 << 26)
    lq.lq_attn_tree(cache, batch, m, q, q, 0.1, positions=t, work=work, stream=0)
    for x in wrong:
        _refused(lq, lq.lq_attn_tree, cache, batch, m, q, q, 0.1, positions=x, work=work, stream=0)
    for x in (OnGpu(5, 1, dtype=I32), OnGpu(6, 1), OnGpu(6, 1, dtype=I32, index=1)):
        _refused(lq, lq.lq_attn_tree, cache, batch, x, q, q, 0.1, work=work, stream=0)
    _refused(lq, lq.lq_attn_tree, cache, batch, m, q, q, 0.1, work=OnGpu(100), stream=0)
    _refused(lq, lq.lq_attn_tree, cache, batch, m, q, q, 0.1, stream=0)
    _refused(lq, lq.lq_attn_tree, cache, batch, m, OnGpu(6, 4, 32), q, 0.1, work=work, stream=0)
    _refused(lq, lq.lq_attn_tree, _kv(lq, 1)[0], batch, m, q, q, 0.1, work=work, stream=0)
    keep, other = OnGpu(2, 4, dtype=I32), OnGpu(2, dtype=I32, at=2 * P)
    lq.lq_tree_accept(batch, t, t, t, keep, ints, ints, other, stream=0)
    for x in wrong:
        _refused(lq, lq.lq_tree_accept, batch, t, x, t, keep, ints, ints, other, stream=0)
    _refused(lq, lq.lq_tree_accept, batch, t, t, t, OnGpu(3, 4, dtype=I32), ints, ints, other, stream=0)
    _refused(lq, lq.lq_tree_accept, batch, t, t, t, keep, OnGpu(3, dtype=I32), ints, other, stream=0)
    lq.lq_kv_keep(cache, batch, keep, ints, stream=0)
    _refused(lq, lq.lq_kv_keep, cache, batch, OnGpu(1, 4, dtype=I32), ints, stream=0)
    _refused(lq, lq.lq_kv_keep, cache, batch, keep, OnGpu(2), stream=0)
    _refused(lq, lq.lq_kv_keep, _kv(lq, 1)[0], batch, keep, ints, stream=0)
    assert calls == ["lq_tree_plan", "lq_attn_tree", "lq_tree_accept", "lq_kv_keep"]


def test_python_beams(lq, calls):
    x, s, i, work = OnGpu(8, 100), OnGpu(8), OnGpu(2, 5, dtype=I32), OnGpu(1 << 20, dtype=torch.uint8)
    good = dict(logits=x, scores=s, beams=4, k=5, out_scores=OnGpu(2, 5), out_parents=i, out_tokens=i, work=work, stream=0)
    lq.lq_beam_select(**good)
    strided = OnGpu(8, 100)
    strided.x = torch.empty(8, 200, device="meta")[:, ::2]
    for kw in (dict(beams=3), dict(beams=0), dict(logits=OnGpu(8, 100, dtype=torch.float16)), dict(logits=torch.zeros(8, 100)), dict(logits=strided),
               dict(scores=OnGpu(7)), dict(scores=OnGpu(8, index=1)), dict(out_scores=OnGpu(2, 4)), dict(out_parents=OnGpu(2, 5)),
               dict(out_tokens=OnGpu(2, 4, dtype=I32)), dict(work=OnGpu(4)), dict(work=OnGpu(1 << 20, index=1)),
               dict(finished=OnGpu(8, dtype=torch.bool)), dict(finished=OnGpu(7, dtype=I32))):
        _refused(lq, lq.lq_beam_select, **{**good, **kw})
    n, t = OnGpu(8, dtype=I32), OnGpu(8, 3, dtype=I32)
    good = dict(parent=n, beams=4, table=t, kv_len=n, page_size=16, table_out=OnGpu(8, 3, dtype=I32, at=2 * P), copies=t, stream=0)
    lq.lq_beam_pages(**good)
    for kw in (dict(beams=3), dict(parent=OnGpu(8)), dict(kv_len=OnGpu(2, dtype=I32)), dict(table=OnGpu(7, 3, dtype=I32)), dict(table=n),
               dict(table_out=OnGpu(8, 4, dtype=I32)), dict(copies=OnGpu(8, 2, dtype=I32)), dict(copies=OnGpu(8, 3, dtype=I32, index=1))):
        _refused(lq, lq.lq_beam_pages, **{**good, **kw})
    cache = _kv(lq)[0]
    lq.lq_kv_copy(cache, t, stream=0)
    for c in (OnGpu(8, 2, dtype=I32), OnGpu(8, 3), OnGpu(8, 3, dtype=I32, index=1)):
        _refused(lq, lq.lq_kv_copy, cache, c, stream=0)
    assert calls == ["lq_beam_select", "lq_beam_pages", "lq_kv_copy"]
    _refused(lq, lq.beam_buffers, 2, 65, 100, 5)


def test_struct_is_the_headers(lq):
    """24 bytes, 128 numbers of 64 bits, 128 bytes."""
    assert ctypes.sizeof(lq.RopeTable) == 24 + 128 * 8 + 128
    assert lq.RopeTable.turns.offset == 24 and lq.RopeTable.axis.offset == 24 + 1024
    assert np.array_equal(np.ctypeslib.as_array(lq.Rope(64, 32).struct.axis), np.zeros(128))
