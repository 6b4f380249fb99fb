"""Host-side checks of the paged cache's and the attention's entry points:
sizes, refusals and no-ops, all before any launch (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import oracle as O
from oracle import attention as A

P = 0x10000  # never dereferenced


def _cache(lq, **kw):
    f = dict(fmt=1, page_size=16, kv_heads=2, head_dim=64, num_pages=4, k=P, v=P)
    f.update(kw)
    return ctypes.byref(lq.KVCacheStruct(**f))


def _batch(lq, **kw):
    f = dict(batch=1, max_pages=2, tokens=3, max_q=0, page_table=P, kv_len=P, q_start=P)
    f.update(kw)
    return ctypes.byref(lq.KVBatchStruct(**f))


@pytest.mark.parametrize("fmt,code,bits", [("f16", 0, 16), ("q8_0", 1, 8.5), ("q4_0", 2, 4.5)])
def test_pool_bytes(lq, fmt, code, bits):
    L = lq.lib()
    assert L.lq_kv_pool_bytes(code, 5, 16, 3, 96) == 5 * 16 * 3 * 96 * bits / 8
    assert L.lq_kv_pool_bytes(code, 1 << 20, 16, 8, 128) == (1 << 20) * 16 * 8 * 128 * bits / 8  # past 32 bits
    for bad in ((code, -1, 16, 1, 64), (code, 1, 0, 1, 64), (code, 1, 16, 0, 64), (code, 1, 16, 1, 48), (code, 1, 16, 1, 288),
                (3, 1, 16, 1, 64), (9, 1, 16, 1, 64)):
        assert L.lq_kv_pool_bytes(*bad) == 0


BAD_CACHES = [dict(fmt=7), dict(fmt=-1), dict(page_size=0), dict(page_size=70000), dict(kv_heads=0), dict(head_dim=0),
              dict(head_dim=40), dict(num_pages=-1), dict(k=None), dict(v=None), dict(k=P + 1), dict(v=P + 1)]
BAD_BATCHES = [dict(batch=-1), dict(tokens=-1), dict(max_pages=-1), dict(max_q=-1), dict(page_table=None), dict(kv_len=None),
               dict(q_start=None), dict(page_table=P + 2), dict(kv_len=P + 1), dict(q_start=P + 3)]


def _calls(lq):
    L = lq.lib()
    return {
        "write": lambda c, b, x=P, ld=128, y=P, ld2=128: L.lq_kv_write(c, b, x, ld, y, ld2, 0),
        "read": lambda c, b, x=P, ld=128, y=P, ld2=128: L.lq_kv_read(c, b, x, ld, y, ld2, 0),
        "attn": lambda c, b, x=P, ld=256, y=P, ld2=256, heads=4, scale=0.1, window=0, sinks=0, lse=0, work=P:
            L.lq_attn_paged(c, b, x, ld, y, ld2, lse, heads, scale, window, sinks, work, 0),
    }


@pytest.mark.parametrize("name", ["write", "read", "attn"])
def test_refusals_of_every_call(lq, name):
    f = _calls(lq)[name]
    c, b = _cache(lq), _batch(lq)
    for bad in BAD_CACHES:
        assert f(_cache(lq, **bad), b) == lq.LQ_ERR_INVALID_ARG, bad
    for bad in BAD_BATCHES:
        assert f(c, _batch(lq, **bad)) == lq.LQ_ERR_INVALID_ARG, bad
    assert f(None, b) == lq.LQ_ERR_INVALID_ARG and f(c, None) == lq.LQ_ERR_INVALID_ARG
    assert f(_cache(lq, fmt=3), b) == lq.LQ_ERR_UNSUPPORTED  # interleaved nibbles
    assert f(_cache(lq, head_dim=288), b) == lq.LQ_ERR_UNSUPPORTED
    assert f(c, b, x=P + 2) == lq.LQ_ERR_INVALID_ARG and f(c, b, y=P + 1) == lq.LQ_ERR_INVALID_ARG
    assert f(c, b, ld=100) == lq.LQ_ERR_INVALID_ARG and f(c, b, ld2=100) == lq.LQ_ERR_INVALID_ARG
    for none in (dict(batch=0), dict(tokens=0)):
        assert f(c, _batch(lq, **none)) == lq.LQ_OK
        assert f(_cache(lq, k=None, v=None), _batch(lq, page_table=None, **none)) == lq.LQ_OK


def test_refusals_of_one_call(lq):
    f = _calls(lq)
    c, b = _cache(lq), _batch(lq)
    assert f["write"](c, b, x=None) == f["write"](c, b, y=None) == f["read"](c, b, x=None, y=None) == lq.LQ_ERR_INVALID_ARG
    for bad in (dict(x=None), dict(y=None), dict(work=None), dict(work=P + 8), dict(lse=P + 2), dict(heads=0), dict(heads=3),
                dict(heads=-2), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert f["attn"](c, b, **bad) == lq.LQ_ERR_INVALID_ARG, bad
    for bad in (-1, 4):
        with pytest.raises(lq.LQError):
            lq.attn_route(bad)


def test_work_bytes(lq):
    L = lq.lib()
    n = L.lq_attn_work_bytes(_cache(lq), _batch(lq), 4)
    assert n > 0 and n % 16 == 0
    assert L.lq_attn_work_bytes(_cache(lq), _batch(lq), 3) == 0
    assert L.lq_attn_work_bytes(_cache(lq, head_dim=33), _batch(lq), 4) == 0


def test_python_wrappers_refuse(lq):
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    table, lens, starts = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for bad in ((table.long(), lens, starts), (table, lens[:1], starts), (table, lens, starts[:2]), (table.t(), lens, starts)):
        with pytest.raises(lq.LQError):
            lq.KVBatch(*bad, 4)
    with pytest.raises(lq.LQError):
        lq.KVCache("q8_0", 2, 16, 1, 33, k=P, v=P)
    with pytest.raises(lq.LQError):
        lq.KVCache("q8_0", 2, 16, 1, 64, k=torch.zeros(10, dtype=torch.uint8), v=P)
    cache, batch = lq.KVCache("q8_0", 2, 16, 1, 64, k=P, v=P), lq.KVBatch(table, lens, starts, 4)
    ok = torch.zeros(4, 1, 64)
    for bad in (ok.double(), ok[:3], torch.zeros(4, 1, 32), torch.zeros(4, 64, 1).transpose(1, 2)[:, :, ::2],
                torch.zeros(4, 2, 64)[:, ::2].transpose(0, 2)):
        with pytest.raises(lq.LQError):
            lq.lq_kv_write(cache, batch, bad, ok, stream=0)
    with pytest.raises(lq.LQError):
        lq.lq_attn_paged(cache, batch, ok, ok, 1.0, stream=0)  # a stream, but no work buffer
    with pytest.raises(lq.LQError):
        lq.lq_attn_paged(cache, batch, ok, ok, 1.0, work=P, lse=torch.zeros(4, 2), stream=0)


# ---- the oracle itself ------------------------------------------------------
def test_oracle_attention_by_hand():
    """Two keys with logits 0 and ln 3: weights 1/4 and 3/4."""
    k = np.array([[0.0, 0.0], [np.log(3.0), 0.0]])
    v = np.array([[4.0, 8.0], [8.0, -4.0]])
    o, lse, bound, _ = A.attend(np.array([1.0, 0.0]), k, v, np.array([True, True]), 1.0)
    assert np.allclose(o, [7.0, -1.0]) and np.isclose(lse, np.log(4.0)) and np.allclose(bound, [7.0, 5.0])
    o, lse, _, _ = A.attend(np.array([1.0, 0.0]), k, v, np.array([True, False]), 1.0)
    assert np.allclose(o, v[0]) and lse == 0.0
    o, lse, _, _ = A.attend(np.array([1.0, 0.0]), k, v, np.array([False, False]), 1.0)
    assert np.all(o == 0) and lse == -np.inf


def test_oracle_visibility():
    assert list(np.flatnonzero(A.visible(5, 9, 0, 3))) == [0, 1, 2, 3, 4, 5]
    assert list(np.flatnonzero(A.visible(7, 9, 2, 3))) == [0, 1, 2, 6, 7]
    assert list(np.flatnonzero(A.visible(1, 9, 5, 3))) == [0, 1]
    assert not A.visible(-1, 9, 2, 3).any()


@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
def test_oracle_cache_rows_are_the_packed_blocks(fmt):
    x = np.random.default_rng(0).standard_normal((5, 96)).astype(np.float32)
    codes, scales = A.cache_rows(fmt, x)
    packed = O.pack(fmt, x).view(np.uint8).reshape(5, -1)
    if fmt == "f16":
        assert np.array_equal(codes, packed)
    else:
        blocks = packed.reshape(5, 3, -1)
        assert np.array_equal(codes.reshape(5, 3, -1), blocks[:, :, 2:])
        assert np.array_equal(scales.view(np.uint8).reshape(5, 3, 2), blocks[:, :, :2])
    big = np.full((1, 32), np.inf, np.float32)
    assert np.all(np.isfinite(A.cache_values(fmt, big)))
