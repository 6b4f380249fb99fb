"""What the Python binding of the paged cache and its attention refuses before
any launch (no GPU needed): scratch buffers that are too small, results of
another type, and tensors that are not where the batch is. GPU tensors are
stood in for by objects that say they are one."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

P = 0x10000  # never dereferenced
I32 = torch.int32


class OnGpu:
    """A tensor's shape and type, said to be on GPU `index` at address P."""

    def __init__(self, *shape, dtype=torch.float32, index=0, at=P):
        self.x = torch.empty(*shape, dtype=dtype, device="meta")
        self.index, self.at = index, at
        self.device = torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.x, name)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.at


def _batch(lq, index=0, **kw):
    f = dict(tokens=4, max_q=0)
    f.update(kw)
    return lq.KVBatch(OnGpu(2, 3, dtype=I32, index=index), OnGpu(2, dtype=I32, index=index), OnGpu(3, dtype=I32, index=index), **f)


@pytest.fixture
def calls(lq, monkeypatch):
    """The C calls that were reached, which do nothing here."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            if name in ("lq_kv_write", "lq_kv_read", "lq_attn_paged"):
                return lambda *a: seen.append(name) or 0
            return getattr(real, name)
    real = lq.lib()
    monkeypatch.setattr(lq, "_lib", Lib())
    return seen


def _need(lq, head_dim):
    c = lq.KVCacheStruct(fmt=1, page_size=16, kv_heads=2, head_dim=head_dim, num_pages=4, k=P, v=P)
    b = lq.KVBatchStruct(batch=1, max_pages=2, tokens=3, max_q=0, page_table=P, kv_len=P, q_start=P)
    return lq.lib().lq_attn_work_bytes(ctypes.byref(c), ctypes.byref(b), 2)


@pytest.mark.parametrize("made_for,used_with", [(64, 128), (96, 128), (96, 64), (32, 256), (224, 64)])
def test_work_of_another_geometry(lq, calls, made_for, used_with):
    """A buffer that is too small is refused, one that is large enough serves."""
    small, large = _need(lq, made_for), _need(lq, used_with)
    assert 0 < small < large
    cache, batch = lq.KVCache("q8_0", 4, 16, 2, used_with, k=P, v=P), _batch(lq)
    q = OnGpu(4, 2, used_with)
    for n in (small, large - 1, 0):
        with pytest.raises(lq.LQError) as e:
            lq.lq_attn_paged(cache, batch, q, q, 1.0, work=OnGpu(n, dtype=torch.uint8), stream=0)
        assert e.value.status == lq.LQ_ERR_INVALID_ARG
    apart = OnGpu(large, 2, dtype=torch.uint8)
    apart.x = apart.x[:, 0]
    with pytest.raises(lq.LQError):
        lq.lq_attn_paged(cache, batch, q, q, 1.0, work=apart, stream=0)
    assert not calls
    lq.lq_attn_paged(cache, batch, q, q, 1.0, work=OnGpu(large, dtype=torch.uint8), stream=0)
    lq.lq_attn_paged(cache, batch, q, q, 1.0, work=OnGpu(-(-large // 4), dtype=torch.float32), stream=0)
    other = lq.KVCache("f16", 4, 16, 2, made_for, k=P, v=P)
    lq.lq_attn_paged(other, batch, OnGpu(4, 2, made_for), OnGpu(4, 2, made_for), 1.0, work=OnGpu(large, dtype=torch.uint8), stream=0)
    assert calls == ["lq_attn_paged"] * 3


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float64, torch.int32])
def test_lse_of_another_type(lq, calls, dtype):
    cache, batch = lq.KVCache("f16", 4, 16, 2, 64, k=P, v=P), _batch(lq)
    q = OnGpu(4, 2, 64)
    with pytest.raises(lq.LQError):
        lq.lq_attn_paged(cache, batch, q, q, 1.0, work=P, lse=OnGpu(4, 2, dtype=dtype), stream=0)
    assert not calls
    lq.lq_attn_paged(cache, batch, q, q, 1.0, work=P, lse=OnGpu(4, 2), stream=0)
    assert calls


def test_tensors_of_another_device(lq, calls):
    """CPU tensors and those of another GPU than the page table's."""
    cache, batch, work = lq.KVCache("f16", 4, 16, 2, 64, k=P, v=P), _batch(lq), OnGpu(1 << 26, dtype=torch.uint8)
    x = OnGpu(4, 2, 64)
    for bad in (torch.zeros(4, 2, 64), OnGpu(4, 2, 64, index=1)):
        for a, b in ((bad, x), (x, bad)):
            for call in (lq.lq_kv_write, lq.lq_kv_read):
                with pytest.raises(lq.LQError):
                    call(cache, batch, a, b, stream=0)
            with pytest.raises(lq.LQError):
                lq.lq_attn_paged(cache, batch, a, b, 1.0, work=work, stream=0)
    for lse in (torch.zeros(4, 2), OnGpu(4, 2, index=1)):
        with pytest.raises(lq.LQError):
            lq.lq_attn_paged(cache, batch, x, x, 1.0, work=work, lse=lse, stream=0)
    for w in (torch.zeros(1 << 26, dtype=torch.uint8), OnGpu(1 << 26, dtype=torch.uint8, index=1)):
        with pytest.raises(lq.LQError):
            lq.lq_attn_paged(cache, batch, x, x, 1.0, work=w, stream=0)
    # a batch on the CPU, with rows given as addresses too; a cache on another GPU
    on_cpu = lq.KVBatch(torch.zeros(2, 3, dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(3, dtype=I32), 4)
    pool = int(lq.lib().lq_kv_pool_bytes(0, 4, 16, 2, 64))
    elsewhere = lq.KVCache("f16", 4, 16, 2, 64, k=OnGpu(pool, dtype=torch.uint8, index=1), v=OnGpu(pool, dtype=torch.uint8, index=1))
    for c, b, rows in ((cache, on_cpu, P), (cache, on_cpu, torch.zeros(4, 2, 64)), (elsewhere, batch, x), (elsewhere, batch, P)):
        for call in (lq.lq_kv_write, lq.lq_kv_read):
            with pytest.raises(lq.LQError):
                call(c, b, rows, rows, stream=0)
        with pytest.raises(lq.LQError):
            lq.lq_attn_paged(c, b, rows, rows, 1.0, work=P, heads=2, stream=0)
    # parts of one object on different devices
    with pytest.raises(lq.LQError):
        lq.KVBatch(OnGpu(2, 3, dtype=I32), OnGpu(2, dtype=I32, index=1), OnGpu(3, dtype=I32), 4)
    with pytest.raises(lq.LQError):
        lq.KVCache("f16", 4, 16, 2, 64, k=torch.zeros(pool, dtype=torch.uint8), v=P)
    with pytest.raises(lq.LQError):
        lq.KVCache("f16", 4, 16, 2, 64, k=OnGpu(pool, dtype=torch.uint8), v=OnGpu(pool, dtype=torch.uint8, index=1))
    assert not calls
    # addresses and tensors of the same GPU go through
    here = lq.KVCache("f16", 4, 16, 2, 64, k=OnGpu(pool, dtype=torch.uint8), v=P)
    for rows in (x, P):
        lq.lq_kv_write(here, batch, rows, rows, stream=0)
        lq.lq_kv_read(here, batch, rows, None, stream=0)
        lq.lq_attn_paged(here, batch, rows, rows, 1.0, work=P, heads=2, stream=0)
    assert calls == ["lq_kv_write", "lq_kv_read", "lq_attn_paged"] * 2


def test_page_table_of_another_rank(lq):
    for table in (torch.zeros(4, dtype=I32), torch.zeros(2, 2, 2, dtype=I32)):
        with pytest.raises(lq.LQError):
            lq.KVBatch(table, torch.zeros(table.shape[0], dtype=I32), torch.zeros(table.shape[0] + 1, dtype=I32), 4)
