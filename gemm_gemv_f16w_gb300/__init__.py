"""Python binding of liblq, the GB300 weight-only matmul library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``liblq.so`` (built in-tree by ``gemm_gemv_f16w_gb300.build``).
The names match the C-ABI in ``include/lq.h``:

    lq_gemv_{f16,q8_0,q4_0}, lq_gemm_{f16,q8_0,q4_0}, lq_matmul_{f16,q8_0,q4_0}
    lq_pack_{f16,q8_0,q4_0}, lq_packed_bytes, lq_last_device_error, ...

Compute calls take torch CUDA tensors (A float32 [M,K], W packed bytes,
C float32 [M,N]) or raw device addresses; the stream defaults to torch's
current stream. A non-OK status raises ``LQError``. If the library is
missing, the first call fails loudly: there is no CPU path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# LQ_LIBRARY=debug loads the bounds-checking build (liblq_debug.so, see build.py)
LIB_PATH = os.path.join(_PKG, "liblq_debug.so" if os.environ.get("LQ_LIBRARY") == "debug" else "liblq.so")

LQ_OK, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_CUDA, LQ_ERR_DEVICE_TIMEOUT, LQ_ERR_BOUNDS = range(6)
FMT = {"f16": 0, "q8_0": 1, "q4_0": 2, "q4_0i": 3}  # q4_0i: the pages' interleaved nibbles
ROUTE_AUTO, ROUTE_STREAM, ROUTE_TENSOR_CORE, ROUTE_GENERIC = range(4)
ROUTE_WARP_MMA = 5         # tensor cores, warp-level MMAs, M = 2..48
COUNT_CHAIN, COUNT_PREPASS = 4, 6  # route_count(): decode-chain launches, route 2's A pre-pass launches

# every symbol include/lq.h declares
EXPORTS = [
    "lq_gemv_f16", "lq_gemv_q8_0", "lq_gemv_q4_0",
    "lq_gemm_f16", "lq_gemm_q8_0", "lq_gemm_q4_0",
    "lq_matmul_f16", "lq_matmul_q8_0", "lq_matmul_q4_0",
    "lq_packed_bytes", "lq_pack_f16", "lq_pack_q8_0", "lq_pack_q4_0",
    "lq_status_string", "lq_last_device_error", "lq_version",
    "lq_debug_force_route", "lq_debug_route_count", "lq_debug_reset_counts",
    "lq_debug_set_wait_limit_ns", "lq_gemm_noalloc", "lq_debug_gemv_plan", "lq_gemv_chain", "lq_debug_gemm_rings",
    "lq_debug_gemm_pairs",
    "lq_gemv_argmax", "lq_argmax_f32", "lq_matmul_residual", "lq_matmul_swiglu",
    "lq_gemv_q4_0i", "lq_gemm_q4_0i", "lq_matmul_q4_0i", "lq_pack_q4_0i", "lq_pack_q8_0_rcp",
    "lq_topk_work_bytes", "lq_topk_f32", "lq_gemv_topk", "lq_debug_chain_waits",
    "lq_kv_pool_bytes", "lq_kv_write", "lq_kv_read", "lq_attn_work_bytes", "lq_attn_paged", "lq_debug_attn_route",
    "lq_rope_init", "lq_rope", "lq_tree_plan", "lq_attn_tree", "lq_tree_accept", "lq_kv_keep",
    "lq_beam_work_bytes", "lq_beam_select", "lq_beam_pages", "lq_kv_copy",
]
_COMPUTE = [n for n in EXPORTS if n.split("_")[1] in ("gemv", "gemm", "matmul")]


class LQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded liblq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        for n in _COMPUTE:
            f = getattr(L, n)
            f.argtypes = [vp, vp, vp, i64, i64, i64, vp]
            f.restype = st
        L.lq_packed_bytes.argtypes = [ctypes.c_int, i64, i64]
        L.lq_packed_bytes.restype = ctypes.c_size_t
        for n in ("lq_pack_f16", "lq_pack_q8_0", "lq_pack_q4_0", "lq_pack_q4_0i", "lq_pack_q8_0_rcp"):
            f = getattr(L, n)
            f.argtypes = [vp, i64, i64, vp]
            f.restype = st
        L.lq_status_string.argtypes = [st]
        L.lq_status_string.restype = ctypes.c_char_p
        L.lq_last_device_error.argtypes = []
        L.lq_last_device_error.restype = st
        L.lq_version.restype = ctypes.c_char_p
        L.lq_debug_force_route.argtypes = [st]
        L.lq_debug_force_route.restype = st
        L.lq_debug_route_count.argtypes = [st]
        L.lq_debug_route_count.restype = ctypes.c_uint64
        L.lq_debug_reset_counts.argtypes = []
        L.lq_debug_reset_counts.restype = None
        L.lq_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.lq_debug_set_wait_limit_ns.restype = None
        L.lq_gemv_chain.argtypes = [st, ctypes.POINTER(GemvProblem), ctypes.c_int, vp]
        L.lq_gemv_chain.restype = st
        L.lq_debug_gemm_rings.argtypes = [ctypes.c_int, ctypes.c_int]
        L.lq_debug_gemm_rings.restype = st
        L.lq_debug_gemm_pairs.argtypes = [ctypes.c_int]
        L.lq_debug_gemm_pairs.restype = None
        L.lq_debug_chain_waits.argtypes = [ctypes.c_int]
        L.lq_debug_chain_waits.restype = None
        L.lq_debug_gemv_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.lq_debug_gemv_plan.restype = st
        L.lq_gemm_noalloc.argtypes = [st, vp, vp, vp, i64, i64, i64, vp]
        L.lq_gemm_noalloc.restype = st
        L.lq_gemv_argmax.argtypes = [st, vp, vp, vp, i64, i64, vp, vp]
        L.lq_gemv_argmax.restype = st
        L.lq_argmax_f32.argtypes = [vp, i64, vp, vp]
        L.lq_argmax_f32.restype = st
        L.lq_matmul_residual.argtypes = [st, vp, vp, vp, vp, i64, i64, i64, vp]
        L.lq_matmul_residual.restype = st
        L.lq_matmul_swiglu.argtypes = [st, vp, vp, vp, i64, i64, i64, vp]
        L.lq_matmul_swiglu.restype = st
        L.lq_topk_work_bytes.argtypes = [i64, ctypes.c_int]
        L.lq_topk_work_bytes.restype = ctypes.c_size_t
        L.lq_topk_f32.argtypes = [vp, i64, ctypes.c_int, vp, vp, vp, vp]
        L.lq_topk_f32.restype = st
        L.lq_gemv_topk.argtypes = [st, vp, vp, vp, i64, i64, ctypes.c_int, vp, vp, vp, vp]
        L.lq_gemv_topk.restype = st
        cp, bp = ctypes.POINTER(KVCacheStruct), ctypes.POINTER(KVBatchStruct)
        L.lq_kv_pool_bytes.argtypes = [ctypes.c_int, i64, i64, i64, i64]
        L.lq_kv_pool_bytes.restype = ctypes.c_size_t
        for n in ("lq_kv_write", "lq_kv_read"):
            f = getattr(L, n)
            f.argtypes = [cp, bp, vp, i64, vp, i64, vp]
            f.restype = st
        L.lq_attn_work_bytes.argtypes = [cp, bp, i64]
        L.lq_attn_work_bytes.restype = ctypes.c_size_t
        L.lq_attn_paged.argtypes = [cp, bp, vp, i64, vp, i64, vp, i64, ctypes.c_float, i64, i64, vp, vp]
        L.lq_attn_paged.restype = st
        rp, f64, c_int = ctypes.POINTER(RopeTable), ctypes.c_double, ctypes.c_int
        L.lq_rope_init.argtypes = [rp, i64, i64, c_int, f64, vp, i64, vp, c_int, f64]
        L.lq_rope.argtypes = [rp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, c_int, vp]
        L.lq_tree_plan.argtypes = [bp, vp, vp, vp, i64, i64, i64, vp]
        L.lq_attn_tree.argtypes = [cp, bp, vp, i64, vp, vp, i64, vp, i64, vp, i64, ctypes.c_float, i64, i64, vp, vp]
        L.lq_tree_accept.argtypes = [bp, vp, vp, vp, vp, i64, vp, vp, vp, vp]
        L.lq_kv_keep.argtypes = [cp, bp, vp, i64, vp, vp]
        L.lq_beam_work_bytes.argtypes = [i64, i64, i64, i64]
        L.lq_beam_work_bytes.restype = ctypes.c_size_t
        L.lq_beam_select.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, ctypes.c_int32, vp, vp, vp, vp, vp]
        L.lq_beam_pages.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, vp, vp]
        L.lq_kv_copy.argtypes = [cp, vp, i64, vp]
        for n in ("lq_rope_init", "lq_rope", "lq_tree_plan", "lq_attn_tree", "lq_tree_accept", "lq_kv_keep", "lq_beam_select",
                  "lq_beam_pages", "lq_kv_copy"):
            getattr(L, n).restype = st
        L.lq_debug_attn_route.argtypes = [st]
        L.lq_debug_attn_route.restype = st
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().lq_status_string(int(s)).decode()


def _check(s: int, what: str) -> None:
    if s != LQ_OK:
        raise LQError(s, what)


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, A, W, C, M, N, K, stream=None) -> None:
    _check(getattr(lib(), name)(_ptr(A), _ptr(W), _ptr(C), int(M), int(N), int(K), _stream(stream)),
           name)


def _make(name):
    def f(A, W, C, M, N, K, stream=None):
        _call(name, A, W, C, M, N, K, stream)
    f.__name__ = name
    f.__doc__ = f"{name}(A, W, C, M, N, K, stream=None): see include/lq.h."
    return f


for _n in _COMPUTE:
    globals()[_n] = _make(_n)


def matmul(fmt: str, A, W, N: int, K: int, out=None, kind: str = "matmul", stream=None):
    """C = A @ W^T for packed W of format ``fmt``; A is float32 CUDA [M, K].

    ``kind`` picks the entry point: "matmul" (router), "gemv" or "gemm".
    """
    import torch
    M = A.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _call(f"lq_{kind}_{fmt}", A, W, out, M, N, K, stream)
    return out


class GemvProblem(ctypes.Structure):
    """One problem of lq_gemv_chain (the lq_gemv_problem struct of lq.h)."""
    _fields_ = [("A", ctypes.c_void_p), ("W", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("after", ctypes.c_int32)]


def gemv_problems(items):
    """ctypes array of lq_gemv_problem from (A, W, C, N, K, after) tuples."""
    arr = (GemvProblem * len(items))()
    for i, (A, W, C, N, K, after) in enumerate(items):
        arr[i] = GemvProblem(_ptr(A), _ptr(W), _ptr(C), int(N), int(K), int(after))
    return arr


def lq_gemv_chain(fmt, problems, stream=None) -> int:
    """Runs lq_gemv_chain on a ctypes array from gemv_problems (or a list of
    tuples); returns the lq_status (LQ_ERR_UNSUPPORTED is not an exception:
    the caller falls back to one lq_gemv_<fmt> per problem)."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    arr = problems if isinstance(problems, ctypes.Array) else gemv_problems(problems)
    st = lib().lq_gemv_chain(f, arr, len(arr), _stream(stream))
    if st not in (LQ_OK, LQ_ERR_UNSUPPORTED):
        _check(st, "lq_gemv_chain")
    return st


def lq_gemm_noalloc(fmt, A, W, C, M, N, K, stream=None):
    """Tensor-core GEMM on the library's fixed workspace (no device
    allocation during the call); see include/lq.h for the limits."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib().lq_gemm_noalloc(f, _ptr(A), _ptr(W), _ptr(C), int(M), int(N), int(K),
                                 _stream(stream)), "lq_gemm_noalloc")


# ---- argmax ---------------------------------------------------------------
ARGMAX_RESULT_BYTES = 24  # sizeof(lq_argmax_result): value, index, 16 bytes of work


def argmax_result(dev=None):
    """A device buffer for one lq_argmax_result (int64 x 3, 8-byte aligned)."""
    import torch
    return torch.zeros(3, dtype=torch.int64, device=dev or "cuda")


def read_argmax(res):
    """(value, index) of an lq_argmax_result buffer (synchronises)."""
    raw = res.detach().cpu().numpy().view(np.uint8)
    return float(raw[0:4].view(np.float32)[0]), int(raw[4:8].view(np.int32)[0])


def lq_gemv_argmax(fmt, A, W, C, N, K, out, stream=None):
    """Fused GEMV (M = 1) + argmax into the device lq_argmax_result `out`
    (argmax_result()); C may be None. See include/lq.h."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib().lq_gemv_argmax(f, _ptr(A), _ptr(W), _ptr(C), int(N), int(K), _ptr(out),
                                _stream(stream)), "lq_gemv_argmax")


def lq_argmax_f32(x, n, out, stream=None):
    """Argmax of n device floats into the device lq_argmax_result `out`."""
    _check(lib().lq_argmax_f32(_ptr(x), int(n), _ptr(out), _stream(stream)), "lq_argmax_f32")


# ---- top-k ----------------------------------------------------------------
def topk_buffers(n, k, dev=None):
    """(values, indices, work) device buffers for a top-k of n entries."""
    import torch
    dev = dev or "cuda"
    nbytes = int(lib().lq_topk_work_bytes(int(n), int(k)))
    if nbytes == 0:
        raise LQError(LQ_ERR_INVALID_ARG, "lq_topk_work_bytes")
    return (torch.empty(k, dtype=torch.float32, device=dev), torch.empty(k, dtype=torch.int32, device=dev),
            torch.empty(nbytes // 8, dtype=torch.int64, device=dev))


def lq_topk_f32(x, n, k, values, indices, work, stream=None):
    _check(lib().lq_topk_f32(_ptr(x), int(n), int(k), _ptr(values), _ptr(indices), _ptr(work),
                             _stream(stream)), "lq_topk_f32")


def lq_gemv_topk(fmt, A, W, C, N, K, k, values, indices, work, stream=None):
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib().lq_gemv_topk(f, _ptr(A), _ptr(W), _ptr(C), int(N), int(K), int(k), _ptr(values),
                              _ptr(indices), _ptr(work), _stream(stream)), "lq_gemv_topk")


# ---- epilogue fusions ----------------------------------------------------
def lq_matmul_residual(fmt, A, W, R, C, M, N, K, stream=None):
    """C = A W^T + R (R may be C); see include/lq.h."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib().lq_matmul_residual(f, _ptr(A), _ptr(W), _ptr(R), _ptr(C), int(M), int(N), int(K),
                                    _stream(stream)), "lq_matmul_residual")


def lq_matmul_swiglu(fmt, A, W, H, M, I, K, stream=None):
    """H = silu(A gate^T) * (A up^T) for W = [gate; up] (2I rows); see
    include/lq.h."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib().lq_matmul_swiglu(f, _ptr(A), _ptr(W), _ptr(H), int(M), int(I), int(K), _stream(stream)),
           "lq_matmul_swiglu")


# ---- paged key/value cache and its attention -----------------------------
class KVCacheStruct(ctypes.Structure):
    """The lq_kv_cache struct of lq.h."""
    _fields_ = [("fmt", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class KVBatchStruct(ctypes.Structure):
    """The lq_kv_batch struct of lq.h."""
    _fields_ = [("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p)]


class KVCache:
    """The K and V pools of a paged cache (lq_kv_cache): allocated here, or
    the caller's own device buffers ``k`` and ``v``."""

    def __init__(self, fmt, num_pages, page_size, kv_heads, head_dim, k=None, v=None, device=None):
        code = FMT[fmt] if isinstance(fmt, str) else int(fmt)
        need = int(lib().lq_kv_pool_bytes(code, int(num_pages), int(page_size), int(kv_heads), int(head_dim)))
        if need == 0 and num_pages != 0:
            raise LQError(LQ_ERR_INVALID_ARG, "lq_kv_pool_bytes")
        pools, where = [], set()
        for pool in (k, v):
            if pool is None:
                import torch
                pool = torch.zeros(need, dtype=torch.uint8, device=device or "cuda")
            if not isinstance(pool, int):
                where.add(pool.get_device())
                if not pool.is_contiguous() or pool.numel() * pool.element_size() < need or min(where) < 0 or len(where) > 1:
                    raise LQError(LQ_ERR_INVALID_ARG, f"KVCache: pools of {need} contiguous bytes on one GPU are needed")
            pools.append(pool)
        self.k, self.v = pools
        self.gpu = where.pop() if where else None  # None: addresses, the caller's affair
        self.work_bytes = 0                        # what lq_attn_paged needs, once it is known
        self.struct = KVCacheStruct(code, int(page_size), int(kv_heads), int(head_dim), int(num_pages),
                                    _ptr(self.k), _ptr(self.v))
        self.ref = ctypes.byref(self.struct)
        self.head_dim, self.width = int(head_dim), int(kv_heads) * int(head_dim)


class KVBatch:
    """The tokens of a call (lq_kv_batch): int32 device tensors page_table
    [batch, max_pages], kv_len [batch] and q_start [batch + 1]."""

    def __init__(self, page_table, kv_len, q_start, tokens, max_q=0):
        self.gpu = page_table.get_device()
        for x, shape in ((page_table, None), (kv_len, (page_table.shape[0],)), (q_start, (page_table.shape[0] + 1,))):
            if str(x.dtype) != "torch.int32" or not x.is_contiguous() or len(x.shape) != (1 if shape else 2) \
                    or (shape and tuple(x.shape) != shape) or x.get_device() != self.gpu:
                raise LQError(LQ_ERR_INVALID_ARG, "KVBatch: contiguous int32 page_table [batch, max_pages], kv_len [batch] "
                                                  "and q_start [batch + 1] on one device")
        self.page_table, self.kv_len, self.q_start, self.tokens, self.batch = page_table, kv_len, q_start, int(tokens), page_table.shape[0]
        self.struct = KVBatchStruct(page_table.shape[0], page_table.shape[1], int(tokens), int(max_q), _ptr(page_table),
                                    _ptr(kv_len), _ptr(q_start))
        self.ref = ctypes.byref(self.struct)


def _elsewhere(cache, batch, what):
    """The cache's pools and the batch's tables have no GPU in common (pools
    given as addresses are taken to be on the batch's)."""
    if batch.gpu < 0 or cache.gpu is not None:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: the cache and the batch's tensors have to be on the same GPU")


def _rows(x, batch, width, what):
    """(address, leading dimension) of f32 rows [tokens, heads, head_dim] or
    [tokens, heads * head_dim]; a raw address is taken as tightly packed."""
    if x is None or isinstance(x, int):
        return x or 0, width
    tokens = batch.tokens
    if x.get_device() != batch.gpu:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: a tensor on {x.device} with a batch of another device")
    shape, strides = x.shape, x.stride()
    rank, rows = len(shape), shape[0]
    ok = rows >= tokens and strides[-1] == 1 and x.dtype.itemsize == 4 and x.is_floating_point()
    if rank == 3:
        ok = ok and shape[1] * shape[2] == width and (strides[1] == shape[2] or shape[1] == 1)
    else:
        ok = ok and rank == 2 and shape[1] == width
    if not ok:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: float32 [tokens, heads, head_dim] with contiguous heads and dims wanted, "
                                          f"got {tuple(shape)} {x.dtype}, strides {strides}")
    return x.data_ptr(), strides[0] if rows > 1 else width


_raw_stream = None


def _current_stream() -> int:
    """The handle of torch's current stream, by the quickest way there is."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.current_stream()  # initialises CUDA
        _raw_stream = (lambda: get(device())) if get and device else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def lq_kv_write(cache, batch, K, V, stream=None) -> None:
    """Stores the batch's tokens in the cache; K, V: float32 [tokens,
    kv_heads, head_dim] (token-strided slices allowed). See include/lq.h."""
    if cache.gpu != batch.gpu:
        _elsewhere(cache, batch, "lq_kv_write")
    k, ldk = _rows(K, batch, cache.width, "lq_kv_write")
    v, ldv = _rows(V, batch, cache.width, "lq_kv_write")
    st = (_lib or lib()).lq_kv_write(cache.ref, batch.ref, k, ldk, v, ldv, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_kv_write")


def lq_kv_read(cache, batch, K, V, stream=None) -> None:
    """Reads the batch's tokens back as float32 into K and V (either may be
    None). See include/lq.h."""
    if cache.gpu != batch.gpu:
        _elsewhere(cache, batch, "lq_kv_read")
    k, ldk = _rows(K, batch, cache.width, "lq_kv_read")
    v, ldv = _rows(V, batch, cache.width, "lq_kv_read")
    st = (_lib or lib()).lq_kv_read(cache.ref, batch.ref, k, ldk, v, ldv, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_kv_read")


def attn_work(cache, batch, heads, device=None):
    """The zero-filled scratch buffer of lq_attn_paged."""
    import torch
    nbytes = int(lib().lq_attn_work_bytes(cache.ref, batch.ref, int(heads)))
    if nbytes == 0:
        raise LQError(LQ_ERR_INVALID_ARG, "lq_attn_work_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or batch.page_table.device)


def _attn_operands(cache, batch, Q, O, lse, work, heads, stream, what):
    """The checks that lq_attn_paged and lq_attn_tree share; (q, ldq, o, ldo,
    lse, heads, work, stream) as the C calls take them."""
    if cache.gpu != batch.gpu:
        _elsewhere(cache, batch, what)
    D = cache.head_dim
    if heads is None:
        heads = Q.shape[1] if Q.dim() == 3 else Q.shape[1] // D
    if work is None:
        if stream is not None:
            raise LQError(LQ_ERR_INVALID_ARG, f"{what}: a call on a stream of its own brings its work buffer")
        work = attn_work(cache, batch, heads)
    elif not isinstance(work, int):
        need = cache.work_bytes
        if need == 0:  # (0 for arguments that the call itself refuses)
            need = cache.work_bytes = int(lib().lq_attn_work_bytes(cache.ref, batch.ref, cache.struct.kv_heads))
        if work.numel() * work.element_size() < need or not work.is_contiguous() or work.get_device() != batch.gpu:
            raise LQError(LQ_ERR_INVALID_ARG, f"{what}: a work buffer of {need} contiguous bytes on the batch's GPU is "
                                              "needed (attn_work)")
    q, ldq = _rows(Q, batch, heads * D, what)
    o, ldo = _rows(O, batch, heads * D, what)
    if lse is not None and not isinstance(lse, int) and (tuple(lse.shape) != (batch.tokens, heads) or not lse.is_contiguous()
                                                         or lse.dtype.itemsize != 4 or not lse.is_floating_point()
                                                         or lse.get_device() != batch.gpu):
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: lse is a contiguous float32 [tokens, heads] on the batch's GPU")
    return q, ldq, o, ldo, _ptr(lse), heads, work, _current_stream() if stream is None else _stream(stream)


def lq_attn_paged(cache, batch, Q, O, scale, window=0, sinks=0, lse=None, work=None, heads=None, stream=None) -> None:
    """Attention of the batch's tokens (Q, O: float32 [tokens, heads,
    head_dim]) over the cache, causal, with an optional sliding window and
    sinks; lse: float32 [tokens, heads] or None; work: attn_work(...), which a
    program keeps (None makes one for this call); a buffer made for a cache of
    other heads is refused if it is smaller than this one's. ``heads`` is
    needed where Q is not a three-dimensional tensor. See include/lq.h."""
    q, ldq, o, ldo, lse, heads, work, stream = _attn_operands(cache, batch, Q, O, lse, work, heads, stream, "lq_attn_paged")
    st = (_lib or lib()).lq_attn_paged(cache.ref, batch.ref, q, ldq, o, ldo, lse, heads, scale, window, sinks, _ptr(work), stream)
    if st:
        _check(st, "lq_attn_paged")


def attn_route(route: int) -> None:
    """lq_attn_paged's kernel: 0 automatic, 1 generic, 2 warp-level MMAs,
    3 tcgen05; for tests and comparisons."""
    _check(lib().lq_debug_attn_route(int(route)), "lq_debug_attn_route")


# ---- rotary positions, drafted trees, beams ----------------------------------
ROPE_MAX_PAIRS, ROPE_MAX_AXES, BEAM_MAX = 128, 4, 64


class RopeTable(ctypes.Structure):
    """The lq_rope_table struct of lq.h."""
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("pairs", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("factor", ctypes.c_float), ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * ROPE_MAX_PAIRS),
                ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS)]


class Rope:
    """The angles of rotary positions (lq_rope_table), which a program keeps:
    ``sections`` pairs by each axis of the positions, in blocks or, with
    ``interleaved``, in turns; ``freqs``: angles a position, or None for
    base^(-2j / rotary_dim); ``adjacent``: pairs (2j, 2j + 1) instead of (j, j +
    rotary_dim / 2). See include/lq.h."""

    def __init__(self, head_dim, rotary_dim=None, base=10000.0, adjacent=False, sections=None, interleaved=False, freqs=None, factor=1.0):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        axes = 1 if sections is None else len(sections)
        cut = None if sections is None else (ctypes.c_int32 * axes)(*[int(x) for x in sections])
        if freqs is not None and len(freqs) != rotary_dim // 2:
            raise LQError(LQ_ERR_INVALID_ARG, "Rope: one frequency a pair, rotary_dim / 2 in all")
        given = None if freqs is None else (ctypes.c_double * len(freqs))(*[float(x) for x in freqs])
        self.struct = RopeTable()
        _check(lib().lq_rope_init(ctypes.byref(self.struct), int(head_dim), int(rotary_dim), 1 if adjacent else 0, float(base), given,
                                  axes, cut, 1 if interleaved else 0, float(factor)), "lq_rope_init")
        self.ref = ctypes.byref(self.struct)
        self.head_dim, self.axes = int(head_dim), axes


_int32 = _float32 = None  # torch's types, once it is there (comparing them is the quickest check)


def _types():
    global _int32, _float32
    import torch
    _int32, _float32 = torch.int32, torch.float32
    return True


def _ints(x, shape, gpu, what, name):
    """The address of a contiguous int32 tensor of this shape on this GPU."""
    if _int32 is None:
        _types()
    if x.dtype is not _int32 or x.shape != shape or x.get_device() != gpu or gpu < 0 or not x.is_contiguous():
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: {name} is a contiguous int32 {list(shape)} on the same GPU, got {list(x.shape)} "
                                          f"{x.dtype} on {x.device}")
    return x.data_ptr()


def _head_rows(x, tokens, D, gpu, what):
    """(address, leading dimension, heads) of float32 rows [tokens, heads, D] or
    [tokens, heads * D] on one GPU."""
    shape, strides = x.shape, x.stride()
    rank = len(shape)
    ok = x.dtype is _float32 and x.get_device() == gpu >= 0
    if ok and rank == 3:
        n, heads, d = shape
        ok = n == tokens and d == D and strides[2] == 1 and (strides[1] == D or heads == 1)
    elif ok and rank == 2:
        n, width = shape
        heads = width // D
        ok = n == tokens and heads * D == width and strides[1] == 1
    if not ok or rank < 2 or rank > 3:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: float32 [{tokens}, heads, {D}] with contiguous heads and dims on one GPU wanted, "
                                          f"got {tuple(shape)} {x.dtype} on {x.device}, strides {strides}")
    return x.data_ptr(), strides[0] if tokens > 1 else heads * D, heads


def lq_rope(rope, positions, Q, K=None, q_out=None, k_out=None, inverse=False, stream=None) -> None:
    """Turns the rows of Q and, if given, K (float32 [tokens, heads, head_dim],
    slices of a fused projection's rows allowed) by their positions (int32
    [tokens] or [axes, tokens]; one row expanded to all axes will do), in
    place or into q_out and k_out. See include/lq.h."""
    if _int32 is None:
        _types()
    tokens, gpu, D, axes = Q.shape[0], Q.get_device(), rope.head_dim, rope.axes
    shape, ldp = positions.shape, positions.stride()
    if shape != (axes, tokens) and (axes > 1 or shape != (tokens,)) or positions.dtype is not _int32 or positions.get_device() != gpu \
            or tokens > 1 and ldp[-1] != 1:
        raise LQError(LQ_ERR_INVALID_ARG, f"lq_rope: int32 positions [{rope.axes}, {tokens}] on Q's GPU, contiguous along the tokens")
    q, ldq, heads = _head_rows(Q, tokens, D, gpu, "lq_rope")
    qo, ldqo, n = (q, ldq, heads) if q_out is None else _head_rows(q_out, tokens, D, gpu, "lq_rope")
    k = ldk = ko = ldko = kv_heads = m = 0
    if K is not None:
        k, ldk, kv_heads = _head_rows(K, tokens, D, gpu, "lq_rope")
        ko, ldko, m = (k, ldk, kv_heads) if k_out is None else _head_rows(k_out, tokens, D, gpu, "lq_rope")
    if n != heads or m != kv_heads or (K is None and k_out is not None):
        raise LQError(LQ_ERR_INVALID_ARG, "lq_rope: q_out and k_out have the shapes of Q and K")
    st = (_lib or lib()).lq_rope(rope.ref, tokens, positions.data_ptr(), ldp[0], q, ldq, qo, ldqo,
                                 heads, k, ldk, ko, ldko, kv_heads, 1 if inverse else 0,
                                 _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_rope")


def lq_tree_plan(batch, parent, positions=None, mask=None, window=0, sinks=0, stream=None) -> None:
    """Positions (int32 [tokens]) and masks (int32 [tokens, words], a bit a row
    of the sequence) of the batch's new tokens from their parents (int32
    [tokens]). kv_len must lie within the table's pages. See include/lq.h."""
    t, g = batch.tokens, batch.gpu
    p = _ints(parent, (t,), g, "lq_tree_plan", "parent")
    pos = 0 if positions is None else _ints(positions, (t,), g, "lq_tree_plan", "positions")
    words = 0 if mask is None else mask.shape[-1]
    m = 0 if mask is None else _ints(mask, (t, words), g, "lq_tree_plan", "mask")
    st = (_lib or lib()).lq_tree_plan(batch.ref, p, pos, m, words, window, sinks, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_tree_plan")


def lq_attn_tree(cache, batch, mask, Q, O, scale, positions=None, window=0, sinks=0, lse=None, work=None, heads=None, stream=None) -> None:
    """lq_attn_paged where a row sees of its sequence's new tokens those that its
    mask names (lq_tree_plan); positions are needed with a window. See
    include/lq.h."""
    t = batch.tokens
    q, ldq, o, ldo, lse, heads, work, stream = _attn_operands(cache, batch, Q, O, lse, work, heads, stream, "lq_attn_tree")
    words = mask.shape[-1]
    m = _ints(mask, (t, words), batch.gpu, "lq_attn_tree", "mask")
    pos = 0 if positions is None else _ints(positions, (t,), batch.gpu, "lq_attn_tree", "positions")
    st = (_lib or lib()).lq_attn_tree(cache.ref, batch.ref, m, words, pos, q, ldq, o, ldo, lse, heads, scale, window, sinks, _ptr(work), stream)
    if st:
        _check(st, "lq_attn_tree")


def lq_tree_accept(batch, parent, token, target, keep, count, next_token, kept_len, stream=None) -> None:
    """The path of the tree that the model's choices (target) confirm:
    its rows in keep (int32 [batch, max_keep], -1 behind them), their number in
    count, the choice after the last in next_token and the length of the cache
    with the path in kept_len (int32 [batch] each). kv_len must lie within the
    table's pages. See include/lq.h."""
    what, g, t, b, most = "lq_tree_accept", batch.gpu, (batch.tokens,), (batch.batch,), keep.shape[-1]
    st = (_lib or lib()).lq_tree_accept(batch.ref, _ints(parent, t, g, what, "parent"), _ints(token, t, g, what, "token"),
                                        _ints(target, t, g, what, "target"), _ints(keep, (batch.batch, most), g, what, "keep"), most,
                                        _ints(count, b, g, what, "count"), _ints(next_token, b, g, what, "next_token"),
                                        _ints(kept_len, b, g, what, "kept_len"), _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, what)


def lq_kv_keep(cache, batch, keep, count, stream=None) -> None:
    """Moves the rows keep[i, : count[i]] of each sequence's new tokens to the
    front of them, in the cache. See include/lq.h."""
    if cache.gpu != batch.gpu:
        _elsewhere(cache, batch, "lq_kv_keep")
    b, most = batch.batch, keep.shape[-1]
    st = (_lib or lib()).lq_kv_keep(cache.ref, batch.ref, _ints(keep, (b, most), batch.gpu, "lq_kv_keep", "keep"), most,
                                    _ints(count, (b,), batch.gpu, "lq_kv_keep", "count"),
                                    _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_kv_keep")


def beam_buffers(groups, beams, vocab, k, device=None):
    """(scores, parents, tokens, work) device buffers of lq_beam_select, which a
    program keeps."""
    import torch
    nbytes = int(lib().lq_beam_work_bytes(int(groups), int(beams), int(vocab), int(k)))
    if nbytes == 0:
        raise LQError(LQ_ERR_INVALID_ARG, "lq_beam_work_bytes")
    device = device or "cuda"
    return (torch.empty(groups, k, dtype=torch.float32, device=device), torch.empty(groups, k, dtype=torch.int32, device=device),
            torch.empty(groups, k, dtype=torch.int32, device=device), torch.empty(nbytes, dtype=torch.uint8, device=device))


_beam_work_bytes = {}  # by (groups, beams, vocab, k): a number that depends on these alone


def lq_beam_select(logits, scores, beams, k, out_scores, out_parents, out_tokens, work, finished=None, pad=0, stream=None) -> None:
    """The k best continuations of each group of ``beams`` rows of logits
    (float32 [groups * beams, vocab], rows may be strided) by scores (float32
    [groups * beams]) + log softmax: out_scores, out_parents, out_tokens
    [groups, k], work: beam_buffers(...). out_scores may be scores where k is
    beams. finished: int32 [groups * beams] or None. See include/lq.h."""
    what = "lq_beam_select"
    (n, vocab), gpu = logits.shape, logits.get_device()
    groups = n // beams if beams > 0 else 0
    ok = gpu >= 0 and groups * beams == n and (logits.stride(1) == 1 or vocab == 1)
    if _int32 is None:
        _types()
    ok = ok and logits.dtype is _float32
    for x, shape in ((scores, (n,)), (out_scores, (groups, k))):
        ok = ok and x.dtype is _float32 and x.shape == shape and x.get_device() == gpu and x.is_contiguous()
    if not ok:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: float32 logits [groups * beams, vocab], contiguous scores [groups * beams] and "
                                          "out_scores [groups, k] on one GPU")
    sizes = (groups, beams, vocab, k)
    need = _beam_work_bytes.get(sizes)
    if need is None:  # (0 for sizes that the call itself refuses)
        need = _beam_work_bytes[sizes] = int(lib().lq_beam_work_bytes(*sizes))
    if work.numel() * work.element_size() < need or not work.is_contiguous() or work.get_device() != gpu:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: a work buffer of {need} contiguous bytes on the logits' GPU is needed (beam_buffers)")
    done = 0 if finished is None else _ints(finished, (n,), gpu, what, "finished")
    st = (_lib or lib()).lq_beam_select(logits.data_ptr(), logits.stride(0) if n > 1 else vocab, scores.data_ptr(), groups, beams, vocab, k,
                                        done, pad, out_scores.data_ptr(), _ints(out_parents, (groups, k), gpu, what, "out_parents"),
                                        _ints(out_tokens, (groups, k), gpu, what, "out_tokens"), work.data_ptr(),
                                        _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, what)


def lq_beam_pages(parent, beams, table, kv_len, page_size, table_out, copies, stream=None) -> None:
    """Page tables (int32 [groups * beams, max_pages]) of the beams that go on
    from parent (int32 [groups * beams]), and the copies of last pages that this
    takes (int32 [groups * beams, 3], for lq_kv_copy). See include/lq.h."""
    what, n, gpu = "lq_beam_pages", parent.shape[0], parent.get_device()
    if beams < 1 or n % beams != 0 or table.dim() != 2:
        raise LQError(LQ_ERR_INVALID_ARG, f"{what}: parents and tables of groups * beams rows")
    width = table.shape[1]
    st = (_lib or lib()).lq_beam_pages(_ints(parent, (n,), gpu, what, "parent"), n // beams, beams, _ints(table, (n, width), gpu, what, "table"),
                                       width, _ints(kv_len, (n,), gpu, what, "kv_len"), page_size,
                                       _ints(table_out, (n, width), gpu, what, "table_out"), _ints(copies, (n, 3), gpu, what, "copies"),
                                       _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, what)


def lq_kv_copy(cache, copies, stream=None) -> None:
    """Copies the first tokens of pages of the cache to other pages: copies is
    int32 [n, 3] of (from, to, tokens), as lq_beam_pages gives them. See
    include/lq.h."""
    gpu = copies.get_device() if cache.gpu is None else cache.gpu
    st = (_lib or lib()).lq_kv_copy(cache.ref, _ints(copies, (copies.shape[0], 3), gpu, "lq_kv_copy", "copies"), copies.shape[0],
                                    _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "lq_kv_copy")


# ---- host packers --------------------------------------------------------
def packed_bytes(fmt: str, N: int, K: int) -> int:
    return int(lib().lq_packed_bytes(FMT[fmt], int(N), int(K)))


def pack(fmt: str, W, reciprocal: bool = False) -> np.ndarray:
    """Pack f32 weights [N, K] (numpy or CPU torch) on the host.

    Returns uint16 [N, K] for f16 and uint8 [N, K/32*34 or *18] otherwise.
    fmt "q4_0i" stores the pages' interleaved nibble order; reciprocal=True
    packs Q8_0 with the pages' q = round(x * (1/d)).
    """
    if hasattr(W, "detach"):
        W = W.detach().cpu().numpy()
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    nbytes = packed_bytes(fmt, N, K)
    if nbytes == 0 and N * K > 0:
        raise LQError(LQ_ERR_INVALID_ARG, f"lq_pack_{fmt}")
    if fmt == "f16":
        out = np.empty((N, K), dtype=np.uint16)
    else:
        out = np.empty((N, nbytes // max(N, 1)), dtype=np.uint8)
    name = "lq_pack_q8_0_rcp" if (reciprocal and fmt == "q8_0") else f"lq_pack_{fmt}"
    _check(getattr(lib(), name)(W.ctypes.data, N, K, out.ctypes.data), name)
    return out


def lq_pack_f16(W) -> np.ndarray:
    return pack("f16", W)


def lq_pack_q4_0i(W) -> np.ndarray:
    return pack("q4_0i", W)


def lq_pack_q8_0_rcp(W) -> np.ndarray:
    return pack("q8_0", W, reciprocal=True)


def lq_pack_q8_0(W) -> np.ndarray:
    return pack("q8_0", W)


def lq_pack_q4_0(W) -> np.ndarray:
    return pack("q4_0", W)


# ---- status and test hooks -----------------------------------------------
def last_device_error() -> int:
    return int(lib().lq_last_device_error())


def version() -> str:
    return lib().lq_version().decode()


def force_route(route: int) -> None:
    _check(lib().lq_debug_force_route(int(route)), "lq_debug_force_route")


def route_count(route: int) -> int:
    return int(lib().lq_debug_route_count(int(route)))


def reset_counts() -> None:
    lib().lq_debug_reset_counts()


def set_wait_limit_ns(ns: int) -> None:
    lib().lq_debug_set_wait_limit_ns(int(ns))


def gemv_plan(ctas_per_sm: int = 0, rows_per_stage: int = 0, smem_bytes: int = 0) -> None:
    """Override the decode GEMV's launch plan (0 = automatic); tuning only."""
    _check(lib().lq_debug_gemv_plan(int(ctas_per_sm), int(rows_per_stage), int(smem_bytes)),
           "lq_debug_gemv_plan")


def chain_waits(on: bool) -> None:
    """Dependent problems of lq_gemv_chain wait inside one launch (True) or
    start a new launch (False, the default); for comparisons."""
    lib().lq_debug_chain_waits(1 if on else 0)


def gemm_pairs(on: bool) -> None:
    """Let the tensor-core GEMM pair CTAs on 256-row MMAs where they fit
    (True) or never (False, the default); for comparisons."""
    lib().lq_debug_gemm_pairs(1 if on else 0)


def gemm_rings(a_stages: int = 0, raw_stages: int = 0) -> None:
    """Override the tensor-core GEMM's ring depths (0 = automatic); tuning only."""
    _check(lib().lq_debug_gemm_rings(int(a_stages), int(raw_stages)), "lq_debug_gemm_rings")
