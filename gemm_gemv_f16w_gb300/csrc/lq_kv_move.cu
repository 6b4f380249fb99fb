// Moving tokens inside the paged cache: lq_kv_keep (the accepted path of a
// draft), lq_kv_copy and lq_beam_pages (beams that go on from one another).
//
// Codes and scales are moved as they are: nothing is rounded anew.
//
// Keep. Row keep[k] of a sequence's new tokens goes to the place of row k; keep[]
// ascends, so k <= keep[k]. A CTA has one head of K or V of a sequence and takes the
// rows in order, as many at a time as its threads hold in registers (1024 pieces of
// 16 bytes, or of one scale): all loads, a barrier, all stores. What a store overwrites
// is the source of rows of its own or an earlier time only, so the move is in place.
// 256 rows of Q8_0, 8 heads of 128, moved by one: 15 us (44 when a thread
// takes all rows of its column in order); the accepted paths of 32 sequences 3.4.
//
// Pages. The beams of a group have one length; all pages before its last, partly
// filled one are full and shared, that page and those behind are each
// beam's own. Of the children of a beam the first goes on in its parent's own
// pages. There are as many further children as beams without a child: the m-th
// takes the m-th such beam's own pages and, for the last page's tokens, a copy.
// So no copy's target is another's source, no spare pages are needed, and every
// page keeps exactly one owner.
//
// Copy. One CTA for each side and head of a copy; a (page, head) is contiguous,
// so it moves two runs of bytes. What bounds both is HBM for many beams and the
// launch and the chain list -> page -> bytes for few.
#include <algorithm>

#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

__device__ unsigned g_move_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_move_err, 0u, code); }

constexpr int kKeepThreads = 128;
constexpr int kKeepPieces = 8;  // of a thread at a time
constexpr int kCopyThreads = 256;
constexpr int kMapThreads = 256;

struct KeepArgs {
  kv::Cache c;
  kv::Batch b;
  const int* keep;  // [batch][most]
  const int* count;
  int most;
  int code_columns, columns;  // pieces of a token's head: of the codes, and with the scales
  int rows;                   // at a time: columns * rows pieces
};

// T: a piece of the codes.
template <class T>
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a) {
  // where the rows' codes come from and go to (-1: they stay), and their scales
  __shared__ long long src[kKeepThreads], dst[kKeepThreads], scale_src[kKeepThreads], scale_dst[kKeepThreads];
  __shared__ int stop;
  pdl_wait();
  pdl_launch_dependents();
  const int i = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const kv::Seq s = kv::sequence(a.b, a.c.page_size, i);
  const int base = s.len - s.rows;
  const int* const keep = a.keep + static_cast<long long>(i) * a.most;
  const int count = min(min(a.count[i], a.most), s.rows);
  const int side = static_cast<int>(blockIdx.y) / a.c.kv_heads, head = static_cast<int>(blockIdx.y) - side * a.c.kv_heads;
  unsigned char* const pool = (side ? a.c.v : a.c.k) + head * a.c.head_bytes;
#pragma unroll 1
  for (int k0 = 0; k0 < count; k0 += a.rows) {
    const int n = min(a.rows, count - k0);
    bool good = true;
    if (tid < n) {
      const int k = k0 + tid, from = keep[k];
      good = from >= 0 && from < s.rows && (k == 0 ? true : from > keep[k - 1]);
      const int p_src = base + from, p_dst = base + k;
      int page_src = -1, page_dst = -1;
      if (good && from != k && p_dst >= 0) {
        page_src = kv::page_of(a.c, a.b, i, p_src);
        page_dst = kv::page_of(a.c, a.b, i, p_dst);
      }
      const bool moves = page_src >= 0 && page_dst >= 0 && LQ_IN_BOUNDS(page_src < a.c.num_pages && page_dst < a.c.num_pages);
      const long long scales = static_cast<long long>(a.c.page_size) * a.c.row_bytes;
      const int s_src = moves ? p_src % a.c.page_size : 0, s_dst = moves ? p_dst % a.c.page_size : 0;
      src[tid] = moves ? page_src * a.c.page_bytes + static_cast<long long>(s_src) * a.c.row_bytes : -1;
      dst[tid] = moves ? page_dst * a.c.page_bytes + static_cast<long long>(s_dst) * a.c.row_bytes : -1;
      scale_src[tid] = moves ? page_src * a.c.page_bytes + scales + s_src * (a.c.head_dim / 16) : -1;
      scale_dst[tid] = moves ? page_dst * a.c.page_bytes + scales + s_dst * (a.c.head_dim / 16) : -1;
    }
    // the list ends at the first entry that does not ascend
    if (tid == 0) stop = n;
    __syncthreads();
    if (tid < n && !good) atomicMin(&stop, tid);
    __syncthreads();
    const int m = stop, pieces = m * a.columns;
    T x[kKeepPieces];
    unsigned char* to[kKeepPieces];
    bool scale[kKeepPieces];
#pragma unroll
    for (int j = 0; j < kKeepPieces; ++j) {
      const int e = j * kKeepThreads + tid, r = e / a.columns, column = e - r * a.columns;
      to[j] = nullptr;
      scale[j] = column >= a.code_columns;
      if (e < pieces && src[r] >= 0) {
        if (scale[j]) {
          const int at = (column - a.code_columns) * 2;
          to[j] = pool + scale_dst[r] + at;
          *reinterpret_cast<unsigned short*>(&x[j]) = *reinterpret_cast<const unsigned short*>(pool + scale_src[r] + at);
        } else {
          const int at = column * static_cast<int>(sizeof(T));
          to[j] = pool + dst[r] + at;
          x[j] = *reinterpret_cast<const T*>(pool + src[r] + at);
        }
      }
    }
    __syncthreads();  // all has been read
#pragma unroll
    for (int j = 0; j < kKeepPieces; ++j) {
      if (!to[j]) continue;
      if (scale[j]) {
        *reinterpret_cast<unsigned short*>(to[j]) = *reinterpret_cast<const unsigned short*>(&x[j]);
      } else {
        *reinterpret_cast<T*>(to[j]) = x[j];
      }
    }
    __syncthreads();  // and written, before the next rows are read
    if (m < n) break;
  }
}

struct CopyArgs {
  kv::Cache c;
  const int* copies;  // [n][3]: from page, to page, tokens
};

// bytes (a multiple of sizeof(T)) from one place to another by the whole block
template <class T>
__device__ __forceinline__ void copy_run(unsigned char* to, const unsigned char* from, long long bytes) {
  const long long n = bytes / static_cast<int>(sizeof(T));
  T* const dst = reinterpret_cast<T*>(to);
  const T* const src = reinterpret_cast<const T*>(from);
#pragma unroll 1
  for (long long k = threadIdx.x; k < n; k += kCopyThreads * 8) {
    T x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j * kCopyThreads < n) x[j] = src[k + j * kCopyThreads];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j * kCopyThreads < n) dst[k + j * kCopyThreads] = x[j];
  }
}

template <class T>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int* const c = a.copies + static_cast<long long>(blockIdx.x) * 3;
  const int src = c[0], dst = c[1], rows = min(c[2], a.c.page_size);
  if (rows <= 0 || src < 0 || dst < 0 || src >= a.c.num_pages || dst >= a.c.num_pages || src == dst) return;
  const int head = static_cast<int>(blockIdx.y), h = head < a.c.kv_heads ? head : head - a.c.kv_heads;
  unsigned char* const pool = head < a.c.kv_heads ? a.c.k : a.c.v;
  const unsigned char* const from = pool + src * a.c.page_bytes + h * a.c.head_bytes;
  unsigned char* const to = pool + dst * a.c.page_bytes + h * a.c.head_bytes;
  if (!LQ_IN_BOUNDS(h < a.c.kv_heads)) return;
  copy_run<T>(to, from, static_cast<long long>(rows) * a.c.row_bytes);
  const long long scales = static_cast<long long>(a.c.page_size) * a.c.row_bytes;
  if (a.c.head_bytes > scales) copy_run<unsigned short>(to + scales, from + scales, static_cast<long long>(rows) * (a.c.head_dim / 16));
}

struct PagesArgs {
  const int* parent;  // [groups * beams]
  const int* table;   // [groups * beams][max_pages]
  const int* len;     // [groups * beams]
  int* out;
  int* copies;  // [groups * beams][3]
  int beams, max_pages, page_size;
};

// grid: x = group, y = part of its tables' entries
__global__ void __launch_bounds__(kMapThreads) pages_kernel(const PagesArgs a) {
  __shared__ int parent[LQ_BEAM_MAX], place[LQ_BEAM_MAX], free_list[LQ_BEAM_MAX];
  __shared__ unsigned bits[2][LQ_BEAM_MAX / 32];  // beams without a child; further children
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.beams, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const long long first = static_cast<long long>(blockIdx.x) * n;
  if (tid < LQ_BEAM_MAX) {
    const int p = tid < n ? a.parent[first + tid] : -1;
    parent[tid] = p >= 0 && p < n ? p : -1;
  }
  __syncthreads();
  if (tid < LQ_BEAM_MAX) {
    bool childless = tid < n, further = tid < n && parent[tid] < 0;
    for (int b = 0; b < n; ++b) {
      childless = childless && parent[b] != tid;
      further = further || (tid < n && b < tid && parent[b] == parent[tid]);
    }
    const unsigned c = __ballot_sync(0xffffffffu, childless), f = __ballot_sync(0xffffffffu, further);
    if (lane == 0) {
      bits[0][warp] = c;
      bits[1][warp] = f;
    }
  }
  __syncthreads();
  // how many of a kind are before this thread's beam, and whether it is one
  auto rank = [&](const unsigned (&of)[LQ_BEAM_MAX / 32], bool& is) {
    int before = __popc(of[warp] & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += __popc(of[w]);
    is = (of[warp] >> lane) & 1u;
    return before;
  };
  bool is = false;
  if (tid < n) {
    const int before = rank(bits[0], is);
    if (is) free_list[before] = tid;
  }
  __syncthreads();
  if (tid < n) {  // whose own pages it goes on in
    const int before = rank(bits[1], is);
    place[tid] = is ? free_list[before] : parent[tid];
  }
  __syncthreads();
  const int len = max(a.len[first], 0), whole = len / a.page_size, rows = len - whole * a.page_size;
  const int from = static_cast<int>(blockIdx.y) * kMapThreads, step = static_cast<int>(gridDim.y) * kMapThreads;
  const int entries = n * a.max_pages;
#pragma unroll 4
  for (int x = from + tid; x < entries; x += step) {
    const int b = x / a.max_pages, e = x - b * a.max_pages;
    const int of = e < whole && parent[b] >= 0 ? parent[b] : place[b];  // full pages are the parent's
    if (LQ_IN_BOUNDS(of >= 0 && of < n)) a.out[first * a.max_pages + x] = a.table[(first + of) * a.max_pages + e];
  }
  if (blockIdx.y == 0 && tid < n) {
    const bool copies = parent[tid] >= 0 && place[tid] != parent[tid] && rows > 0 && whole < a.max_pages;
    int* const c = a.copies + (first + tid) * 3;
    c[0] = copies ? a.table[(first + parent[tid]) * a.max_pages + whole] : -1;
    c[1] = copies ? a.table[(first + place[tid]) * a.max_pages + whole] : -1;
    c[2] = copies ? rows : 0;
  }
}

lq_status launch(const void* kernel, dim3 grid, unsigned threads, void* args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* list[1] = {args};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, list);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

// 16-byte steps where every (page, head) begins on a 16-byte boundary.
bool wide(const kv::Cache& c) { return c.head_bytes % 16 == 0 && aligned_to(c.k, 16) && aligned_to(c.v, 16); }

}  // namespace

unsigned read_clear_move_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_move_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_move_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

lq_status lq_kv_keep(const lq_kv_cache* cache, const lq_kv_batch* batch, const int32_t* keep, int64_t max_keep, const int32_t* count,
                     void* stream) {
  bool noop;
  const lq_status st = kv_check(cache, batch, &noop);
  if (st != LQ_OK) return st;
  if (max_keep < 1) return LQ_ERR_INVALID_ARG;
  if (max_keep > (1LL << 24)) return LQ_ERR_UNSUPPORTED;
  if (noop) return LQ_OK;
  if (!keep || !count || !aligned_to(keep, 4) || !aligned_to(count, 4)) return LQ_ERR_INVALID_ARG;
  KeepArgs a = {};
  a.c = kv_cache_view(*cache);
  a.b = kv_batch_view(*batch);
  a.keep = keep;
  a.count = count;
  a.most = static_cast<int>(max_keep);
  const bool w = wide(a.c);
  a.code_columns = a.c.row_bytes / (w ? 16 : 2);
  a.columns = a.code_columns + (cache->fmt == LQ_FMT_F16 ? 0 : a.c.head_dim / 32);  // (at most 264)
  a.rows = std::min(kKeepThreads, kKeepThreads * kKeepPieces / a.columns);
  const dim3 grid(static_cast<unsigned>(a.b.batch), static_cast<unsigned>(2 * a.c.kv_heads));
  const void* kernel = w ? reinterpret_cast<const void*>(keep_kernel<uint4>) : reinterpret_cast<const void*>(keep_kernel<unsigned short>);
  return launch(kernel, grid, kKeepThreads, &a, static_cast<cudaStream_t>(stream));
}

lq_status lq_kv_copy(const lq_kv_cache* cache, const int32_t* copies, int64_t n, void* stream) {
  lq_kv_batch any = {};  // no tokens: the cache alone is checked
  bool noop;
  const lq_status st = kv_check(cache, &any, &noop);
  if (st != LQ_OK) return st;
  if (n < 0) return LQ_ERR_INVALID_ARG;
  if (n == 0 || cache->num_pages == 0) return LQ_OK;
  if (!cache->k || !cache->v || !aligned_to(cache->k, 2) || !aligned_to(cache->v, 2) || !copies || !aligned_to(copies, 4))
    return LQ_ERR_INVALID_ARG;
  const int64_t most = (1LL << 31) - 1;
  if (cache->head_dim > 256 || cache->num_pages > most || cache->kv_heads > 4096 || n > most) return LQ_ERR_UNSUPPORTED;
  CopyArgs a = {};
  a.c = kv_cache_view(*cache);
  a.copies = copies;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(2 * a.c.kv_heads));
  const void* kernel = wide(a.c) ? reinterpret_cast<const void*>(copy_kernel<uint4>) : reinterpret_cast<const void*>(copy_kernel<unsigned short>);
  return launch(kernel, grid, kCopyThreads, &a, static_cast<cudaStream_t>(stream));
}

lq_status lq_beam_pages(const int32_t* parent, int64_t groups, int64_t beams, const int32_t* table, int64_t max_pages,
                        const int32_t* kv_len, int64_t page_size, int32_t* table_out, int32_t* copies, void* stream) {
  if (groups < 0 || beams < 1 || max_pages < 0 || page_size < 1 || page_size > 65536) return LQ_ERR_INVALID_ARG;
  const int64_t most = 1LL << 30;  // (each by itself, too: the products are to fit 64 bits)
  if (beams > LQ_BEAM_MAX || groups > most || max_pages > most || groups * beams > most || max_pages * page_size > most ||
      beams * max_pages > most)
    return LQ_ERR_UNSUPPORTED;
  if (groups == 0) return LQ_OK;
  for (const void* p : {static_cast<const void*>(parent), static_cast<const void*>(kv_len), static_cast<const void*>(copies)})
    if (!p || !aligned_to(p, 4)) return LQ_ERR_INVALID_ARG;
  if (max_pages > 0 && (!table || !table_out || !aligned_to(table, 4) || !aligned_to(table_out, 4) || table == table_out))
    return LQ_ERR_INVALID_ARG;
  PagesArgs a = {};
  a.parent = parent;
  a.table = table;
  a.len = kv_len;
  a.out = table_out;
  a.copies = copies;
  a.beams = static_cast<int>(beams);
  a.max_pages = static_cast<int>(max_pages);
  a.page_size = static_cast<int>(page_size);
  // (four entries a thread)
  const int64_t parts = std::min<int64_t>(std::max<int64_t>((beams * max_pages + 4 * kMapThreads - 1) / (4 * kMapThreads), 1), 1024);
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(parts));
  return launch(reinterpret_cast<const void*>(pages_kernel), grid, kMapThreads, &a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
