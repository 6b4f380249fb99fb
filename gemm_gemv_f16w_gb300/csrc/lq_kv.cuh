// The paged key/value cache as the kernels see it: where a token's codes and
// scales are, which rows belong to which sequence, and what a code stands for.
#pragma once
#include <cuda_fp16.h>

#include "lq_device.cuh"
#include "lq_internal.h"

namespace lq {
namespace kv {

// One pool geometry (K and V share it). A (page, head) is head_bytes of
// contiguous memory: page_size rows of row_bytes codes, then page_size rows
// of head_dim / 32 f16 scales (quantised formats).
struct Cache {
  unsigned char* k;
  unsigned char* v;
  long long head_bytes;
  long long page_bytes;  // kv_heads * head_bytes
  int page_size, kv_heads, head_dim, num_pages;
  int row_bytes;
};

struct Batch {
  const int* table;
  const int* kv_len;
  const int* q_start;
  int batch, max_pages, tokens;
};

__host__ __device__ constexpr int code_row_bytes(int fmt, int head_dim) {
  return fmt == LQ_FMT_F16 ? 2 * head_dim : (fmt == LQ_FMT_Q8_0 ? head_dim : head_dim / 2);
}

// Sequence i: its rows of the call [row0, row0 + rows) and its length, both
// clipped to what exists.
struct Seq {
  int row0, rows, len;
};
__device__ __forceinline__ Seq sequence(const Batch& b, int page_size, int i) {
  Seq s;
  s.row0 = min(max(b.q_start[i], 0), b.tokens);
  s.rows = min(max(b.q_start[i + 1], s.row0), b.tokens) - s.row0;
  const long long most = static_cast<long long>(b.max_pages) * page_size;
  s.len = static_cast<int>(min(static_cast<long long>(max(b.kv_len[i], 0)), most));
  return s;
}

// The sequence that row t belongs to (-1: none), found by the whole warp: 32
// entries of q_start at a time narrow the range 32-fold.
__device__ __forceinline__ int find_sequence(const Batch& b, int t, int lane) {
  int lo = 0, n = b.batch;  // the answer, if any, is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool before = lane * step < n && b.q_start[i] <= t;
    const unsigned mask = __ballot_sync(0xffffffffu, before);
    const int last = mask == 0u ? 0 : 31 - __clz(static_cast<int>(mask));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return b.q_start[lo] <= t && t < b.q_start[lo + 1] ? lo : -1;
}

// a / b (both not negative), by 32-bit division where both fit: less code and
// time than the 64-bit one, which a call of ordinary size never needs.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Page of position p of sequence i, or -1 where there is none.
__device__ __forceinline__ int page_of(const Cache& c, const Batch& b, int i, int p) {
  const int at = p / c.page_size;
  if (p < 0 || at >= b.max_pages) return -1;
  const int page = b.table[static_cast<long long>(i) * b.max_pages + at];
  return page >= 0 && page < c.num_pages ? page : -1;
}

// The visible positions of a query at position p: [0, sink_end) and
// [begin, p]; empty ranges where there are none.
struct Visible {
  int sink_end, begin;
};
__device__ __forceinline__ Visible visible(int p, int window, int sinks) {
  Visible v;
  v.begin = window > 0 ? max(0, p - window + 1) : 0;
  v.sink_end = min(sinks, v.begin);
  return v;
}

}  // namespace kv

// The host's checks and views of the caller's structs (lq_kv.cu).
lq_status kv_check(const lq_kv_cache* cache, const lq_kv_batch* batch, bool* noop);
kv::Cache kv_cache_view(const lq_kv_cache& c);
kv::Batch kv_batch_view(const lq_kv_batch& b);
}  // namespace lq
