// Host-side declarations of the attention kernels.
#pragma once
#include "lq_kv.cuh"

namespace lq {

// A call of lq_attn_paged (already validated).
struct AttnArgs {
  kv::Cache c;
  kv::Batch b;
  const float* Q;
  float* O;
  float* lse;  // may be null
  long long ldq, ldo;
  int heads, group;  // query heads; query heads per key/value head
  float scale;
  int window, sinks;  // window 0: none
  // lq_attn_tree: what rows see of their sequence's new tokens (null: up to themselves),
  // mask_words a row, and the rows' positions (null without a window)
  const uint32_t* mask;
  const int* positions;
  int mask_words;
};

namespace tree {
// Bits at .. at + 31 of a row's mask; bits that it does not have are 0.
__device__ __forceinline__ uint32_t bits(const AttnArgs& a, int t, int at) {
  const uint32_t* const row = a.mask + static_cast<long long>(t) * a.mask_words;
  const int w = at >> 5, shift = at & 31;
  const uint32_t lo = w >= 0 && w < a.mask_words ? row[w] : 0u;
  const uint32_t hi = shift != 0 && w + 1 >= 0 && w + 1 < a.mask_words ? row[w + 1] : 0u;
  return __funnelshift_r(lo, hi, shift);
}
// The position of row t, of a sequence whose new tokens are base .. len - 1.
__device__ __forceinline__ int position(const AttnArgs& a, int t, int base, int len) {
  return a.window > 0 ? max(min(a.positions[t], len - 1), base) : base;
}
}  // namespace tree

// Route counters (lq_debug_route_count): 8 generic, 9 rows x 16-key tiles on
// warp-level MMAs, 10 row tiles on tcgen05.
constexpr int kAttnRouteGeneric = 8, kAttnRouteWarp = 9, kAttnRouteTile = 10;

lq_status launch_attn_generic(const AttnArgs& a, int fmt, cudaStream_t stream);

// The work buffer: arrival counters (zero between calls), then partial results.
constexpr int kAttnMaxCtas = 256;
constexpr size_t kAttnCounterBytes = 4096;  // counters by CTA, and by slot (two a CTA)
static_assert(3 * kAttnMaxCtas * sizeof(int) <= kAttnCounterBytes);

// Rows of 8 on warp-level MMAs (lq_attn_warp.cu); `rows`: the most rows
// (tokens * group) a sequence is expected to have, small_rows: sequences with
// more are left to another kernel (0: none are). LQ_ERR_UNSUPPORTED outside
// its geometries.
bool attn_warp_eligible(const AttnArgs& a);
size_t attn_warp_work_bytes();
lq_status launch_attn_warp(const AttnArgs& a, int fmt, int rows, int small_rows, void* work, cudaStream_t stream);
lq_status launch_attn_warp_tree(const AttnArgs& a, int fmt, int rows, int small_rows, void* work, cudaStream_t stream);  // with a mask

// Tiles of 128 rows on tcgen05 (lq_attn_tile.cu); sequences with at most
// small_rows rows are left to another kernel (0: none are).
bool attn_tile_eligible(const AttnArgs& a);
size_t attn_tile_work_bytes(int head_dim);
lq_status launch_attn_tile(const AttnArgs& a, int fmt, int small_rows, void* work, cudaStream_t stream);
lq_status launch_attn_tile_tree(const AttnArgs& a, int fmt, int small_rows, void* work, cudaStream_t stream);  // with a mask

}  // namespace lq
