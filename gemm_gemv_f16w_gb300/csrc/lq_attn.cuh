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
};

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

// Tiles of 128 rows on tcgen05 (lq_attn_tile.cu); sequences with at most
// small_rows rows are left to another kernel (0: none are).
bool attn_tile_eligible(const AttnArgs& a);
size_t attn_tile_work_bytes(int head_dim);
lq_status launch_attn_tile(const AttnArgs& a, int fmt, int small_rows, void* work, cudaStream_t stream);

}  // namespace lq
