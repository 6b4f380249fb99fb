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

}  // namespace lq
