// lq_attn_paged: argument checks, the choice of a kernel, and the generic
// kernel that takes every geometry.
//
// Generic kernel: one CTA per (row, query head). Its eight warps stride over
// the visible keys, a lane holding the dims lane, lane + 32, ... of the query
// and the running output; a warp-wide sum gives each logit, and a running
// maximum and sum (softmax in one pass over the keys) rescale the output when
// the maximum grows. The warps' partial results are joined through shared
// memory. It is bound by its serial chain of loads and shuffles per key and
// reads a shared head's keys once per query head: one f16 sequence of 513
// positions, 32 heads over 8 of 128, takes 66 us (the warp-level kernel 10),
// 64 sequences of 8192 take 5.1 ms (0.34; with heads of 96, which only this
// kernel takes, 4.4).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lq_attn.cuh"

namespace lq {
namespace {

__device__ unsigned g_attn_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_attn_err, 0u, code); }

std::atomic<int> g_attn_route{0};

constexpr int kGWarps = 8;
constexpr int kMaxDim = 256;
// Rows (tokens x query heads a key/value head) of a sequence up to which the
// warp-level kernel runs: it reads the keys once for every 16 rows, and its
// time grows with the rows; the tile kernel's is that of 256 (heads of 256: 128) rows. 32 heads
// over 8, 16 sequences of 4096 | one of 32768, us, warp-level / tile:
//   rows           32               48               64               128
//   f16, 64    31/59 | 32/50    38/59 | 38/55    47/59 | 46/50    79/59 | 80/51
//   f16, 128   54/82 | 61/75    67/81 | 81/84    89/82 | 102/76   147/83 | 188/78
//   Q8_0, 64   35/83 | 35/72    42/83 | 43/76    52/83 | 53/72    89/83 | 94/72
//   Q8_0, 128  53/165 | 55/138  67/167 | 72/150  85/172 | 91/142  147/185 | 169/149
//   Q4_0, 128  54/140 | 54/128  68/141 | 73/137  86/141 | 93/127  150/149 | 175/128
// 16 sequences of 4096, 2 | 4 heads of 256:
//   rows           32               48              80                96
//   f16, 256   33/57 | 62/77    45/57 | 84/76   69/58 | 128/78    79/60 | 152/79
//   Q8_0, 256  31/89 | 58/170   42/88 | 79/175  62/90 | 120/184   73/91 | 141/189
// One number a format is a compromise: where the two cross also depends on the
// head dim and on how many sequences share the SMs. f16 of 64 dims crosses at 64
// rows (a few us given away from 49 on), and 16 sequences of Q8_0, 128 dims, would
// gain from the warp-level kernel up to 128 rows, where one sequence loses.
int few_rows(int fmt, int head_dim) { return fmt == LQ_FMT_F16 ? 48 : (head_dim == 256 ? 96 : 80); }

template <int FMT>
__global__ void __launch_bounds__(kGWarps * 32) attn_generic_kernel(const AttnArgs a) {
  __shared__ float part[kGWarps][kMaxDim + 2];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = static_cast<int>(blockIdx.x / a.heads), h = static_cast<int>(blockIdx.x % a.heads);
  const int D = a.c.head_dim, blocks = D / 32, hk = h / a.group;
  const int i = kv::find_sequence(a.b, t, lane);
  if (i < 0) return;  // the whole CTA
  const kv::Seq s = kv::sequence(a.b, a.c.page_size, i);
  const int p = s.len - s.rows + (t - s.row0);
  const kv::Visible see = kv::visible(p, a.window, a.sinks);

  float q[kMaxDim / 32], acc[kMaxDim / 32];
  bool odd = false;  // the query is not finite
  const float* qrow = a.Q + t * a.ldq + static_cast<long long>(h) * D;
#pragma unroll
  for (int b = 0; b < kMaxDim / 32; ++b) {
    const float x = b < blocks ? qrow[b * 32 + lane] : 0.0f;
    odd = odd || !isfinite(x);
    q[b] = x * a.scale;
    acc[b] = 0.0f;
  }
  odd = __any_sync(0xffffffffu, odd);
  float m = -INFINITY, l = 0.0f;
  bool any = false;
  // keys 0 .. sink_end-1, then begin .. p, dealt to the warps in turn
  const int count = p < 0 ? 0 : see.sink_end + (p - see.begin + 1);
  const long long scale_at = static_cast<long long>(a.c.page_size) * a.c.row_bytes;
  for (int n = warp; n < count; n += kGWarps) {
    const int j = n < see.sink_end ? n : see.begin + (n - see.sink_end);
    const int page = kv::page_of(a.c, a.b, i, j);
    if (page < 0) continue;
    const int slot = j % a.c.page_size;
    const long long at = page * a.c.page_bytes + hk * a.c.head_bytes;
    float v[kMaxDim / 32], x = 0.0f;
#pragma unroll
    for (int b = 0; b < kMaxDim / 32; ++b) {
      if (b >= blocks) break;
      float kd;
      const unsigned char* kr = a.c.k + at + static_cast<long long>(slot) * a.c.row_bytes;
      const unsigned char* vr = a.c.v + at + static_cast<long long>(slot) * a.c.row_bytes;
      if constexpr (FMT == LQ_FMT_F16) {
        kd = __half2float(reinterpret_cast<const __half*>(kr)[b * 32 + lane]);
        v[b] = __half2float(reinterpret_cast<const __half*>(vr)[b * 32 + lane]);
      } else {
        const float ks = __half2float(reinterpret_cast<const __half*>(a.c.k + at + scale_at)[slot * blocks + b]);
        const float vs = __half2float(reinterpret_cast<const __half*>(a.c.v + at + scale_at)[slot * blocks + b]);
        if constexpr (FMT == LQ_FMT_Q8_0) {
          kd = ks * static_cast<float>(static_cast<signed char>(kr[b * 32 + lane]));
          v[b] = vs * static_cast<float>(static_cast<signed char>(vr[b * 32 + lane]));
        } else {
          const int at4 = b * 16 + (lane & 15), shift = (lane >> 4) * 4;
          kd = ks * static_cast<float>(static_cast<int>((kr[at4] >> shift) & 15) - 8);
          v[b] = vs * static_cast<float>(static_cast<int>((vr[at4] >> shift) & 15) - 8);
        }
      }
      x = fmaf(q[b], kd, x);
    }
    x = warp_sum(x);
    any = true;
    const float to = fmaxf(m, x);
    const float base = to == -INFINITY ? 0.0f : to;  // every logit so far is -inf
    const float keep = expf(m - base), w = expf(x - base);
    m = to;
    l = l * keep + w;
#pragma unroll
    for (int b = 0; b < kMaxDim / 32; ++b)
      if (b < blocks) acc[b] = acc[b] * keep + w * v[b];
  }
#pragma unroll
  for (int b = 0; b < kMaxDim / 32; ++b)
    if (b < blocks) part[warp][b * 32 + lane] = acc[b];
  if (lane == 0) {
    part[warp][kMaxDim] = any ? m : -INFINITY;
    part[warp][kMaxDim + 1] = l;
  }
  const bool seen = __syncthreads_or(any ? 1 : 0) != 0;  // (if not, the sum is zero)
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kGWarps; ++w) top = fmaxf(top, part[w][kMaxDim]);
  const float base = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < kGWarps; ++w) sum += part[w][kMaxDim + 1] * expf(part[w][kMaxDim] - base);
  // nothing but logits of -inf: zeros, unless a query that is not finite made them
  if (sum == 0.0f && seen && odd) sum = NAN;
  float* orow = a.O + t * a.ldo + static_cast<long long>(h) * D;
  for (int d = threadIdx.x; d < D; d += kGWarps * 32) {
    float o = 0.0f;
    for (int w = 0; w < kGWarps; ++w) o += part[w][d] * expf(part[w][kMaxDim] - base);
    if (LQ_IN_BOUNDS(t < a.b.tokens && h < a.heads)) orow[d] = sum == 0.0f ? 0.0f : o / sum;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<long long>(t) * a.heads + h] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

}  // namespace

lq_status launch_attn_generic(const AttnArgs& a, int fmt, cudaStream_t stream) {
  const long long ctas = static_cast<long long>(a.b.tokens) * a.heads;
  if (ctas > (1LL << 31) - 1) return LQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kGWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*kernel)(AttnArgs) = fmt == LQ_FMT_F16    ? attn_generic_kernel<LQ_FMT_F16>
                             : fmt == LQ_FMT_Q8_0 ? attn_generic_kernel<LQ_FMT_Q8_0>
                                                  : attn_generic_kernel<LQ_FMT_Q4_0>;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_route(kAttnRouteGeneric);
  return cuda_status(e);
}

unsigned read_clear_attn_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_attn_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

size_t lq_attn_work_bytes(const lq_kv_cache* cache, const lq_kv_batch* batch, int64_t heads) {
  bool noop;
  if (kv_check(cache, batch, &noop) != LQ_OK) return 0;
  if (heads < 1 || heads % cache->kv_heads != 0 || heads > 65536) return 0;
  return std::max(attn_warp_work_bytes(), attn_tile_work_bytes(cache->head_dim));
}

lq_status lq_attn_paged(const lq_kv_cache* cache, const lq_kv_batch* batch, const float* Q, int64_t ldq,
                        float* O, int64_t ldo, float* lse, int64_t heads, float scale, int64_t window,
                        int64_t sinks, void* work, void* stream) {
  bool noop;
  lq_status st = kv_check(cache, batch, &noop);
  if (st != LQ_OK) return st;
  if (heads < 1 || heads % cache->kv_heads != 0 || window < 0 || sinks < 0 || !std::isfinite(scale))
    return LQ_ERR_INVALID_ARG;
  if (noop) return LQ_OK;
  const int64_t width = heads * cache->head_dim;
  if (!Q || !O || !work || !aligned_to(Q, 4) || !aligned_to(O, 4) || !aligned_to(lse, 4) || !aligned_to(work, 16))
    return LQ_ERR_INVALID_ARG;
  if (ldq < width || ldo < width) return LQ_ERR_INVALID_ARG;
  if (heads > 65536 || batch->tokens * heads > (1LL << 31) - 1) return LQ_ERR_UNSUPPORTED;
  AttnArgs a = {};
  a.c = kv_cache_view(*cache);
  a.b = kv_batch_view(*batch);
  a.Q = Q;
  a.O = O;
  a.lse = lse;
  a.ldq = ldq;
  a.ldo = ldo;
  a.heads = static_cast<int>(heads);
  a.group = static_cast<int>(heads / cache->kv_heads);
  a.scale = scale;
  const int64_t most = 1LL << 30;  // past every position (kv_check)
  a.window = static_cast<int>(std::min(window, most));
  a.sinks = static_cast<int>(std::min(sinks, most));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int route = g_attn_route.load();
  // (without pages the other kernels have no address that they may read)
  if (route == 1 || a.c.num_pages == 0) return launch_attn_generic(a, cache->fmt, s);
  // the most rows (tokens x query heads a key/value head) of a sequence, as
  // far as the host knows
  const int64_t q = batch->max_q > 0 ? std::min(batch->max_q, batch->tokens) : batch->tokens;
  const int rows = static_cast<int>(std::min<int64_t>(q * a.group, 1 << 30));
  if (route == 2) return launch_attn_warp(a, cache->fmt, rows, 0, work, s);
  if (route == 3) return launch_attn_tile(a, cache->fmt, 0, work, s);
  if (!attn_warp_eligible(a)) return launch_attn_generic(a, cache->fmt, s);
  const int few = few_rows(cache->fmt, cache->head_dim);
  if (rows <= few || !attn_tile_eligible(a)) return launch_attn_warp(a, cache->fmt, rows, 0, work, s);
  // one sequence: all of it is one kernel's; else each kernel takes its own
  const int split = a.b.batch > 1 ? few : 0;
  if (split) {
    st = launch_attn_warp(a, cache->fmt, split, split, work, s);
    if (st != LQ_OK) return st;
  }
  return launch_attn_tile(a, cache->fmt, split, work, s);
}

lq_status lq_debug_attn_route(int route) {
  if (route < 0 || route > 3) return LQ_ERR_INVALID_ARG;
  g_attn_route.store(route);
  return LQ_OK;
}

}  // extern "C"
