// Rotary positions with one or several axes: lq_rope_init, lq_rope.
//
// Mathematics. Pair j of a head's first rotary_dim values is turned by the angle
// t = pos[axis(j)] * freq_j:
//     y_a = f (x_a cos t - x_b sin t),   y_b = f (x_b cos t + x_a sin t).
// Angles of far positions have to be reduced with more bits than f32 has: at
// position 10^6 an f32 product is off by 0.06. Here a frequency is held as turns
// a position in units of 2^-64, so that the 64-bit integer product with the
// position is the angle modulo one turn by itself (the frequency is off by 1.5 units
// at most, the angle by 2^-32 of a turn at any 32-bit position). Of its upper 32 bits the
// nearest quarter is taken off in integers and turned by exactly; what is left, an eighth
// of a turn at most, goes to sincospif in f32, which rounds it by 2^-28 of a turn at most
// (the whole angle in f32 would be off by 2^-26).
//
// Split. A warp takes one token and a range of its heads; a lane owns a unit of
// eight values (four pairs) at the same place of every head, so that cosines
// and sines are computed once and stay in registers for all of the warp's heads.
// Loads of four heads are on their way before the first is used. Values behind
// the rotary ones are copied by lanes of their own (in place: not touched).
// With many tokens a warp takes all heads; with few, heads are spread over more
// warps until there are about eight an SM (32 tokens of 32 + 8 heads of 128, one
// warp a token: 5.7 us, spread: 2.5; 300 tokens: 5.9 and 3.7).
//
// What bounds it: each value is read and written once, HBM for prompts (16383 tokens
// of 32 + 8 heads of 128, three axes: 102 us, 6.56 TB/s, 98 % of a copy; pairs of
// neighbours 106; 64 dims of 16 + 2 heads of 256: 93); a launch and one round of loads
// for a step.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "lq_device.cuh"
#include "lq_internal.h"

namespace lq {
namespace {

__device__ unsigned g_rope_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_rope_err, 0u, code); }

constexpr int kWarps = 4;
constexpr int kHeadsAhead = 4;  // heads whose loads are on their way together

struct RopeArgs {
  lq_rope_table r;
  const int32_t* pos;
  const float* in[2];  // Q, K
  float* out[2];
  long long ldp, ld_in[2], ld_out[2];
  long long tokens;
  int heads[2];
  int head_dim, half;  // half: pairs
  int units;           // of a head, rotated ones first
  int splits, per;     // warps a token; heads a warp
  float sign;
};

// W: values of a lane's vector; a unit is two of them.
template <int W>
struct Vec {
  float v[W];
};
template <int W>
__device__ __forceinline__ Vec<W> load(const float* at) {
  Vec<W> x;
  if constexpr (W == 4) {
    const float4 f = *reinterpret_cast<const float4*>(at);
    x.v[0] = f.x;
    x.v[1] = f.y;
    x.v[2] = f.z;
    x.v[3] = f.w;
  } else {
    x.v[0] = *at;
  }
  return x;
}
template <int W>
__device__ __forceinline__ void store(float* at, const Vec<W>& x) {
  if constexpr (W == 4) {
    *reinterpret_cast<float4*>(at) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  } else {
    *at = x.v[0];
  }
}

template <int W, bool ADJACENT>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long t = item / a.splits;
  if (t >= a.tokens) return;
  const int h0 = static_cast<int>(item - t * a.splits) * a.per, all = a.heads[0] + a.heads[1], h1 = min(h0 + a.per, all);
  // lanes of a head: the power of two that holds its units (32 at a time where it has more)
  int lanes = 1;
  while (lanes < a.units && lanes < 32) lanes *= 2;
  const int rotated = a.half / W;
#pragma unroll 1
  for (int u = lane % lanes; u - lane % lanes < a.units; u += lanes) {
    const bool turns = u < rotated;
    float c[W], s[W];  // of the unit's W pairs
    int at0, at1;
    if (turns) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int j = u * W + i;
        const long long p = a.pos[a.r.axis[j] * a.ldp + t];
        const unsigned long long turn = static_cast<unsigned long long>(p) * a.r.turns[j];
        const unsigned part = static_cast<unsigned>((turn + (1ull << 31)) >> 32), quarter = (part + (1u << 29)) >> 30;
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int>(part - (quarter << 30))) * 0x1p-31f, &sn, &cs);
        const float x = quarter & 1u ? sn : cs, y = quarter & 1u ? cs : sn;
        c[i] = quarter == 1u || quarter == 2u ? -x : x;
        s[i] = quarter >= 2u ? -y : y;
        c[i] *= a.r.factor;
        s[i] *= a.r.factor * a.sign;
      }
      at0 = ADJACENT ? 2 * W * u : W * u;
      at1 = ADJACENT ? at0 + W : a.half + W * u;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
      }
      at0 = 2 * a.half + 2 * W * (u - rotated);
      at1 = at0 + W;
    }
    const bool mine = u < a.units && LQ_IN_BOUNDS(at1 + W <= a.head_dim);
    const int step = 32 / lanes;  // heads at a time
#pragma unroll 1
    for (int h = h0 + lane / lanes; h < h1; h += step * kHeadsAhead) {
      Vec<W> x[kHeadsAhead][2];
#pragma unroll
      for (int n = 0; n < kHeadsAhead; ++n) {
        const int hh = h + n * step, side = hh < a.heads[0] ? 0 : 1;
        if (mine && hh < h1) {
          const float* from = a.in[side] + t * a.ld_in[side] + static_cast<long long>(side ? hh - a.heads[0] : hh) * a.head_dim;
          x[n][0] = load<W>(from + at0);
          x[n][1] = load<W>(from + at1);
        }
      }
#pragma unroll
      for (int n = 0; n < kHeadsAhead; ++n) {
        const int hh = h + n * step, side = hh < a.heads[0] ? 0 : 1;
        if (mine && hh < h1) {
          float* to = a.out[side] + t * a.ld_out[side] + static_cast<long long>(side ? hh - a.heads[0] : hh) * a.head_dim;
          Vec<W> y[2] = {x[n][0], x[n][1]};
          if (turns) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
              // pair i of the unit: (x0[i], x1[i]), or neighbours of the 2 W values
              const int e0 = ADJACENT ? 2 * i : i, e1 = ADJACENT ? 2 * i + 1 : W + i;
              const float p = x[n][e0 / W].v[e0 % W], q = x[n][e1 / W].v[e1 % W];
              y[e0 / W].v[e0 % W] = fmaf(p, c[i], -(q * s[i]));
              y[e1 / W].v[e1 % W] = fmaf(q, c[i], p * s[i]);
            }
          }
          store<W>(to + at0, y[0]);
          store<W>(to + at1, y[1]);
        }
      }
    }
  }
}

// What lq_rope_init makes; anything else was not made by it.
bool table_fits(const lq_rope_table& r) {
  if (r.head_dim < 2 || r.head_dim % 2 != 0 || r.head_dim > 65536) return false;
  if (r.rotary_dim < 2 || r.rotary_dim % 2 != 0 || r.rotary_dim > r.head_dim || r.rotary_dim > 2 * LQ_ROPE_MAX_PAIRS) return false;
  if ((r.pairs != LQ_ROPE_HALVES && r.pairs != LQ_ROPE_ADJACENT) || r.axes < 1 || r.axes > LQ_ROPE_MAX_AXES || !std::isfinite(r.factor))
    return false;
  for (int j = 0; j < r.rotary_dim / 2; ++j)
    if (r.axis[j] >= r.axes) return false;
  return true;
}

}  // namespace

unsigned read_clear_rope_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_rope_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

lq_status lq_rope_init(lq_rope_table* table, int64_t head_dim, int64_t rotary_dim, int pairs, double base, const double* freqs,
                       int64_t axes, const int32_t* sections, int interleaved, double factor) {
  if (!table || head_dim < 2 || head_dim % 2 != 0 || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > head_dim)
    return LQ_ERR_INVALID_ARG;
  if (pairs != LQ_ROPE_HALVES && pairs != LQ_ROPE_ADJACENT) return LQ_ERR_INVALID_ARG;
  if (axes < 1 || (axes > 1 && !sections) || !std::isfinite(factor) || !std::isfinite(static_cast<float>(factor)))
    return LQ_ERR_INVALID_ARG;
  if (!freqs && (!std::isfinite(base) || base <= 0.0)) return LQ_ERR_INVALID_ARG;
  if (rotary_dim > 2 * LQ_ROPE_MAX_PAIRS || axes > LQ_ROPE_MAX_AXES || head_dim > 65536) return LQ_ERR_UNSUPPORTED;
  const int half = static_cast<int>(rotary_dim / 2);
  if (sections) {
    int64_t sum = 0;
    for (int64_t x = 0; x < axes; ++x) {
      if (sections[x] < 0) return LQ_ERR_INVALID_ARG;
      // in turns, an axis's last pair, number axes * (section - 1) + its index, has to exist
      if (interleaved && x > 0 && sections[x] > 0 && axes * (sections[x] - 1) + x >= half) return LQ_ERR_INVALID_ARG;
      sum += sections[x];
    }
    if (sum != half) return LQ_ERR_INVALID_ARG;
  }
  lq_rope_table r;
  std::memset(&r, 0, sizeof(r));
  r.head_dim = static_cast<int32_t>(head_dim);
  r.rotary_dim = static_cast<int32_t>(rotary_dim);
  r.pairs = pairs;
  r.axes = static_cast<int32_t>(axes);
  r.factor = static_cast<float>(factor);
  int axis = 0, left = sections ? sections[0] : half;
  for (int j = 0; j < half; ++j) {
    const double freq = freqs ? freqs[j] : std::pow(base, -2.0 * j / static_cast<double>(rotary_dim));
    if (!(std::fabs(freq) <= 4294967296.0)) return LQ_ERR_INVALID_ARG;
    // |freq| / (2 pi) in two doubles, modulo 1, in units of 2^-64
    constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;
    const double size = std::fabs(freq), high = size * kHigh, low = std::fma(size, kHigh, -high) + size * kLow;
    const double part = high - std::floor(high);  // exact
    const uint64_t turn = static_cast<uint64_t>(std::ldexp(part, 64)) +
                          static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(std::ldexp(low, 64))));
    r.turns[j] = freq < 0.0 ? 0 - turn : turn;
    if (sections && interleaved) {
      const int turns = j % static_cast<int>(axes);
      r.axis[j] = static_cast<uint8_t>(j < axes * static_cast<int64_t>(sections[turns]) ? turns : 0);
    } else {
      while (left == 0) left = sections[++axis];
      r.axis[j] = static_cast<uint8_t>(axis);
      --left;
    }
  }
  *table = r;
  return LQ_OK;
}

lq_status lq_rope(const lq_rope_table* table, int64_t tokens, const int32_t* positions, int64_t ldp, const float* Q, int64_t ldq,
                  float* QO, int64_t ldqo, int64_t heads, const float* K, int64_t ldk, float* KO, int64_t ldko, int64_t kv_heads,
                  int inverse, void* stream) {
  if (!table || !table_fits(*table) || tokens < 0 || heads < 0 || kv_heads < 0) return LQ_ERR_INVALID_ARG;
  if (tokens == 0 || heads + kv_heads == 0) return LQ_OK;
  const int64_t d = table->head_dim;
  if (heads > 65536 || kv_heads > 65536 || tokens > (1LL << 30)) return LQ_ERR_UNSUPPORTED;
  // (ldp 0: all axes go by one row, which is only read)
  if (!positions || !aligned_to(positions, 4) || (table->axes > 1 && ldp != 0 && ldp < tokens)) return LQ_ERR_INVALID_ARG;
  RopeArgs a = {};
  a.r = *table;
  a.pos = positions;
  a.ldp = ldp;
  a.tokens = tokens;
  a.head_dim = table->head_dim;
  a.half = table->rotary_dim / 2;
  a.sign = inverse ? -1.0f : 1.0f;
  const float* in[2] = {Q, K};
  float* out[2] = {QO, KO};
  const int64_t li[2] = {ldq, ldk}, lo[2] = {ldqo, ldko}, n[2] = {heads, kv_heads};
  bool vec = d % 8 == 0 && table->rotary_dim % 8 == 0, in_place = true;
  for (int i = 0; i < 2; ++i) {
    if (n[i] == 0) continue;
    if (!in[i] || !out[i] || !aligned_to(in[i], 4) || !aligned_to(out[i], 4) || li[i] < n[i] * d || lo[i] < n[i] * d)
      return LQ_ERR_INVALID_ARG;
    if (in[i] == out[i] && li[i] != lo[i] && tokens > 1) return LQ_ERR_INVALID_ARG;  // rows would run into one another
    in_place = in_place && in[i] == out[i];
    vec = vec && aligned_to(in[i], 16) && aligned_to(out[i], 16) && li[i] % 4 == 0 && lo[i] % 4 == 0;
    a.in[i] = in[i];
    a.out[i] = out[i];
    a.ld_in[i] = li[i];
    a.ld_out[i] = lo[i];
    a.heads[i] = static_cast<int>(n[i]);
  }
  const int w = vec ? 4 : 1;
  a.units = static_cast<int>((in_place ? table->rotary_dim : d) / (2 * w));  // in place the other values stay
  // heads a warp: all of a token's, fewer while there are not eight warps an SM
  int lanes = 1;
  while (lanes < a.units && lanes < 32) lanes *= 2;
  const int all = a.heads[0] + a.heads[1], step = 32 / lanes;
  const int64_t want = 8LL * std::max(device_info().sm_count, 1);
  const int most = (all + step - 1) / step;
  const int splits = static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, want / tokens)));
  a.per = ((all + splits - 1) / splits + step - 1) / step * step;
  a.splits = (all + a.per - 1) / a.per;
  const int64_t items = tokens * a.splits, ctas = (items + kWarps - 1) / kWarps;
  if (ctas > (1LL << 31) - 1) return LQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool adjacent = table->pairs == LQ_ROPE_ADJACENT;
  void (*kernel)(RopeArgs) = vec ? (adjacent ? rope_kernel<4, true> : rope_kernel<4, false>)
                                 : (adjacent ? rope_kernel<1, true> : rope_kernel<1, false>);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

}  // extern "C"
