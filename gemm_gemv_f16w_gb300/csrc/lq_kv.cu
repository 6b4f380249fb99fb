// Writing tokens into the paged key/value cache and reading them back.
//
// One pass over the data: 4 bytes an element come in or go out as f32, and
// 2 (f16), 1.0625 (Q8_0) or 0.5625 (Q4_0) as codes and scales: HBM is the
// floor (for a decode step, the launch), and instruction issue the first
// bound: a warp has about 40 cycles for 128 elements. A warp takes 1024
// consecutive elements of one token's heads, four per lane and load, so that
// a block of 32 is eight neighbouring lanes: its largest magnitude is three
// shuffles away, four codes of a lane leave as one 4-byte store (Q4_0: the
// low-nibble lanes fetch their partners' codes with one shuffle), and the
// loads of all groups are in flight before the first is used. The eight
// warps of a CTA take 16 consecutive tokens, whose rows are neighbours in a page.
//
// The rounding rules are those of the host packers (lq_pack.cpp), and the
// codes are theirs bit for bit, without a division an element: the scale
// top / 127 comes from the rounded reciprocal by Markstein's correction (the
// remainder top - 127 q is exact, q + remainder / 127 rounds correctly:
// tests/test_kv_scale_cpu.py, for every mantissa), and x / d from an approximate
// reciprocal, whose error (3e-5 at most) cannot change a code unless x / d is
// within 1e-4 of a half. Blocks with such an element (one in 160), with values
// beyond the cache's range, NaNs or scales near f32's smallest take the exact
// divisions.
//
// 16384 tokens, 8 heads of 128, Q8_0: written in 42 us (4.0 TB/s; 59 % of the
// issue slots, the loads' latency for the rest), written and read back in 69 (107
// with the divisions for all). 37 thousand such tokens read back: 61 us (6.2 TB/s,
// 92 % of a copy). One token of each of eight sequences written and read back: 7.5
// us from a graph, two launches.
#include <algorithm>

#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

__device__ unsigned g_kv_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_kv_err, 0u, code); }

constexpr int kKvWarps = 8;
constexpr int kKvTokens = 16;  // tokens of a CTA
constexpr int kKvGroups = 8;  // 128-element groups of a warp
constexpr float kTiny = 1.0842021724855044e-19f;  // 2^-63: remainders and reciprocals stay normal above

struct KvArgs {
  kv::Cache c;
  kv::Batch b;
  const float* in[2];  // K, V rows (write)
  float* out[2];       // K, V rows (read; null: skip)
  long long ld[2];
  int width;           // kv_heads * head_dim
  int sides, only;     // 2: K and V; 1: only K (0) or only V (1)
  unsigned by_dim;     // ceil(2^32 / head_dim): e / head_dim is the high word of e * by_dim (e < 2^24)
};

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float clamped(float x) { return fminf(fmaxf(x, -65504.0f), 65504.0f); }

// Destination of four codes: one store where the pool is aligned for it.
template <bool VEC, class T>
__device__ __forceinline__ void store4(unsigned char* at, const T (&q)[4]) {
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(q);
    else
      *reinterpret_cast<unsigned*>(at) = *reinterpret_cast<const unsigned*>(q);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<T*>(at)[j] = q[j];
  }
}

// Quantises and stores the lane's four elements x (elements e .. e + 3 of the
// head's row; lanes 8i .. 8i + 7 hold one block). `row` and `scales` are the
// token's codes and scales; null drops the store (all lanes still take part
// in the shuffles).
template <int FMT, bool VEC>
__device__ __forceinline__ void put(const float4& x4, int e, unsigned char* row, __half* scales, int lane) {
  const float x[4] = {x4.x, x4.y, x4.z, x4.w};
  if constexpr (FMT == LQ_FMT_F16) {
    alignas(8) __half h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __float2half_rn(x[j] == x[j] ? clamped(x[j]) : x[j]);
    if (row) store4<VEC>(row + 2 * e, h);
  } else {
    // (a NaN is lost here and found by the test of the quotients)
    const float mine = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    float top = mine;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // the block's first element of at least this magnitude (the whole warp asks)
    auto first_of = [&](float size) {
      const unsigned holders = __ballot_sync(0xffffffffu, mine >= size) >> (lane & 24);
      const int first = __ffs(static_cast<int>(holders & 0xFFu)) - 1;
      float own = x[3];
#pragma unroll
      for (int j = 2; j >= 0; --j) own = fabsf(x[j]) >= size ? x[j] : own;
      return __shfl_sync(0xffffffffu, own, (lane & 24) + first);
    };
    float m = top;
    if constexpr (FMT == LQ_FMT_Q4_0) m = first_of(top);  // the largest gives the scale its sign
    // q = m / 127, or m / -8 (exact)
    constexpr float kBy127 = 1.0f / 127.0f;
    float d = m * -0.125f;
    if constexpr (FMT == LQ_FMT_Q8_0) {
      const float q = m * kBy127;
      d = __fmaf_rn(__fmaf_rn(-127.0f, q, m), kBy127, q);
    }
    const float by_d = top == 0.0f ? 0.0f : reciprocal(d);
    constexpr float kMagic = 12582912.0f + (FMT == LQ_FMT_Q4_0 ? 8.0f : 0.0f);  // 1.5 2^23: the sum's low byte is the code
    unsigned t[4];
    bool plain = top <= 65504.0f && (top == 0.0f || top >= kTiny);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y = x[j] * by_d;
      if constexpr (FMT == LQ_FMT_Q4_0) y = y > 7.25f ? 7.25f : y;  // 7.5 .. 8 is code 15 too (a NaN stays)
      const float r = y + kMagic;
      plain = plain && fabsf((r - kMagic) - y) < 0.4999f;  // no half near, no NaN
      t[j] = __float_as_uint(r);
    }
    bool bad = false;
    unsigned word = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    if (__any_sync(0xffffffffu, !plain)) {  // by the definition's own divisions
      // a NaN in the block: of its eight lanes, any
      bad = ((__ballot_sync(0xffffffffu, x[0] != x[0] || x[1] != x[1] || x[2] != x[2] || x[3] != x[3]) >> (lane & 24)) & 0xFFu) != 0u;
      // of several values beyond the range the first counts: once clamped they are equal
      if constexpr (FMT == LQ_FMT_Q4_0) m = first_of(fminf(top, 65504.0f));
      d = FMT == LQ_FMT_Q8_0 ? __fdiv_rn(fminf(top, 65504.0f), 127.0f) : __fdiv_rn(clamped(m), -8.0f);
      word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int v = FMT == LQ_FMT_Q8_0 ? 0 : 8;
        if (!bad && d != 0.0f) {
          const float y = __fdiv_rn(clamped(x[j]), d);
          v = FMT == LQ_FMT_Q8_0 ? max(-127, min(127, static_cast<int>(roundf(y)))) : min(15, static_cast<int>(__fadd_rn(y, 8.5f)));
        }
        word |= (static_cast<unsigned>(v) & 0xFFu) << (8 * j);
      }
    }
    if constexpr (FMT == LQ_FMT_Q4_0) {
      word &= 0x0F0F0F0Fu;
      word |= __shfl_down_sync(0xffffffffu, word, 4) << 4;  // elements + 16
    }
    alignas(4) unsigned char q[4];
    *reinterpret_cast<unsigned*>(q) = word;
    if constexpr (FMT == LQ_FMT_Q8_0) {
      if (row) store4<VEC>(row + e, q);
    } else {
      if (row && (lane & 4) == 0) store4<VEC>(row + (e >> 5) * 16 + (e & 15), q);
    }
    if (row && (lane & 7) == 0) scales[e >> 5] = bad ? __ushort_as_half(0x7E00) : __float2half_rn(d);
  }
}

// The codes (and scale) of the four elements e .. e + 3 of a stored row, and
// the values that they stand for.
struct Four {
  uint2 codes;
  unsigned short scale;
};
template <int FMT, bool VEC>
__device__ __forceinline__ Four take4(const unsigned char* row, const __half* scales, int e) {
  Four f;
  f.codes = make_uint2(0u, 0u);
  f.scale = 0;
  if constexpr (FMT == LQ_FMT_F16) {
    if constexpr (VEC) {
      f.codes = __ldg(reinterpret_cast<const uint2*>(row + 2 * e));
    } else {
      const unsigned short* at = reinterpret_cast<const unsigned short*>(row) + e;
      f.codes = make_uint2(at[0] | static_cast<unsigned>(at[1]) << 16, at[2] | static_cast<unsigned>(at[3]) << 16);
    }
  } else {
    const unsigned char* at = FMT == LQ_FMT_Q8_0 ? row + e : row + (e >> 5) * 16 + (e & 15);
    if constexpr (VEC) {
      f.codes.x = __ldg(reinterpret_cast<const unsigned*>(at));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f.codes.x |= static_cast<unsigned>(at[j]) << (8 * j);
    }
    f.scale = __ldg(reinterpret_cast<const unsigned short*>(scales) + (e >> 5));
  }
  return f;
}
template <int FMT>
__device__ __forceinline__ float4 values4(const Four& f, int e) {
  if constexpr (FMT == LQ_FMT_F16) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f.codes.x)), y = __half22float2(*reinterpret_cast<const __half2*>(&f.codes.y));
    return make_float4(x.x, x.y, y.x, y.y);
  } else {
    const float d = __half2float(__ushort_as_half(f.scale));
    const unsigned w = FMT == LQ_FMT_Q8_0 ? f.codes.x ^ 0x80808080u : ((e & 16) ? f.codes.x >> 4 : f.codes.x) & 0x0F0F0F0Fu;
    constexpr float kBias = FMT == LQ_FMT_Q8_0 ? kMagicS8 : kMagicQ4;
    return make_float4(d * (s8_to_magic(w, 0) - kBias), d * (s8_to_magic(w, 1) - kBias), d * (s8_to_magic(w, 2) - kBias),
                       d * (s8_to_magic(w, 3) - kBias));
  }
}

// grid: x = groups of kKvTokens tokens, y = sides * (segment of kKvGroups * 128 elements) + side
template <int FMT, bool VEC, bool WRITE>
__global__ void __launch_bounds__(kKvWarps * 32) kv_kernel(const KvArgs a) {
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = a.sides == 2 ? static_cast<int>(blockIdx.y & 1u) : a.only;
  const int segment = static_cast<int>(a.sides == 2 ? blockIdx.y >> 1 : blockIdx.y);
  const int first = segment * (kKvGroups * 128) + lane * 4;
  // where the CTA's tokens are, a lane each (the chain of loads behind that is
  // paid once for a warp's two tokens); -2: the token is no sequence's
  const int t0 = static_cast<int>(blockIdx.x) * kKvTokens;
  int my_page = -2, my_slot = 0;
  if (lane < kKvTokens && t0 + lane < a.b.tokens) {
    const int t = t0 + lane;
    int lo = 0, n = a.b.batch;  // the last sequence that begins at or before t is in [lo, lo + n)
    while (n > 1) {
      const int half = n / 2;
      const bool right = a.b.q_start[lo + half] <= t;
      lo = right ? lo + half : lo;
      n = right ? n - half : half;
    }
    if (a.b.q_start[lo] <= t && t < a.b.q_start[lo + 1]) {
      const kv::Seq s = kv::sequence(a.b, a.c.page_size, lo);
      const int p = s.len - s.rows + (t - s.row0);
      my_page = p >= 0 ? kv::page_of(a.c, a.b, lo, p) : -1;
      my_slot = max(p, 0) % a.c.page_size;
    }
  }
#pragma unroll 1
  for (int tt = warp; tt < kKvTokens && t0 + tt < a.b.tokens; tt += kKvWarps) {
    const int t = t0 + tt;
    float4 x[kKvGroups];
    if constexpr (WRITE) {
      const float* in = a.in[which] + t * a.ld[which];
#pragma unroll
      for (int g = 0; g < kKvGroups; ++g) {
        const int e = first + g * 128;
        x[g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (e < a.width) {
          if constexpr (VEC) {
            x[g] = *reinterpret_cast<const float4*>(in + e);
          } else {
            x[g] = make_float4(in[e], in[e + 1], in[e + 2], in[e + 3]);
          }
        }
      }
    }
    const int page = __shfl_sync(0xffffffffu, my_page, tt), slot = __shfl_sync(0xffffffffu, my_slot, tt);
    const int D = a.c.head_dim;
    const unsigned head_bytes = static_cast<unsigned>(a.c.head_bytes);  // at most 2^16 tokens of 512 bytes
    // the token's codes and scales of head 0
    unsigned char* codes = nullptr;
    __half* scale0 = nullptr;
    if (page >= 0 && LQ_IN_BOUNDS(page < a.c.num_pages)) {
      unsigned char* at = (which ? a.c.v : a.c.k) + page * a.c.page_bytes;
      codes = at + static_cast<long long>(slot) * a.c.row_bytes;
      scale0 = reinterpret_cast<__half*>(at + static_cast<long long>(a.c.page_size) * a.c.row_bytes) + slot * (D / 32);
    }
    auto place = [&](int e, unsigned char*& row, __half*& scales) {  // the head of element e; its element there
      const unsigned h = __umulhi(static_cast<unsigned>(e), a.by_dim);
      row = nullptr;
      scales = nullptr;
      if (codes && e < a.width && LQ_IN_BOUNDS(h < static_cast<unsigned>(a.c.kv_heads))) {
        const unsigned long long at = static_cast<unsigned long long>(h) * head_bytes;
        row = codes + at;
        scales = reinterpret_cast<__half*>(reinterpret_cast<unsigned char*>(scale0) + at);
      }
      return e - static_cast<int>(h) * D;
    };
    unsigned char* row;
    __half* scales;
    if constexpr (WRITE) {
#pragma unroll
      for (int g = 0; g < kKvGroups; ++g) {
        const int e = first + g * 128;
        if (e - lane * 4 >= a.width) break;  // the warp's last group
        const int r = place(e, row, scales);
        put<FMT, VEC>(x[g], r, row, scales, lane);
      }
    } else if (page != -2) {
      float* const out0 = a.out[which] + t * a.ld[which] + first;
      Four got[kKvGroups];  // all on their way before the first is used
#pragma unroll
      for (int g = 0; g < kKvGroups; ++g) {
        got[g].codes = make_uint2(0u, 0u);
        got[g].scale = 0;
        const int r = place(first + g * 128, row, scales);
        if (row) got[g] = take4<FMT, VEC>(row, scales, r);
      }
#pragma unroll
      for (int g = 0; g < kKvGroups; ++g) {
        const int e = first + g * 128;
        if (e >= a.width) break;
        const int r = e - static_cast<int>(__umulhi(static_cast<unsigned>(e), a.by_dim)) * D;
        // (no place: zeros; a 4-bit code of zero stands for -8 d, d is zero too)
        const float4 v = values4<FMT>(got[g], r);
        float* out = out0 + g * 128;
        if constexpr (VEC) {
          *reinterpret_cast<float4*>(out) = v;
        } else {
          out[0] = v.x;
          out[1] = v.y;
          out[2] = v.z;
          out[3] = v.w;
        }
      }
    }
  }
}

template <bool WRITE>
lq_status launch(int fmt, KvArgs& a, cudaStream_t stream) {
  a.by_dim = static_cast<unsigned>(((1ull << 32) + a.c.head_dim - 1) / a.c.head_dim);
  a.sides = WRITE || (a.out[0] && a.out[1]) ? 2 : 1;
  a.only = !WRITE && !a.out[0] ? 1 : 0;
  const unsigned segments = static_cast<unsigned>((a.width + kKvGroups * 128 - 1) / (kKvGroups * 128));
  bool vec = a.c.head_bytes % 16 == 0 && aligned_to(a.c.k, 16) && aligned_to(a.c.v, 16);
  for (int i = 0; i < 2; ++i) {
    const void* p = WRITE ? static_cast<const void*>(a.in[i]) : static_cast<const void*>(a.out[i]);
    vec = vec && (!p || (a.ld[i] % 4 == 0 && aligned_to(p, 16)));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.b.tokens + kKvTokens - 1) / kKvTokens),
                     static_cast<unsigned>(a.sides) * segments);
  cfg.blockDim = dim3(kKvWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*kernel)(KvArgs) = nullptr;
  switch (fmt) {
    case LQ_FMT_F16: kernel = vec ? kv_kernel<LQ_FMT_F16, true, WRITE> : kv_kernel<LQ_FMT_F16, false, WRITE>; break;
    case LQ_FMT_Q8_0: kernel = vec ? kv_kernel<LQ_FMT_Q8_0, true, WRITE> : kv_kernel<LQ_FMT_Q8_0, false, WRITE>; break;
    default: kernel = vec ? kv_kernel<LQ_FMT_Q4_0, true, WRITE> : kv_kernel<LQ_FMT_Q4_0, false, WRITE>; break;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

}  // namespace

lq_status kv_check(const lq_kv_cache* cache, const lq_kv_batch* batch, bool* noop) {
  *noop = false;
  if (!cache || !batch) return LQ_ERR_INVALID_ARG;
  const lq_kv_cache& c = *cache;
  const lq_kv_batch& b = *batch;
  if (c.fmt == LQ_FMT_Q4_0I) return LQ_ERR_UNSUPPORTED;
  if (c.fmt != LQ_FMT_F16 && c.fmt != LQ_FMT_Q8_0 && c.fmt != LQ_FMT_Q4_0) return LQ_ERR_INVALID_ARG;
  if (c.page_size < 1 || c.page_size > 65536 || c.kv_heads < 1 || c.num_pages < 0) return LQ_ERR_INVALID_ARG;
  if (c.head_dim < 32 || c.head_dim % 32 != 0) return LQ_ERR_INVALID_ARG;
  if (b.batch < 0 || b.tokens < 0 || b.max_q < 0 || b.max_pages < 0) return LQ_ERR_INVALID_ARG;
  if (b.batch == 0 || b.tokens == 0) {
    *noop = true;
    return LQ_OK;
  }
  if (!c.k || !c.v || !aligned_to(c.k, 2) || !aligned_to(c.v, 2)) return LQ_ERR_INVALID_ARG;
  if (!b.page_table || !b.kv_len || !b.q_start) return LQ_ERR_INVALID_ARG;
  if (!aligned_to(b.page_table, 4) || !aligned_to(b.kv_len, 4) || !aligned_to(b.q_start, 4)) return LQ_ERR_INVALID_ARG;
  // 32-bit token, page and row indices inside the kernels
  const long long most = (1LL << 31) - 1;
  if (static_cast<int64_t>(b.max_pages) * c.page_size > (1LL << 30)) return LQ_ERR_UNSUPPORTED;
  if (c.head_dim > 256 || c.num_pages > most || b.tokens > (1LL << 30) || c.kv_heads > 4096) return LQ_ERR_UNSUPPORTED;
  return LQ_OK;
}

kv::Cache kv_cache_view(const lq_kv_cache& c) {
  kv::Cache v;
  v.k = static_cast<unsigned char*>(c.k);
  v.v = static_cast<unsigned char*>(c.v);
  v.row_bytes = kv::code_row_bytes(c.fmt, c.head_dim);
  v.head_bytes = static_cast<long long>(c.page_size) * (v.row_bytes + (c.fmt == LQ_FMT_F16 ? 0 : c.head_dim / 32 * 2));
  v.page_bytes = v.head_bytes * c.kv_heads;
  v.page_size = c.page_size;
  v.kv_heads = c.kv_heads;
  v.head_dim = c.head_dim;
  v.num_pages = static_cast<int>(c.num_pages);
  return v;
}

kv::Batch kv_batch_view(const lq_kv_batch& b) {
  kv::Batch v;
  v.table = b.page_table;
  v.kv_len = b.kv_len;
  v.q_start = b.q_start;
  v.batch = b.batch;
  v.max_pages = b.max_pages;
  v.tokens = static_cast<int>(b.tokens);
  return v;
}

unsigned read_clear_kv_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_kv_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

size_t lq_kv_pool_bytes(int fmt, int64_t num_pages, int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  if (fmt != LQ_FMT_F16 && fmt != LQ_FMT_Q8_0 && fmt != LQ_FMT_Q4_0) return 0;
  if (num_pages < 0 || num_pages > (1LL << 31) - 1 || page_size < 1 || page_size > 65536) return 0;
  if (kv_heads < 1 || kv_heads > 4096 || head_dim < 32 || head_dim % 32 != 0 || head_dim > 256) return 0;
  const size_t row = static_cast<size_t>(kv::code_row_bytes(fmt, static_cast<int>(head_dim))) +
                     (fmt == LQ_FMT_F16 ? 0 : static_cast<size_t>(head_dim) / 32 * 2);
  const unsigned __int128 bytes = static_cast<unsigned __int128>(row) * static_cast<size_t>(page_size) *
                                  static_cast<size_t>(kv_heads) * static_cast<size_t>(num_pages);
  return bytes > (static_cast<unsigned __int128>(1) << 62) ? 0 : static_cast<size_t>(bytes);
}

lq_status lq_kv_write(const lq_kv_cache* cache, const lq_kv_batch* batch, const float* K, int64_t ldk,
                      const float* V, int64_t ldv, void* stream) {
  bool noop;
  lq_status st = kv_check(cache, batch, &noop);
  if (st != LQ_OK || noop) return st;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (!K || !V || !aligned_to(K, 4) || !aligned_to(V, 4) || ldk < width || ldv < width) return LQ_ERR_INVALID_ARG;
  KvArgs a = {};
  a.c = kv_cache_view(*cache);
  a.b = kv_batch_view(*batch);
  a.in[0] = K;
  a.in[1] = V;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.width = static_cast<int>(width);
  return launch<true>(cache->fmt, a, static_cast<cudaStream_t>(stream));
}

lq_status lq_kv_read(const lq_kv_cache* cache, const lq_kv_batch* batch, float* K, int64_t ldk, float* V,
                     int64_t ldv, void* stream) {
  bool noop;
  lq_status st = kv_check(cache, batch, &noop);
  if (st != LQ_OK || noop) return st;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (!K && !V) return LQ_ERR_INVALID_ARG;
  if (!aligned_to(K, 4) || !aligned_to(V, 4) || (K && ldk < width) || (V && ldv < width)) return LQ_ERR_INVALID_ARG;
  KvArgs a = {};
  a.c = kv_cache_view(*cache);
  a.b = kv_batch_view(*batch);
  a.out[0] = K;
  a.out[1] = V;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.width = static_cast<int>(width);
  return launch<false>(cache->fmt, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
