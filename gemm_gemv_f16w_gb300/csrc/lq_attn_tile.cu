// Attention of many rows (chunks, whole prompts) over the paged cache, on the
// 5th-generation tensor cores.
//
// Mathematics as in lq_attn_warp.cu: one pass over the keys with a running
// maximum M (set 11 below the largest base-2 logit, moved when a tile passes
// it by 15), weights p = 2^(x - M) and their sum, in f32; every product with
// f32's precision from f16 operands in two parts (x = hi + lo):
//   S = (q_hi + q_lo) (k_hi + k_lo)   for f16 caches k_lo = 0
//   O = p_hi v_hi + p_lo v_hi + p_hi v_lo
// q is scaled by a power of two per row to the top of f16's range first.
// Q8_0 and Q4_0 values d * code have at most 18 significant bits and are
// multiples of 2^-24, so hi (rounded toward zero, which keeps values up to
// 2 * 65504 in range) and lo hold them exactly.
//
// A unit is (sequence, key/value head, 256 query rows (token, head of the
// group)): two row tiles of 128 share every key tile. Key tiles are 128 "rows
// of shared memory": 128 keys (f16), or 64 keys, hi parts and then lo parts
// (quantised), so that both run the same MMAs: S[128 x 128] = Q K^T with K as
// it lies (K-major), and O[128 x D] = P V with P from tensor memory and V as
// it lies (its keys are the contraction: an MN-major operand), one layout and
// one loader for both. Tensor memory: S of the two row tiles (256 columns; P's
// parts overwrite S in place, 16 columns a 16 keys) and their O (2 D columns).
// O starts from zero in every tile and is added to the f32 sums that the
// softmax threads keep in registers (thread = row, D sums): the tensor core's
// own accumulation truncates, which over thousands of keys would show.
//
// Roles (four warpgroups, registers moved between them): two softmax groups,
// one per row tile; four loader warps (16-byte asynchronous copies for f16;
// loads, exact dequantisation and swizzled stores otherwise); one thread that
// issues MMAs: QK of both row tiles, then PV of both, so that one tile's
// softmax runs under the other's MMAs.
//
// What bounds it: the tensor cores, at two (f16) or 3.5 (quantised: 2 x 2
// products for S, 3 for O) MMAs a product of the plain formula. All units'
// key tiles are dealt in equal contiguous ranges to one CTA an SM; a unit
// that spans CTAs is joined from partial sums by the last one to arrive, in
// the order of the keys.
// Every wait is bounded; on timeout the kernel records LQ_ERR_DEVICE_TIMEOUT,
// lets its copies and MMAs finish, frees TMEM and returns.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lq_attn.cuh"
#include "lq_tcgen05.cuh"

namespace lq {
namespace {

__device__ unsigned g_attnt_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_attnt_err, 0u, code); }

constexpr int kThreads = 512;
constexpr int kRows = 256;          // query rows of a unit: two tiles of 128
constexpr int kLoaders = 128;       // loader threads
constexpr int kMinTiles = 4;        // key tiles worth a CTA
constexpr int kInfo = 16;           // tiles of bookkeeping kept
constexpr int kMaxBatch = 4096;     // sequences whose totals fit in shared memory
constexpr float kNoMax = -1e30f;    // M before the first key
constexpr float kLift = 11.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TileParams {
  AttnArgs a;
  int* counters;
  float* parts;
  int small_rows;  // sequences with at most this many rows are another kernel's
  int vec_q, vec_o;
  unsigned long long wait_ns;
  unsigned wait_iters;
};

template <int FMT, int D>
struct Geo {
  static constexpr int KT = FMT == LQ_FMT_F16 ? 128 : 64;  // keys of a tile
  static constexpr int ROW = FMT == LQ_FMT_F16 ? 2 * D : (FMT == LQ_FMT_Q8_0 ? D : D / 2);
  static constexpr int HALVES = D / 64;                    // 64-dim column groups
  static constexpr int GROUP = 128 * 128;                  // bytes of a group: 128 rows of 128 bytes
  static constexpr int UNIT = HALVES * GROUP;              // K or V of a tile
  static constexpr int NU = D == 128 ? 3 : 6;              // ring of units
  static constexpr int QPART = HALVES * GROUP;             // hi or lo of a row tile
  static constexpr int Q = 4 * QPART;                      // [row tile][hi, lo]
  static constexpr int SMEM = Q + NU * UNIT + 1024 + 1024;  // alignment, barriers
  static constexpr int SLOT = kRows * (D + 2);             // floats of a partial result
  // registers a thread of the warpgroups: together the launch's 4 * 128
  static constexpr int REG_SOFTMAX = D == 128 ? 200 : 168, REG_LOAD = D == 128 ? 72 : 128, REG_MMA = D == 128 ? 40 : 48;
  static_assert(2 * REG_SOFTMAX + REG_LOAD + REG_MMA <= 512);
};

struct Bars {
  uint64_t full[6], empty[6];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort;
  int last;
  int start_i, start_h, start_rt, start_k;
  long long total;
  uint64_t join;             // the softmax threads of a unit that spans CTAs
  // first key; bit g: the page of keys 16 g .. is there, kTwo, kFirst
  int2 info[kInfo];
  uint32_t bad[kInfo][4];    // keys whose values are not finite (kept out of the MMA)
};
static_assert(sizeof(Bars) <= 1024);
constexpr uint32_t kTwo = 1u << 8;    // both row tiles of the unit have rows
constexpr uint32_t kFirst = 1u << 9;  // the unit's first tile here

__device__ __forceinline__ uint64_t desc_mn(uint32_t at) {  // 128-byte swizzle, MN-major: 64-dim groups, 8-key groups
  uint64_t d = 0;
  d |= static_cast<uint64_t>((at & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((128u * 128u) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// One lane of a converged warp, the same every time; the compiler knows that
// it is one, and keeps the MMAs' descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2(h);
  lo = h2(__floats2half2_rn(x - f.x, y - f.y));
}
// Four int8 codes (a word) as two f16 pairs: (code + 128) in the mantissa of
// 1024, less 1152; both steps are exact.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t& p0, uint32_t& p1) {
  const __half2 bias = __half2half2(__ushort_as_half(0xE480));  // -1152
  w ^= 0x80808080u;
  p0 = h2(__hadd2(as_h2(__byte_perm(w, 0x64646464u, 0x4140)), bias));
  p1 = h2(__hadd2(as_h2(__byte_perm(w, 0x64646464u, 0x4342)), bias));
}
// The nibbles of four bytes, less 8, as f16 pairs: low nibbles, high nibbles.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& l0, uint32_t& l1, uint32_t& h0, uint32_t& h1) {
  const __half2 bias = __half2half2(__ushort_as_half(0xE408));  // -1032
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  l0 = h2(__hadd2(as_h2(__byte_perm(lo, 0x64646464u, 0x4140)), bias));
  l1 = h2(__hadd2(as_h2(__byte_perm(lo, 0x64646464u, 0x4342)), bias));
  h0 = h2(__hadd2(as_h2(__byte_perm(hi, 0x64646464u, 0x4140)), bias));
  h1 = h2(__hadd2(as_h2(__byte_perm(hi, 0x64646464u, 0x4342)), bias));
}
// The exact split of a dequantised pair: hi toward zero, lo the rest.
__device__ __forceinline__ void split2_rz(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  const float2 f = __half22float2(as_h2(hi));
  lo = h2(__floats2half2_rn(x - f.x, y - f.y));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A unit of this kernel and the part [k0, k1) of its n key tiles.
struct Work {
  int i, h, rt, row_tiles;
  kv::Seq s;
  int n, sink_tiles, first;  // tiles [0, sink_tiles) and [first, ...)
  int k0, k1;
  int p0, p1;  // positions of its first and last row
};

template <int KT>
__device__ __forceinline__ void unit_tiles(Work& w, const AttnArgs& a) {
  const int rows = w.s.rows * a.group, rho0 = w.rt * kRows;
  w.p0 = w.s.len - w.s.rows + rho0 / a.group;
  w.p1 = w.s.len - w.s.rows + min(rho0 + kRows - 1, rows - 1) / a.group;
  const kv::Visible v = kv::visible(max(w.p0, 0), a.window, a.sinks);
  w.first = v.begin / KT;
  w.sink_tiles = min((v.sink_end + KT - 1) / KT, w.first);
  w.n = w.p1 < 0 ? 1 : w.sink_tiles + w.p1 / KT + 1 - w.first;  // one empty tile where there is no key
}

__device__ __forceinline__ bool takes(const kv::Seq& s, const TileParams& P) {
  return s.rows > 0 && s.rows * P.a.group > P.small_rows;
}

// Walks a CTA's range of tiles unit by unit; every role walks for itself.
template <int KT>
struct Walk {
  Work w;
  long long left;  // tiles of the range from w.k0 on
  __device__ __forceinline__ void enter(const TileParams& P, int i) {
    for (;; ++i) {
      w.s = kv::sequence(P.a.b, P.a.c.page_size, i);
      if (takes(w.s, P)) break;
    }
    w.i = i;
    w.row_tiles = (w.s.rows * P.a.group + kRows - 1) / kRows;
  }
  __device__ __forceinline__ void begin(const TileParams& P, const Bars* b, long long tiles) {
    enter(P, b->start_i);
    w.h = b->start_h;
    w.rt = b->start_rt;
    left = tiles;
    unit_tiles<KT>(w, P.a);
    w.k0 = b->start_k;
    w.k1 = static_cast<int>(min(static_cast<long long>(w.n), w.k0 + left));
  }
  __device__ __forceinline__ bool next(const TileParams& P) {
    left -= w.k1 - w.k0;
    if (left <= 0) return false;
    if (++w.rt == w.row_tiles) {
      w.rt = 0;
      if (++w.h == P.a.c.kv_heads) {
        w.h = 0;
        enter(P, w.i + 1);
      }
    }
    unit_tiles<KT>(w, P.a);
    w.k0 = 0;
    w.k1 = static_cast<int>(min(static_cast<long long>(w.n), left));
    return true;
  }
  __device__ __forceinline__ int key_of(int k) const { return (k < w.sink_tiles ? k : w.first + (k - w.sink_tiles)) * KT; }
};

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tile_kernel(const __grid_constant__ TileParams P) {
  using G = Geo<FMT, D>;
  constexpr int KT = G::KT, NU = G::NU;
  constexpr bool QUANT = FMT != LQ_FMT_F16;
  extern __shared__ unsigned char raw_smem[];
  unsigned char* const smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  unsigned char* const ring = smem + G::Q;
  Bars* const bar = reinterpret_cast<Bars*>(ring + NU * G::UNIT);
  const AttnArgs& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;

  if (tid == 0) {
    for (int u = 0; u < NU; ++u) {
      mbar_init(&bar->full[u], kLoaders);
      mbar_init(&bar->empty[u], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&bar->q_ready[q], 128);
      mbar_init(&bar->s_full[q], 2);  // the MMAs, and the issuing thread (what the loaders wrote)
      mbar_init(&bar->p_ready[q], 128);
      mbar_init(&bar->o_full[q], 2);
    }
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->join, 256);
    bar->abort = 0;
    for (int k = 0; k < kInfo; ++k)
      for (int j = 0; j < 4; ++j) bar->bad[k][j] = 0;
    fence_barrier_init();
  }
  pdl_wait();

  // ---- this CTA's range of all units' tiles -----------------------------------
  long long* const totals = reinterpret_cast<long long*>(ring);
  for (int i = warp; i < a.b.batch; i += kThreads / 32) {
    Work w;
    w.s = kv::sequence(a.b, a.c.page_size, i);
    long long sum = 0;
    if (takes(w.s, P)) {
      const int rts = (w.s.rows * a.group + kRows - 1) / kRows;
      for (w.rt = lane; w.rt < rts; w.rt += 32) {
        unit_tiles<KT>(w, a);
        sum += w.n;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) totals[i] = sum * a.c.kv_heads;
  }
  __syncthreads();
  auto scan32 = [&](long long mine) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, mine, o);
      if (lane >= o) mine += up;
    }
    return mine;
  };
  if (warp == 0) {
    long long total = 0;
    for (int i = lane; i < a.b.batch; i += 32) total += totals[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinTiles));
    long long x = per * blockIdx.x;
    if (lane == 0) bar->total = total;
    if (x < total) {
      int i = 0;
      for (int base = 0;; base += 32) {
        const long long mine = base + lane < a.b.batch ? totals[base + lane] : 0, incl = scan32(mine);
        const unsigned past = __ballot_sync(0xffffffffu, x < incl);
        if (past) {
          const int at = __ffs(static_cast<int>(past)) - 1;
          i = base + at;
          x -= __shfl_sync(0xffffffffu, incl - mine, at);
          break;
        }
        x -= __shfl_sync(0xffffffffu, incl, 31);
      }
      const long long head = totals[i] / a.c.kv_heads;
      const int h = static_cast<int>(x / head);
      x -= h * head;
      Work w;
      w.s = kv::sequence(a.b, a.c.page_size, i);
      for (int base = 0;; base += 32) {
        w.rt = base + lane;
        unit_tiles<KT>(w, a);
        const long long mine = w.rt * kRows < w.s.rows * a.group ? w.n : 0, incl = scan32(mine);
        const unsigned past = __ballot_sync(0xffffffffu, x < incl);
        if (past) {
          const int at = __ffs(static_cast<int>(past)) - 1;
          const long long k = x - __shfl_sync(0xffffffffu, incl - mine, at);
          if (lane == 0) {
            bar->start_i = i;
            bar->start_h = h;
            bar->start_rt = base + at;
            bar->start_k = static_cast<int>(k);
          }
          break;
        }
        x -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  if (warp == 12) {
    tc::tmem_alloc(&bar->tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bar->tmem;
  const long long total = bar->total;
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinTiles));
  const long long x0 = per * blockIdx.x;
  const long long mine = min(per, total - x0);  // tiles of this CTA

  auto wait = [&](uint64_t* b, uint32_t parity) {  // by whole warps
    const bool ok = __all_sync(0xffffffffu, mbar_wait(b, parity, P.wait_ns, P.wait_iters));
    if (!ok) {
      if (lane == 0) record_error(kDevErrTimeout);
      bar->abort = 1;
    }
    return ok;
  };

  if (wg < 2) {
    // ================= softmax: thread = query row =================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::REG_SOFTMAX));
    const int q = wg, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + q * 128, o_at = tmem + lanes + 256 + q * D;
    unsigned char* const q_hi = smem + q * 2 * G::QPART;
    unsigned char* const q_lo = q_hi + G::QPART;
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
    uint32_t tile = 0, tiles_q = 0, joins = 0;  // tiles done by the CTA, by this row tile
    Walk<KT> walk;
    bool on = mine > 0;
    if (on) walk.begin(P, bar, mine);
    while (on) {
      const Work& w = walk.w;
      const int rho = w.rt * kRows + q * 128 + r, rows_all = w.s.rows * a.group;
      const bool active = w.rt * kRows + q * 128 < rows_all;  // the row tile has rows
      const bool row = rho < rows_all;
      const int t = w.s.row0 + (row ? rho / a.group : 0);
      const int head = w.h * a.group + (row ? rho % a.group : 0);
      const int pos = w.s.len - w.s.rows + min(rho, rows_all - 1) / a.group;
      float om[D], M = kNoMax, l = 0.0f, f = 0.0f;
      const long long src_off = t * a.ldq + static_cast<long long>(head) * D;
      if (active) {
        // the warp's 32 query rows, one or two at a time: scaled to the top of
        // f16's range, in two parts
        constexpr int LPR = D / 4, RPI = 32 / LPR;  // lanes a row, rows at a time
        const int sub = lane / LPR, l4 = lane % LPR;
        const uint32_t live = __ballot_sync(0xffffffffu, row);
        const uint32_t col = (l4 >> 4) * G::GROUP + (l4 & 1) * 8;  // column group, half of a 16-byte chunk
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += RPI) {
          const int rr = r0 + sub;
          const float* src = a.Q + __shfl_sync(0xffffffffu, src_off, rr) + l4 * 4;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if ((live >> rr) & 1u) {
            if (P.vec_q) {
              v = ldg128f(src);
            } else {
              v = make_float4(src[0], src[1], src[2], src[3]);
            }
          }
          float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int ex = static_cast<int>(__float_as_uint(top) >> 23);
          const int es = ex == 0 || ex == 255 ? 127 : min(max(127 + 127 + 14 - ex, 1), 253);
          const float sigma = __uint_as_float(static_cast<unsigned>(es) << 23);
          const float fr = __shfl_sync(0xffffffffu, fabsf(a.scale) * kLog2e / sigma, (lane % RPI) * LPR);
          if (lane / RPI == r0 / RPI) f = fr;
          uint2 hi, lo;
          split2(v.x * (sigma * sign), v.y * (sigma * sign), hi.x, lo.x);
          split2(v.z * (sigma * sign), v.w * (sigma * sign), hi.y, lo.y);
          const uint32_t at = col + tc::sw128_offset((warp & 3) * 32 + rr, (l4 >> 1) & 7);
          *reinterpret_cast<uint2*>(q_hi + at) = hi;
          *reinterpret_cast<uint2*>(q_lo + at) = lo;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar->q_ready[q]);
#pragma unroll
        for (int d = 0; d < D; ++d) om[d] = 0.0f;
      }
      for (int k = w.k0; k < w.k1; ++k, ++tile) {
        if (!active) continue;
        const uint32_t parity = tiles_q++ & 1u;
        if (!wait(&bar->s_full[q], parity)) goto out;
        tc::fence_after_sync();
        const int2 info = bar->info[tile % kInfo];
        const int j0 = info.x;
        const uint32_t pages = static_cast<uint32_t>(info.y) & 0xFFu;
        constexpr uint32_t kAll = (1u << (KT / 16)) - 1u;
        const bool clear = pages == kAll && j0 + KT - 1 <= pos &&
                           (a.window == 0 || j0 > pos - a.window || j0 + KT <= a.sinks);
        const bool edge = __any_sync(0xffffffffu, !clear);
        auto sees = [&](int j) {  // key j of the tile
          const int key = j0 + j;
          return ((pages >> (j >> 4)) & 1u) && key <= pos && (a.window == 0 || key > pos - a.window || key < a.sinks);
        };
        // raw sums of keys j .. j + 15: asked for, and (after wait_ld) put together
        auto ask = [&](int j, uint32_t (&s)[16], uint32_t (&s2)[16]) {
          tmem_ld16(s_at + j, s);
          if constexpr (QUANT) tmem_ld16(s_at + 64 + j, s2);
        };
        auto sum = [&](uint32_t (&s)[16], uint32_t (&s2)[16]) {
          if constexpr (QUANT) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 x = fadd2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                     make_float2(__uint_as_float(s2[i]), __uint_as_float(s2[i + 1])));
              s[i] = __float_as_uint(x.x);
              s[i + 1] = __float_as_uint(x.y);
            }
          }
        };
        uint32_t sa[16], sb[16], sa2[16], sb2[16];  // two chunks in turn
        float top = -INFINITY;
        auto largest = [&](int j, uint32_t (&s)[16], uint32_t (&s2)[16], bool masked) {
          sum(s, s2);
          if (!masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, __uint_as_float(s[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sees(j + i) ? __uint_as_float(s[i]) * f : -INFINITY);
          }
        };
        if (!edge) {
          ask(0, sa, sa2);
#pragma unroll
          for (int j = 0; j < KT; j += 32) {
            tc::wait_ld();
            ask(j + 16, sb, sb2);
            largest(j, sa, sa2, false);
            tc::wait_ld();
            if (j + 32 < KT) ask(j + 32, sa, sa2);
            largest(j + 16, sb, sb2, false);
          }
          top *= f;
        } else {
#pragma unroll 1
          for (int j = 0; j < KT; j += 16) {
            ask(j, sa, sa2);
            tc::wait_ld();
            largest(j, sa, sa2, true);
          }
        }
        float keep = 1.0f;
        if (top > M + 15.0f) {
          const float to = fmaxf(M, top - kLift);
          keep = ex2(M - to);
          M = to;
          l *= keep;
        }
        // weights, in two parts, over the logits: 16 columns a 16 keys
        const float2 ff = make_float2(f, f), mm = make_float2(-M, -M);
        float2 l2 = make_float2(0.0f, 0.0f);
        auto weights = [&](int j, uint32_t (&s)[16], uint32_t (&s2)[16], bool masked) {
          sum(s, s2);
          uint32_t w16[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), ff, mm);
            float2 p = make_float2(ex2(x.x), ex2(x.y));
            if (masked) {
              p.x = sees(j + i) ? p.x : 0.0f;
              p.y = sees(j + i + 1) ? p.y : 0.0f;
            }
            l2 = fadd2(l2, p);
            const __half2 h = __floats2half2_rn(p.x, p.y);
            const float2 hf = __half22float2(h);
            const float2 r2 = fadd2(p, make_float2(-hf.x, -hf.y));
            w16[i / 2] = h2(h);
            w16[8 + i / 2] = h2(__floats2half2_rn(r2.x, r2.y));
          }
          tmem_st16(s_at + j, w16);
        };
        if (!edge) {
          ask(0, sa, sa2);
#pragma unroll
          for (int j = 0; j < KT; j += 32) {
            tc::wait_ld();
            ask(j + 16, sb, sb2);
            weights(j, sa, sa2, false);
            tc::wait_ld();
            if (j + 32 < KT) ask(j + 32, sa, sa2);
            weights(j + 16, sb, sb2, false);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < KT; j += 16) {
            ask(j, sa, sa2);
            tc::wait_ld();
            weights(j, sa, sa2, true);
          }
        }
        l += l2.x + l2.y;
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bar->p_ready[q]);
        if (!wait(&bar->o_full[q], parity)) goto out;
        tc::fence_after_sync();
        {
          const float2 kk = make_float2(keep, keep);
          auto add = [&](int d, const uint32_t (&o)[16]) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 x = ffma2(make_float2(om[d + i], om[d + i + 1]), kk, make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])));
              om[d + i] = x.x;
              om[d + i + 1] = x.y;
            }
          };
          tmem_ld16(o_at, sa);
#pragma unroll
          for (int d = 0; d < D; d += 32) {
            tc::wait_ld();
            tmem_ld16(o_at + d + 16, sb);
            add(d, sa);
            tc::wait_ld();
            if (d + 32 < D) tmem_ld16(o_at + d + 32, sa);
            add(d + 16, sb);
          }
        }
        tc::fence_before_sync();
        // values that are not finite reach the rows that see them here
        for (int word = 0; word < KT / 32; ++word) {
          uint32_t bits = bar->bad[tile % kInfo][word];
          while (bits) {
            const int j = word * 32 + __ffs(static_cast<int>(bits)) - 1;
            bits &= bits - 1;
            if (!row || !sees(j)) continue;
            const int page = kv::page_of(a.c, a.b, w.i, j0 + j);
            if (page < 0) continue;
            const int slot = (j0 + j) % a.c.page_size;
            const unsigned char* at = a.c.v + page * a.c.page_bytes + w.h * a.c.head_bytes;
            const __half* h16 = QUANT ? reinterpret_cast<const __half*>(at + static_cast<long long>(a.c.page_size) * G::ROW) + slot * (D / 32)
                                      : reinterpret_cast<const __half*>(at) + static_cast<long long>(slot) * D;
#pragma unroll
            for (int d = 0; d < D; ++d) {
              const float v = __half2float(h16[QUANT ? d / 32 : d]);
              if (!(fabsf(v) <= 65504.0f)) om[d] += QUANT ? v - v : v;  // a block's scale: NaN
            }
          }
        }
      }
      {
        // ---- the unit's result, or its part -------------------------------------
        // rows go out through the query rows' shared memory (their MMAs are done; a
        // warp's rows of all parts are its own): whole rows, 16 bytes a lane
        auto write_rows = [&]() {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // 0: the row sees nothing; NaN stays
          __syncwarp();
#pragma unroll
          for (int d = 0; d < D; d += 4)
            *reinterpret_cast<float4*>(q_hi + (d / 32) * G::GROUP + tc::sw128_offset(r, (d / 4) & 7)) =
                make_float4(om[d] * inv, om[d + 1] * inv, om[d + 2] * inv, om[d + 3] * inv);
          __syncwarp();
          constexpr int LPR = D / 4, RPI = 32 / LPR;
          const int sub = lane / LPR, l4 = lane % LPR;
          const uint32_t live = __ballot_sync(0xffffffffu, row && LQ_IN_BOUNDS(t < a.b.tokens && head < a.heads));
          const long long off = t * a.ldo + static_cast<long long>(head) * D;
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += RPI) {
            const int rr = r0 + sub;
            float* out = a.O + __shfl_sync(0xffffffffu, off, rr) + l4 * 4;
            const float4 v =
                *reinterpret_cast<const float4*>(q_hi + (l4 >> 3) * G::GROUP + tc::sw128_offset((warp & 3) * 32 + rr, l4 & 7));
            if ((live >> rr) & 1u) {
              if (P.vec_o) {
                *reinterpret_cast<float4*>(out) = v;
              } else {
                out[0] = v.x;
                out[1] = v.y;
                out[2] = v.z;
                out[3] = v.w;
              }
            }
          }
          if (row && a.lse) a.lse[static_cast<long long>(t) * a.heads + head] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
        };
        const bool whole = w.k0 == 0 && w.k1 == w.n;
        if (whole) {
          if (active) write_rows();
        } else {
          // the unit's CTAs are c0 .. c1; c0's slot 2 c0 + 1, the others' 2 c
          const long long unit_x = x0 + (mine - walk.left) - w.k0;
          const int c0 = static_cast<int>(unit_x / per), c1 = static_cast<int>((unit_x + w.n - 1) / per);
          const int rr = q * 128 + r;
          auto slot_of = [&](int c) { return P.parts + static_cast<long long>(c == c0 ? 2 * c0 + 1 : 2 * c) * G::SLOT; };
          if (row) {
            float* to = slot_of(static_cast<int>(blockIdx.x));
#pragma unroll
            for (int d = 0; d < D; d += 4)
              reinterpret_cast<float4*>(to)[(d / 4) * kRows + rr] = make_float4(om[d], om[d + 1], om[d + 2], om[d + 3]);
            to[D * kRows + rr] = M;
            to[(D + 1) * kRows + rr] = l;
          }
          __threadfence();
          mbar_arrive(&bar->join);
          if (!wait(&bar->join, joins++ & 1u)) goto out;
          if (tid == 0) {
            const int before = atomicAdd(P.counters + c0, 1);
            bar->last = before == c1 - c0;
            if (before == c1 - c0) P.counters[c0] = 0;
          }
          mbar_arrive(&bar->join);
          if (!wait(&bar->join, joins++ & 1u)) goto out;
          if (bar->last && active) {
            __threadfence();
            M = kNoMax;
            for (int c = c0; row && c <= c1; ++c) M = fmaxf(M, __ldcg(slot_of(c) + D * kRows + rr));
            l = 0.0f;
#pragma unroll
            for (int d = 0; d < D; ++d) om[d] = 0.0f;
            for (int c = c0; row && c <= c1; ++c) {
              const float* from = slot_of(c);
              const float scale = ex2(__ldcg(from + D * kRows + rr) - M);
              l = fmaf(scale, __ldcg(from + (D + 1) * kRows + rr), l);
#pragma unroll
              for (int d = 0; d < D; d += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(from) + (d / 4) * kRows + rr);
                om[d] = fmaf(scale, v.x, om[d]);
                om[d + 1] = fmaf(scale, v.y, om[d + 1]);
                om[d + 2] = fmaf(scale, v.z, om[d + 2]);
                om[d + 3] = fmaf(scale, v.w, om[d + 3]);
              }
            }
            write_rows();
          }
        }
      }
      on = walk.next(P);
    }
  out:;
  } else if (wg == 2) {
    // ================= loader ========================================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::REG_LOAD));
    const int tl = tid & 127;
    uint32_t unit = 0, tile = 0;
    uint32_t pending = 0;  // f16: units issued whose copies are not yet reported
    bool alive = true;
    Walk<KT> walk;
    bool on = mine > 0;
    if (on) walk.begin(P, bar, mine);

    // the values of a unit's chunks that this thread copied: those that are not
    // finite are taken out and their keys noted
    auto screen = [&](uint32_t at_unit, uint32_t tile_no) {
      constexpr int CH = D / 8, PASS = kLoaders / CH, N = KT / PASS;
      const int row0 = tl / CH, ch = tl % CH;
#pragma unroll 1
      for (int n = 0; n < N; ++n) {
        const int row = row0 + n * PASS;
        unsigned char* at = ring + at_unit + (ch >> 3) * G::GROUP + tc::sw128_offset(row, ch & 7);
        uint4 v = *reinterpret_cast<uint4*>(at);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((w[j] & 0x7C00u) == 0x7C00u) {
            w[j] &= 0xFFFF0000u;
            bad = true;
          }
          if ((w[j] & 0x7C000000u) == 0x7C000000u) {
            w[j] &= 0xFFFFu;
            bad = true;
          }
        }
        if (bad) {
          *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
          atomicOr(&bar->bad[tile_no % kInfo][row >> 5], 1u << (row & 31));
        }
      }
    };
    uint32_t pend_unit = 0, pend_tile = 0;
    bool pend_screen = false;
    auto report = [&]() {  // f16: the oldest pending unit has landed
      if (pend_screen) screen((pend_unit % NU) * G::UNIT, pend_tile);
      fence_proxy_async_smem();
      mbar_arrive(&bar->full[pend_unit % NU]);
      pending = 0;
    };

    while (on && alive) {
      const Work& w = walk.w;
      const kv::Visible v0 = kv::visible(max(w.p0, 0), a.window, a.sinks);
      auto group_at = [&](int j) -> long long {
        const int key = j + lane * 16;
        const int page = lane < KT / 16 ? kv::page_of(a.c, a.b, w.i, key) : -1;
        return page < 0 ? -1 : page * a.c.page_bytes + w.h * a.c.head_bytes + static_cast<long long>(key % a.c.page_size) * G::ROW;
      };
      long long ahead = -1;
      for (int k = w.k0; k < w.k1 && alive; ++k, ++tile) {
        const int j0 = walk.key_of(k);
        // the tile's groups of 16 keys, one lane each: where their rows begin (-1: nowhere)
        const long long base = k == w.k0 ? group_at(j0) : ahead;
        if (k + 1 < w.k1) ahead = group_at(walk.key_of(k + 1));
        const uint32_t pages = __ballot_sync(0xffffffffu, base >= 0);
        const bool mixed = w.s.rows > 1 && !(j0 + KT - 1 <= w.p0 && (a.window == 0 || j0 > w.p1 - a.window || j0 + KT <= a.sinks));
        if (tl == 0) {
          bar->info[tile % kInfo] = make_int2(
              j0, static_cast<int>(pages | (w.rt * kRows + 128 < w.s.rows * a.group ? kTwo : 0u) | (k == w.k0 ? kFirst : 0u)));
          for (int j = 0; j < 4; ++j) bar->bad[(tile + kInfo / 2) % kInfo][j] = 0;
        }
        const bool all = pages == (1u << (KT / 16)) - 1u && j0 + KT - 1 <= w.p1 && (j0 >= v0.begin || j0 + KT <= v0.sink_end);
        auto some_row_sees = [&](int key) { return all || (key <= w.p1 && (key >= v0.begin || key < v0.sink_end)); };
        if constexpr (!QUANT) {
          constexpr int CH = D / 8, PASS = kLoaders / CH, N = KT / PASS;  // chunks a row, rows a pass, passes
          const int row0 = tl / CH, ch = tl % CH;
          for (int side = 0; side < 2; ++side, ++unit) {
            uint64_t* const e = &bar->empty[unit % NU];
            const uint32_t parity = ((unit / NU) & 1u) ^ 1u;
            if (pending && !__all_sync(0xffffffffu, mbar_test_wait(e, parity))) {  // about to wait: report what landed
              wait_copies<0>();
              report();
            }
            if (!wait(e, parity)) {
              alive = false;
              break;
            }
            const unsigned char* pool = side ? a.c.v : a.c.k;
            const uint32_t dst = smem_u32(ring) + (unit % NU) * G::UNIT + (ch >> 3) * G::GROUP + tc::sw128_offset(row0, ch & 7);
            const unsigned char* const src = pool + row0 * G::ROW + ch * 16;
#pragma unroll 4
            for (int n = 0; n < N; ++n) {  // rows row0 + n PASS: the same place in a swizzle atom, one group of 16 a pass
              const long long at = __shfl_sync(0xffffffffu, base, n * PASS / 16);
              const bool there = at >= 0 && some_row_sees(j0 + row0 + n * PASS);
              copy16(dst + n * PASS * 128, src + max(at, 0ll) + (n * PASS % 16) * G::ROW, there);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (pending) {
              wait_copies<1>();
              report();
            }
            pending = 1;
            pend_unit = unit;
            pend_tile = tile;
            pend_screen = side == 1 && mixed;
          }
        } else {
          // 16 codes a chunk: Q8_0 16 bytes (elements 16 c ..), Q4_0 8 bytes of a
          // block (elements 8 (c & 1) .. of both its halves)
          constexpr int CH = D / 16, PASS = kLoaders / CH, N = KT / PASS;
          const int row0 = tl / CH, ch = tl % CH;
          uint4 raw[2][N];
          __half sc[2][N];
#pragma unroll
          for (int n = 0; n < N; ++n) {  // PASS = 16 or 32 rows a pass
            const int row = row0 + n * PASS;
            const long long at = __shfl_sync(0xffffffffu, base, row >> 4);
            const bool there = at >= 0 && some_row_sees(j0 + row);
            // the scales lie after the page's codes: slot * D / 32 of them in
            const long long slot = (j0 + (row & ~15)) % a.c.page_size;
            const long long sat = at - slot * G::ROW + static_cast<long long>(a.c.page_size) * G::ROW + (slot + (row & 15)) * (D / 16) + (ch >> 1) * 2;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
              raw[side][n] = make_uint4(0u, 0u, 0u, 0u);
              sc[side][n] = __ushort_as_half(0);
              const unsigned char* pool = side ? a.c.v : a.c.k;
              if (there) {
                if constexpr (FMT == LQ_FMT_Q8_0) {
                  raw[side][n] = *reinterpret_cast<const uint4*>(pool + at + (row & 15) * G::ROW + ch * 16);
                } else {
                  const uint2 x = *reinterpret_cast<const uint2*>(pool + at + (row & 15) * G::ROW + ch * 8);
                  raw[side][n].x = x.x;
                  raw[side][n].y = x.y;
                }
                sc[side][n] = *reinterpret_cast<const __half*>(pool + sat);
              }
            }
          }
          for (int side = 0; side < 2; ++side, ++unit) {
            if (!wait(&bar->empty[unit % NU], ((unit / NU) & 1u) ^ 1u)) {
              alive = false;
              break;
            }
            unsigned char* const dst = ring + (unit % NU) * G::UNIT;
#pragma unroll
            for (int n = 0; n < N; ++n) {
              const int row = row0 + n * PASS;
              __half d = side ? sc[1][n] : sc[0][n];
              if (side == 1 && mixed && !(fabsf(__half2float(d)) <= 65504.0f)) {
                d = __ushort_as_half(0);
                atomicOr(&bar->bad[tile % kInfo][row >> 5], 1u << (row & 31));
              }
              const uint4 x = side ? raw[1][n] : raw[0][n];
              const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
              uint32_t hi[8], lo[8];
              if constexpr (FMT == LQ_FMT_Q8_0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) codes8(w4[i], hi[2 * i], hi[2 * i + 1]);
              } else {  // pairs (0, 1), (2, 3), ... of the low nibbles, then of the high ones
#pragma unroll
                for (int i = 0; i < 2; ++i) codes4(w4[i], hi[2 * i], hi[2 * i + 1], hi[4 + 2 * i], hi[4 + 2 * i + 1]);
              }
              const __half2 d2 = __half2half2(d);
              if (!(fabsf(__half2float(d)) >= (FMT == LQ_FMT_Q8_0 ? 515.5f : 8188.0f))) {
                // code * d in f16, and what it leaves: exact by the fused multiply-add
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const __half2 c2 = as_h2(hi[i]), prod = __hmul2_rn(c2, d2);
                  hi[i] = h2(prod);
                  lo[i] = h2(__hfma2(c2, d2, __hneg2(prod)));
                }
              } else {  // the top of f16's range: rounded toward zero, through f32
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float2 c2 = __half22float2(as_h2(hi[i]));
                  const float df = __half2float(d);
                  split2_rz(c2.x * df, c2.y * df, hi[i], lo[i]);
                }
              }
              // 16-byte chunks of the row: the second column group's threads start with their second
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const int part = s ^ ((ch >> 2) & 1);
                const int c16 = FMT == LQ_FMT_Q8_0 ? 2 * ch + part : (ch >> 1) * 4 + (ch & 1) + 2 * part;
                const uint32_t at = (c16 >> 3) * G::GROUP;
                const uint4 vh = part ? make_uint4(hi[4], hi[5], hi[6], hi[7]) : make_uint4(hi[0], hi[1], hi[2], hi[3]);
                const uint4 vl = part ? make_uint4(lo[4], lo[5], lo[6], lo[7]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
                *reinterpret_cast<uint4*>(dst + at + tc::sw128_offset(row, c16 & 7)) = vh;
                *reinterpret_cast<uint4*>(dst + at + tc::sw128_offset(64 + row, c16 & 7)) = vl;
              }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar->full[unit % NU]);
          }
        }
      }
      if (alive) on = walk.next(P);
    }
    wait_copies<0>();
    if (pending) report();
  } else {
    // ================= MMA issue =======================================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::REG_MMA));
    if (warp == 12) {
      constexpr uint32_t kQK = tc::idesc_f16_f32(128, 128);
      constexpr uint32_t kPV = tc::idesc_f16_f32(128, D) | (1u << 16);  // B is MN-major
      const uint32_t q_at = smem_u32(smem), ring_at = smem_u32(ring);
      uint32_t seen[2] = {0, 0}, units[2] = {0, 0};  // tiles, units of a row tile
      bool alive = true;
      auto at_unit = [&](uint32_t u) { return ring_at + (u % NU) * G::UNIT; };
      // S = Q K^T of row tile q with the keys of ring unit u
      auto qk = [&](int q, uint32_t u, bool first) {
        if (first) alive = wait(&bar->q_ready[q], (q ? units[1]++ : units[0]++) & 1u);
        if (!alive) return;
        tc::fence_after_sync();
        if (elect_one()) {
          const uint64_t b0 = tc::desc_sw128_kmajor(at_unit(u));
          const uint64_t a0 = tc::desc_sw128_kmajor(q_at + q * 2 * G::QPART);
#pragma unroll 1
          for (int part = 1; part >= 0; --part)  // low parts first
#pragma unroll 4
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t off = (c >> 2) * G::GROUP + (c & 3) * 32;
              tc::mma_bf16(tmem + q * 128, a0 + ((part * G::QPART + off) >> 4), b0 + (off >> 4), kQK, part == 1 && c == 0 ? 0u : 1u);
            }
          tc::commit(&bar->s_full[q]);
          mbar_arrive(&bar->s_full[q]);
        }
        __syncwarp();
      };
      // O = P V of row tile q with the values of ring unit u
      auto pv = [&](int q, uint32_t u) {
        alive = wait(&bar->p_ready[q], (q ? seen[1]++ : seen[0]++) & 1u);
        if (!alive) return;
        tc::fence_after_sync();
        if (elect_one()) {
          const uint64_t b0 = desc_mn(at_unit(u));
          const uint32_t p = tmem + q * 128, o = tmem + 256 + q * D;
          constexpr int KS = KT / 16;
#pragma unroll 4
          for (int c = 0; c < KS; ++c)  // p_lo v_hi
            tc::mma_f16_ts(o, p + 16 * c + 8, b0 + c * 128, kPV, c == 0 ? 0u : 1u);
          if constexpr (QUANT) {
#pragma unroll 4
            for (int c = 0; c < KS; ++c)  // p_hi v_lo
              tc::mma_f16_ts(o, p + 16 * c, b0 + (KS + c) * 128, kPV, 1u);
          }
#pragma unroll 4
          for (int c = 0; c < KS; ++c)  // p_hi v_hi
            tc::mma_f16_ts(o, p + 16 * c, b0 + c * 128, kPV, 1u);
          tc::commit(&bar->o_full[q]);
          mbar_arrive(&bar->o_full[q]);
        }
        __syncwarp();
      };
      auto filled = [&](uint32_t u) { return wait(&bar->full[u % NU], (u / NU) & 1u); };
      auto release = [&](uint32_t u) {
        if (elect_one()) tc::commit(&bar->empty[u % NU]);
        __syncwarp();
      };
      // Order: PV of a row tile, then its next QK, while the other's softmax
      // runs. MMAs of one thread run in order, so that QK may overwrite the P
      // that the PV before it reads. Between units both PVs come first: the
      // next queries are written when both row tiles are done.
      uint32_t flags = 0;
      if (mine > 0) {
        alive = filled(0);
        if (alive) {
          flags = static_cast<uint32_t>(bar->info[0].y);
          qk(0, 0, true);
          if (alive && (flags & kTwo)) qk(1, 0, true);
          if (alive) release(0);
        }
      }
#pragma unroll 1
      for (uint32_t tile = 0; tile < mine && alive; ++tile) {
        const uint32_t v = 2 * tile + 1, k = v + 1;
        const bool two = (flags & kTwo) != 0, more = tile + 1 < mine;
        alive = filled(v);
        if (alive) pv(0, v);
        if (!alive) break;
        uint32_t next = 0;
        if (more) {
          alive = filled(k);
          if (!alive) break;
          next = static_cast<uint32_t>(bar->info[(tile + 1) % kInfo].y);
          if (!(next & kFirst)) qk(0, k, false);
        }
        if (alive && two) pv(1, v);
        if (!alive) break;
        release(v);
        if (more) {
          if (next & kFirst) qk(0, k, true);
          if (alive && (next & kTwo)) qk(1, k, (next & kFirst) != 0);
          if (alive) release(k);
          flags = next;
        }
      }
      // everything issued has to be done before the tensor memory is freed
      if (elect_one()) tc::commit(&bar->drain);
      __syncwarp();
      mbar_wait(&bar->drain, 0, kDrainWaitNs);
    }
  }
  pdl_launch_dependents();
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

template <int FMT, int D>
lq_status run(const TileParams& p, int ctas, cudaStream_t stream) {
  using G = Geo<FMT, D>;
  static std::atomic<bool> ready[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return LQ_ERR_CUDA;
  if (!ready[dev].load()) {
    if (cudaFuncSetAttribute(attn_tile_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM) != cudaSuccess) {
      cudaGetLastError();
      return LQ_ERR_CUDA;
    }
    ready[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tile_kernel<FMT, D>, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_route(kAttnRouteTile);
  return cuda_status(e);
}

template <int FMT>
lq_status pick(const TileParams& p, int ctas, cudaStream_t stream) {
  return p.a.c.head_dim == 64 ? run<FMT, 64>(p, ctas, stream) : run<FMT, 128>(p, ctas, stream);
}

}  // namespace

size_t attn_tile_work_bytes(int head_dim) {
  const int ctas = std::min(std::max(device_info().sm_count, 152), kAttnMaxCtas);
  if (head_dim != 64 && head_dim != 128) return 0;
  return kAttnCounterBytes + static_cast<size_t>(ctas) * 2 * kRows * (head_dim + 2) * 4;
}

bool attn_tile_eligible(const AttnArgs& a) {
  const int d = a.c.head_dim;
  return (d == 64 || d == 128) && a.c.page_size % 16 == 0 && aligned_to(a.c.k, 16) && aligned_to(a.c.v, 16) && a.b.batch <= kMaxBatch;
}

lq_status launch_attn_tile(const AttnArgs& a, int fmt, int small_rows, void* work, cudaStream_t stream) {
  if (!attn_tile_eligible(a)) return LQ_ERR_UNSUPPORTED;
  TileParams p;
  p.a = a;
  p.counters = static_cast<int*>(work);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(work) + kAttnCounterBytes);
  p.small_rows = small_rows;
  p.vec_q = a.ldq % 4 == 0 && aligned_to(a.Q, 16);
  p.vec_o = a.ldo % 4 == 0 && aligned_to(a.O, 16);
  p.wait_ns = wait_limit_ns();
  p.wait_iters = wait_limit_iters();
  const int ctas = std::max(1, std::min(device_info().sm_count, kAttnMaxCtas));
  switch (fmt) {
    case LQ_FMT_F16: return pick<LQ_FMT_F16>(p, ctas, stream);
    case LQ_FMT_Q8_0: return pick<LQ_FMT_Q8_0>(p, ctas, stream);
    default: return pick<LQ_FMT_Q4_0>(p, ctas, stream);
  }
}

unsigned read_clear_attn_tile_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attnt_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_attnt_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq
