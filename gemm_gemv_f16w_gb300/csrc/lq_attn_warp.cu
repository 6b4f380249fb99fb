// Attention of few rows (decoding, drafted tokens) over the paged cache: the
// keys and values are streamed once, f32-accurate products on warp-level MMAs.
//
// Mathematics. A unit is (sequence, key/value head, 8 * NR query rows: the
// (token, head of the group) pairs of that head). Over tiles of 16 keys, with
// a running maximum M of the base-2 logits x and sums l, o:
//     x_j = scale log2(e) q . k_j,   p_j = 2^(x_j - M),   l += p_j,   o += p_j v_j
// M is set 11 below the maximum and moves (l and o are rescaled) only when a
// tile's maximum passes it by 15: the result is the same, the largest p is
// between 2^11 and 2^15, so that even weights of 2^-20 of the largest keep
// their bits in f16, and most tiles skip the step.
//
// f32 from f16 operands: the 16 rows of mma.m16n8k16 hold 8 query rows twice,
// rows 0..7 the high f16 part of the other operand's values and rows 8..15
// the low part (x - f16(x)), so one MMA gives both products and a thread finds
// them in its own registers. q is scaled to the top of f16's range by a power
// of two per row first, so that its low part keeps its bits. Cached codes are
// exact in f16: f16 values themselves, int8 and 4-bit codes placed in the
// mantissa of 1024 by byte-permutes and one exact packed add. Their scales d
// stay in f32: S = sum_b d_jb (q_b . code_jb) over the blocks b of 32 dims,
// and in the value product they go to the weights, P_b = p_j d_jb (in two f16
// parts; M then goes by x_j + log2 max_b |d_jb|, so that P <= 2^15 whatever
// the values' size). One M for all blocks is the choice here: the parts' last
// step is 2^-24 and the largest P at least 2^11, so that blocks whose scales
// are 2^-k of the row's largest keep 36 - k bits of their weights. Each step's
// value product starts from zero and is added to the f32 sums in registers: the
// MMA's own accumulation truncates, which over thousands of keys would show.
//
// Split. Each warp streams its own tiles by 16-byte asynchronous copies into a
// private ring (rows padded so that the fragment loads hit all banks), no
// barrier between warps until a unit ends; besides the steps in use the rings
// have 64 to 128 KB on the way to an SM (f16 128, but 64 for two row groups of
// 128 dims; quantised 90 to 108, but 68 for Q8_0 of 256 dims); a page is looked
// up 16 keys at a time, 32 tiles ahead. The tiles of all units
// are dealt in equal contiguous ranges to one CTA an SM, whatever the batch's
// lengths (a unit's start counted as tiles): a CTA whose range covers a whole
// unit writes its rows, others leave partial sums (M, l, o), and the last one
// to arrive joins them in the order of the keys.
//
// What bounds it. Every key and value is read once for all rows that share it,
// so HBM is the floor. f16: 64 sequences of 8192 positions, 8 heads of 128,
// take 342 us (6.29 TB/s, 93 % of a copy); one of 131071, 2 heads of 256, 61 us
// (4.43 TB/s: 27 tiles a warp, of whose time a fifth is start and join). Q8_0:
// the same batch with mixed lengths up to 8192 131 us (4.63 TB/s, 69 %), bound
// by issue: the MMAs' and conversions' instructions and their fixed latency, at
// the 12 warps that registers and stages allow. Q4_0 has half the bytes and the
// same work: 128 us. Four tokens of 16 sequences of up to 6000, Q4_0: 50 us. One
// token over 513 positions takes 9.6 us: launch, page lookup, one round of
// loads, the join of the warps.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lq_attn.cuh"

namespace lq {
namespace {

// The same kernels twice: this file, and with the rows' masks of lq_attn_tree
// lq_attn_warp_tree.cu, which includes it.
#ifdef LQ_ATTN_TREE
constexpr bool kTree = true;
#else
constexpr bool kTree = false;
#endif

__device__ unsigned g_attnw_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_attnw_err, 0u, code); }

constexpr int kTile = 16;            // keys of a tile: never crosses a page
// Tiles worth a CTA: fewer make more partial results to join. One f16 sequence of 1600 | 3000
// positions, 8 heads of 128: 8: 16.2 | 15.6 us, 16: 12.8 | 16.5, 32: 14.8 | 15.5.
constexpr int kMinTiles = 16;
constexpr int kJoin = 8;              // partial results that one CTA joins at once
constexpr float kNoMax = -3.402823466e38f;  // M before the first key: no finite logit is lower
constexpr float kLift = 11.0f;       // how far M stays below the maximum
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSmemMax = 232448;

struct WarpParams {
  AttnArgs a;
  int* counters;  // one per CTA; zero between calls
  float* parts;   // two slots per CTA
  int small_rows;  // sequences with more rows (tokens * group) are another kernel's; 0: all are ours
  int vec;         // O rows take 16-byte stores
};

template <int FMT, int D, int NR>
struct Geo {
  // warps: what registers and stages allow. A step of 64 sequences of up to 8192, Q8_0, heads
  // of 128: 12 warps of 168 registers 162 us, 8 warps 172, 16 warps 190 (with one tile a step);
  // Q4_0, heads of 64: 12 warps 100 us, 8 warps 108.
  static constexpr int W = FMT == LQ_FMT_F16 && D == 256 ? 4 : (FMT != LQ_FMT_F16 && D <= 128 && NR == 1 ? 12 : 8);
  // tiles a step: two where a tile's work does not cover the step's own. The same step in us
  // with two | one: Q8_0 of 64 104 | 110, Q4_0 of 64 100 | 105, f16 of 64 117 | 112, Q4_0 of 128 157 | 148
  static constexpr int TPS = FMT != LQ_FMT_F16 && D == 64 ? 2 : 1;
  static constexpr int ROW = FMT == LQ_FMT_F16 ? 2 * D : (FMT == LQ_FMT_Q8_0 ? D : D / 2);
  // pitches: the eight rows (or 4 x 32, 8 x 16 bytes) of a fragment load fall
  // into different banks
  static constexpr int KP = FMT == LQ_FMT_Q8_0 ? ROW + 32 : ROW + 16;
  static constexpr int VP = ROW + 16;
  static constexpr int SB = FMT == LQ_FMT_F16 ? 0 : kTile * (D / 32) * 2;  // scales of a tile, one side
  static constexpr int TILE = kTile * (KP + VP) + 2 * SB;
  static constexpr int HEAD = 16;  // per stage: first position and visible keys of each tile
  static constexpr int STAGE = TPS * TILE + HEAD;
  static constexpr int R = 8 * NR;
  // tiles up to which few units are better not split (8 heads of f16, 513 positions: 9.8 us,
  // split 12.5; 1100 positions: 13.4 and 12.9)
  static constexpr int WHOLE = 6 * W;
  static constexpr int QF = NR * (D / 16) * 512;           // fragments of the query rows
  // partial sums of the warps that are joined at once: half of them, two where the sums are large
  static constexpr int JOINS = NR * D <= 256 ? W / 2 : 2;
  static constexpr int MERGE = JOINS * R * (D + 2) * 4;
  static constexpr int FIXED = QF + MERGE + 2048;
  static constexpr int FIT = (kSmemMax - FIXED) / (W * STAGE);
  static constexpr int S = FIT > 6 ? 6 : FIT;
  static_assert(S >= 2 && STAGE % 16 == 0 && QF % 16 == 0 && MERGE % 16 == 0);
  static constexpr int SMEM = W * S * STAGE + FIXED;
  static constexpr int SLOT = R * (D + 2);  // floats of a partial result
  // Tiles that a unit counts for besides its own where the tiles are dealt: its start and its
  // join. With 0 | 8 | 16 | 32 | 48 | 64, us: the step of 64 sequences of up to 8192, Q8_0, heads
  // of 128, 153 | 149 | 142 | 132 | 134 | 137; of up to 4096, f16, heads of 64, 70 | 65 | 62 | 56 |
  // 56 | 57; 16 of up to 2000, Q8_0, 2 heads of 256, 23 | 18 | 17 | 17 | 19 | 19.
  static constexpr int START = D == 256 ? 16 : 32;
  static constexpr bool QREG = NR * D <= 128 && W <= 8;  // query fragments in registers
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A B: the first of a sum, without registers that hold zeros.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
// 16 bytes, or zeros where `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

// A pair as two f16 pairs, high parts and what they leave.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 r = ffma2(__half22float2(h), make_float2(-1.0f, -1.0f), x);
  hi = h2(h);
  lo = h2(__floats2half2_rn(r.x, r.y));
}
// N words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4);
  if constexpr (N == 1) {
    w[0] = lds32(at);
  } else if constexpr (N == 2) {
    const uint2 v = lds64(at);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = lds128(at);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}
// f16 number i of packed words.
template <int N>
__device__ __forceinline__ float half_at(const uint32_t (&w)[N], int i) {
  const __half2 h = as_h2(w[i >> 1]);
  return (i & 1) ? __high2float(h) : __low2float(h);
}

// Four int8 codes (a word) as two f16 pairs: (code + 128) in the mantissa of
// 1024, less 1152; both steps are exact.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t& p0, uint32_t& p1) {
  const __half2 bias = __half2half2(__ushort_as_half(0xE480));  // -1152
  w ^= 0x80808080u;
  p0 = h2(__hadd2(as_h2(__byte_perm(w, 0x64646464u, 0x4140)), bias));
  p1 = h2(__hadd2(as_h2(__byte_perm(w, 0x64646464u, 0x4342)), bias));
}
// The low (high) nibbles of bytes 0 and 2 of w, less 8, as an f16 pair: in
// the mantissa of 1024 (times 16 for the high ones).
__device__ __forceinline__ uint32_t nibbles_lo(uint32_t w) {
  return h2(__hadd2(as_h2((w & 0x000F000Fu) | 0x64006400u), __half2half2(__ushort_as_half(0xE408))));  // -1032
}
__device__ __forceinline__ uint32_t nibbles_hi(uint32_t w) {
  return h2(__hfma2(as_h2((w & 0x00F000F0u) | 0x64006400u), __half2half2(__ushort_as_half(0x2C00)),  // 1/16
                    __half2half2(__ushort_as_half(0xD480))));                                        // -72
}

// Where element e of a query row goes among the MMA fragments: the lane's
// quarter c, the MMA of its block of 32, the register pair and the half, in
// the order in which a lane reads a key's codes.
template <int FMT>
__device__ __forceinline__ void q_place(int e, int& mma, int& c, int& pair, int& half) {
  const int i = e & 31;
  if constexpr (FMT == LQ_FMT_F16) {
    mma = i >> 4;
    pair = (i >> 3) & 1;
    c = (i & 7) >> 1;
    half = i & 1;
  } else if constexpr (FMT == LQ_FMT_Q8_0) {
    c = i >> 3;
    mma = (i >> 2) & 1;
    pair = (i >> 1) & 1;
    half = i & 1;
  } else {  // low nibbles 0..15, high 16..31; a word gives bytes (0, 2), (1, 3)
    mma = i >> 4;
    c = (i & 15) >> 2;
    pair = i & 1;
    half = (i >> 1) & 1;
  }
}

// Dim of output register pair element (n-tile nt, column 2c + j) of a lane.
template <int FMT>
__device__ __forceinline__ int o_dim(int nt, int c, int j) {
  if constexpr (FMT == LQ_FMT_F16) return nt * 8 + 2 * c + j;
  const int b = nt >> 2, i = nt & 3, n = 2 * c + j;
  if constexpr (FMT == LQ_FMT_Q8_0) return b * 32 + 4 * n + i;
  return b * 32 + (i >> 1) * 16 + 2 * n + (i & 1);
}

// The keys of a unit: tiles [0, sink_tiles) and [first, first + n - sink_tiles).
struct Tiles {
  int sink_tiles, first, n;
};
__device__ __forceinline__ Tiles tiles_of(const kv::Seq& s, int window, int sinks) {
  Tiles t;
  const int p0 = s.len - s.rows;  // the first token's position
  const kv::Visible v = kv::visible(max(p0, 0), window, sinks);
  t.first = v.begin / kTile;
  t.sink_tiles = min((v.sink_end + kTile - 1) / kTile, t.first);
  t.n = max(1, t.sink_tiles + (s.len + kTile - 1) / kTile - t.first);  // one empty tile where there is no key
  return t;
}

// A CTA's piece: tiles [k0, k1) of a unit.
struct Piece {
  int i, h, rt, row_tiles;  // sequence, key/value head, row tile of row_tiles
  kv::Seq s;
  Tiles t;
  int k0, k1;
};

template <int FMT, int D, int NR>
__global__ void __launch_bounds__(Geo<FMT, D, NR>::W * 32, 1) attn_warp_kernel(const WarpParams P) {
  using G = Geo<FMT, D, NR>;
  constexpr int W = G::W, TPS = G::TPS, S = G::S, R = G::R, NB = D / 32, START = G::START;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* const merge_at = smem + W * S * G::STAGE;
  float* const merge = reinterpret_cast<float*>(merge_at);
  const uint32_t qf = smem_u32(merge_at + G::MERGE);
  unsigned char* const qf_ptr = merge_at + G::MERGE;
  float* const row_f = reinterpret_cast<float*>(qf_ptr + G::QF);  // [R] logit factor of a row
  long long* const scan = reinterpret_cast<long long*>(row_f + 16);  // [W + 4]
  float* const row_m = row_f + 128;                                   // [R] of the joined result
  float* const row_l = row_m + 16;
  int* const last_flag = reinterpret_cast<int*>(row_l + 16);

  const AttnArgs& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int group = a.group, H = a.c.kv_heads, page_size = a.c.page_size;
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end

  // ---- this CTA's share of all tiles ----------------------------------------
  struct Cost {
    long long tiles;  // of a sequence, all heads and row tiles, with START more a unit
    int units, n;     // its units, and their tiles each
  };
  auto cost = [&](int i) {
    Cost c = {0, 0, 0};
    if (i >= a.b.batch) return c;
    const kv::Seq s = kv::sequence(a.b, page_size, i);
    const int rows = s.rows * group;
    if (rows == 0 || (P.small_rows && rows > P.small_rows)) return c;
    c.units = (rows + R - 1) / R * H;
    c.n = tiles_of(s, a.window, a.sinks).n;
    c.tiles = static_cast<long long>(c.units) * (c.n + START);
    return c;
  };
  // inclusive sums over the block's threads, and the block's total in scan[W]
  auto block_scan = [&](long long mine, long long& all) {
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();  // scan[] is free
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w == warp) incl += all;
      all += scan[w];
    }
    return incl;
  };
  const Cost first = cost(tid);
  long long total, units;
  const long long first_incl = block_scan(first.tiles, total), unit_incl = block_scan(first.units, units);
  const long long first_all = total;
  const bool one_pass = a.b.batch <= W * 32;  // every sequence has a thread
  const bool short_units = !__syncthreads_or(first.n > G::WHOLE);
#pragma unroll 1
  for (int base = W * 32; base < a.b.batch; base += W * 32) {
    long long all;
    block_scan(cost(base + tid).tiles, all);
    total += all;
  }
  // Few short units: a CTA takes one whole unit (joining parts costs more than
  // the tiles: one f16 sequence of 513 positions, 8 heads, 9.7 us against 12.9
  // in parts of 16 tiles). Otherwise all tiles in equal ranges.
  const bool whole_units = one_pass && short_units && units <= gridDim.x;
  long long per = max(kv::quotient(total + gridDim.x - 1, gridDim.x), static_cast<long long>(kMinTiles));
  // One tree, whose units are all alike (several sequences' are not): where the parts of a
  // unit would be joined in two rounds, a few more than kJoin - 1 of them, ranges that make
  // one round of it, though some SMs stay idle. 7 tokens of 32 heads
  // over 8 of 128, f16 | Q8_0: over 2000 positions 13.9 | 14.7 us against 15.8 | 16.8, over 4000 16.8 |
  // 18.5 against 17.6 | 19.1; over 8000 21.7 | 24.8 against 21.2 | 23.9. Of 264 shapes of heads
  // of 64 and 128 that it applies to (3 to 24 tokens, 16 to 64 heads over 2 to 8, 1200 to 4400
  // positions, three formats) times are 0.84 to 1.03 of those without it, 0.985 in the mean;
  // heads of 256 gain nothing (180 shapes, 0.93 to 1.05, 1.00) and do without.
  constexpr int kShortTiles = 300;
  if (kTree && D < 256 && a.b.batch == 1) {
    const Cost one = cost(0);
    if (one.n <= kShortTiles && one.units * (kJoin - 1) * 10 >= static_cast<int>(gridDim.x) * 6)
      per = max(per, static_cast<long long>((one.n + START + kJoin - 2) / (kJoin - 1)));
  }
  long long x0 = per * blockIdx.x, x1 = min(x0 + per, total);
  if (whole_units) {
    if (blockIdx.x >= units) return;
    if (blockIdx.x >= unit_incl - first.units && blockIdx.x < unit_incl) {
      const long long within = (blockIdx.x - (unit_incl - first.units)) * (first.n + START);
      scan[W + 2] = first_incl - first.tiles + within;
      scan[W + 3] = first.n + START;
    }
    __syncthreads();
    x0 = scan[W + 2];
    x1 = x0 + scan[W + 3];
  }
  if (x0 >= x1) return;
  // the sequence that x0 falls into
  long long before = 0;
#pragma unroll 1
  for (int base = 0;; base += W * 32) {
    long long mine = first.tiles, all = first_all, incl = first_incl;
    if (base > 0) {
      mine = cost(base + tid).tiles;
      incl = block_scan(mine, all);
    }
    incl += before;
    const bool here = x0 < before + all;
    if (here && x0 >= incl - mine && x0 < incl) {
      scan[W] = base + tid;
      scan[W + 1] = x0 - (incl - mine);
    }
    if (here) break;
    before += all;
  }
  __syncthreads();
  Piece pc;
  auto enter = [&](int i) {  // the first sequence from i on that has work here
    for (;; ++i) {
      pc.s = kv::sequence(a.b, page_size, i);
      const int rows = pc.s.rows * group;
      if (rows != 0 && !(P.small_rows && rows > P.small_rows)) break;
    }
    pc.i = i;
    pc.row_tiles = (pc.s.rows * group + R - 1) / R;
    pc.t = tiles_of(pc.s, a.window, a.sinks);
  };
  enter(static_cast<int>(scan[W]));
  {
    const long long off = scan[W + 1], unit = kv::quotient(off, pc.t.n + START);
    const int at = static_cast<int>(off - unit * (pc.t.n + START));
    x0 += max(START - at, 0);  // the place of its first tile
    if (x0 >= x1) return;      // the start alone is here: the next CTA's
    pc.h = static_cast<int>(kv::quotient(unit, pc.row_tiles));
    pc.rt = static_cast<int>(unit - static_cast<long long>(pc.h) * pc.row_tiles);
    pc.k0 = max(at - START, 0);
    pc.k1 = static_cast<int>(min(static_cast<long long>(pc.t.n), pc.k0 + (x1 - x0)));
  }

  // ---- a warp's steps of a piece ---------------------------------------------
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * S * G::STAGE);
  unsigned char* const ring_ptr = smem + warp * S * G::STAGE;
  // 32 of the warp's tiles, lane -> (step lane / TPS, tile lane % TPS): where its
  // codes and scales begin, its first key and the keys that some row sees
  long long code_at = 0, scale_at = 0;
  int first_key = 0;
  uint32_t seen = 0;
  constexpr int IDS = 32 / TPS;
  auto look_up = [&](int m) {  // the warp's steps m .. m + IDS - 1
    const int k = pc.k0 + (warp + W * (m + lane / TPS)) * TPS + lane % TPS;
    first_key = (k < pc.t.sink_tiles ? k : pc.t.first + (k - pc.t.sink_tiles)) * kTile;
    const int page = k < pc.k1 ? kv::page_of(a.c, a.b, pc.i, first_key) : -1;
    const int slot = first_key % page_size;
    const long long head = max(page, 0) * a.c.page_bytes + pc.h * a.c.head_bytes;
    code_at = head + static_cast<long long>(slot) * G::ROW;
    scale_at = head + static_cast<long long>(page_size) * G::ROW + slot * (NB * 2);
    const int p0 = pc.s.len - pc.s.rows, j0 = first_key;
    const kv::Visible v = kv::visible(max(p0, 0), a.window, a.sinks);
    uint32_t mask = 0xFFFFu;
    if (pc.s.len - j0 < kTile) mask = pc.s.len > j0 ? (1u << (pc.s.len - j0)) - 1u : 0u;
    if (j0 < v.begin) {  // keys before the first row's window: sinks only
      const uint32_t in = v.begin - j0 >= kTile ? 0u : ~((1u << (v.begin - j0)) - 1u);
      const uint32_t sink = v.sink_end - j0 >= kTile ? 0xFFFFu : (v.sink_end > j0 ? (1u << (v.sink_end - j0)) - 1u : 0u);
      mask &= in | sink;
    }
    seen = page >= 0 && LQ_IN_BOUNDS(page < a.c.num_pages && slot + kTile <= page_size && pc.h < H) ? mask : 0u;
  };
  constexpr int CH = G::ROW / 16;     // 16-byte chunks of a row
  constexpr int CN = kTile * CH / 32; // chunks a lane
  static_assert(CN >= 1);
  const int row0 = lane / CH, col0 = lane % CH;  // the lane's first chunk; the others are 32 / CH rows on
  auto load = [&](int m) {  // the copies of step m (a group even if empty)
    if (m % IDS == 0) look_up(m);
    if (pc.k0 + (warp + W * m) * TPS < pc.k1) {
      const uint32_t stage = ring + static_cast<uint32_t>(m % S) * G::STAGE;
#pragma unroll
      for (int t = 0; t < TPS; ++t) {
        const int from = (m % IDS) * TPS + t;
        const long long at = __shfl_sync(0xffffffffu, code_at, from);
        const uint32_t mask = __shfl_sync(0xffffffffu, seen, from);
        const int j0 = __shfl_sync(0xffffffffu, first_key, from);
        const uint32_t dst = stage + G::HEAD + t * G::TILE;
        const uint32_t kd = dst + row0 * G::KP + col0 * 16, vd = dst + kTile * G::KP + row0 * G::VP + col0 * 16;
        const unsigned char* ks = a.c.k + at + lane * 16;
        const unsigned char* vs = a.c.v + at + lane * 16;
        if (mask == 0xFFFFu) {
#pragma unroll
          for (int n = 0; n < CN; ++n) {
            cp_async16(kd + n * (32 / CH) * G::KP, ks + n * 512);
            cp_async16(vd + n * (32 / CH) * G::VP, vs + n * 512);
          }
        } else {
#pragma unroll
          for (int n = 0; n < CN; ++n) {
            const bool there = (mask >> (row0 + n * (32 / CH))) & 1u;
            copy16(kd + n * (32 / CH) * G::KP, ks + n * 512, there);
            copy16(vd + n * (32 / CH) * G::VP, vs + n * 512, there);
          }
        }
        if constexpr (FMT != LQ_FMT_F16) {
          const long long sat = __shfl_sync(0xffffffffu, scale_at, from);
          constexpr int SC = G::SB / 16;  // chunks of a side's scales
          const int side = lane / SC;
          if (side < 2)
            copy16(dst + kTile * (G::KP + G::VP) + side * G::SB + (lane % SC) * 16,
                   (side ? a.c.v : a.c.k) + sat + (lane % SC) * 16, mask != 0u);
        }
        if (lane == 0)
          *reinterpret_cast<int2*>(ring_ptr + (m % S) * G::STAGE + t * 8) = make_int2(j0, static_cast<int>(mask));
      }
    }
    commit_copies();
  };

#pragma unroll
  for (int m = 0; m < S - 1; ++m) load(m);

  const float qscale = a.scale * kLog2e;
  // the unit's query rows: asked for early, and stored as MMA fragments in
  // shared memory (two parts, scaled to the top of f16's range) once it is free
  constexpr int RPW = (R + W - 1) / W;  // rows a warp
  float qv[RPW][NB];
  auto ask_queries = [&]() {
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int rho = pc.rt * R + warp + i * W;
      const bool there = warp + i * W < R && rho < pc.s.rows * group;
      const int token = there ? rho / group : 0;
      const float* src = a.Q + (pc.s.row0 + token) * a.ldq + static_cast<long long>(pc.h * group + (there ? rho - token * group : 0)) * D;
#pragma unroll
      for (int b = 0; b < NB; ++b) qv[i][b] = there ? src[b * 32 + lane] : 0.0f;
    }
  };
  auto store_queries = [&]() {
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * W;
      if (r >= R) break;
      float top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) top = fmaxf(top, fabsf(qv[i][b]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // sigma: a power of two that takes the largest |q| to [2^14, 2^15)
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int es = ex == 0 || ex == 255 ? 127 : min(max(127 + 127 + 14 - ex, 1), 253);
      const float sigma = __uint_as_float(static_cast<unsigned>(es) << 23);
      if (lane == 0) row_f[r] = qscale / sigma;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float x = qv[i][b] * sigma;
        const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
        int mma, cc, pair, half;
        q_place<FMT>(lane, mma, cc, pair, half);
        unsigned char* at = qf_ptr + (((r >> 3) * NB + b) * 2 + mma) * 512 + ((r & 7) * 4 + cc) * 16 + pair * 8 + half * 2;
        *reinterpret_cast<__half*>(at) = hi;
        *reinterpret_cast<__half*>(at + 4) = lo;
      }
    }
  };
  ask_queries();
  for (;;) {
    store_queries();
    const int rho0 = pc.rt * R, rows_all = pc.s.rows * group;
    __syncthreads();
    uint32_t qr[G::QREG ? NR * NB * 2 : 1][4];
    if constexpr (G::QREG) {
#pragma unroll
      for (int i = 0; i < NR * NB * 2; ++i) {
        const uint4 v = lds128(qf + i * 512 + lane * 16);
        qr[i][0] = v.x;
        qr[i][1] = v.y;
        qr[i][2] = v.z;
        qr[i][3] = v.w;
      }
    }
    float f[NR], M[NR];
    float2 l[NR], om[NR][D / 8];
    int pos[NR], row_t[kTree ? NR : 1];  // a tree's rows: the row of the call
    const int tree_base = pc.s.len - pc.s.rows;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      f[n] = row_f[n * 8 + g];
      M[n] = kNoMax;
      l[n] = make_float2(0.0f, 0.0f);
      pos[n] = pc.s.len - pc.s.rows + min(rho0 + n * 8 + g, rows_all - 1) / group;
      if constexpr (kTree) {
        row_t[n] = pc.s.row0 + pos[n] - tree_base;
        pos[n] = tree::position(a, row_t[n], tree_base, pc.s.len);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) om[n][i] = make_float2(0.0f, 0.0f);
    }
    // (a tree: keys before the new tokens, and the largest position there can be)
    const int p_first = kTree ? tree_base - 1 : pc.s.len - pc.s.rows + rho0 / group;
    const int p_last = kTree ? pc.s.len - 1 : pc.s.len - pc.s.rows + min(rho0 + R - 1, rows_all - 1) / group;

    const int steps = (pc.k1 - pc.k0 + TPS - 1) / TPS;
    int m = 0;
    for (int st = warp; st < steps; st += W, ++m) {
      wait_copies<S - 2>();
      __syncwarp();
      const uint32_t stage = ring + static_cast<uint32_t>(m % S) * G::STAGE;
      const uint32_t t0 = stage + G::HEAD;
      int j0[TPS];
      bool edge = false, mixed = false;
      uint32_t any[TPS];
#pragma unroll
      for (int t = 0; t < TPS; ++t) {
        const uint2 hd = lds64(stage + t * 8);
        j0[t] = static_cast<int>(hd.x);
        any[t] = hd.y;
        const bool clear = j0[t] + kTile - 1 <= p_first &&
                           (a.window == 0 || j0[t] > p_last - a.window || j0[t] + kTile <= a.sinks);
        edge = edge || any[t] != 0xFFFFu || !clear;
        mixed = mixed || (!clear && (kTree || pc.s.rows > 1));
      }
      // ---- logits ---------------------------------------------------------------
      constexpr int NT = TPS * 2;  // n-tiles of 8 keys
      constexpr bool MANY = NR * D > 256;
      float2 x[NR][NT];
      auto query = [&](int n, int i, uint32_t (&q4)[4]) {  // MMA i of a row tile's query
        if constexpr (G::QREG) {
#pragma unroll
          for (int j = 0; j < 4; ++j) q4[j] = qr[n * NB * 2 + i][j];
        } else {
          const uint4 v = lds128(qf + (n * NB * 2 + i) * 512 + lane * 16);
          q4[0] = v.x;
          q4[1] = v.y;
          q4[2] = v.z;
          q4[3] = v.w;
        }
      };
      if constexpr (FMT == LQ_FMT_F16) {
        float acc[NR][NT][4];
        const uint32_t at = t0 + (lane & 7) * G::KP + (lane >> 3) * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t q4[NR][2][4];
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) query(n, 2 * b + h, q4[n][h]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t kf[4];
            ldmatrix4(kf, at + (nt >> 1) * G::TILE + (nt & 1) * 8 * G::KP + b * 64);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              if (b == 0) {
                mma_f16_first(acc[n][nt], q4[n][0], kf[0], kf[1]);
              } else {
                mma_f16(acc[n][nt], q4[n][0], kf[0], kf[1]);
              }
              mma_f16(acc[n][nt], q4[n][1], kf[2], kf[3]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            x[n][nt] = fmul2(fadd2(make_float2(acc[n][nt][0], acc[n][nt][1]), make_float2(acc[n][nt][2], acc[n][nt][3])), make_float2(f[n], f[n]));
      } else {
        uint32_t kd[NT][2][NB / 2];  // scales of the keys 2c, 2c + 1 of each 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            lds_words(t0 + (nt >> 1) * G::TILE + kTile * (G::KP + G::VP) + ((nt & 1) * 8 + 2 * c + j) * (NB * 2), kd[nt][j]);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) x[n][nt] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t q4[MANY ? 1 : NR][2][4], kfs[MANY ? NT : 1][4];
          if constexpr (!MANY) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h) query(n, 2 * b + h, q4[n][h]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t row = t0 + (nt >> 1) * G::TILE + ((nt & 1) * 8 + g) * G::KP;
            uint32_t kf[4];
            if constexpr (FMT == LQ_FMT_Q8_0) {
              const uint2 w = lds64(row + b * 32 + c * 8);
              codes8(w.x, kf[0], kf[1]);
              codes8(w.y, kf[2], kf[3]);
            } else {
              const uint32_t w = lds32(row + b * 16 + c * 4), w8 = w >> 8;
              kf[0] = nibbles_lo(w);
              kf[1] = nibbles_lo(w8);
              kf[2] = nibbles_hi(w);
              kf[3] = nibbles_hi(w8);
            }
            if constexpr (MANY) {
#pragma unroll
              for (int j = 0; j < 4; ++j) kfs[nt][j] = kf[j];
              continue;
            }
            const float2 d = make_float2(half_at(kd[nt][0], b), half_at(kd[nt][1], b));
#pragma unroll
            for (int n = 0; n < (MANY ? 0 : NR); ++n) {
              float acc[4];
              mma_f16_first(acc, q4[n][0], kf[0], kf[1]);
              mma_f16(acc, q4[n][1], kf[2], kf[3]);
              x[n][nt] = ffma2(d, fadd2(make_float2(acc[0], acc[1]), make_float2(acc[2], acc[3])), x[n][nt]);
            }
          }
          if constexpr (MANY) {  // (queries a row group at a time: fewer registers)
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              query(n, 2 * b, q4[0][0]);
              query(n, 2 * b + 1, q4[0][1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 d = make_float2(half_at(kd[nt][0], b), half_at(kd[nt][1], b));
                float acc[4];
                mma_f16_first(acc, q4[0][0], kfs[nt][0], kfs[nt][1]);
                mma_f16(acc, q4[0][1], kfs[nt][2], kfs[nt][3]);
                x[n][nt] = ffma2(d, fadd2(make_float2(acc[0], acc[1]), make_float2(acc[2], acc[3])), x[n][nt]);
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) x[n][nt] = fmul2(x[n][nt], make_float2(f[n], f[n]));
      }
      // ---- masks: bit 2 nt + j of vis[n] is key 8 nt + 2c + j for the lane's row --
      uint32_t vis[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) vis[n] = 0xFFFFFFFFu;
      if (edge) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          uint32_t named[TPS];  // the tile's keys among the new tokens that the row's mask names
          if constexpr (kTree) {
#pragma unroll
            for (int t = 0; t < TPS; ++t) named[t] = tree::bits(a, row_t[n], j0[t] - tree_base);
          }
#pragma unroll
          for (int nt = 0; nt < TPS * 2; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int at = (nt & 1) * 8 + 2 * c + j, key = j0[nt >> 1] + at;
              const bool in_window = a.window == 0 || key > pos[n] - a.window || key < a.sinks;
              bool see;
              if constexpr (kTree) {
                see = ((any[nt >> 1] >> at) & 1u) && (key < tree_base ? in_window : ((named[nt >> 1] >> at) & 1u) != 0u);
              } else {
                see = ((any[nt >> 1] >> at) & 1u) && key <= pos[n] && in_window;
              }
              if (!see) {
                vis[n] &= ~(1u << (2 * nt + j));
                if (j == 0) x[n][nt].x = -INFINITY; else x[n][nt].y = -INFINITY;
              }
            }
        }
      }
      // ---- values' scales: thread's keys 2c, 2c + 1 of each 8 --------------------
      uint32_t vd[FMT == LQ_FMT_F16 ? 1 : NT][2][FMT == LQ_FMT_F16 ? 1 : NB / 2];
      float2 ld[NT];  // log2 of the largest |d| of a key
      if constexpr (FMT != LQ_FMT_F16) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            lds_words(t0 + (nt >> 1) * G::TILE + kTile * (G::KP + G::VP) + G::SB + ((nt & 1) * 8 + 2 * c + j) * (NB * 2), vd[nt][j]);
            __half2 top = as_h2(vd[nt][j][0] & 0x7FFF7FFFu);
#pragma unroll
            for (int w = 1; w < NB / 2; ++w) top = __hmax2(top, as_h2(vd[nt][j][w] & 0x7FFF7FFFu));
            const float e = fmaxf(lg2(fmaxf(__low2float(top), __high2float(top))), -24.0f);
            if (j == 0) ld[nt].x = e; else ld[nt].y = e;
          }
        }
      }
      // ---- running maximum, weights ----------------------------------------------
      float2 p[NR][NT];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float top = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 y = FMT == LQ_FMT_F16 ? x[n][nt] : fadd2(x[n][nt], ld[nt]);
          top = fmaxf(top, fmaxf(y.x, y.y));
        }
        // (a difference of neighbours is exact, M + 15 need not be)
        if (__any_sync(0xffffffffu, top - M[n] > 15.0f)) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          float to = fmaxf(M[n], top - kLift);
          to = top - to > 15.0f ? top : to;  // past 2^27 the step itself is 16
          const float keep = ex2(M[n] - to);
          M[n] = to;
          l[n] = fmul2(l[n], make_float2(keep, keep));
#pragma unroll
          for (int i = 0; i < D / 8; ++i) om[n][i] = fmul2(om[n][i], make_float2(keep, keep));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 y = fadd2(x[n][nt], make_float2(-M[n], -M[n]));
          p[n][nt] = make_float2(ex2(y.x), ex2(y.y));
          l[n] = fadd2(l[n], p[n][nt]);
        }
      }
      // ---- weighted values ---------------------------------------------------------
      if constexpr (FMT == LQ_FMT_F16) {
        bool slow = false;
        if (mixed) {  // a value that is not finite may be invisible to some of the rows
          uint32_t bad = 0;
#pragma unroll 1
          for (int t = 0; t < TPS; ++t)
#pragma unroll 1
            for (int i = lane; i < kTile * D / 8; i += 32) {
              const uint4 v = lds128(t0 + t * G::TILE + kTile * G::KP + (i / (D / 8)) * G::VP + (i % (D / 8)) * 16);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int h = 0; h < 4; ++h) bad |= (w[h] & 0x7C00u) == 0x7C00u || (w[h] & 0x7C000000u) == 0x7C000000u ? 1u : 0u;
            }
          slow = __any_sync(0xffffffffu, bad != 0u);
        }
        if (!slow) {
          uint32_t pa[NR][TPS][4];
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int t = 0; t < TPS; ++t) {
              split2(p[n][2 * t], pa[n][t][0], pa[n][t][1]);
              split2(p[n][2 * t + 1], pa[n][t][2], pa[n][t][3]);
            }
          const uint32_t at = t0 + kTile * G::KP + ((lane & 7) + ((lane >> 3) & 1) * 8) * G::VP + (lane >> 4) * 16;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            float acc[NR][2][4];
#pragma unroll
            for (int t = 0; t < TPS; ++t) {
              uint32_t vf[4];
              ldmatrix4_trans(vf, at + t * G::TILE + d * 32);
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                if (t == 0) {
                  mma_f16_first(acc[n][0], pa[n][t], vf[0], vf[1]);
                  mma_f16_first(acc[n][1], pa[n][t], vf[2], vf[3]);
                } else {
                  mma_f16(acc[n][0], pa[n][t], vf[0], vf[1]);
                  mma_f16(acc[n][1], pa[n][t], vf[2], vf[3]);
                }
              }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                om[n][2 * d + h] = fadd2(om[n][2 * d + h], fadd2(make_float2(acc[n][h][0], acc[n][h][1]), make_float2(acc[n][h][2], acc[n][h][3])));
          }
        } else {  // key by key, leaving out what a row does not see
#pragma unroll
          for (int nt = 0; nt < TPS * 2; ++nt)
#pragma unroll 1
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t row = t0 + (nt >> 1) * G::TILE + kTile * G::KP + ((nt & 1) * 8 + kk) * G::VP;
              const int from = (lane & ~3) | (kk >> 1);
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                const float w0 = __shfl_sync(0xffffffffu, p[n][nt].x, from), w1 = __shfl_sync(0xffffffffu, p[n][nt].y, from);
                const uint32_t vv = __shfl_sync(0xffffffffu, vis[n], from);
                const float w = (kk & 1) ? w1 : w0;
                if ((vv >> (2 * nt + (kk & 1))) & 1u) {
#pragma unroll
                  for (int i = 0; i < D / 8; ++i) {
                    const float2 v = __half22float2(as_h2(lds32(row + i * 16 + c * 4)));
                    om[n][i] = ffma2(make_float2(w, w), v, om[n][i]);
                  }
                }
              }
            }
        }
      } else {
        auto add_values = [&](const bool masked) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float acc[MANY ? 1 : NR][4][4];
#pragma unroll
          for (int t = 0; t < TPS; ++t) {
            const uint32_t tv = t0 + t * G::TILE + kTile * G::KP;
            uint32_t pa[MANY ? 1 : NR][4];
            auto weigh = [&](int n, int u, uint32_t (&to)[4]) {  // row group n's weights times the block's scales
              const int nt = 2 * t + u;
              float2 w = fmul2(p[n][nt], make_float2(half_at(vd[nt][0], b), half_at(vd[nt][1], b)));
              if (masked) {  // the scale of a key that the row does not see may be NaN
                w.x = (vis[n] >> (2 * nt)) & 1u ? w.x : 0.0f;
                w.y = (vis[n] >> (2 * nt + 1)) & 1u ? w.y : 0.0f;
              }
              split2(w, to[2 * u], to[2 * u + 1]);
            };
            if constexpr (!MANY) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < NR; ++n) weigh(n, u, pa[n]);
            }
            uint32_t vf[4][2];  // n-tile, register
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t row = tv + (u * 8 + 2 * c) * G::VP;
              if constexpr (FMT == LQ_FMT_Q8_0) {
                const uint32_t w0 = lds32(row + b * 32 + g * 4), w1 = lds32(row + G::VP + b * 32 + g * 4);
                codes8(__byte_perm(w0, w1, 0x5140), vf[0][u], vf[1][u]);
                codes8(__byte_perm(w0, w1, 0x7362), vf[2][u], vf[3][u]);
              } else {
                const uint32_t w = __byte_perm(lds16(row + b * 16 + g * 2), lds16(row + G::VP + b * 16 + g * 2), 0x5410), w8 = w >> 8;
                vf[0][u] = nibbles_lo(w);
                vf[1][u] = nibbles_lo(w8);
                vf[2][u] = nibbles_hi(w);
                vf[3][u] = nibbles_hi(w8);
              }
            }
            if constexpr (MANY) {
              static_assert(!MANY || TPS == 1);
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                weigh(n, 0, pa[0]);
                weigh(n, 1, pa[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  mma_f16_first(acc[0][i], pa[0], vf[i][0], vf[i][1]);
                  om[n][4 * b + i] = fadd2(om[n][4 * b + i], fadd2(make_float2(acc[0][i][0], acc[0][i][1]), make_float2(acc[0][i][2], acc[0][i][3])));
                }
              }
            }
#pragma unroll
            for (int n = 0; n < (MANY ? 0 : NR); ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (t == 0) {
                  mma_f16_first(acc[n][i], pa[n], vf[i][0], vf[i][1]);
                } else {
                  mma_f16(acc[n][i], pa[n], vf[i][0], vf[i][1]);
                }
              }
          }
#pragma unroll
          for (int n = 0; n < (MANY ? 0 : NR); ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              om[n][4 * b + i] = fadd2(om[n][4 * b + i], fadd2(make_float2(acc[n][i][0], acc[n][i][1]), make_float2(acc[n][i][2], acc[n][i][3])));
        }
        };
        if (!edge) {  // (two copies: merged into one, every tile pays for the masks)
          add_values(false);
        } else {
          add_values(true);
        }
      }
      __syncwarp();  // every lane has read the slot that the next copies take
      load(m + S - 1);
    }

    // ---- the next piece's copies start before this one is joined -----------------
    const Piece done = pc;
    x0 += done.k1 - done.k0 + START;
    const bool more = x0 < x1;
    if (more) {
      pc.k0 = 0;
      if (++pc.rt == pc.row_tiles) {
        pc.rt = 0;
        if (++pc.h == H) {
          pc.h = 0;
          enter(pc.i + 1);
        }
      }
      pc.k1 = static_cast<int>(min(static_cast<long long>(pc.t.n), x1 - x0));
#pragma unroll 1
      for (int n = 0; n < S - 1; ++n) load(n);
      ask_queries();
    }

    // ---- join the warps, pairwise, half of them at a time -----------------------------------
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      l[n].x += l[n].y;
      l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, 1);
      l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, 2);
    }
#pragma unroll
    for (int n_left = W; n_left > 1; n_left = (n_left + 1) / 2) {
      const int half = (n_left + 1) / 2;
#pragma unroll
      for (int w0 = 0; w0 < n_left - half; w0 += G::JOINS) {
        if (warp >= half + w0 && warp < min(half + w0 + G::JOINS, n_left)) {
          float* at = merge + (warp - half - w0) * (R * (D + 2));
#pragma unroll
          for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(at + ((n * (D / 8) + i) * 32 + lane) * 2) = om[n][i];
            if (c == 0) {
              at[R * D + n * 8 + g] = M[n];
              at[R * D + R + n * 8 + g] = l[n].x;
            }
          }
        }
        __syncthreads();
        if (warp >= w0 && warp < min(w0 + G::JOINS, n_left - half)) {
          const float* at = merge + (warp - w0) * (R * (D + 2));
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float om2 = at[R * D + n * 8 + g], l2 = at[R * D + R + n * 8 + g];
            const float to = fmaxf(M[n], om2), f1 = ex2(M[n] - to), f2 = ex2(om2 - to);
            M[n] = to;
            l[n].x = l[n].x * f1 + l2 * f2;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const float2 o2 = *reinterpret_cast<const float2*>(at + ((n * (D / 8) + i) * 32 + lane) * 2);
              om[n][i] = ffma2(om[n][i], make_float2(f1, f1), fmul2(o2, make_float2(f2, f2)));
            }
          }
        }
        __syncthreads();
      }
    }
    // warp 0 lays the rows out: [R][D], then M and l
    if (warp == 0) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int r = n * 8 + g;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) merge[r * D + o_dim<FMT>(i, c, j)] = j == 0 ? om[n][i].x : om[n][i].y;
        if (c == 0) {
          row_m[r] = M[n];
          row_l[r] = l[n].x;
        }
      }
    }
    __syncthreads();

    const int d_rho0 = done.rt * R, d_rows = min(R, done.s.rows * group - d_rho0);
    auto row_out = [&](int r) {
      const int rho = d_rho0 + r, t = done.s.row0 + rho / group, h = done.h * group + rho % group;
      return make_int2(t, h);
    };
    auto finish = [&](int r, int d4, float4 o, float sum) {  // four dims of a row
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // 0: the row sees nothing; NaN stays
      const int2 th = row_out(r);
      float* at = a.O + th.x * a.ldo + static_cast<long long>(th.y) * D + d4 * 4;
      if (!LQ_IN_BOUNDS(th.x < a.b.tokens && th.y < a.heads)) return;
      o.x *= inv;
      o.y *= inv;
      o.z *= inv;
      o.w *= inv;
      if (P.vec) {
        *reinterpret_cast<float4*>(at) = o;
      } else {
        at[0] = o.x;
        at[1] = o.y;
        at[2] = o.z;
        at[3] = o.w;
      }
    };
    auto finish_lse = [&](int r, float top, float sum) {
      if (!a.lse) return;
      const int2 th = row_out(r);
      a.lse[static_cast<long long>(th.x) * a.heads + th.y] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };

    const bool whole = done.k0 == 0 && done.k1 == done.t.n;
    if (whole) {
      for (int e = tid; e < d_rows * (D / 4); e += W * 32) {
        const int r = e / (D / 4);
        finish(r, e % (D / 4), *reinterpret_cast<const float4*>(merge + e * 4), row_l[r]);
      }
      if (tid < d_rows) finish_lse(tid, row_m[tid], row_l[tid]);
    } else {
      // partial sums: the unit's CTAs are c0 .. c1, c0's slot 2 c0 + 1, the others' 2 c
      const long long unit_x0 = x0 - START - done.k1, unit_x1 = unit_x0 + done.t.n - 1;
      const int c0 = static_cast<int>(kv::quotient(unit_x0, per)), parts = static_cast<int>(kv::quotient(unit_x1, per)) - c0 + 1;
      auto slot_of = [&](int q) { return q == 0 ? 2 * c0 + 1 : 2 * (c0 + q); };
      auto part_at = [&](int slot) { return P.parts + static_cast<long long>(slot) * G::SLOT; };
      const int me = static_cast<int>(blockIdx.x) - c0;
      float* mine = part_at(slot_of(me));
      for (int e = tid; e < R * (D / 4); e += W * 32)
        reinterpret_cast<float4*>(mine)[e] = *reinterpret_cast<const float4*>(merge + e * 4);
      if (tid < R) {
        mine[R * D + tid] = row_m[tid];
        mine[R * D + R + tid] = row_l[tid];
      }
      // Counts this CTA in; true for the last of n, which leaves the counter at zero.
      auto last_of = [&](int* counter, int n) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int before_us = atomicAdd(counter, 1);
          *last_flag = before_us == n - 1;
          if (before_us == n - 1) *counter = 0;
        }
        __syncthreads();
        const bool last = *last_flag != 0;
        if (last) __threadfence();
        return last;
      };
      // Joins n parts, the q-th in slot_at(q), in the order of the keys: into the
      // first's slot, or (into == null) the output.
      auto combine = [&](auto&& slot_at, int n, float* into) {
        if (n <= kJoin) {  // one round of loads
          for (int e = tid; e < d_rows * (D / 4); e += W * 32) {
            const int r = e / (D / 4);
            float m[kJoin], ls[kJoin];
            float4 v[kJoin];
#pragma unroll
            for (int q = 0; q < kJoin; ++q) {
              const float* at = part_at(slot_at(min(q, n - 1)));
              m[q] = __ldcg(at + R * D + r);
              ls[q] = __ldcg(at + R * D + R + r);
              v[q] = __ldcg(reinterpret_cast<const float4*>(at) + e);
            }
            float top = m[0], sum = 0.0f;
#pragma unroll
            for (int q = 1; q < kJoin; ++q) top = fmaxf(top, m[q]);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < kJoin; ++q) {
              if (q < n) {
                const float w = ex2(m[q] - top);
                sum = fmaf(w, ls[q], sum);
                o.x = fmaf(w, v[q].x, o.x);
                o.y = fmaf(w, v[q].y, o.y);
                o.z = fmaf(w, v[q].z, o.z);
                o.w = fmaf(w, v[q].w, o.w);
              }
            }
            if (into) {
              reinterpret_cast<float4*>(into)[e] = o;
              row_m[r] = top;
              row_l[r] = sum;
            } else {
              finish(r, e % (D / 4), o, sum);
              if (e % (D / 4) == 0) finish_lse(r, top, sum);
            }
          }
          if (into) {
            __syncthreads();  // every thread has read the parts' maxima
            if (tid < R) {
              into[R * D + tid] = tid < d_rows ? row_m[tid] : kNoMax;
              into[R * D + R + tid] = tid < d_rows ? row_l[tid] : 0.0f;
            }
          }
          return;
        }
        for (int r = warp; r < R; r += W) {
          float top = kNoMax;
          for (int q = lane; q < n; q += 32) top = fmaxf(top, __ldcg(part_at(slot_at(q)) + R * D + r));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          float sum = 0.0f;
          for (int q = lane; q < n; q += 32) {
            const float w = ex2(__ldcg(part_at(slot_at(q)) + R * D + r) - top);
            sum = fmaf(w, __ldcg(part_at(slot_at(q)) + R * D + R + r), sum);
          }
          sum = warp_sum(sum);
          if (lane == 0) {
            row_m[r] = top;
            row_l[r] = sum;
          }
        }
        __syncthreads();
        for (int e = tid; e < d_rows * (D / 4); e += W * 32) {
          const int r = e / (D / 4);
          const float top = row_m[r];
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
          for (int q = 0; q < n; ++q) {
            const float* at = part_at(slot_at(q));
            const float w = ex2(__ldcg(at + R * D + r) - top);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(at) + e);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
          }
          if (into) {
            reinterpret_cast<float4*>(into)[e] = o;
          } else {
            finish(r, e % (D / 4), o, row_l[r]);
          }
        }
        if (into) {
          __syncthreads();  // every thread has read the parts' maxima
          if (tid < R) {
            into[R * D + tid] = row_m[tid];
            into[R * D + R + tid] = row_l[tid];
          }
        } else if (tid < d_rows) {
          finish_lse(tid, row_m[tid], row_l[tid]);
        }
      };
      // Up to kJoin parts are joined by the last CTA of them; more in groups of
      // kJoin first, so that no CTA reads more than a few dozen of them.
      if (parts <= kJoin) {
        if (last_of(P.counters + c0, parts)) combine(slot_of, parts, static_cast<float*>(nullptr));
      } else {
        const int g0 = me / kJoin * kJoin, groups = (parts + kJoin - 1) / kJoin;
        if (last_of(P.counters + kAttnMaxCtas + slot_of(g0), min(kJoin, parts - g0))) {
          combine([&](int q) { return slot_of(g0 + q); }, min(kJoin, parts - g0), part_at(slot_of(g0)));
          if (last_of(P.counters + c0, groups)) combine([&](int q) { return slot_of(q * kJoin); }, groups, static_cast<float*>(nullptr));
        }
      }
    }
    if (!more) return;
    __syncthreads();  // merge, row_f and the fragments are free
  }
}

template <int FMT, int D, int NR>
lq_status run(const WarpParams& p, int ctas, cudaStream_t stream) {
  using G = Geo<FMT, D, NR>;
  static std::atomic<bool> ready[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return LQ_ERR_CUDA;
  if (!ready[dev].load()) {
    if (cudaFuncSetAttribute(attn_warp_kernel<FMT, D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM) != cudaSuccess) {
      cudaGetLastError();
      return LQ_ERR_CUDA;
    }
    ready[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(G::W * 32);
  cfg.dynamicSmemBytes = G::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_warp_kernel<FMT, D, NR>, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_route(kAttnRouteWarp);
  return cuda_status(e);
}

template <int FMT>
lq_status pick(const WarpParams& p, int nr, int ctas, cudaStream_t stream) {
  switch (p.a.c.head_dim) {
    case 64: return nr == 1 ? run<FMT, 64, 1>(p, ctas, stream) : run<FMT, 64, 2>(p, ctas, stream);
    case 128: return nr == 1 ? run<FMT, 128, 1>(p, ctas, stream) : run<FMT, 128, 2>(p, ctas, stream);
    default:
#ifdef LQ_ATTN_TREE
      if constexpr (FMT != LQ_FMT_F16)
        if (nr == 2) return run<FMT, 256, 2>(p, ctas, stream);
#endif
      return run<FMT, 256, 1>(p, ctas, stream);
  }
}

}  // namespace

#ifndef LQ_ATTN_TREE
// Counters, then two slots of up to 16 rows a CTA.
size_t attn_warp_work_bytes() {
  const int ctas = std::max(device_info().sm_count, 152);
  return kAttnCounterBytes + static_cast<size_t>(ctas) * 2 * 16 * (256 + 2) * 4;
}

bool attn_warp_eligible(const AttnArgs& a) {
  const int d = a.c.head_dim;
  return (d == 64 || d == 128 || d == 256) && a.c.page_size % kTile == 0 && aligned_to(a.c.k, 16) && aligned_to(a.c.v, 16);
}

lq_status launch_attn_warp(const AttnArgs& a, int fmt, int rows, int small_rows, void* work, cudaStream_t stream) {
  if (a.mask) return launch_attn_warp_tree(a, fmt, rows, small_rows, work, stream);
#else
lq_status launch_attn_warp_tree(const AttnArgs& a, int fmt, int rows, int small_rows, void* work, cudaStream_t stream) {
#endif
  if (!attn_warp_eligible(a)) return LQ_ERR_UNSUPPORTED;
  WarpParams p;
  p.a = a;
  p.counters = static_cast<int*>(work);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(work) + kAttnCounterBytes);
  p.small_rows = small_rows;
  p.vec = a.ldo % 4 == 0 && aligned_to(a.O, 16);
  const int ctas = std::max(1, std::min(device_info().sm_count, kAttnMaxCtas));
  // row groups that share a tile's keys. Two of 256 dims are for trees of quantised caches: few other
  // calls have the rows. Q4_0, 16 sequences of 4096 | one of 32768, 4 heads over one, us with two | one:
  // 32 rows 58 | 64, 39 | 39; 64: 95 | 115, 59 | 63; 128: 173 | 217, 93 | 109; 24: 57 | 50, 38 | 33; in f16
  // 64 rows take 138 | 142, 74 | 77, and the tile kernel 57 for the first.
  const int nr = a.c.head_dim == 256 ? (kTree && rows > 32 ? 2 : 1) : (rows > 8 ? 2 : 1);
  switch (fmt) {
    case LQ_FMT_F16: return pick<LQ_FMT_F16>(p, nr, ctas, stream);
    case LQ_FMT_Q8_0: return pick<LQ_FMT_Q8_0>(p, nr, ctas, stream);
    default: return pick<LQ_FMT_Q4_0>(p, nr, ctas, stream);
  }
}

#ifdef LQ_ATTN_TREE
unsigned read_clear_attn_warp_tree_error() {
#else
unsigned read_clear_attn_warp_error() {
#endif
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attnw_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_attnw_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq
