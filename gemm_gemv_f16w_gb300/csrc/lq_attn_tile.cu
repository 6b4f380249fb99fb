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
// group)): two row tiles of 128 share every key tile (heads of 256: below). Key tiles are 128 "rows
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
// Heads of 256: O of one row tile fills half of the tensor memory, its queries 128
// KB of shared memory, so a unit is 128 rows and a key tile 64 rows. Both
// softmax groups work on that row tile: each takes the maximum over all keys (the
// same bits in both), weighs its half of the keys (P has columns of its own) and
// sums its half of O's dims; QK of the next tile (S in two places in turn) runs
// under the softmax. 2048 tokens over 16384 positions, 16 heads over 2, run at
// 607 TFLOP/s of the plain formula in f16, 195 in Q8_0 (tiles of 32 keys only).
//
// Roles (four warpgroups, registers moved between them): two softmax groups,
// one per row tile; four loader warps (16-byte asynchronous copies for f16;
// loads, exact dequantisation and swizzled stores otherwise); one thread that
// issues MMAs: QK of both row tiles, then PV of both, so that one tile's
// softmax runs under the other's MMAs.
//
// Split: all units' key tiles are dealt in equal contiguous ranges to one CTA an
// SM; a unit that spans CTAs is joined from partial sums by the last one to
// arrive, in the order of the keys.
//
// What bounds it. The floor are the tensor cores at two (f16) or 3.5 (quantised:
// 2 x 2 products for S, 3 for O) MMAs a product of the plain formula; they are
// busy for half of the cycles. The rest is each row tile's own chain: S has to
// be read, the weights of 128 keys a thread computed and written, and O
// added before that tile's next MMAs, and the other tile's work covers half of it;
// without the weights' arithmetic, or without either product, the time stays
// within 10 %. 1024 tokens over 16384 positions, 32 heads over 8 of 128, f16: 357 us
// (746 TFLOP/s of the plain formula, two MMAs a product); 2048 over 16384, Q8_0:
// 1380 us (374 TFLOP/s), where the loaders' conversions (two parts of every element
// for every CTA that reads it) take as long as the MMAs. A unit's start and end add
// 10 us: 128 KB of queries come in and as much goes out at about 20 bytes a cycle an
// SM, and asking for the queries a tile earlier changed nothing. So 3 prompts of up
// to 4001 tokens, f16, take 463 us (557 TFLOP/s), and a prompt of 8192 under a window
// of 1024, 32 heads over 8 of 64, whose units have nine tiles, 238.
// Every wait is bounded; on timeout the kernel records LQ_ERR_DEVICE_TIMEOUT,
// lets its copies and MMAs finish, frees TMEM and returns. The roles' hand-overs
// are modelled in tests/test_attn_tile_protocol_cpu.py.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstring>
#include <type_traits>

#include "lq_attn.cuh"
#include "lq_tcgen05.cuh"

namespace lq {
namespace {

__device__ unsigned g_attnt_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_attnt_err, 0u, code); }

constexpr int kThreads = 512;
constexpr int kLoaders = 128;       // loader threads
// Key tiles worth a CTA: one f16 sequence, 512 of 1000 | 500 of 500 tokens, 32 heads over 8
// of 128: 2: 54.7 | 48.5 us, 4: 48.7 | 54.8, 8: 72.0 | 93.4.
constexpr int kMinTiles = 4;
constexpr int kInfo = 8;            // tiles of bookkeeping kept
constexpr int kUnits = 8;           // units of bookkeeping kept
constexpr int kMaxBatch = 4096;     // sequences whose totals fit in shared memory
constexpr float kNoMax = -3.402823466e38f;  // M before the first key: no finite logit is lower
constexpr float kLift = 11.0f;
constexpr float kLarge = 65536.0f;  // maxima from here on: logits are rounded before M is taken off
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TileParams {
  AttnArgs a;
  int* counters;
  float* parts;
  int small_rows;  // sequences with at most this many rows are another kernel's
  int vec_q, vec_o;
  int tma;         // f16: the tensor maps of the pools are there
  unsigned wait_hint, wait_clocks;  // how long a poll may block (ns), how long a wait may last (SM cycles)
};

template <int FMT, int D>
struct Geo {
  static constexpr bool ONE = D == 256;                    // one row tile a unit, shared by both softmax groups
  static constexpr int ROWS = ONE ? 128 : 256;             // query rows of a unit
  static constexpr int KROWS = ONE ? 64 : 128;             // rows of a key tile in shared memory
  static constexpr int KT = FMT == LQ_FMT_F16 ? KROWS : KROWS / 2;  // keys of a tile
  static constexpr int DO = ONE ? 128 : D;                 // output dims of a softmax thread
  static constexpr int ROW = FMT == LQ_FMT_F16 ? 2 * D : (FMT == LQ_FMT_Q8_0 ? D : D / 2);
  static constexpr int HALVES = D / 64;                    // 64-dim column groups
  static constexpr int GROUP = 128 * 128;                  // bytes of a group of queries: 128 rows of 128 bytes
  static constexpr int KGROUP = KROWS * 128;               // of keys or values
  static constexpr int UNIT = HALVES * KGROUP;             // K or V of a tile
  static constexpr int NU = D == 64 ? 6 : 3;               // ring of units
  static constexpr int QPART = HALVES * GROUP;             // hi or lo of a row tile
  static constexpr int Q = ROWS / 64 * QPART;              // [row tile][hi, lo]
  static constexpr int SMEM = Q + NU * UNIT + 1024 + 2048;  // alignment, barriers
  // Key tiles that a unit's start and end cost. One prompt of 4096 tokens with 0 | 2 | 4 | 6 |
  // 9, us: f16, heads of 64 244 | 196 | 184 | 188 | 197, of 128 364 | 294 | 243 | 245 | 255;
  // Q8_0 318 | 273 | 253 | 261 | 267, 506 | 453 | 441 | 448 | 454. Heads of 256: f16 with 7 |
  // 10 | 13 318 | 308 | 316, Q8_0 with 4 | 5 | 7 767 | 761 | 768.
  static constexpr int START = D != 256 ? 4 : (FMT == LQ_FMT_F16 ? 10 : 5);
  static constexpr int SLOT = ROWS * (D + 2);              // floats of a partial result
  // Quantised tiles: their loaders convert, and at 72 registers they wait on their own
  // chains. 2048 tokens over 16384 positions, 32 query heads over 8 of 128, Q8_0: 1652 us
  // with (200, 72), 1529 with (192, 88), 1740 with (176, 120). In f16 the loaders only
  // issue copies: 3 prompts of 4001 take 594 us with (200, 72), 602 with (192, 88).
  static constexpr bool QUANT = FMT != LQ_FMT_F16;
  // registers a thread of the warpgroups: together no more than the launch's 4 * 128
  static constexpr int REG_SOFTMAX = D != 64 ? (QUANT ? 192 : 200) : 168, REG_LOAD = D != 64 ? (QUANT ? 88 : 72) : 128,
                       REG_MMA = D != 64 ? 40 : 48;
  static_assert(2 * REG_SOFTMAX + REG_LOAD + REG_MMA <= 512);
};

// What the loaders know of a unit and tell the softmax threads.
struct UnitInfo {
  int tiles;         // key tiles of it here; 0: no more units
  int rho0, rows;    // its first row, and all rows of its sequence and head
  int row0, pos0;    // the sequence's first row of the call, and that row's position
  int head0;         // the first query head
  int seq, kv_head;
  int c0, c1, slot;  // the CTAs it spans and this one's slot of partial sums; c0 == c1: it is whole here
  int pad;           // 48 bytes
};

// What the planning warp knows of a key tile and tells the loaders and, through
// the MMAs' barriers, the softmax threads.
struct TileInfo {
  int j0;                     // first key
  uint32_t flags;
  int p1, begin, sink_end;    // keys that rows of the unit see: [begin, p1] and [0, sink_end)
  int ends;                   // the unit that ends with this tile here; -1: it goes on
  // where the rows of each group of 16 keys begin: f16 their row of the pool,
  // quantised the byte offsets of codes and scales (2 entries a group); -1: nowhere
  alignas(16) long long at[8];
};
static_assert(offsetof(TileInfo, at) % 16 == 0 && sizeof(TileInfo) % 16 == 0);

struct Bars {
  uint64_t full[6], empty[6];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2];
  uint64_t unit[kUnits], unit_free[kUnits];
  uint64_t join;  // the softmax threads of a unit that spans CTAs
  uint64_t drain;
  uint32_t tmem;
  int last;
  int start_i, start_h, start_rt, start_k;
  long long per, start_x, ends[2];  // tiles a CTA; the place of the first unit; tiles before the range's ends
  uint64_t told[kInfo], done[kInfo];   // a tile is described / its units are filled
  alignas(16) TileInfo info[kInfo];
  alignas(16) uint32_t bad[kInfo][4];  // keys whose values are not finite (kept out of the MMA)
  alignas(16) UnitInfo units[kUnits];
};
static_assert(sizeof(Bars) <= 2048 && offsetof(Bars, info) % 16 == 0 && offsetof(Bars, bad) % 16 == 0);
// TileInfo.flags: bit g < 8: the page of keys 16 g .. is there
constexpr uint32_t kTwo = 1u << 8;     // both row tiles of the unit have rows
constexpr uint32_t kFirst = 1u << 9;   // the unit's first tile here
constexpr uint32_t kMixed = 1u << 10;  // some key is seen by some of the rows only
constexpr uint32_t kAll = 1u << 11;    // every key is there and seen by some row

// Shared-memory matrix descriptors, 128-byte swizzle, as words: the low one has
// the address (>> 4) and the leading byte offset, the high one the stride
// (1024: groups of 8 rows) and the mode. Queries and keys are K-major (leading
// offset unused); values are MN-major: 64-dim groups a key tile's rows apart, 8-key groups.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t at) { return ((at & 0x3FFFFu) >> 4) | (1u << 16); }
template <int GROUP_BYTES>
__device__ __forceinline__ uint32_t desc_mn(uint32_t at) {
  return ((at & 0x3FFFFu) >> 4) | ((static_cast<uint32_t>(GROUP_BYTES) >> 4) << 16);
}
// D[tmem] = A B or (ADD) D + A B, f16, A from shared memory or from tensor memory.
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "n"(kDescHigh), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "n"(kDescHigh), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st1(uint32_t at, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(r) : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t at) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for the phase of `parity` for at most `clocks` cycles of the SM (below
// 2^32, so that 32 bits tell). As little code as can be: the roles' loops
// share the instruction cache.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint32_t hint, uint32_t clocks) {
  const uint32_t at = smem_u32(bar), t0 = static_cast<uint32_t>(clock());
  uint32_t ok;
  do {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(hint)
        : "memory");
  } while (ok == 0u && static_cast<uint32_t>(clock()) - t0 < clocks);
  return ok != 0u;
}
__device__ __forceinline__ void arrive_many(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
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
  int p0, p1;                // positions of its first and last row
  int begin, sink_end;       // keys that its rows see: [begin, p1] and [0, sink_end)
};

template <int KT, int ROWS>
__device__ __forceinline__ void unit_tiles(Work& w, const AttnArgs& a) {
  const int rows = w.s.rows * a.group, rho0 = w.rt * ROWS;
  w.p0 = w.s.len - w.s.rows + rho0 / a.group;
  w.p1 = w.s.len - w.s.rows + min(rho0 + ROWS - 1, rows - 1) / a.group;
  const kv::Visible v = kv::visible(max(w.p0, 0), a.window, a.sinks);
  w.begin = v.begin;
  w.sink_end = v.sink_end;
  w.first = v.begin / KT;
  w.sink_tiles = min((v.sink_end + KT - 1) / KT, w.first);
  w.n = w.p1 < 0 ? 1 : w.sink_tiles + w.p1 / KT + 1 - w.first;  // one empty tile where there is no key
}

__device__ __forceinline__ bool takes(const kv::Seq& s, const TileParams& P) {
  return s.rows > 0 && s.rows * P.a.group > P.small_rows;
}

// The first sequence from i on that has work here.
template <int ROWS>
__device__ __forceinline__ void enter(Work& w, const TileParams& P, int i) {
  for (;; ++i) {
    w.s = kv::sequence(P.a.b, P.a.c.page_size, i);
    if (takes(w.s, P)) break;
  }
  w.i = i;
  w.row_tiles = (w.s.rows * P.a.group + ROWS - 1) / ROWS;
}

__device__ __forceinline__ long long scan32(long long mine, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, mine, o);
    if (lane >= o) mine += up;
  }
  return mine;
}

// This CTA's range of all units' tiles, in the order (sequence, key/value head, row
// tile, key tile). A unit counts as START tiles more than it has, ahead of its own:
// its start costs about that much, and without it the CTAs that get the many short
// units of a prompt's beginning are the last to end. Warps 0 and 1 look for the
// range's two ends: the tiles before each, and where the first one is.
template <int KT, int ROWS, int START>
__device__ __forceinline__ void plan(const TileParams& P, Bars* bar, long long* totals, int warp, int lane) {
  const AttnArgs& a = P.a;
  int* const units = reinterpret_cast<int*>(totals + kMaxBatch);
#pragma unroll 1
  for (int i = warp; i < a.b.batch; i += kThreads / 32) {
    Work w;
    w.s = kv::sequence(a.b, a.c.page_size, i);
    long long sum = 0;
    const int rts = takes(w.s, P) ? (w.s.rows * a.group + ROWS - 1) / ROWS : 0;
#pragma unroll 1
    for (w.rt = lane; w.rt < rts; w.rt += 32) {
      unit_tiles<KT, ROWS>(w, a);
      sum += w.n + START;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      totals[i] = sum;  // of one head
      units[i] = rts;
    }
  }
  __syncthreads();
  if (warp > 1) return;
  long long all = 0;
#pragma unroll 1
  for (int i = lane; i < a.b.batch; i += 32) all += totals[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  all *= a.c.kv_heads;
  const long long per = max(kv::quotient(all + gridDim.x - 1, gridDim.x), static_cast<long long>(kMinTiles));
  const long long end = min(per * (blockIdx.x + warp), all);
  long long x = end, before = 0;  // place in the unit in the end; units before it
  int i = 0, h = 0, rt = 0;
#pragma unroll 1
  for (int base = 0; base < a.b.batch; base += 32) {  // the sequence
    const bool is = base + lane < a.b.batch;
    const long long here = is ? totals[base + lane] * a.c.kv_heads : 0, incl = scan32(here, lane);
    const long long us = scan32(is ? static_cast<long long>(units[base + lane]) * a.c.kv_heads : 0, lane);
    const unsigned past = __ballot_sync(0xffffffffu, x < incl);
    const int at = past ? __ffs(static_cast<int>(past)) - 1 : 31;
    const long long skip = __shfl_sync(0xffffffffu, incl - (past ? here : 0), at);
    x -= skip;
    if (past) {
      i = base + at;
      before += __shfl_sync(0xffffffffu, us, at) - static_cast<long long>(units[i]) * a.c.kv_heads;
      break;
    }
    before += __shfl_sync(0xffffffffu, us, 31);
  }
  if (end < all) {
    h = static_cast<int>(kv::quotient(x, totals[i]));
    x -= h * totals[i];
    Work w;
    w.s = kv::sequence(a.b, a.c.page_size, i);
#pragma unroll 1
    for (int base = 0;; base += 32) {  // the row tile
      w.rt = base + lane;
      unit_tiles<KT, ROWS>(w, a);
      const long long here = w.rt < units[i] ? w.n + START : 0, incl = scan32(here, lane);
      const unsigned past = __ballot_sync(0xffffffffu, x < incl);
      if (past) {
        const int at = __ffs(static_cast<int>(past)) - 1;
        rt = base + at;
        x -= __shfl_sync(0xffffffffu, incl - here, at);
        break;
      }
      x -= __shfl_sync(0xffffffffu, incl, 31);
    }
    before += static_cast<long long>(h) * units[i] + rt;
  }
  if (lane == 0) {
    // tiles before the end: its place less the starts before it
    bar->ends[warp] = end - x - START * before + max(x - START, 0ll);
    if (warp == 0) {
      bar->per = per;
      bar->start_i = i;
      bar->start_h = h;
      bar->start_rt = rt;
      bar->start_k = static_cast<int>(max(x - START, 0ll));
      bar->start_x = end - x;
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ TileParams P, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using G = Geo<FMT, D>;
  constexpr int KT = G::KT, NU = G::NU, ROWS = G::ROWS, DO = G::DO;
  constexpr bool ONE = G::ONE;
  constexpr bool QUANT = FMT != LQ_FMT_F16;
  extern __shared__ unsigned char raw_smem[];
  unsigned char* const smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  unsigned char* const ring = smem + G::Q;
  Bars* const bar = reinterpret_cast<Bars*>(ring + NU * G::UNIT);
  const AttnArgs& a = P.a;
  // (from lane 0 by a shuffle: the compiler then knows that a warp has one role,
  // and keeps its addresses and descriptors in uniform registers)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), wg = warp >> 2;

  if (tid == 0) {
    for (int u = 0; u < NU; ++u) {
      mbar_init(&bar->full[u], kLoaders);
      mbar_init(&bar->empty[u], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&bar->q_ready[q], ONE ? 256 : 128);
      mbar_init(&bar->s_full[q], 2);  // the MMAs, and the issuing thread (what the loaders wrote)
      mbar_init(&bar->p_ready[q], ONE ? 256 : 128);
      mbar_init(&bar->o_full[q], 2);
    }
    for (int u = 0; u < kUnits; ++u) {
      mbar_init(&bar->unit[u], 1);
      mbar_init(&bar->unit_free[u], 256);
    }
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->join, 256);
    for (int k = 0; k < kInfo; ++k) {
      mbar_init(&bar->told[k], 1);
      mbar_init(&bar->done[k], kLoaders);
    }
    for (int k = 0; k < kInfo; ++k) *reinterpret_cast<uint4*>(bar->bad[k]) = make_uint4(0u, 0u, 0u, 0u);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  plan<KT, ROWS, G::START>(P, bar, reinterpret_cast<long long*>(ring), warp, lane);
  if (warp == 12) {
    tc::tmem_alloc(&bar->tmem, 512);
    tc::tmem_relinquish();
  }
  fence_proxy_async_smem();  // the totals lay where copies will land
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar->tmem, 0);
  const int mine = __shfl_sync(0xffffffffu, static_cast<int>(min(bar->ends[1] - bar->ends[0], 1ll << 30)), 0);  // key tiles here

  bool in_time = true;  // no wait of this warp has run out
  auto wait = [&](uint64_t* b, uint32_t parity) {  // by whole warps
    in_time = __all_sync(0xffffffffu, wait_for(b, parity, P.wait_hint, P.wait_clocks));
    return in_time;
  };

  if (wg < 2) {
    // ================= softmax: thread = query row =================================
    // One row tile: both groups look at every key for the maximum, each weighs its
    // half of the keys and sums its half of the output's dims.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::REG_SOFTMAX));
    const int q = wg, r = tid & 127, half = q;
    const int rq = ONE ? 0 : q, row_at = rq * 128 + r, dim0 = ONE ? half * DO : 0;  // row tile, row of the unit, first dim
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + rq * 128, p_at = ONE ? s_at + 128 : s_at, o_at = tmem + lanes + 256 + q * DO;
    unsigned char* const q_hi = smem + rq * 2 * G::QPART;
    unsigned char* const q_lo = q_hi + G::QPART;
    // the column groups of the queries' two parts that are this softmax group's own:
    // its rows come and go through them, 32 floats a group
    auto own = [&](int s) { return q_hi + (ONE ? (s >> 1) * 4 + 2 * half + (s & 1) : s) * G::GROUP; };
    uint32_t tile = 0, tiles_q = 0, joins = 0;  // tiles done by the CTA, by this row tile
#pragma unroll 1
    for (uint32_t un = 0;; ++un) {
      if (!wait(&bar->unit[un % kUnits], (un / kUnits) & 1u)) break;
      const UnitInfo& w = bar->units[un % kUnits];
      const int tiles = w.tiles;
      if (tiles == 0) break;
      const int rho = w.rho0 + row_at;
      const bool active = w.rho0 + rq * 128 < w.rows;  // the row tile has rows
      const bool row = rho < w.rows;
      const int token = min(rho, w.rows - 1) / a.group;
      const int t = w.row0 + token, head = w.head0 + (min(rho, w.rows - 1) - token * a.group), pos = w.pos0 + token;
      float om[DO], M = kNoMax, l = 0.0f, f = 0.0f;
      if (active) {
        // The warp's 32 query rows come as f32 into the very bytes of shared memory
        // that their two f16 parts will take (rows of 128 bytes in the group's own
        // column groups), and each thread turns its row: no other thread's bytes.
        constexpr int LPR = DO / 4, RPI = 32 / LPR;  // lanes a row, rows at a time
        const int l4 = lane % LPR;
        const long long off = t * a.ldq + static_cast<long long>(head) * D + dim0;
        const uint32_t live = __ballot_sync(0xffffffffu, row);
        unsigned char* const land = own(l4 >> 3) + (warp & 3) * 32 * 128 + (l4 & 7) * 16;
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += RPI) {
          const int rr = r0 + lane / LPR;
          const float* src = a.Q + __shfl_sync(0xffffffffu, off, rr) + l4 * 4;
          const bool there = (live >> rr) & 1u;
          if (P.vec_q) {
            copy16(smem_u32(land + rr * 128), there ? src : a.Q, there);
          } else {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (there) v = make_float4(src[0], src[1], src[2], src[3]);
            *reinterpret_cast<float4*>(land + rr * 128) = v;
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        wait_copies<0>();
        __syncwarp();
        // 16-byte chunks in an order of the row's own, so that eight rows hit all banks
        float4 v[DO / 4];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < DO / 4; ++j) {
          v[j] = *reinterpret_cast<const float4*>(own(j >> 3) + r * 128 + (((j ^ r) & 7) << 4));
          top = fmaxf(top, fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w))));
        }
        if constexpr (ONE) {  // the other half's
          tmem_st1(p_at + 2 + half, __float_as_uint(top));
          tc::wait_st();
          tc::fence_before_sync();
          mbar_arrive(&bar->join);
          if (!wait(&bar->join, joins++ & 1u)) break;
          tc::fence_after_sync();
          const uint32_t other = tmem_ld1(p_at + 2 + (half ^ 1));
          tc::wait_ld();
          tc::fence_before_sync();
          top = fmaxf(top, __uint_as_float(other));
        }
        // scaled to the top of f16's range by a power of two; f takes S back to base-2 logits
        const int ex = static_cast<int>(__float_as_uint(top) >> 23);
        const int es = ex == 0 || ex == 255 ? 127 : min(max(127 + 127 + 14 - ex, 1), 253);
        const float sigma = __uint_as_float(static_cast<unsigned>(es) << 23);
        f = __uint_as_float(static_cast<unsigned>(254 - es) << 23) * fabsf(a.scale) * kLog2e;
        const float sg = a.scale < 0.0f ? -sigma : sigma;
        const bool odd = r & 1;
#pragma unroll
        for (int j = 0; j < DO / 4; j += 2) {
          const float4 x = odd ? v[j + 1] : v[j], y = odd ? v[j] : v[j + 1];  // dims in order
          uint4 hi, lo;
          split2(x.x * sg, x.y * sg, hi.x, lo.x);
          split2(x.z * sg, x.w * sg, hi.y, lo.y);
          split2(y.x * sg, y.y * sg, hi.z, lo.z);
          split2(y.z * sg, y.w * sg, hi.w, lo.w);
          const int c8 = (j >> 3 & 1) * 4 + (((j >> 1) ^ (r >> 1)) & 3);  // 16-byte chunk of the 64-dim group
          const uint32_t at = (ONE ? 2 * half + (j >> 4) : j >> 4) * G::GROUP + r * 128 + ((c8 ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(q_hi + at) = hi;
          *reinterpret_cast<uint4*>(q_lo + at) = lo;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar->q_ready[rq]);
#pragma unroll
        for (int d = 0; d < DO; ++d) om[d] = 0.0f;
      }
      bool ok = true;
      if (!active) tile += tiles;
#pragma unroll 1
      for (int k = 0; k < (active ? tiles : 0); ++k, ++tile, ++tiles_q) {
        // (one row tile: S of the next tile comes while this one's lies here, in turn)
        const uint32_t s_now = s_at + (ONE ? (tiles_q & 1u) * 64 : 0);
        ok = ONE ? wait(&bar->s_full[tiles_q & 1u], (tiles_q >> 1) & 1u) : wait(&bar->s_full[rq], tiles_q & 1u);
        if (!ok) break;
        tc::fence_after_sync();
        const int j0 = bar->info[tile % kInfo].j0;
        const uint32_t pages = bar->info[tile % kInfo].flags & 0xFFu;
        const bool clear = pages == (1u << (KT / 16)) - 1u && j0 + KT - 1 <= pos &&
                           (a.window == 0 || j0 > pos - a.window || j0 + KT <= a.sinks);
        const bool edge = __any_sync(0xffffffffu, !clear);
        // bit i: the row sees key j + i of the tile (i < 32; j a multiple of 16)
        auto vis32 = [&](int j) -> uint32_t {
          const int last = pos - j0 - j;  // keys up to here are not ahead of the row
          uint32_t m = last < 0 ? 0u : (last >= 31 ? 0xFFFFFFFFu : (2u << last) - 1u);
          if (a.window != 0) {
            const int from = last >= a.window ? last - a.window + 1 : 0;  // keys from here on are in the window
            const int sink = min(max(a.sinks - j0 - j, 0), 32);           // keys below are sinks
            m &= (from >= 32 ? 0u : 0xFFFFFFFFu << from) | (sink >= 32 ? 0xFFFFFFFFu : (1u << sink) - 1u);
          }
          const uint32_t pg = pages >> (j >> 4);
          return m & ((pg & 1u ? 0xFFFFu : 0u) | (pg & 2u ? 0xFFFF0000u : 0u));
        };
        // Over the raw sums of the tile's keys from `from` on, 16 at a time. (Asking for the
        // next 16 ahead of time costs more in register moves than it hides.)
        auto each = [&](auto&& what, bool masked, int from, int to) {
#pragma unroll 1
          for (int j = from; j < to; j += 16) {
            uint32_t s[16];
            tmem_ld16(s_now + j, s);
            const uint32_t vis = masked ? vis32(j) : 0u;
            if constexpr (QUANT) {
              uint32_t low[16];
              tmem_ld16(s_now + KT + j, low);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 x = fadd2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                       make_float2(__uint_as_float(low[i]), __uint_as_float(low[i + 1])));
                s[i] = __float_as_uint(x.x);
                s[i + 1] = __float_as_uint(x.y);
              }
            } else {
              tc::wait_ld();
            }
            what(j, s, vis);
          }
        };
        float top = -INFINITY;
        // (two loops each: merged into one, the masks cost every tile 1.4 times as much)
        if (!edge) {
          each([&](int, uint32_t (&s)[16], uint32_t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, __uint_as_float(s[i]));
          }, false, 0, KT);
        } else {
          each([&](int, uint32_t (&s)[16], uint32_t vis) {
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, (vis >> i) & 1u ? __uint_as_float(s[i]) : -INFINITY);
          }, true, 0, KT);
        }
        top = top == -INFINITY ? top : top * f;
        float keep = 1.0f;
        if (top - M > 15.0f) {  // (exact between neighbours, which M + 15 need not be)
          float to = fmaxf(M, top - kLift);
          to = top - to > 15.0f ? top : to;  // past 2^27 the step itself is 16
          keep = ex2(M - to);
          M = to;
          l *= keep;
        }
        // Weights, in two parts, over the logits: 16 columns a 16 keys. s f - M in one
        // step saves the rounding of s f, but M comes from the rounded product of the
        // largest s: where that rounding counts (past 2^24 it can be an exponent and
        // more, and weights would leave f16's range) every product is rounded. (By
        // scalar multiplications: packed ones are merged with the addition after all.)
        const bool large = __any_sync(0xffffffffu, fabsf(M) >= kLarge);
        const float2 ff = make_float2(f, f), mm = make_float2(-M, -M), minus = make_float2(-1.0f, -1.0f);
        float2 l2 = make_float2(0.0f, 0.0f);
        auto weights = [&](int j, uint32_t (&s)[16], uint32_t vis, bool masked, bool rounded) {
          uint32_t w16[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 raw = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
            const float2 x = rounded ? fadd2(make_float2(__fmul_rn(raw.x, f), __fmul_rn(raw.y, f)), mm) : ffma2(raw, ff, mm);
            float2 p = make_float2(ex2(x.x), ex2(x.y));
            if (masked) {
              p.x = (vis >> i) & 1u ? p.x : 0.0f;
              p.y = (vis >> (i + 1)) & 1u ? p.y : 0.0f;
            }
            l2 = fadd2(l2, p);
            const __half2 h = __floats2half2_rn(p.x, p.y);
            const float2 r2 = ffma2(__half22float2(h), minus, p);
            w16[i / 2] = h2(h);
            w16[8 + i / 2] = h2(__floats2half2_rn(r2.x, r2.y));
          }
          tmem_st16(p_at + j, w16);
        };
        const int from = ONE ? half * (KT / 2) : 0, to = ONE ? from + KT / 2 : KT;
        if (large) {
          each([&](int j, uint32_t (&s)[16], uint32_t vis) { weights(j, s, vis, true, true); }, true, from, to);
        } else if (!edge) {
          each([&](int j, uint32_t (&s)[16], uint32_t) { weights(j, s, 0u, false, false); }, false, from, to);
        } else {
          each([&](int j, uint32_t (&s)[16], uint32_t vis) { weights(j, s, vis, true, false); }, true, from, to);
        }
        l += l2.x + l2.y;
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bar->p_ready[rq]);
        ok = wait(&bar->o_full[rq], tiles_q & 1u);
        if (!ok) break;
        tc::fence_after_sync();
        const uint4 bad = *reinterpret_cast<const uint4*>(bar->bad[tile % kInfo]);
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          const float2 kk = make_float2(keep, keep);
          uint32_t sa[16], sb[16];
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
          for (int d = 0; d < DO; d += 32) {
            tc::wait_ld();
            tmem_ld16(o_at + d + 16, sb);
            add(d, sa);
            tc::wait_ld();
            if (d + 32 < DO) tmem_ld16(o_at + d + 32, sa);
            add(d + 16, sb);
          }
          if (pass == 1 || (bad.x | bad.y | bad.z | bad.w) == 0u) break;
          // values that are not finite were kept out of the MMA: once more, with
          // their sums over the keys that each row sees in O's place
#pragma unroll 1
          for (int d = 0; d < DO; d += 16) {
            float o[16] = {};
#pragma unroll 1
            for (int j = 0; j < KT; ++j) {
              const uint32_t word = j < 32 ? bad.x : (j < 64 ? bad.y : (j < 96 ? bad.z : bad.w));
              if (!((word >> (j & 31)) & 1u) || !((vis32(j & ~31) >> (j & 31)) & 1u)) continue;
              const int page = kv::page_of(a.c, a.b, w.seq, j0 + j);
              if (page < 0) continue;
              const int slot = (j0 + j) % a.c.page_size;
              const unsigned char* at = a.c.v + page * a.c.page_bytes + w.kv_head * a.c.head_bytes;
              const __half* h16 = QUANT ? reinterpret_cast<const __half*>(at + static_cast<long long>(a.c.page_size) * G::ROW) + slot * (D / 32) + (dim0 + d) / 32
                                        : reinterpret_cast<const __half*>(at) + static_cast<long long>(slot) * D + dim0 + d;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float v = __half2float(h16[QUANT ? 0 : i]);
                if (!(fabsf(v) <= 65504.0f)) o[i] += QUANT ? v - v : v;  // a block's scale: NaN
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) sa[i] = __float_as_uint(o[i]);
            tmem_st16(o_at + d, sa);
          }
          tc::wait_st();
          keep = 1.0f;
        }
        tc::fence_before_sync();
      }
      if (!ok) break;

      // ---- the unit's result, or its part -----------------------------------------
      bool writes = active;
      if constexpr (ONE) {  // the groups' sums of weights, by tensor memory that held P
        tmem_st1(p_at + half, __float_as_uint(l));
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bar->join);
        if (!wait(&bar->join, joins++ & 1u)) break;
        tc::fence_after_sync();
        const uint32_t other = tmem_ld1(p_at + (half ^ 1));
        tc::wait_ld();
        l = half == 0 ? l + __uint_as_float(other) : __uint_as_float(other) + l;
        tc::fence_before_sync();
      }
      if (w.c0 != w.c1) {
        auto slot_of = [&](int slot) { return P.parts + static_cast<long long>(slot) * G::SLOT; };  // [dim / 4][row][4], then M and l
        constexpr int kSums = D * ROWS;
        if (row) {
          float* to = slot_of(w.slot);
#pragma unroll
          for (int d = 0; d < DO; d += 4)
            *reinterpret_cast<float4*>(to + (dim0 + d) * ROWS + row_at * 4) = make_float4(om[d], om[d + 1], om[d + 2], om[d + 3]);
          if (!ONE || half == 0) *reinterpret_cast<float2*>(to + kSums + row_at * 2) = make_float2(M, l);
        }
        __threadfence();
        mbar_arrive(&bar->join);
        if (!wait(&bar->join, joins++ & 1u)) break;
        if (tid == 0) {
          const int before = atomicAdd(P.counters + w.c0, 1);
          bar->last = before == w.c1 - w.c0;
          if (before == w.c1 - w.c0) P.counters[w.c0] = 0;
        }
        mbar_arrive(&bar->join);
        if (!wait(&bar->join, joins++ & 1u)) break;
        writes = active && bar->last;
        if (writes && row) {  // in the order of the keys
          __threadfence();
          M = kNoMax;
          l = 0.0f;
#pragma unroll
          for (int d = 0; d < DO; ++d) om[d] = 0.0f;
#pragma unroll 1
          for (int c = w.c0; c <= w.c1; ++c) {
            const float* from = slot_of(c == w.c0 ? 2 * c + 1 : 2 * c);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + kSums + row_at * 2));
            const float to = fmaxf(M, ml.x), f1 = ex2(M - to), f2 = ex2(ml.x - to);
            M = to;
            l = l * f1 + ml.y * f2;
#pragma unroll
            for (int d = 0; d < DO; d += 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(from + (dim0 + d) * ROWS + row_at * 4));
              om[d] = om[d] * f1 + v.x * f2;
              om[d + 1] = om[d + 1] * f1 + v.y * f2;
              om[d + 2] = om[d + 2] * f1 + v.z * f2;
              om[d + 3] = om[d + 3] * f1 + v.w * f2;
            }
          }
        }
      }
      if (writes) {
        // rows go out through the query rows' shared memory (their MMAs are done; a
        // warp's rows of all parts are its own): whole rows, 16 bytes a lane
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // 0: the row sees nothing; NaN stays
        __syncwarp();
#pragma unroll
        for (int d = 0; d < DO; d += 4)
          *reinterpret_cast<float4*>(own(d / 32) + tc::sw128_offset(r, (d / 4) & 7)) =
              make_float4(om[d] * inv, om[d + 1] * inv, om[d + 2] * inv, om[d + 3] * inv);
        __syncwarp();
        constexpr int LPR = DO / 4, RPI = 32 / LPR;
        const int l4 = lane % LPR;
        const uint32_t live = __ballot_sync(0xffffffffu, row && LQ_IN_BOUNDS(t < a.b.tokens && head < a.heads));
        const long long off = t * a.ldo + static_cast<long long>(head) * D + dim0;
        const unsigned char* const from = own(l4 >> 3);
#pragma unroll 8
        for (int r0 = 0; r0 < 32; r0 += RPI) {
          const int rr = r0 + lane / LPR;
          float* out = a.O + __shfl_sync(0xffffffffu, off, rr) + l4 * 4;
          const float4 v = *reinterpret_cast<const float4*>(from + tc::sw128_offset((warp & 3) * 32 + rr, l4 & 7));
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
        if (row && a.lse && (!ONE || half == 0)) a.lse[static_cast<long long>(t) * a.heads + head] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
        __syncwarp();
      }
      mbar_arrive(&bar->unit_free[un % kUnits]);
    }
  } else if (wg == 2) {
    // ================= loader ========================================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::REG_LOAD));
    const int tl = tid & 127;
    constexpr int CPR = QUANT ? D / 16 : D / 8;          // chunks a row: 16 codes, or 16 bytes of f16
    constexpr int PASS = kLoaders / CPR, N = KT / PASS;  // rows a pass, passes
    const int row0 = tl / CPR, ch = tl % CPR;
    bool alive = true;

    // the values of a unit's chunks that this thread copied: those that are not
    // finite are taken out and their keys noted
    auto screen = [&](uint32_t at_unit, uint32_t tile_no) {
#pragma unroll 1
      for (int n = 0; n < N; ++n) {
        const int row = row0 + n * PASS;
        unsigned char* at = ring + at_unit + (ch >> 3) * G::KGROUP + tc::sw128_offset(row, ch & 7);
        uint4 v = *reinterpret_cast<uint4*>(at);
        uint32_t w4[4] = {v.x, v.y, v.z, v.w};
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((w4[j] & 0x7C00u) == 0x7C00u) {
            w4[j] &= 0xFFFF0000u;
            bad = true;
          }
          if ((w4[j] & 0x7C000000u) == 0x7C000000u) {
            w4[j] &= 0xFFFFu;
            bad = true;
          }
        }
        if (bad) {
          *reinterpret_cast<uint4*>(at) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
          atomicOr(&bar->bad[tile_no % kInfo][row >> 5], 1u << (row & 31));
        }
      }
    };

    uint32_t unit = 0, pend = 0;  // ring units filled; f16: unit whose copies are not yet reported, plus one
    uint32_t pend_tile = 0;       // its tile
    uint32_t boxed = 0;           // f16, bit i: the copy engine fills the i-th unit from the last
    bool pend_screen = false;
    using Raw = typename std::conditional<FMT == LQ_FMT_Q8_0, uint4, uint2>::type;
    Raw ahead[2];
    __half sc_ahead[2];
    bool there[2];
    // Quantised: codes and scales of the tile's two passes `it`, K's and then V's.
    auto fetch = [&](int it, const TileInfo& c) {
      const int side = it / (N / 2), nn = it % (N / 2);
      const unsigned char* const pool = (side ? a.c.v : a.c.k) + ch * (G::ROW * 16 / D);
      const unsigned char* const scales = (side ? a.c.v : a.c.k) + (ch >> 1) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row0 + (2 * nn + i) * PASS;
        const longlong2 at = *reinterpret_cast<const longlong2*>(&c.at[2 * (row >> 4)]);
        const int key = c.j0 + row;
        // unconditional loads (a branch around them holds the loop up): a key that
        // is not there reads the pool's first bytes, its scale becomes zero at use
        there[i] = at.x >= 0 && key <= c.p1 && (key >= c.begin || key < c.sink_end);
        ahead[i] = *reinterpret_cast<const Raw*>(pool + (there[i] ? at.x + (row & 15) * G::ROW : 0));
        sc_ahead[i] = *reinterpret_cast<const __half*>(scales + (there[i] ? at.y + (row & 15) * (D / 16) : 0));
      }
    };
    auto report = [&]() {  // f16: the pending unit has landed
      const uint32_t u = pend - 1;
      if (pend_screen) screen((u % NU) * G::UNIT, pend_tile);
      fence_proxy_async_smem();
      mbar_arrive(&bar->full[u % NU]);
      pend = 0;
    };
    // Units go in the order of their use. One row tile: the next tile's K before this
    // one's V, so a step is K of its tile and V of the tile before.
    const uint32_t tiles = static_cast<uint32_t>(max(mine, 0)), steps = tiles > 0 ? tiles + (ONE ? 1 : 0) : 0;
#pragma unroll 1
    for (uint32_t step = 0; step < steps && alive; ++step) {  // loader
      const int first = ONE && step == tiles ? 1 : 0, last = ONE && step == 0 ? 1 : 2;  // sides
      if ((!QUANT || step == 0) && step < tiles) {
        alive = wait(&bar->told[step % kInfo], (step / kInfo) & 1u);
        if (!alive) break;
        if constexpr (QUANT) fetch(0, bar->info[step % kInfo]);
      }
      if constexpr (!QUANT) {
#pragma unroll 1
        for (int side = first; side < last; ++side, ++unit) {
          const TileInfo& c = bar->info[(step - (ONE ? side : 0)) % kInfo];
          uint64_t* const e = &bar->empty[unit % NU];
          const uint32_t parity = ((unit / NU) & 1u) ^ 1u;
          uint64_t* const fl = &bar->full[unit % NU];
          // every key is every row's: the copy engine's boxes of 16 keys x 64 dims, all
          // by one warp (which arrives for the others, so that it can see them land)
          const bool boxes = P.tma && (c.flags & (kAll | kMixed)) == kAll;
          if (pend && (boxes || !__all_sync(0xffffffffu, mbar_test_wait(e, parity)))) {  // report what landed before waiting
            wait_copies<0>();
            report();
          }
          alive = wait(e, parity);
          if (!alive) break;
          boxed = boxed << 1 | (boxes ? 1u : 0u);
          if (boxes) {
            if (warp == 8) {
              if (lane == 0) {
                mbar_arrive_expect_tx(fl, G::UNIT);
                arrive_many(fl, kLoaders - 1);
              }
              __syncwarp();
              if (lane < KT / 16) {
                const int r16 = static_cast<int>(c.at[lane]);
#pragma unroll
                for (int h = 0; h < G::HALVES; ++h)
                  tc::tma_load_2d(ring + (unit % NU) * G::UNIT + h * G::KGROUP + lane * 2048, side ? &mv : &mk, h * 64, r16, fl);
              }
              __syncwarp();
            }
            continue;
          }
          // (passes of eight rows and more stay at the same place of a swizzle atom)
          const uint32_t dst = smem_u32(ring) + (unit % NU) * G::UNIT + (ch >> 3) * G::KGROUP + (PASS % 8 == 0 ? tc::sw128_offset(row0, ch & 7) : 0);
          const unsigned char* const src = (side ? a.c.v : a.c.k) + row0 * G::ROW + ch * 16;
#pragma unroll 4
          for (int n = 0; n < N; ++n) {  // rows row0 + n PASS: one group of 16 a pass
            const long long at = c.at[n * PASS / 16];
            const int key = c.j0 + row0 + n * PASS;
            const bool there = at >= 0 && key <= c.p1 && (key >= c.begin || key < c.sink_end);
            copy16(PASS % 8 == 0 ? dst + n * PASS * 128 : dst + (n * PASS / 8) * 1024 + tc::sw128_offset(row0 + n * PASS % 8, ch & 7), src + max(at, 0ll) * G::ROW + (n * PASS % 16) * G::ROW, there);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (pend) {
            wait_copies<1>();
            report();
          }
          pend = unit + 1;
          pend_screen = side == 1 && (c.flags & kMixed);
          pend_tile = step - (ONE ? side : 0);
        }
      } else {
        // Two passes at a time, K's and then V's, in a small loop (straight code for
        // all passes is bound by instruction fetches); two are on their way.
#pragma unroll 1
        for (int it = first * (N / 2); it < last * (N / 2); ++it) {
          const int side = it / (N / 2), nn = it % (N / 2);
          if (nn == 0) {
            alive = wait(&bar->empty[unit % NU], ((unit / NU) & 1u) ^ 1u);
            if (!alive) break;
          }
          unsigned char* const dst = ring + (unit % NU) * G::UNIT;
          alignas(16) uint32_t w4[2][4];
          __half d2[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<Raw*>(w4[i]) = ahead[i];
            d2[i] = there[i] ? sc_ahead[i] : __ushort_as_half(0);
          }
          const uint32_t tile = step - (ONE ? side : 0);
          if (it + 1 < last * (N / 2)) {
            fetch(it + 1, bar->info[(step - (ONE ? (it + 1) / (N / 2) : 0)) % kInfo]);
          } else if (step + 1 < tiles) {
            alive = wait(&bar->told[(step + 1) % kInfo], ((step + 1) / kInfo) & 1u);
            if (!alive) break;
            fetch(0, bar->info[(step + 1) % kInfo]);
          } else if (ONE && step + 1 < steps) {
            fetch(N / 2, bar->info[step % kInfo]);
          }
          const bool mixed = side == 1 && (bar->info[tile % kInfo].flags & kMixed);
          // step by step for both passes at once: one chain after the other would
          // leave this warp waiting for its own results
          uint32_t hi[2][8], lo[2][8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (mixed && !(fabsf(__half2float(d2[i])) <= 65504.0f)) {
              const int row = row0 + (2 * nn + i) * PASS;
              d2[i] = __ushort_as_half(0);
              atomicOr(&bar->bad[tile % kInfo][row >> 5], 1u << (row & 31));
            }
            if constexpr (FMT == LQ_FMT_Q8_0) {
#pragma unroll
              for (int n = 0; n < 4; ++n) codes8(w4[i][n], hi[i][2 * n], hi[i][2 * n + 1]);
            } else {  // pairs (0, 1), (2, 3), ... of the low nibbles, then of the high ones
#pragma unroll
              for (int n = 0; n < 2; ++n) codes4(w4[i][n], hi[i][2 * n], hi[i][2 * n + 1], hi[i][4 + 2 * n], hi[i][4 + 2 * n + 1]);
            }
          }
          constexpr float kTop = FMT == LQ_FMT_Q8_0 ? 515.5f : 8188.0f;
          if (!(fabsf(__half2float(d2[0])) >= kTop) && !(fabsf(__half2float(d2[1])) >= kTop)) {
            // code * d in f16, and what it leaves: exact by the fused multiply-add
            const __half2 da = __half2half2(d2[0]), db = __half2half2(d2[1]);
            __half2 prod[2][8];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              prod[0][n] = __hmul2_rn(as_h2(hi[0][n]), da);
              prod[1][n] = __hmul2_rn(as_h2(hi[1][n]), db);
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              lo[0][n] = h2(__hfma2(as_h2(hi[0][n]), da, __hneg2(prod[0][n])));
              lo[1][n] = h2(__hfma2(as_h2(hi[1][n]), db, __hneg2(prod[1][n])));
              hi[0][n] = h2(prod[0][n]);
              hi[1][n] = h2(prod[1][n]);
            }
          } else {  // the top of f16's range: rounded toward zero, through f32
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float df = __half2float(d2[i]);
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const float2 c2 = __half22float2(as_h2(hi[i][n]));
                split2_rz(c2.x * df, c2.y * df, hi[i][n], lo[i][n]);
              }
            }
          }
          // 16-byte chunks of the rows: the second column group's threads start with their second
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = row0 + (2 * nn + i) * PASS;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int part = s ^ ((ch >> 2) & 1);
              const int c16 = FMT == LQ_FMT_Q8_0 ? 2 * ch + part : (ch >> 1) * 4 + (ch & 1) + 2 * part;
              unsigned char* const to = dst + (c16 >> 3) * G::KGROUP + tc::sw128_offset(row, c16 & 7);
              *reinterpret_cast<uint4*>(to) = part ? make_uint4(hi[i][4], hi[i][5], hi[i][6], hi[i][7]) : make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
              *reinterpret_cast<uint4*>(to + KT * 128) = part ? make_uint4(lo[i][4], lo[i][5], lo[i][6], lo[i][7]) : make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
            }
          }
          if (nn == N / 2 - 1) {
            fence_proxy_async_smem();
            mbar_arrive(&bar->full[unit % NU]);
            ++unit;
          }
        }
      }
      if (!alive) break;
      if (!ONE || step > 0) mbar_arrive(&bar->done[(step - (ONE ? 1 : 0)) % kInfo]);
    }
    wait_copies<0>();
    if (pend) report();
    // The copy engine finishes before this warp leaves, whether or not a wait of its
    // own has run out: the MMA warp may have given up on the last units, and nothing
    // may land once the CTA is gone. (They have landed where all went well.)
    if (warp == 8) {
      for (uint32_t i = 0; i < NU; ++i) {
        const uint32_t u = unit - 1 - i;  // the units before `unit` were issued
        if ((boxed >> i) & 1u) mbar_wait(&bar->full[u % NU], (u / NU) & 1u, kDrainWaitNs);
      }
    }
  } else {
    // ================= MMA issue =======================================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::REG_MMA));
    if (warp == 12) {
      constexpr uint32_t kQK = tc::idesc_f16_f32(128, G::KROWS);
      constexpr uint32_t kPV = tc::idesc_f16_f32(128, D) | (1u << 16);  // B is MN-major
      const uint32_t q_desc = desc_k(smem_u32(smem)), k_desc = desc_k(smem_u32(ring)), v_desc = desc_mn<G::KGROUP>(smem_u32(ring));
      uint32_t turn = 0;  // parities: bits 0, 1 tiles of a row tile, bits 2, 3 its units, bit 4 the ring
      uint32_t slot = 0;  // ring unit of the next K or V
      bool alive = true;
      auto filled = [&]() { return wait(&bar->full[slot], (turn >> 4) & 1u); };
      auto advance = [&]() {
        if (++slot == NU) {
          slot = 0;
          turn ^= 16u;
        }
      };
      // S = Q K^T for row tile q, its low parts first; O = P V: p_lo v_hi, (quantised)
      // p_hi v_lo, p_hi v_hi, the small ones first
      auto issue_qk = [&](int q, uint32_t kslot, int buf) {
        const uint32_t b = k_desc + kslot * (G::UNIT >> 4), d = tmem + q * 128 + buf * 64;
        const uint32_t hi = q_desc + q * (2 * G::QPART >> 4), lo = hi + (G::QPART >> 4);
        auto at = [](int c, int group) -> uint32_t { return ((c >> 2) * group + (c & 3) * 32) >> 4; };
        mma_ss<false>(d, lo, b, kQK);
#pragma unroll
        for (int c = 1; c < D / 16; ++c) mma_ss<true>(d, lo + at(c, G::GROUP), b + at(c, G::KGROUP), kQK);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) mma_ss<true>(d, hi + at(c, G::GROUP), b + at(c, G::KGROUP), kQK);
        tc::commit(&bar->s_full[q + buf]);
        mbar_arrive(&bar->s_full[q + buf]);
      };
      auto issue_pv = [&](int q, uint32_t vslot) {
        const uint32_t b = v_desc + vslot * (G::UNIT >> 4);
        const uint32_t p = tmem + q * 128 + (ONE ? 128 : 0), o = tmem + 256 + q * D;
        constexpr int KS = KT / 16;
        mma_ts<false>(o, p + 8, b, kPV);
#pragma unroll
        for (int c = 1; c < KS; ++c) mma_ts<true>(o, p + 16 * c + 8, b + c * 128, kPV);
        if constexpr (QUANT) {
#pragma unroll
          for (int c = 0; c < KS; ++c) mma_ts<true>(o, p + 16 * c, b + (KS + c) * 128, kPV);
        }
#pragma unroll
        for (int c = 0; c < KS; ++c) mma_ts<true>(o, p + 16 * c, b + c * 128, kPV);
        tc::commit(&bar->o_full[q]);
        mbar_arrive(&bar->o_full[q]);
      };
      if constexpr (ONE) {
        // QK of a tile, then PV of the tile before, whose softmax ran meanwhile; between
        // units PV first, as the next queries are written after it
        auto qk = [&](uint32_t kslot, int tile) {
          tc::fence_after_sync();
          if (elect_one()) {
            issue_qk(0, kslot, tile & 1);
            tc::commit(&bar->empty[kslot]);
          }
          __syncwarp();
        };
        auto queries = [&]() {
          const bool there = wait(&bar->q_ready[0], (turn >> 2) & 1u);
          turn ^= 4u;
          return there;
        };
        if (mine > 0) {
          alive = filled() && queries();
          if (alive) {
            qk(slot, 0);
            advance();
          }
        }
#pragma unroll 1
        for (int tile = 0; tile < mine && alive; ++tile) {
          const bool more = tile + 1 < mine;
          bool fresh = false;  // the next tile is a unit's first
          uint32_t kslot = 0;
          if (more) {
            alive = filled();
            if (!alive) break;
            kslot = slot;
            advance();
            fresh = __shfl_sync(0xffffffffu, bar->info[(tile + 1) % kInfo].flags, 0) & kFirst;
            if (!fresh) qk(kslot, tile + 1);
          }
          alive = filled() && wait(&bar->p_ready[0], turn & 1u);
          if (!alive) break;
          turn ^= 1u;
          tc::fence_after_sync();
          if (elect_one()) {
            issue_pv(0, slot);
            tc::commit(&bar->empty[slot]);
          }
          __syncwarp();
          advance();
          if (fresh) {
            alive = queries();
            if (alive) qk(kslot, tile + 1);
          }
        }
      }
      // Order: PV of a row tile, then its next QK, while the other's softmax
      // runs. MMAs of one thread run in order, so that QK may overwrite the P
      // that the PV before it reads. Between units both PVs come first: the
      // next queries are written when both row tiles are done.
      uint32_t flags = 0, vslot = 0, kslot = 0;
#pragma unroll 1
      for (int tile = ONE ? mine : -1; tile < mine && mine > 0 && alive; ++tile) {
        const bool more = tile + 1 < mine;
        uint32_t next = 0;
        bool have = false;
        if (tile >= 0) {
          alive = filled();
          if (!alive) break;
          vslot = slot;
          advance();
        }
#pragma unroll 1
        for (int s = tile < 0 ? 1 : 0; s < 4; ++s) {
          // 0 PV of row tile 0, 1 its QK, 2 PV of row tile 1, 3 its QK; between units 0, 2, 1, 3
          if (more && !have && s > 0) {
            alive = filled();
            if (!alive) break;
            kslot = slot;
            advance();
            next = __shfl_sync(0xffffffffu, bar->info[(tile + 1) % kInfo].flags, 0);
            have = true;
          }
          const int op = (next & kFirst) && (s == 1 || s == 2) ? 3 - s : s;
          const int q = op >> 1;
          if ((op & 1) == 0) {  // O = P V
            if (tile < 0) continue;
            const bool does = q == 0 || (flags & kTwo);
            if (does) {
              alive = wait(&bar->p_ready[q], (turn >> q) & 1u);
              if (!alive) break;
              turn ^= 1u << q;
              tc::fence_after_sync();
            }
            if (elect_one()) {
              if (does) {
                issue_pv(q, vslot);
              }
              if (q == 1) tc::commit(&bar->empty[vslot]);  // the last reader of V
            }
            __syncwarp();
          } else if (more) {  // S = Q K^T of the next tile
            const bool does = q == 0 || (next & kTwo);
            if (does) {
              if (next & kFirst) {
                alive = wait(&bar->q_ready[q], (turn >> (2 + q)) & 1u);
                if (!alive) break;
                turn ^= 4u << q;
              }
              tc::fence_after_sync();
            }
            if (elect_one()) {
              if (does) {
                issue_qk(q, kslot, 0);
              }
              if (q == 1) tc::commit(&bar->empty[kslot]);  // the last reader of K
            }
            __syncwarp();
          }
        }
        if (!alive) break;
        flags = next;
      }
      // everything issued has to be done before the tensor memory is freed
      if (elect_one()) tc::commit(&bar->drain);
      __syncwarp();
      mbar_wait(&bar->drain, 0, kDrainWaitNs);
    } else if (warp == 13) {
      // ---- walks the CTA's tiles a few ahead of the loaders ----------------------------
      const long long per = bar->per;
      long long ux = bar->start_x;  // the unit's place among all tiles and starts
      int left = mine;              // tiles from the walk's on
      uint32_t un = 0;
      int k = 0;
      bool alive = true, first = true;
      Work w;
      if (mine > 0) {
        enter<ROWS>(w, P, bar->start_i);
        w.h = bar->start_h;
        w.rt = bar->start_rt;
        w.k0 = bar->start_k;
      }
#pragma unroll 1
      for (uint32_t tile = 0; left > 0; ++tile, --left) {
        if (first) {  // a unit
          unit_tiles<KT, ROWS>(w, a);
          w.k1 = min(w.n, w.k0 + left);
          if (un >= kUnits) alive = wait(&bar->unit_free[un % kUnits], ((un / kUnits) & 1u) ^ 1u);
          if (!alive) break;
          if (lane == 0) {
            UnitInfo& u = bar->units[un % kUnits];
            u.tiles = w.k1 - w.k0;
            u.rho0 = w.rt * ROWS;
            u.rows = w.s.rows * a.group;
            u.row0 = w.s.row0;
            u.pos0 = w.s.len - w.s.rows;
            u.head0 = w.h * a.group;
            u.seq = w.i;
            u.kv_head = w.h;
            const bool whole = w.k0 == 0 && w.k1 == w.n;
            u.c0 = whole ? 0 : static_cast<int>(kv::quotient(ux + G::START, per));
            u.c1 = whole ? 0 : static_cast<int>(kv::quotient(ux + G::START + w.n - 1, per));
            u.slot = 2 * static_cast<int>(blockIdx.x) + (w.k0 == 0 ? 1 : 0);
            mbar_arrive(&bar->unit[un % kUnits]);
          }
          __syncwarp();
          if (un > 0) {  // its queries, towards the softmax threads
#pragma unroll 1
            for (int r = lane; r < ROWS; r += 32) {
              const int rho = w.rt * ROWS + r, token = rho / a.group;
              const float* src = a.Q + (w.s.row0 + token) * a.ldq + static_cast<long long>(w.h * a.group + rho - token * a.group) * D;
              if (P.vec_q && rho < w.s.rows * a.group) bulk_prefetch_l2(src, D * 4);
            }
          }
          ++un;
          k = w.k0;
        }
        const int j0 = (k < w.sink_tiles ? k : w.first + (k - w.sink_tiles)) * KT;
        // pages of the tile's groups of 16 keys, one lane each
        const int key = j0 + lane * 16;
        const int page = lane < KT / 16 ? kv::page_of(a.c, a.b, w.i, key) : -1;
        const uint32_t pages = __ballot_sync(0xffffffffu, page >= 0);
        // A slot is free when every softmax thread is done with its tile. Within a
        // unit that is when the loaders have filled the tile four on: its V took the
        // place of a unit of the ring whose reader came after the next tile's PV,
        // and so after that tile's weights. A unit's last tile has no next one, and
        // the units that follow may leave the second row tile's group without one:
        // there the whole unit has to be done. (Not so for its other tiles: its last
        // PV may wait for the next unit's first keys.)
        if (tile >= kInfo / 2) {
          alive = wait(&bar->done[(tile - kInfo / 2) % kInfo], ((tile - kInfo / 2) / kInfo) & 1u);
          if (!alive) break;
        }
        TileInfo& ti = bar->info[tile % kInfo];
        if (tile >= kInfo) {
          const uint32_t ended = static_cast<uint32_t>(ti.ends);
          if (ti.ends >= 0) alive = wait(&bar->unit_free[ended % kUnits], (ended / kUnits) & 1u);
          if (!alive) break;
          __syncwarp();  // every lane has read it
        }
        if (lane < KT / 16) {
          const int slot = key % a.c.page_size;
          if constexpr (!QUANT) {
            ti.at[lane] = page < 0 ? -1 : (static_cast<long long>(page) * a.c.kv_heads + w.h) * a.c.page_size + slot;
          } else {
            const long long head = page * a.c.page_bytes + w.h * a.c.head_bytes;
            ti.at[2 * lane] = page < 0 ? -1 : head + static_cast<long long>(slot) * G::ROW;
            ti.at[2 * lane + 1] = head + static_cast<long long>(a.c.page_size) * G::ROW + slot * (D / 16);
          }
        }
        if (lane == 0) {
          const bool every = a.window == 0 || j0 > w.p1 - a.window || j0 + KT <= a.sinks;
          uint32_t flags = pages;
          if (w.rt * ROWS + 128 < w.s.rows * a.group) flags |= kTwo;
          if (first) flags |= kFirst;
          if (w.s.rows > 1 && !(j0 + KT - 1 <= w.p0 && every)) flags |= kMixed;
          if (pages == (1u << (KT / 16)) - 1u && j0 + KT - 1 <= w.p1 && (j0 >= w.begin || j0 + KT <= w.sink_end)) flags |= kAll;
          ti.j0 = j0;
          ti.flags = flags;
          ti.p1 = w.p1;
          ti.begin = w.begin;
          ti.sink_end = w.sink_end;
          ti.ends = k + 1 == w.k1 ? static_cast<int>(un) - 1 : -1;
          *reinterpret_cast<uint4*>(bar->bad[tile % kInfo]) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->told[tile % kInfo]);
        first = ++k == w.k1 && left > 1;
        if (first) {
          ux += G::START + w.n;
          if (++w.rt == w.row_tiles) {
            w.rt = 0;
            if (++w.h == a.c.kv_heads) {
              w.h = 0;
              enter<ROWS>(w, P, w.i + 1);
            }
          }
          w.k0 = 0;
        }
      }
      if (alive && un >= kUnits) alive = wait(&bar->unit_free[un % kUnits], ((un / kUnits) & 1u) ^ 1u);
      if (lane == 0) {  // no more units
        bar->units[un % kUnits].tiles = 0;
        mbar_arrive(&bar->unit[un % kUnits]);
      }
    }
  }
  if (!in_time && lane == 0) record_error(kDevErrTimeout);
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

// An f16 pool as rows of head_dim values, in boxes of 16 rows x 64 dims.
bool pool_map(CUtensorMap* map, const void* pool, const kv::Cache& c) {
  const long long rows = static_cast<long long>(c.num_pages) * c.kv_heads * c.page_size;
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_tiled());
  if (!encode || rows < 16 || rows > (1LL << 31) - 1) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim) * 2};
  const cuuint32_t box[2] = {64, 16}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(pool), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  CUtensorMap maps[2];
  std::memset(maps, 0, sizeof(maps));
  TileParams q = p;
  q.tma = FMT == LQ_FMT_F16 && pool_map(&maps[0], p.a.c.k, p.a.c) && pool_map(&maps[1], p.a.c.v, p.a.c);
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tile_kernel<FMT, D>, q, maps[0], maps[1]);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_route(kAttnRouteTile);
  return cuda_status(e);
}

template <int FMT>
lq_status pick(const TileParams& p, int ctas, cudaStream_t stream) {
  switch (p.a.c.head_dim) {
    case 64: return run<FMT, 64>(p, ctas, stream);
    case 128: return run<FMT, 128>(p, ctas, stream);
    default: return run<FMT, 256>(p, ctas, stream);
  }
}

}  // namespace

size_t attn_tile_work_bytes(int head_dim) {
  const int ctas = std::min(std::max(device_info().sm_count, 152), kAttnMaxCtas);
  const int slot = head_dim == 64    ? Geo<LQ_FMT_F16, 64>::SLOT
                   : head_dim == 128 ? Geo<LQ_FMT_F16, 128>::SLOT
                   : head_dim == 256 ? Geo<LQ_FMT_F16, 256>::SLOT
                                     : 0;
  return slot == 0 ? 0 : kAttnCounterBytes + static_cast<size_t>(ctas) * 2 * slot * 4;
}

bool attn_tile_eligible(const AttnArgs& a) {
  const int d = a.c.head_dim;
  return (d == 64 || d == 128 || d == 256) && a.c.page_size % 16 == 0 && aligned_to(a.c.k, 16) && aligned_to(a.c.v, 16) && a.b.batch <= kMaxBatch;
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
  // the default limit of 2 s as cycles of a fast clock; a debugging limit below
  // one millisecond gives up at the first poll that fails
  const unsigned long long ns = wait_limit_ns();
  p.wait_hint = ns < 1000000ull ? 0u : 10000000u;
  p.wait_clocks = ns < 1000000ull ? 0u : static_cast<unsigned>(std::min(ns * 2, 4200000000ull));
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
