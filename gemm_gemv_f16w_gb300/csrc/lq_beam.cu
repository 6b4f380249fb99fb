// Beam search's selection: lq_beam_select.
//
// Mathematics. Of all continuations (beam b, token j) of a group the k best by
//     score_b + (x_bj - lse_b),   lse_b = log sum_j exp(x_bj).
// Within a beam that is the order of x itself, so one pass over the logits gives
// each part of a row its k best logits and its share of the sum, and only those
// candidates ever get a score. lse_b and the scores are held in two f32 parts (48 bits;
// 64-bit arithmetic is slow on this chip and cost the join 1 to 3 us): beams are compared
// across lse's, where f32's steps (5e-7 at 8) would be ties.
//
// The sum. Of a round of 4096 logits each warp has M, its largest, and S = sum 2^(c (x -
// M)), c = log2(e), in f32; x - M is taken first, so that roundings weigh on distances
// from the maximum only (and a row of the type's lowest value is a row like any other).
// The warps' eight make the round's, and the join adds a row's rounds in two f32 parts.
// Which logits are added together, and in which order, is fixed by their places in the
// row alone: equal rows have equal sums and tie, whichever ranges they are dealt to.
// log S is off by less than 2^-18, in units of 2^-24: a term 4 for 2^y and 9 for y
// (2.3 |y| ln 2, and the mean of |y|, weighed by the terms, is at most 5.6 for 512 of them);
// their sum 9, the warps' 10, the rounds' 10, the logarithm 3. (2^-22 at most in rows of 500 to 2^20
// normal logits.)
//
// The candidates. If each of the 8 warps has ceil(k / 8) maxima (of what a thread has
// seen) at or above a limit, k logits of the part are: the least of the warps'
// ceil(k / 8)-th largest maxima, taken in the 1st, 4th, 16th ... round of 4096 logits,
// costs a vote or two (fewer warps where the row is short). Of the 16 logits that a thread has of a round
// only the largest is noted, and only at or above the limit: the k best logits are
// among the 16 of the k best notes (were one in another, k notes would rank above it),
// and those few are read once more when the part ends. Should the notes run full (rows
// that grow, rows of one value) the warps meet, the best k stay and the limit rises.
// Keys (logit, lower token first) are distinct, so that k of them are well defined and
// the result does not depend on the order in which threads took notes.
//
// Split. The rounds of all rows that are read are dealt to the CTAs in equal
// contiguous ranges; a range's part of a row leaves k candidates, and each round (M, S). Each warp
// streams its own 512 logits of a round by asynchronous copies, two rounds ahead and
// across rows, and no warp waits for another but where a limit is taken or a row ends.
// A second kernel, a CTA a group, joins the parts: the sums of each beam by a warp, a
// limit from the lists' first entries, and the best k of what is at or above it. (Joined by the
// last part to arrive instead, whose range then ends late, 32 groups of 8 beams over a
// vocabulary of 151936 take 67 us.)
//
// What bounds it: logits are read once, HBM. 32 groups of 8 beams, a fifth of them ended,
// vocabulary 151936, k 16: 42 us (the parts 34, the join 7; the logits at a copy's rate
// take 23, those of the live beams 19): the parts begin with the look for the rows that
// count and end with a wait for the slowest warp, and the join is a chain of four
// dependent loads and as many barriers. (With one M and S for a range's part of a row, whose
// roundings then go by the range, 41.) One group of 4 beams, k 8: 10.5 us. An ended beam
// (one candidate, its score as it is) and one with a score of -inf are not read at all.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "lq_argmax.cuh"
#include "lq_device.cuh"
#include "lq_internal.h"

namespace lq {
namespace {

__device__ unsigned g_beam_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_beam_err, 0u, code); }

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 16;                   // logits of a thread and round
constexpr int kRound = kThreads * kPer;
constexpr int kStages = 3;                 // rounds in shared memory
constexpr int kStep = kThreads;            // notes that all warps may take between two looks at their number
constexpr int kNotes = 4 * kStep;
constexpr int kCtas = 152 * 3;             // ranges that the rounds are dealt to
constexpr int kScanRows = 4096;            // rows up to which those that are not read are left out of the deal
constexpr int kPicks = 1024;               // candidates that a join ranks together
constexpr int kAtOnce = 2;                 // of a list, in a join
constexpr int kSumsAtOnce = 2;             // of a lane, in a join
constexpr int kSums = 64;                  // rounds whose sums are in shared memory, a warp's each
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTokenBits = 26;             // of a vocabulary

struct BeamArgs {
  const float* logits;
  const float* scores;
  const int* finished;  // may be null
  float* out_scores;
  int* out_parents;
  int* out_tokens;
  int* per;                     // rounds of a range
  int* number;                  // [rows]: of a row among those that are read
  float2* sums;                 // [rows][rounds]: M and S
  unsigned long long* lists;    // [parts][k], best first, 0: none
  long long ld;
  int rows, beams, vocab, k, pad;
  int rounds;                   // of a row
  int scan;                     // the rows that are not read are left out of the deal
};

// A candidate of the join: its score, then (equal scores) the lower beam, the
// larger logit, the lower token. hi 0: none.
struct Pick {
  unsigned long long hi, lo;
};

__device__ __forceinline__ bool better(const Pick& a, const Pick& b) { return a.hi != b.hi ? a.hi > b.hi : a.lo > b.lo; }
__device__ __forceinline__ bool better(unsigned long long a, unsigned long long b) { return a > b; }
__device__ __forceinline__ bool is(const Pick& p) { return p.hi != 0ull; }
__device__ __forceinline__ bool is(unsigned long long k) { return k != 0ull; }

// A number in two parts, the first its value in f32.
struct Pair {
  float hi, lo;
};

// A part's shared memory besides the rounds.
struct Notes {
  unsigned long long key[kNotes];  // the largest of a thread's round
  unsigned long long all[LQ_BEAM_MAX * kPer];  // the logits of the best notes' rounds
  unsigned long long few[kThreads];
  float2 sum[kSums][kWarps];  // M and S of what a warp has of a round
  unsigned limit[kWarps];
};
struct Join {
  Pick pick[kPicks];
  Pick few[kThreads];
  Pair lse[LQ_BEAM_MAX];
  unsigned limit[kWarps];
  float score[LQ_BEAM_MAX], base[LQ_BEAM_MAX];  // base NaN: an ended beam
  int start[LQ_BEAM_MAX + 1], part[LQ_BEAM_MAX];  // lists before a beam's, and its first part
  int count;
};
constexpr int kRing = kStages * kRound * 4;
constexpr int kSmem = kRing + static_cast<int>(sizeof(Notes));

// Rows before row r that are read (s.before: of r / q; q: rows a thread counted).
struct Scan {
  int before[kThreads + 1];
  int warp[kWarps];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of the warp's values, of those that are numbers.
__device__ __forceinline__ float max_of_warp(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned hi = static_cast<unsigned>(key >> 32);
  return __uint_as_float((hi & 0x80000000u) ? (hi & 0x7FFFFFFFu) : ~hi);
}
__device__ __forceinline__ unsigned ordered(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);  // -0 as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// A key's place in the order by its upper 32 bits alone: a float as `ordered` has it.
__device__ __forceinline__ unsigned upper(unsigned long long k) { return static_cast<unsigned>(k >> 32); }
__device__ __forceinline__ unsigned upper(const Pick& p) { return upper(p.hi); }

// The q-th largest (1 <= q <= 32) of the warp's values, one a lane.
__device__ __forceinline__ unsigned nth_of_warp(unsigned x, int q, int lane) {
  unsigned top = __reduce_max_sync(0xffffffffu, x);
#pragma unroll 1
  for (; q > 1; --q) {
    const unsigned holders = __ballot_sync(0xffffffffu, x == top);
    if (lane == __ffs(static_cast<int>(holders)) - 1) x = 0u;  // (taken out; below every float)
    top = __reduce_max_sync(0xffffffffu, x);
  }
  return top;
}

// Leaves the best min(k, n) of n distinct keys, best first, in key[0 .. ), by the
// whole block; few[kThreads] is scratch.
template <class K>
__device__ __noinline__ int best_of(K* key, K* few, int n, int k) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  __shared__ int fewer;
  __shared__ unsigned limit[kWarps];
  // More than 256: each thread's best; with ceil(k / 8) of each warp's at or above a key, k
  // are, and what is below it goes. If too many stay, the k-th of the threads' bests itself
  // is taken: no more than k threads have keys at or above it, at most k / 256 of the keys
  // stay, rounded up a thread, and the loop ends.
  for (int turn = 0; n > kThreads; ++turn) {
    K mine = {};
    for (int i = tid; i < n; i += kThreads) mine = better(key[i], mine) ? key[i] : mine;
    few[tid] = mine;
    const unsigned nth = nth_of_warp(upper(mine), (k + kWarps - 1) / kWarps, lane);
    if (lane == 0) limit[warp] = nth;
    if (tid == 0) fewer = 0;
    __syncthreads();
    unsigned lim = limit[0];
    for (int w = 1; w < kWarps; ++w) lim = min(lim, limit[w]);
    K least = {};
    if (turn > 0) {
      int before = 0;
      for (int j = 0; j < kThreads; ++j) before += better(few[j], mine) ? 1 : 0;
      __syncthreads();
      if (before == k - 1) few[0] = mine;
      __syncthreads();
      least = few[0];
    }
    // in place: a round of the block's reads lies ahead of its writes
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      K x = {};
      if (i0 + tid < n) x = key[i0 + tid];
      __syncthreads();
      if (is(x) && upper(x) >= lim && !better(least, x)) key[atomicAdd(&fewer, 1)] = x;
      __syncthreads();
    }
    n = fewer;
    __syncthreads();
  }
  K x = {};
  int rank = k;
  if (tid < n) {
    x = key[tid];
    rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += better(key[j], x) ? 1 : 0;
  }
  __syncthreads();
  if (rank < k) key[rank] = x;
  __syncthreads();
  return min(n, k);
}

__device__ __forceinline__ Pair sum_of(float a, float b) {  // exactly
  const float t = a + b, v = t - a;
  return {t, (a - (t - v)) + (b - v)};
}
__device__ __forceinline__ Pair sum_of(const Pair& a, float b) {
  const Pair t = sum_of(a.hi, b);
  return sum_of(t.hi, t.lo + a.lo);
}
__device__ __forceinline__ Pair sum_of(const Pair& a, const Pair& b) {
  const Pair t = sum_of(a.hi, b.hi);
  return sum_of(t.hi, t.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Pick pick_of(const Pair& score, int beam, unsigned long long key) {
  Pick p = {0ull, 0ull};
  if (!(fabsf(score.hi) < INFINITY)) return p;
  p.hi = static_cast<unsigned long long>(ordered(score.hi)) << 32 | ordered(score.lo);
  const unsigned token = 0xFFFFFFFFu - static_cast<unsigned>(key);
  p.lo = (static_cast<unsigned long long>(LQ_BEAM_MAX - 1 - beam) << 58) | ((key >> 32) << kTokenBits) | ((1u << kTokenBits) - 1u - token);
  return p;
}

__device__ __forceinline__ bool is_read(const BeamArgs& a, int row) {
  return a.scores[row] > -INFINITY && !(a.finished && a.finished[row] != 0);
}

// Logits above `value` are noted, and those equal to it whose tokens are below `token`.
struct Limit {
  float value;
  int token;
};
// The notes are full, or this warp has taken all of its own (done): the warps meet until
// none has more. The best k stay; what follows has to rank above the least of them. (Not
// inlined, so that all warps meet at one and the same barrier.)
__device__ __noinline__ bool meet_warps(Notes& s, int& count, int k, bool done, Limit& limit) {
  if (!__syncthreads_or(!done)) return false;
  const int kept = best_of(s.key, s.few, count, k);
  if (kept == k) {
    limit.value = value_of(s.key[k - 1]);
    limit.token = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned>(s.key[k - 1]));
  }
  if (threadIdx.x == 0) count = kept;
  __syncthreads();
  return true;
}

// How the rounds are dealt: CTA c has rounds [c per, (c + 1) per) of the rows that are
// read, in order; the part of the l-th such row that CTA c has is number l + c.
struct Deal {
  int per, rounds;
  __device__ __forceinline__ int cta_of(long long x) const {  // (the 32-bit division where it will do)
    return (x >> 31) == 0 ? static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(per)) : static_cast<int>(x / per);
  }
  __device__ __forceinline__ int first_cta(int l) const { return cta_of(static_cast<long long>(l) * rounds); }
  __device__ __forceinline__ int last_cta(int l) const { return cta_of(static_cast<long long>(l) * rounds + rounds - 1); }
};

// The group's k best from its parts' lists.
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamArgs a) {
  __shared__ Join s;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int group = static_cast<int>(blockIdx.x), row0 = group * a.beams;
  if (warp == 0) {  // two beams a lane
    int n[2], before = 0;
    Deal deal;
    deal.per = __ldcg(a.per);
    deal.rounds = a.rounds;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = 2 * lane + h;
      n[h] = 0;
      if (b < a.beams) {
        const float score = a.scores[row0 + b];
        const int ended = a.finished ? a.finished[row0 + b] : 0;
        const int l = __ldcg(a.number + row0 + b);  // (of a row that is read; asked for with the others)
        s.score[b] = score;
        if (ended != 0) {
          s.base[b] = NAN;  // its logits give no candidate
        } else if (!a.scan || score > -INFINITY) {
          const int c0 = deal.first_cta(l);
          s.part[b] = l + c0;
          n[h] = deal.last_cta(l) - c0 + 1;
          s.base[b] = 0.0f;
        }
      }
      before += n[h];
    }
    int incl = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    s.start[2 * lane] = incl - before;
    s.start[2 * lane + 1] = incl - before + n[0];
    if (lane == 31) s.start[LQ_BEAM_MAX] = incl;
    if (lane == 0) s.count = 0;
  }
  __syncthreads();
  const int lists = s.start[LQ_BEAM_MAX];
  auto beam_of = [&](int list) {
    int b = 0;
#pragma unroll 1
    for (int step = LQ_BEAM_MAX / 2; step > 0; step /= 2)
      if (b + step < a.beams && s.start[b + step] <= list) b += step;
    return b;
  };
  auto key_of = [&](int list, int b, int at) {
    return at < a.k ? __ldcg(a.lists + static_cast<long long>(s.part[b] + list - s.start[b]) * a.k + at) : 0ull;
  };
  // The first entries of the lists, one a thread and as many of each list as there are
  // threads for (a warp's are of every eighth place: beams that are far ahead are in every
  // warp), and the next ones of a thread's own list: asked for before the sums.
  const int m = lists > 0 ? max(1, min(a.k, kThreads / lists)) : 1, place = lane * kWarps + warp, mine = place / m;
  const int covered = kThreads / m, mine_beam = mine < lists ? beam_of(mine) : 0, own_beam = tid < lists ? beam_of(tid) : 0;
  const unsigned long long mine_key = mine < min(lists, covered) ? key_of(mine, mine_beam, place - mine * m) : 0ull;
  unsigned long long key[kAtOnce];
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) key[i] = tid < lists ? key_of(tid, own_beam, (tid < covered ? m : 0) + i) : 0ull;
#pragma unroll 1
  for (int b = warp; b < a.beams; b += kWarps) {
    if (s.start[b + 1] == s.start[b]) continue;  // not read
    const float2* const sums = a.sums + static_cast<long long>(row0 + b) * a.rounds;
    float top = -INFINITY;
    Pair sum = {0.0f, 0.0f};
#pragma unroll 1
    for (int i0 = lane; i0 < a.rounds; i0 += 32 * kSumsAtOnce) {
      float2 m[kSumsAtOnce];
      float to = top;
#pragma unroll
      for (int i = 0; i < kSumsAtOnce; ++i) m[i] = i0 + 32 * i < a.rounds ? __ldcg(sums + i0 + 32 * i) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int i = 0; i < kSumsAtOnce; ++i) to = fmaxf(to, m[i].x);
      const float ref = to == -INFINITY ? 0.0f : to, less = expf(top - ref);
      sum.hi = __fmul_rn(sum.hi, less);
      sum.lo = __fmul_rn(sum.lo, less);
#pragma unroll
      for (int i = 0; i < kSumsAtOnce; ++i) sum = sum_of(sum, __fmul_rn(m[i].y, expf(m[i].x - ref)));
      top = to;
    }
    const float all = max_of_warp(top), ref = all == -INFINITY ? 0.0f : all, less = expf(top - ref);
    sum.hi = __fmul_rn(sum.hi, less);
    sum.lo = __fmul_rn(sum.lo, less);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Pair other = {__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)};
      sum = sum_of(sum, other);
    }
    // log sum: f32's logarithm, and by how much it misses the sum
    const float l = logf(sum.hi), part = expf(-l), miss = fmaf(sum.hi, part, -1.0f) + sum.lo * part;
    if (lane == 0) {
      const Pair all_of = sum_of(sum_of(ref, l), miss);
      s.lse[b] = s.base[b] != s.base[b] ? Pair{NAN, 0.0f} : all_of;
    }
  }
  __syncthreads();
  auto scored = [&](unsigned long long key, int b) {
    const Pick none = {0ull, 0ull};
    if (key == 0ull) return none;
    const Pair d = sum_of(value_of(key), -s.lse[b].hi), t = sum_of(s.score[b], d.hi);
    return pick_of(sum_of(t, d.lo - s.lse[b].lo), b, key);
  };
  // ended beams: one candidate each
  if (tid < a.beams && s.base[tid] != s.base[tid]) {
    const Pick p = pick_of(Pair{s.score[tid], 0.0f}, tid, amax::make_key(0.0f, static_cast<unsigned>(a.pad)));
    if (is(p)) s.pick[atomicAdd(&s.count, 1)] = p;
  }
  // A limit: with ceil(k / 8) of each warp's entries at or above it, k are.
  const Pick p = scored(mine_key, mine_beam);
  const unsigned nth = nth_of_warp(upper(p), (a.k + kWarps - 1) / kWarps, lane);
  if (lane == 0) s.limit[warp] = nth;
  __syncthreads();
  unsigned limit = s.limit[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) limit = min(limit, s.limit[w]);
  limit = max(limit, 1u);  // (scores' own are above it)
  if (upper(p) >= limit) s.pick[atomicAdd(&s.count, 1)] = p;
  // The lists are sorted: a thread goes down the rest of each of its own until it is below.
#pragma unroll 1
  for (int i0 = 0; i0 < lists; i0 += kThreads) {
    const int list = i0 + tid, at0 = list < covered ? m : 0;
    bool on = list < lists;
    const int b = i0 == 0 ? own_beam : (on ? beam_of(list) : 0);
#pragma unroll 1
    for (int at = 0; at < a.k; at += kAtOnce) {
      if (i0 + at > 0) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) key[i] = on ? key_of(list, b, at0 + at + i) : 0ull;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const Pick x = scored(key[i], b);
        on = on && upper(x) >= limit;
        if (on) {
          const int to = atomicAdd(&s.count, 1);
          if (LQ_IN_BOUNDS(to < kPicks)) s.pick[to] = x;
        }
      }
      const bool more = __syncthreads_or(on);
      const int have = s.count;
      __syncthreads();  // everyone has read it
      if (have > kPicks - kAtOnce * kThreads) {
        const int kept = best_of(s.pick, s.few, have, a.k);
        if (tid == 0) s.count = kept;
        __syncthreads();
      }
      if (!more) break;
    }
  }
  __syncthreads();
  const int n = best_of(s.pick, s.few, s.count, a.k);
  if (tid < a.k) {
    const long long out = static_cast<long long>(group) * a.k + tid;
    const bool some = tid < n;
    const Pick x = s.pick[some ? tid : 0];
    constexpr unsigned kTokens = (1u << kTokenBits) - 1u;
    a.out_scores[out] = some ? value_of(x.hi) : -INFINITY;
    a.out_parents[out] = some ? LQ_BEAM_MAX - 1 - static_cast<int>(x.lo >> 58) : -1;
    a.out_tokens[out] = some ? static_cast<int>(kTokens - (static_cast<unsigned>(x.lo) & kTokens)) : -1;
  }
}

// 16 (or 4) bytes; what is beyond `bytes` is zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3) beam_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Notes& s = *reinterpret_cast<Notes*>(raw + kRing);
  __shared__ Scan scan;
  __shared__ int count;  // notes taken
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const int R = a.rounds;

  // ---- the rows that are read, and this CTA's range of their rounds -----------------
  const int q = a.scan ? (a.rows + kThreads - 1) / kThreads : 1;
  int live = a.rows;
  if (a.scan) {
    int mine = 0;
    for (int r = tid * q; r < min(tid * q + q, a.rows); ++r) mine += is_read(a, r) ? 1 : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan.warp[warp] = incl;
    __syncthreads();
    live = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) incl += live;
      live += scan.warp[w];
    }
    scan.before[tid + 1] = incl;
    if (tid == 0) scan.before[0] = 0;
    __syncthreads();
  }
  auto is_live = [&](int r) { return !a.scan || is_read(a, r); };
  Deal deal;
  deal.rounds = R;
  deal.per = static_cast<int>(max((static_cast<long long>(live) * R + ctas - 1) / ctas, 1ll));
  if (cta == 0 && tid == 0) *a.per = deal.per;
  const long long x0 = static_cast<long long>(cta) * deal.per, x1 = min(x0 + deal.per, static_cast<long long>(live) * R);
  if (x0 >= x1) return;
  int number = static_cast<int>(x0 / R), round = static_cast<int>(x0 - static_cast<long long>(number) * R);  // of the row; in it
  int row = number;
  if (a.scan) {  // the number-th row that is read
    int at = 0;
    for (int step = kThreads / 2; step > 0; step /= 2)
      if (scan.before[at + step] <= number) at += step;
    row = at * q;
    for (int skip = number - scan.before[at];; ++row)
      if (is_read(a, row) && skip-- == 0) break;
  }
  int left = static_cast<int>(x1 - x0);

  // ---- copies, ahead of the work -------------------------------------------------------
  float* const ring = reinterpret_cast<float*>(raw) + warp * (kRound / kWarps);
  int copy_row = row, copy_round = round, copy_left = left, copy_stage = 0;
  auto copy = [&]() {
    if (copy_left > 0) {
      const int base = copy_round * kRound + warp * (kRound / kWarps);
      const float* const from = a.logits + copy_row * a.ld;
      const uint32_t to = smem_u32(ring + copy_stage * kRound);
      const int inside = a.vocab - base;  // logits of the row from there on
#pragma unroll
      for (int n = 0; n < (VEC ? kPer / 4 : kPer); ++n) {
        const int e = VEC ? (n * 32 + lane) * 4 : n * 32 + lane;
        const int bytes = max(0, min(inside - e, VEC ? 4 : 1)) * 4;
        const float* const at = bytes > 0 && LQ_IN_BOUNDS(copy_row >= 0 && copy_row < a.rows) ? from + base + e : a.logits;
        if constexpr (VEC) {
          copy16(to + e * 4, at, bytes);
        } else {
          copy4(to + e * 4, at, bytes);
        }
      }
      --copy_left;
      if (++copy_round == R) {
        copy_round = 0;
        ++copy_row;
        if (copy_left > 0)
          while (!is_live(copy_row)) ++copy_row;
      }
      copy_stage = copy_stage + 1 == kStages ? 0 : copy_stage + 1;
    }
    commit_copies();
  };
#pragma unroll
  for (int n = 0; n < kStages - 1; ++n) copy();

  int stage = 0;
  // ---- the parts of rows ------------------------------------------------------------------
#pragma unroll 1
  while (left > 0) {
    if (tid == 0) {
      count = 0;
      a.number[row] = number;
    }
    __syncthreads();
    const int rounds = min(R - round, left);  // here
    float highest = -INFINITY;
    float lim = -3.402823466e38f;     // logits above are noted, and those equal to it
    int lim_token = 1 << kTokenBits;  // whose tokens are below this one
    auto meet = [&](bool done) {
      Limit limit = {lim, lim_token};
      const bool more = meet_warps(s, count, a.k, done, limit);
      lim = limit.value;
      lim_token = limit.token;
      return more;
    };
    // The warps' sums of n rounds, the last of them round `last`, become the rounds'. (No
    // fused operation: the compiler might form it in one place and not in another.)
    auto add_warps = [&](int n, int last) {
      if (tid >= n) return;
      const float2* const of = s.sum[tid];
      float all = of[0].x, term[kWarps];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = fmaxf(all, of[w].x);
      const float ref = all == -INFINITY ? 0.0f : all;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) term[w] = __fmul_rn(of[w].y, ex2((of[w].x - ref) * kLog2e));
#pragma unroll
      for (int half = kWarps / 2; half > 0; half /= 2)
#pragma unroll
        for (int w = 0; w < half; ++w) term[w] += term[w + half];
      a.sums[static_cast<long long>(row) * R + (last - n + 1 + tid)] = make_float2(all, term[0]);
    };
    int next_limit = 0;
#pragma unroll 1
    for (int i = 0; i < rounds; ++i, ++round) {
      if (i > 0 && i % kSums == 0) {
        while (meet(true)) {
        }
        add_warps(kSums, round - 1);
        __syncthreads();
      }
      wait_copies<kStages - 2>();
      if constexpr (!VEC) __syncwarp();  // what other lanes have copied
      float v[kPer];
      const float* const at = ring + stage * kRound;
#pragma unroll
      for (int n = 0; n < kPer / 4; ++n) {
        const float4 f = *reinterpret_cast<const float4*>(at + (n * 32 + lane) * 4);
        v[4 * n] = f.x;
        v[4 * n + 1] = f.y;
        v[4 * n + 2] = f.z;
        v[4 * n + 3] = f.w;
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
      copy();
      const int base = round * kRound + warp * (kRound / kWarps);  // token of the warp's first
      if (base + kRound / kWarps > a.vocab) {
#pragma unroll
        for (int n = 0; n < kPer; ++n)
          if (base + ((n / 4) * 32 + lane) * 4 + n % 4 >= a.vocab) v[n] = -INFINITY;
      }
      float top = v[0];
#pragma unroll
      for (int n = 1; n < kPer; ++n) top = fmaxf(top, v[n]);
      // the sum
      const float whole = max_of_warp(top), ref = whole == -INFINITY ? 0.0f : whole;
      float2 term[kPer / 2];
#pragma unroll
      for (int n = 0; n < kPer / 2; ++n) {
        const float2 y = fmul2(fadd2(make_float2(v[2 * n], v[2 * n + 1]), make_float2(-ref, -ref)), make_float2(kLog2e, kLog2e));
        term[n] = make_float2(ex2(y.x), ex2(y.y));
      }
#pragma unroll
      for (int half = kPer / 4; half > 0; half /= 2)
#pragma unroll
        for (int n = 0; n < half; ++n) term[n] = fadd2(term[n], term[n + half]);
      const float sum = warp_sum(term[0].x + term[0].y);
      if (lane == 0) s.sum[i % kSums][warp] = make_float2(whole, sum);
      // the candidates
      highest = fmaxf(highest, top);
      if (i == next_limit) {
        while (i > 0 && meet(true)) {
        }
        // (of the warps that have logits: a row may end within its first round)
        const int warps = i > 0 ? kWarps : max(1, min(kWarps, (a.vocab - round * kRound + kRound / kWarps - 1) / (kRound / kWarps)));
        const int of_each = (a.k + warps - 1) / warps;
        const unsigned nth = nth_of_warp(ordered(highest), min(of_each, 32), lane);
        if (lane == 0) s.limit[warp] = nth;
        __syncthreads();
        unsigned lowest = s.limit[0];
        for (int w = 1; w < warps; ++w) lowest = min(lowest, s.limit[w]);
        const float least = of_each <= 32 ? value_of(static_cast<unsigned long long>(lowest) << 32) : -INFINITY;
        if (least > lim) {
          lim = least;
          lim_token = 1 << kTokenBits;
        }
        next_limit = 4 * i + 3;
      }
      if (whole >= lim) {
        // (eight warps take no more than kStep notes between this and their next looks)
        while (__shfl_sync(0xffffffffu, *static_cast<volatile int*>(&count), 0) > kNotes - kStep) meet(false);
        if (top >= lim) {
          int n = kPer - 1;  // the first of the largest
#pragma unroll
          for (int m = kPer - 2; m >= 0; --m) n = v[m] == top ? m : n;
          const int j = base + ((n / 4) * 32 + lane) * 4 + n % 4;
          if (top > lim || j < lim_token) {
            const int to_note = atomicAdd(&count, 1);
            if (LQ_IN_BOUNDS(to_note < kNotes)) s.key[to_note] = amax::make_key(top, static_cast<unsigned>(j));
          }
        }
        __syncwarp();
      }
    }
    left -= rounds;
    while (meet(true)) {
    }
    add_warps((rounds - 1) % kSums + 1, round - 1);
    const int notes = best_of(s.key, s.few, count, a.k);  // (a barrier, too)
    if (tid == 0) count = 0;
    __syncthreads();
    // the logits of the notes' rounds that are no worse than the last note
    const unsigned long long least = notes == a.k ? s.key[a.k - 1] : 1ull;
    for (int e = tid; e < notes * kPer; e += kThreads) {
      const int j = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned>(s.key[e / kPer])), n = e % kPer;
      const int within = j % (kRound / kWarps), first = j - within;  // of the warp's 512
      const int token = first + (n / 4) * 128 + within % 128 / 4 * 4 + n % 4;
      if (token >= a.vocab || !LQ_IN_BOUNDS(token >= 0)) continue;
      const float x = a.logits[row * a.ld + token];
      const unsigned long long key = x > -INFINITY ? amax::make_key(x, static_cast<unsigned>(token)) : 0ull;
      if (key >= least) {
        const int to = atomicAdd(&count, 1);
        if (LQ_IN_BOUNDS(to < LQ_BEAM_MAX * kPer)) s.all[to] = key;
      }
    }
    __syncthreads();
    const int n = best_of(s.all, s.few, count, a.k);
    const int part = number + cta;
    if (tid < a.k) a.lists[static_cast<long long>(part) * a.k + tid] = tid < n ? s.all[tid] : 0ull;
    __syncthreads();  // the notes are free
    if (round == R && left > 0) {
      round = 0;
      ++number;
      do ++row;
      while (!is_live(row));
    }
  }
}

int64_t row_rounds(int64_t vocab) { return (vocab + kRound - 1) / kRound; }
bool sizes_fit(int64_t groups, int64_t beams, int64_t vocab, int64_t k) {
  return groups >= 1 && beams >= 1 && beams <= LQ_BEAM_MAX && vocab >= 1 && vocab <= (1LL << kTokenBits) && k >= 1 && k <= LQ_BEAM_MAX &&
         groups * beams <= (1LL << 24);
}
size_t number_bytes(int64_t rows) { return (static_cast<size_t>(rows + 1) * 4 + 15) / 16 * 16; }

}  // namespace

unsigned read_clear_beam_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_beam_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_beam_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

size_t lq_beam_work_bytes(int64_t groups, int64_t beams, int64_t vocab, int64_t k) {
  if (groups < 1 || groups > (1LL << 24) || !sizes_fit(groups, beams, vocab, k)) return 0;
  const size_t lists = static_cast<size_t>(groups * beams) + kCtas;  // a part ends where a row or a range does
  return number_bytes(groups * beams) + lists * static_cast<size_t>(k) * 8 +
         static_cast<size_t>(groups * beams) * static_cast<size_t>(row_rounds(vocab)) * sizeof(float2);
}

lq_status lq_beam_select(const float* logits, int64_t ld, const float* scores, int64_t groups, int64_t beams, int64_t vocab, int64_t k,
                         const int32_t* finished, int32_t pad, float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* work,
                         void* stream) {
  if (groups < 0 || beams < 1 || vocab < 1 || k < 1 || ld < vocab) return LQ_ERR_INVALID_ARG;
  if (finished && (pad < 0 || pad >= vocab)) return LQ_ERR_INVALID_ARG;
  if (groups > (1LL << 24)) return LQ_ERR_UNSUPPORTED;
  if (groups == 0) return LQ_OK;
  if (!sizes_fit(groups, beams, vocab, k)) return LQ_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(scores), static_cast<const void*>(out_scores),
                        static_cast<const void*>(out_parents), static_cast<const void*>(out_tokens)})
    if (!p || !aligned_to(p, 4)) return LQ_ERR_INVALID_ARG;
  if (!work || !aligned_to(work, 16) || !aligned_to(finished, 4)) return LQ_ERR_INVALID_ARG;
  // a group's scores are read before its results are written, which are in their place
  // only where there are as many
  const uintptr_t in = reinterpret_cast<uintptr_t>(scores), out = reinterpret_cast<uintptr_t>(out_scores);
  if (in < out + groups * k * sizeof(float) && out < in + groups * beams * sizeof(float) && !(in == out && k == beams)) return LQ_ERR_INVALID_ARG;
  BeamArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.scores = scores;
  a.finished = finished;
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  const int64_t rows = groups * beams;
  a.rows = static_cast<int>(rows);
  a.beams = static_cast<int>(beams);
  a.vocab = static_cast<int>(vocab);
  a.k = static_cast<int>(k);
  a.pad = pad;
  a.rounds = static_cast<int>(row_rounds(vocab));
  a.scan = rows <= kScanRows;
  a.per = static_cast<int*>(work);
  a.number = a.per + 1;
  a.lists = reinterpret_cast<unsigned long long*>(static_cast<char*>(work) + number_bytes(rows));
  a.sums = reinterpret_cast<float2*>(a.lists + (rows + kCtas) * k);
  const int64_t ctas = std::min<int64_t>(rows * a.rounds, kCtas);
  const bool vec = aligned_to(logits, 16) && ld % 4 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<bool> ready[2][kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return LQ_ERR_CUDA;
  void (*const kernel)(BeamArgs) = vec ? beam_kernel<true> : beam_kernel<false>;
  if (!ready[vec][dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
      cudaGetLastError();
      return LQ_ERR_CUDA;
    }
    ready[vec][dev].store(true);
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  cfg.gridDim = dim3(static_cast<unsigned>(groups));
  cfg.dynamicSmemBytes = 0;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, beam_join_kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

}  // extern "C"
