// Beam search's selection: lq_beam_select.
//
// Mathematics. Of all continuations (beam b, token j) of a group the k best by
//     score_b + (x_bj - lse_b),   lse_b = log sum_j exp(x_bj).
// Within a beam that is the order of x itself, so one pass over the logits gives
// each part of a row its k best logits and its share of the sum, and only those
// candidates ever get a score. lse_b and the scores are held in 64 bits: beams
// are compared across lse's, where f32's steps (5e-7 at 8) would be ties.
//
// The sum. A thread keeps a running maximum M and S = sum 2^(c (x - M)), c = log2(e),
// in f32; x - M is taken first, so that roundings weigh on distances from the maximum
// only (and a row of the type's lowest value is a row like any other). Of the
// terms' errors (2^-22 each) the sum of a vocabulary keeps next to nothing.
//
// The candidates. The k-th largest of the 256 threads' first maxima (16 logits
// each) is at most the part's k-th largest logit: from then on only logits above it
// are noted, in shared memory, a few per cent of k more than are needed. The
// notes hold one round of 4096 logits whatever they are; should they run full
// (rows that grow, rows of one value) the best k are picked and the limit is raised.
// Keys (logit, lower token first) are distinct, so that k of them are well defined and
// the result does not depend on the order in which threads took notes.
//
// Split. A row is cut into parts so that all parts fill the SMs evenly (plan_parts);
// the last part of a group to arrive joins them: the sums of each beam by a
// warp, then k rounds in which the best of all lists' heads is taken.
//
// What bounds it: logits are read once, HBM. An ended beam (one candidate, its score
// as it is) and one with a score of -inf are not read at all.
#include <algorithm>
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
constexpr int kNotes = kRound + 1024;      // room for a round behind what was noted before
constexpr int kSlots = 152 * 4;            // CTAs that the parts are planned for
constexpr int kMaxParts = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTokenBits = 26;             // of a vocabulary

struct BeamArgs {
  const float* logits;
  const float* scores;
  const int* finished;  // may be null
  float* out_scores;
  int* out_parents;
  int* out_tokens;
  int* counters;                // [groups]; zero between calls
  float2* sums;                 // [rows][parts]: M and S
  unsigned long long* lists;    // [rows][parts][k], best first, 0: none
  long long ld;
  int beams, vocab, k, pad, parts, chunk;
};

// A candidate of the join: its score, then (equal scores) the lower beam, the
// larger logit, the lower token. hi 0: none.
struct Pick {
  unsigned long long hi, lo;
};

// Shared memory, first of a part, then of the join.
struct Notes {
  unsigned long long key[kNotes];
  alignas(16) unsigned long long few[kThreads];
  float2 sum[kWarps];
};
struct Join {
  double lse[LQ_BEAM_MAX];
  unsigned char taken[LQ_BEAM_MAX * kMaxParts];  // of a list
  Pick win[2][kWarps];
  int win_list[2][kWarps];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned hi = static_cast<unsigned>(key >> 32);
  return __uint_as_float((hi & 0x80000000u) ? (hi & 0x7FFFFFFFu) : ~hi);
}
// The next float above a finite one.
__device__ __forceinline__ float above(float x) {
  if (x == 0.0f) return __uint_as_float(1u);
  const int i = __float_as_int(x);
  return __int_as_float(x > 0.0f ? i + 1 : i - 1);
}

// The k-th largest of the block's keys, one a thread (distinct or zero); 0 if
// there are fewer. few[] is scratch; every thread takes part.
__device__ __forceinline__ unsigned long long kth_of_block(unsigned long long mine, int k, unsigned long long* few, unsigned long long* out) {
  const int tid = static_cast<int>(threadIdx.x);
  few[tid] = mine;
  if (tid == 0) *out = 0ull;
  __syncthreads();
  int before = 0;
#pragma unroll 8
  for (int j = 0; j < kThreads; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(few + j);
    before += (o.x > mine ? 1 : 0) + (o.y > mine ? 1 : 0);
  }
  if (mine != 0ull && before == k - 1) *out = mine;
  __syncthreads();
  const unsigned long long t = *out;
  __syncthreads();  // few and out are free
  return t;
}

// Leaves the best min(k, n) of the n noted keys, best first, in key[0 .. ).
__device__ __forceinline__ int best_notes(Notes& s, int n, int k) {
  const int tid = static_cast<int>(threadIdx.x);
  __shared__ unsigned long long limit;
  __shared__ int fewer;
  // No more than k threads have a largest key at or above the k-th largest of
  // them, and every one of the best k is at or above it: at most k / 256 of the
  // notes stay, rounded up a thread, so that the loop ends.
  while (n > kThreads) {
    unsigned long long mine = 0ull;
    for (int i = tid; i < n; i += kThreads) mine = s.key[i] > mine ? s.key[i] : mine;
    const unsigned long long least = kth_of_block(mine, k, s.few, &limit);
    // in place: a round of the block's reads lies ahead of its writes
    if (tid == 0) fewer = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const unsigned long long key = i0 + tid < n ? s.key[i0 + tid] : 0ull;
      __syncthreads();
      if (key != 0ull && key >= least) s.key[atomicAdd(&fewer, 1)] = key;
      __syncthreads();
    }
    n = fewer;
    __syncthreads();
  }
  const unsigned long long key = tid < n ? s.key[tid] : 0ull;
  int rank = 0;
  for (int j = 0; j < n; ++j) rank += s.key[j] > key ? 1 : 0;
  __syncthreads();
  if (key != 0ull && rank < k) s.key[rank] = key;
  __syncthreads();
  return min(n, k);
}

__device__ __forceinline__ bool better(const Pick& a, const Pick& b) { return a.hi != b.hi ? a.hi > b.hi : a.lo > b.lo; }
__device__ __forceinline__ Pick pick_of(double score, int beam, unsigned long long key) {
  Pick p = {0ull, 0ull};
  if (!(score > -INFINITY)) return p;  // -inf, NaN
  score += 0.0;                        // -0 as +0
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(score));
  p.hi = (u >> 63) ? ~u : (u | (1ull << 63));
  const unsigned token = 0xFFFFFFFFu - static_cast<unsigned>(key);
  p.lo = (static_cast<unsigned long long>(LQ_BEAM_MAX - 1 - beam) << 58) | ((key >> 32) << kTokenBits) | ((1u << kTokenBits) - 1u - token);
  return p;
}

// The group's k best from the parts' lists, by the whole block.
__device__ void join(const BeamArgs& a, Join& s, int group) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int row0 = group * a.beams, lists = a.beams * a.parts;
  for (int b = warp; b < a.beams; b += kWarps) {
    const bool read = !(a.finished && a.finished[row0 + b] != 0) && a.scores[row0 + b] > -INFINITY;
    double l = 0.0;
    if (read) {
      float2 mine[kMaxParts / 32];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kMaxParts / 32; ++i) {
        const int p = i * 32 + lane;
        mine[i] = p < a.parts ? __ldcg(a.sums + static_cast<long long>(row0 + b) * a.parts + p) : make_float2(-INFINITY, 0.0f);
        top = fmaxf(top, mine[i].x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kMaxParts / 32; ++i)
        if (i * 32 + lane < a.parts) sum += mine[i].y * expf(mine[i].x - base);
      sum = warp_sum(sum);
      l = static_cast<double>(base) + log(static_cast<double>(sum));
    }
    if (lane == 0) s.lse[b] = l;
  }
  for (int i = tid; i < lists; i += kThreads) s.taken[i] = 0;
  __syncthreads();
  auto head = [&](int list, int taken) -> Pick {
    const Pick none = {0ull, 0ull};
    const int b = list / a.parts, part = list - b * a.parts;
    const float score = a.scores[row0 + b];
    if (a.finished && a.finished[row0 + b] != 0) {  // as it is, with the padding token
      if (part != 0 || taken != 0) return none;
      return pick_of(static_cast<double>(score), b, amax::make_key(0.0f, static_cast<unsigned>(a.pad)));
    }
    if (!(score > -INFINITY) || taken >= a.k) return none;
    const unsigned long long key = __ldcg(a.lists + (static_cast<long long>(row0 + b) * a.parts + part) * a.k + taken);
    if (key == 0ull) return none;
    return pick_of(static_cast<double>(score) + (static_cast<double>(value_of(key)) - s.lse[b]), b, key);
  };
  // a thread's lists: tid, tid + 256, ...; the best of their heads
  auto best_here = [&](int& which) {
    Pick p = {0ull, 0ull};
    which = -1;
    for (int i = tid; i < lists; i += kThreads) {
      const Pick c = head(i, s.taken[i]);
      if (better(c, p)) {
        p = c;
        which = i;
      }
    }
    return p;
  };
  int which;
  Pick mine = best_here(which);
  for (int r = 0; r < a.k; ++r) {
    Pick p = mine;
    int list = which;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Pick q;
      q.hi = __shfl_xor_sync(0xffffffffu, p.hi, o);
      q.lo = __shfl_xor_sync(0xffffffffu, p.lo, o);
      const int other = __shfl_xor_sync(0xffffffffu, list, o);
      if (better(q, p)) {
        p = q;
        list = other;
      }
    }
    if (lane == 0) {
      s.win[r & 1][warp] = p;
      s.win_list[r & 1][warp] = list;
    }
    __syncthreads();
    p = s.win[r & 1][0];
    list = s.win_list[r & 1][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      if (better(s.win[r & 1][w], p)) {
        p = s.win[r & 1][w];
        list = s.win_list[r & 1][w];
      }
    }
    const long long out = static_cast<long long>(group) * a.k + r;
    if (tid == 0) {
      const bool none = p.hi == 0ull;
      const unsigned long long u = (p.hi >> 63) ? (p.hi & ~(1ull << 63)) : ~p.hi;
      const double score = __longlong_as_double(static_cast<long long>(u));
      a.out_scores[out] = none ? -INFINITY : static_cast<float>(score);
      a.out_parents[out] = none ? -1 : LQ_BEAM_MAX - 1 - static_cast<int>(p.lo >> 58);
      a.out_tokens[out] = none ? -1 : static_cast<int>(((1u << kTokenBits) - 1u) - static_cast<unsigned>(p.lo & ((1u << kTokenBits) - 1u)));
    }
    if (list >= 0 && list % kThreads == tid) {  // its owner
      ++s.taken[list];
      mine = best_here(which);
    }
  }
}

// grid: x = part + parts * row
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 4) beam_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Notes& s = *reinterpret_cast<Notes*>(raw);
  __shared__ unsigned long long limit;
  __shared__ int last, count;  // count: notes taken
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int row = static_cast<int>(blockIdx.x) / a.parts, part = static_cast<int>(blockIdx.x) - row * a.parts;
  const bool read = !(a.finished && a.finished[row] != 0) && a.scores[row] > -INFINITY;
  if (read) {
    const int c0 = min(part * a.chunk, a.vocab), c1 = min(c0 + a.chunk, a.vocab);
    const float* const x0 = a.logits + row * a.ld;
    float M = -INFINITY, S = 0.0f;
    float lim = -3.402823466e38f;   // logits from here on are noted
    int noted = 0;
    if (tid == 0) count = 0;
#pragma unroll 1
    for (int base = c0; base < c1; base += kRound) {
      float v[kPer];
#pragma unroll
      for (int q = 0; q < kPer / 4; ++q) {
        if constexpr (VEC) {  // (parts begin on multiples of four)
          const int j = base + (q * kThreads + tid) * 4;
          if (j + 3 < c1 && LQ_IN_BOUNDS(j >= 0 && j + 3 < a.vocab)) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(x0 + j));
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * q + i] = j + i < c1 ? x0[j + i] : -INFINITY;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = base + (4 * q + i) * kThreads + tid;
            v[4 * q + i] = j < c1 && LQ_IN_BOUNDS(j >= 0 && j < a.vocab) ? __ldcs(x0 + j) : -INFINITY;
          }
        }
      }
      float top = v[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top = fmaxf(top, v[i]);
      // the sum
      const float to = fmaxf(M, top), ref = to == -INFINITY ? 0.0f : to;
      S *= ex2((M - ref) * kLog2e);
      M = to;
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 y = fmul2(fadd2(make_float2(v[i], v[i + 1]), make_float2(-ref, -ref)), make_float2(kLog2e, kLog2e));
        sum = fadd2(sum, make_float2(ex2(y.x), ex2(y.y)));
      }
      S += sum.x + sum.y;
      // the candidates
      if (base == c0) {
        // (a thread's number tells equal maxima apart)
        const unsigned long long t = kth_of_block(top > -INFINITY ? amax::make_key(top, static_cast<unsigned>(tid)) : 0ull, a.k, s.few, &limit);
        if (t != 0ull) lim = value_of(t);
      } else {
        __syncthreads();  // the count of the round before is whole
        noted = count;
        if (noted + kRound > kNotes) {  // full: the best k stay, and what follows has to beat them all
          __syncthreads();
          noted = best_notes(s, noted, a.k);
          if (noted == a.k) lim = fmaxf(lim, value_of(s.key[a.k - 1]) < INFINITY ? above(value_of(s.key[a.k - 1])) : INFINITY);
          if (tid == 0) count = noted;
        }
        __syncthreads();
      }
      if (top >= lim) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (v[i] >= lim) {
            const int j = VEC ? base + ((i / 4) * kThreads + tid) * 4 + i % 4 : base + i * kThreads + tid;
            const int at = atomicAdd(&count, 1);
            if (LQ_IN_BOUNDS(at < kNotes)) s.key[at] = amax::make_key(v[i], static_cast<unsigned>(j));
          }
        }
      }
    }
    __syncthreads();
    const int n = best_notes(s, c0 < c1 ? count : 0, a.k);
    const long long at = static_cast<long long>(row) * a.parts + part;
    if (tid < a.k) a.lists[at * a.k + tid] = tid < n ? s.key[tid] : 0ull;
    // the block's sum
    float top = M;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    const float w = warp_sum(S * ex2((M - ref) * kLog2e));
    if (lane == 0) s.sum[warp] = make_float2(top, w);
    __syncthreads();
    if (tid == 0) {
      float all = -INFINITY, total = 0.0f;
      for (int i = 0; i < kWarps; ++i) all = fmaxf(all, s.sum[i].x);
      const float r = all == -INFINITY ? 0.0f : all;
      for (int i = 0; i < kWarps; ++i) total += s.sum[i].y * ex2((s.sum[i].x - r) * kLog2e);
      a.sums[at] = make_float2(all, total);
    }
  }
  // the last of the group's parts joins them
  const int group = row / a.beams;
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const int all = a.beams * a.parts, before = atomicAdd(a.counters + group, 1);
    last = before == all - 1;
    if (last) a.counters[group] = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  join(a, *reinterpret_cast<Join*>(raw), group);
}

// Parts of a row: as many as make the CTAs' rounds fewest, counting a CTA's start
// and end as three rounds of its own.
int plan_parts(int64_t rows, int64_t vocab) {
  const int64_t rounds = (vocab + kRound - 1) / kRound;
  int best = 1;
  double least = 1e300;
  for (int64_t p = 1; p <= std::min<int64_t>(rounds, kMaxParts); ++p) {
    const int64_t each = (rounds + p - 1) / p, waves = (rows * p + kSlots - 1) / kSlots;
    const double cost = static_cast<double>(waves) * static_cast<double>(each + 3);
    if (cost < least) {
      least = cost;
      best = static_cast<int>(p);
    }
  }
  return best;
}

bool sizes_fit(int64_t groups, int64_t beams, int64_t vocab, int64_t k) {
  return groups >= 1 && beams >= 1 && beams <= LQ_BEAM_MAX && vocab >= 1 && vocab <= (1LL << kTokenBits) && k >= 1 && k <= LQ_BEAM_MAX &&
         groups * beams <= (1LL << 24);
}
size_t counter_bytes(int64_t groups) { return (static_cast<size_t>(groups) * 4 + 255) / 256 * 256; }

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
  const size_t lists = static_cast<size_t>(groups * beams) * plan_parts(groups * beams, vocab);
  return counter_bytes(groups) + lists * (sizeof(float2) + static_cast<size_t>(k) * 8);
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
  BeamArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.scores = scores;
  a.finished = finished;
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  a.beams = static_cast<int>(beams);
  a.vocab = static_cast<int>(vocab);
  a.k = static_cast<int>(k);
  a.pad = pad;
  const int64_t rows = groups * beams;
  a.parts = plan_parts(rows, vocab);
  a.chunk = static_cast<int>((((vocab + a.parts - 1) / a.parts) + 3) / 4 * 4);
  a.counters = static_cast<int*>(work);
  a.lists = reinterpret_cast<unsigned long long*>(static_cast<char*>(work) + counter_bytes(groups));
  a.sums = reinterpret_cast<float2*>(a.lists + rows * a.parts * k);
  const int64_t ctas = rows * a.parts;
  if (ctas > (1LL << 31) - 1) return LQ_ERR_UNSUPPORTED;
  const bool vec = aligned_to(logits, 16) && ld % 4 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Notes);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static_assert(sizeof(Notes) <= 47 * 1024 && sizeof(Join) <= sizeof(Notes));
  cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? beam_kernel<true> : beam_kernel<false>, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

}  // extern "C"
