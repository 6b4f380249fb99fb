// A tree of drafted tokens: lq_tree_plan, lq_tree_accept.
//
// The tree is given by parents: parent[t] is the number, within its sequence's
// rows, of the row that row t follows; it has to be smaller than t's own, else t
// is a root. So every walk towards a root ends, and the ancestors come in
// descending order.
//
// Plan: one thread a row walks to its root, counts the steps (its depth) and
// writes the bits of its ancestors a word at a time as the walk passes them,
// without any array. It is bound by the walk's chain of loads, so a block brings
// the parents that its rows can come by into shared memory first (sequences of
// up to kNear rows; beyond, they are read where they lie): one sequence of 2000 rows
// and depths of up to 447 takes 62 us, 90 from global memory; 32 of up to 61 take 3.9.
//
// Accept: one warp a sequence. The path starts at row 0; the next row is the
// lowest one behind the last whose parent it is and whose token is what the model
// chose there. Children follow their parents, so one pass over the rows finds the
// whole path, 128 at a time with all that is known of them in registers: 2000 rows
// take 7.9 us, 32 sequences of up to 61 rows 2.2 (a choice that is read after its row is
// known: 14.6 and 3.7).
#include "lq_device.cuh"
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

__device__ unsigned g_tree_err;
__device__ __forceinline__ void record_error(unsigned code) { atomicCAS(&g_tree_err, 0u, code); }

constexpr int kPlanThreads = 128;
constexpr int kNear = 8192;      // parents in shared memory
constexpr int kAcceptGroups = 4; // of 32 rows, asked for together

struct PlanArgs {
  kv::Batch b;
  const int* parent;
  int* positions;  // may be null
  uint32_t* mask;  // may be null
  int words, window, sinks;
};

// The last sequence that begins at or before row t; -1 if t is none's.
__device__ __forceinline__ int sequence_of(const kv::Batch& b, int t) {
  int lo = 0, n = b.batch;
  while (n > 1) {
    const int half = n / 2;
    const bool right = b.q_start[lo + half] <= t;
    lo = right ? lo + half : lo;
    n = right ? n - half : half;
  }
  return b.q_start[lo] <= t && t < b.q_start[lo + 1] ? lo : -1;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int near[kNear];
  __shared__ int lowest;  // the first row that the block's rows can come by
  pdl_wait();
  pdl_launch_dependents();  // the next kernel's launch runs under this one; it waits for its end
  const int t0 = static_cast<int>(blockIdx.x) * kPlanThreads, t = t0 + static_cast<int>(threadIdx.x);
  const int i = t < a.b.tokens ? sequence_of(a.b, t) : -1;
  const int row0 = i >= 0 ? max(a.b.q_start[i], 0) : t;
  if (threadIdx.x == 0) lowest = row0;
  __syncthreads();
  const int from = min(lowest, t0), to = min(t0 + kPlanThreads, a.b.tokens);
  const bool is_near = to - from <= kNear;
  if (is_near) {
#pragma unroll 4
    for (int r = from + static_cast<int>(threadIdx.x); r < to; r += kPlanThreads) near[r - from] = a.parent[r];
  }
  __syncthreads();
  if (i < 0) return;
  const int rows = min(a.b.q_start[i + 1], a.b.tokens) - row0;
  const int base = max(a.b.kv_len[i], 0) - rows, row = t - row0;
  const int* const parent = is_near && row0 >= from ? near + (row0 - from) : a.parent + row0;
  auto above = [&](int r) {  // its parent, or -1
    const int p = LQ_IN_BOUNDS(row0 + r >= 0 && row0 + r < a.b.tokens) ? parent[r] : -1;
    return p < r ? p : -1;
  };
  int depth = 0;
  if (a.window > 0 || !a.mask) {
    for (int r = above(row); r >= 0; r = above(r)) ++depth;
  }
  if (a.mask) {
    uint32_t* const out = a.mask + static_cast<long long>(t) * a.words;
    const int whole = depth;  // (with a window)
    int word = a.words - 1, steps = 0;
    uint32_t bits = 0;
    for (int r = row; r >= 0; r = above(r), ++steps) {
      const int w = r >> 5;
      for (; word > w; --word) {
        out[word] = bits;
        bits = 0;
      }
      const bool see = a.window == 0 || steps < a.window || base + (whole - steps) < a.sinks;
      if (w == word && see) bits |= 1u << (r & 31);  // (w > word: beyond the mask's bits)
    }
    for (; word >= 0; --word) {
      out[word] = bits;
      bits = 0;
    }
    depth = steps - 1;
  }
  if (a.positions) a.positions[t] = base + depth;
}

struct AcceptArgs {
  kv::Batch b;
  const int* parent;
  const int* token;
  const int* target;
  int* keep;  // [batch][most]
  int* count;
  int* next;
  int* kept_len;
  int most;
};

__global__ void __launch_bounds__(32) accept_kernel(const AcceptArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = static_cast<int>(blockIdx.x), lane = static_cast<int>(threadIdx.x);
  const int row0 = min(max(a.b.q_start[i], 0), a.b.tokens), rows = min(max(a.b.q_start[i + 1], row0), a.b.tokens) - row0;
  int* const keep = a.keep + static_cast<long long>(i) * a.most;
  int n = 0, last = -1, chosen = -1;
  if (rows > 0) {
    if (lane == 0) keep[0] = 0;
    n = 1;
    last = 0;
    chosen = a.target[row0];
#pragma unroll 1
    for (int r0 = 0; r0 < rows && n < a.most; r0 += 32 * kAcceptGroups) {
      int parent[kAcceptGroups], token[kAcceptGroups], target[kAcceptGroups];
#pragma unroll
      for (int g = 0; g < kAcceptGroups; ++g) {
        const int r = r0 + g * 32 + lane;
        const bool there = r < rows && LQ_IN_BOUNDS(row0 + r < a.b.tokens);
        parent[g] = there ? a.parent[row0 + r] : -1;
        token[g] = there ? a.token[row0 + r] : 0;
        target[g] = there ? a.target[row0 + r] : 0;
      }
#pragma unroll
      for (int g = 0; g < kAcceptGroups; ++g) {
        while (n < a.most) {
          const int r = r0 + g * 32 + lane;
          const unsigned which = __ballot_sync(0xffffffffu, r > last && r < rows && parent[g] == last && token[g] == chosen);
          if (which == 0u) break;
          const int from = __ffs(static_cast<int>(which)) - 1;
          last = r0 + g * 32 + from;
          chosen = __shfl_sync(0xffffffffu, target[g], from);
          if (lane == 0) keep[n] = last;
          ++n;
        }
      }
    }
  }
  for (int k = n + lane; k < a.most; k += 32) keep[k] = -1;
  if (lane == 0) {
    a.count[i] = n;
    a.next[i] = chosen;
    a.kept_len[i] = max(a.b.kv_len[i], 0) - rows + n;
  }
}

lq_status launch(const void* kernel, unsigned ctas, unsigned threads, void* args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = use_pdl() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* list[1] = {args};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, list);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

}  // namespace

// What both calls need of a batch; its pages and max_q do not matter here.
static lq_status tree_check(const lq_kv_batch* batch, bool* noop) {
  *noop = false;
  if (!batch || batch->batch < 0 || batch->tokens < 0) return LQ_ERR_INVALID_ARG;
  if (batch->tokens > (1LL << 30)) return LQ_ERR_UNSUPPORTED;
  *noop = batch->batch == 0;
  if (*noop) return LQ_OK;
  if (!batch->kv_len || !batch->q_start || !aligned_to(batch->kv_len, 4) || !aligned_to(batch->q_start, 4)) return LQ_ERR_INVALID_ARG;
  return LQ_OK;
}

unsigned read_clear_tree_error() {
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_tree_err, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_tree_err, &zero, sizeof(zero));
  return v;
}

}  // namespace lq

using namespace lq;

extern "C" {

lq_status lq_tree_plan(const lq_kv_batch* batch, const int32_t* parent, int32_t* positions, uint32_t* mask, int64_t mask_words,
                       int64_t window, int64_t sinks, void* stream) {
  bool noop;
  const lq_status st = tree_check(batch, &noop);
  if (st != LQ_OK) return st;
  if (mask_words < 0 || window < 0 || sinks < 0 || (mask && mask_words < 1)) return LQ_ERR_INVALID_ARG;
  if (mask_words > LQ_TREE_MAX_WORDS) return LQ_ERR_UNSUPPORTED;
  if (noop || batch->tokens == 0) return LQ_OK;
  if (!parent || (!positions && !mask) || !aligned_to(parent, 4) || !aligned_to(positions, 4) || !aligned_to(mask, 4))
    return LQ_ERR_INVALID_ARG;
  PlanArgs a = {};
  a.b = kv_batch_view(*batch);
  a.parent = parent;
  a.positions = positions;
  a.mask = mask;
  a.words = static_cast<int>(mask_words);
  const int64_t most = 1LL << 30;
  a.window = static_cast<int>(window < most ? window : most);
  a.sinks = static_cast<int>(sinks < most ? sinks : most);
  const unsigned ctas = static_cast<unsigned>((batch->tokens + kPlanThreads - 1) / kPlanThreads);
  return launch(reinterpret_cast<const void*>(plan_kernel), ctas, kPlanThreads, &a, static_cast<cudaStream_t>(stream));
}

lq_status lq_tree_accept(const lq_kv_batch* batch, const int32_t* parent, const int32_t* token, const int32_t* target, int32_t* keep,
                         int64_t max_keep, int32_t* count, int32_t* next, int32_t* kept_len, void* stream) {
  bool noop;
  const lq_status st = tree_check(batch, &noop);
  if (st != LQ_OK) return st;
  if (max_keep < 1) return LQ_ERR_INVALID_ARG;
  if (max_keep > (1LL << 24)) return LQ_ERR_UNSUPPORTED;
  if (noop) return LQ_OK;
  for (const void* p : {static_cast<const void*>(parent), static_cast<const void*>(token), static_cast<const void*>(target)})
    if ((!p && batch->tokens > 0) || !aligned_to(p, 4)) return LQ_ERR_INVALID_ARG;
  for (const void* p : {keep, count, next, kept_len})
    if (!p || !aligned_to(p, 4)) return LQ_ERR_INVALID_ARG;
  if (kept_len == batch->kv_len) return LQ_ERR_INVALID_ARG;  // the calls that follow need both
  AcceptArgs a = {};
  a.b = kv_batch_view(*batch);
  a.parent = parent;
  a.token = token;
  a.target = target;
  a.keep = keep;
  a.count = count;
  a.next = next;
  a.kept_len = kept_len;
  a.most = static_cast<int>(max_keep);
  return launch(reinterpret_cast<const void*>(accept_kernel), static_cast<unsigned>(batch->batch), 32, &a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
