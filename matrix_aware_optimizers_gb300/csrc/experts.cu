// Routing of an expert layer: scores and choice of experts, the plan of the copies' places,
// the combination of the experts' outputs, and the gradients.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "experts.h"
#include "internal.h"

namespace mao {
namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// Unsigned integers in the order of the floats; 0 for -inf and NaN, which are never chosen.
__device__ __forceinline__ uint32_t order_of(float key) {
  if (!(key > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(key + 0.0f);  // -0 counts as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// ------------------------------------------------------------------ choice of experts
//
// One warp per token; lane l holds experts 32 i + l. The softmax is one maximum, one sum. Keys
// are compared as ordered integers.
//
// The instructions bound it (1097 per token of 256 experts in 8 runs with sigmoid scores and a bias,
// 89% of the issue slots), not its 17 MB: 16,384 tokens take 17.7 us in a graph of calls, and 12.4 with
// softmax scores and neither bias nor runs. The gradient takes 6.6 us for sigmoid scores, of which it
// reads only the chosen logits, and 8.6 for softmax. Choosing the best one by one over all keys took
// 35 us against 20 (both with a filled L2).

constexpr int ROUTE_WARPS = 4;

template <int VPL>
__device__ __forceinline__ void load_logits(const void* base, int64_t row, int64_t ld, int dtype,
                                            int experts, int lane, float (&x)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    x[i] = e < experts ? load_elem(base, row * ld + e, dtype) : -INFINITY;
  }
}

// Scores of a token's experts from its logits (softmax over the warp, or sigmoid).
template <int VPL>
__device__ __forceinline__ void scores_of(const float (&x)[VPL], int score, float (&p)[VPL]) {
  if (score == MAO_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = __fdividef(1.0f, 1.0f + expf(-x[i]));
    // the quotient is within 4 units in the last place, but 0 once its divisor passes 2^126: from
    // x = -87.4 down the score is e^x
    bool low = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) low = low || (p[i] == 0.0f && x[i] > -INFINITY);
    if (low) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (p[i] == 0.0f) p[i] = expf(x[i]);
    }
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;  // every expert masked: all scores 0
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    p[i] = expf(x[i] - m);
    sum += p[i];
  }
  sum = warp_sum(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < VPL; ++i) p[i] *= inv;
}

// Lane j's j-th best key of the warp (its index, or -1 where none is left). At least top_k
// lanes hold a key that is no smaller than the top_k-th largest of the lanes' largest keys, so
// only keys from there on can be chosen: usually about top_k of them, which are ranked against
// one another, one to a lane. With more than 32 (many ties) the best are taken one by one.
// `scratch`: 64 words of shared memory.
template <int VPL>
__device__ __forceinline__ int best_of(uint32_t (&u)[VPL], int top_k, int lane, float* scratch) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = max(m, u[i]);
  uint32_t least = 0u;
  for (int j = 0; j < top_k; ++j) {
    const uint32_t top = __reduce_max_sync(FULL, m);
    if (top == 0u) {  // fewer than top_k lanes hold anything: every key counts
      least = 1u;
      break;
    }
    least = top;
    if (m == top) m = 0u;
  }
  __syncwarp();
  uint2* list = reinterpret_cast<uint2*>(scratch);
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t who = __ballot_sync(FULL, u[i] >= least);
    if (u[i] >= least) {
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (at < 32) list[at] = make_uint2(u[i], uint32_t(32 * i + lane));
    }
    n += __popc(who);
  }
  __syncwarp();
  int id = -1;
  if (n <= 32) {
    // listed by rising index, so of equal keys the one listed first is better
    const uint2 mine = lane < n ? list[lane] : make_uint2(0u, 0u);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t o = __shfl_sync(FULL, mine.x, j);
      rank += (o > mine.x || (o == mine.x && j < lane)) ? 1 : 0;
    }
    __syncwarp();
    int* place = reinterpret_cast<int*>(scratch);
    if (lane < n) place[rank] = int(mine.y);
    __syncwarp();
    if (lane < n && lane < top_k) id = place[lane];
    return id;
  }
  for (int j = 0; j < top_k; ++j) {
    uint32_t best = 0u;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (u[i] > best) {
        best = u[i];
        at = 32 * i + lane;
      }
    const uint32_t top = __reduce_max_sync(FULL, best);
    if (top == 0u) break;
    const int e = __reduce_min_sync(FULL, best == top ? at : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (32 * i + lane == e) u[i] = 0u;
    if (lane == j) id = e;
  }
  return id;
}

template <int VPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_kernel(const RouteParams p) {
  extern __shared__ float sm[];
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + warp;
  if (t >= p.tokens) return;
  float* score_sm = sm + warp * 2 * 32 * VPL;
  float* key_sm = score_sm + 32 * VPL;
  float x[VPL], s[VPL];
  load_logits<VPL>(p.logits, t, p.ld, p.dtype, p.experts, lane, x);
  scores_of<VPL>(x, p.score, s);
  uint32_t u[VPL];
  const bool plain = !p.bias && p.groups == 1;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    float key = plain ? x[i] : s[i];
    if (p.bias && e < p.experts) key += p.bias[e];
    if (!(x[i] > -INFINITY)) key = -INFINITY;
    score_sm[e] = s[i];
    u[i] = order_of(key);
    if (p.groups > 1) key_sm[e] = u[i] ? key : -INFINITY;
  }
  __syncwarp();
  if (p.groups > 1) {
    // `per` lanes score a run together, each every per-th key from a place of its own, so
    // that the lanes' reads spread over the banks
    const int size = p.experts / p.groups;
    const int shift = 31 - __clz(32 / p.groups), per = 1 << shift;
    const int g = lane >> shift, sub = lane & (per - 1);
    float first = -INFINITY, second = -INFINITY;
    if (g < p.groups) {
      const int mine = (size - sub + per - 1) >> shift;  // keys of this lane
      const float* run = key_sm + g * size + sub;
      int at = g < mine ? g : 0;
      for (int i = 0; i < mine; ++i) {
        const float k = run[at << shift];
        at = at + 1 == mine ? 0 : at + 1;
        second = fmaxf(second, fminf(first, k));
        first = fmaxf(first, k);
      }
    }
    for (int o = per >> 1; o; o >>= 1) {
      const float f = __shfl_xor_sync(FULL, first, o), s2 = __shfl_xor_sync(FULL, second, o);
      second = fmaxf(fmaxf(second, s2), fminf(first, f));
      first = fmaxf(first, f);
    }
    float run = first;
    if (p.group_score == MAO_GROUP_TOP2 && second > -INFINITY) run += second;
    const uint32_t ru = order_of(run);
    int better = 0;  // runs ahead of run `lane`
    const uint32_t my = __shfl_sync(FULL, ru, (lane << shift) & 31);
    for (int h = 0; h < p.groups; ++h) {
      const uint32_t o = __shfl_sync(FULL, ru, h << shift);
      better += (o > my || (o == my && h < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(FULL, lane < p.groups && better < p.keep);
    // e / size by a float product: exact, half a unit is kept to either side
    const float inv = 1.0f / float(size);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = 32 * i + lane;
      const int run = int((float(e) + 0.5f) * inv);
      if (!((kept >> (run & 31)) & 1u)) u[i] = 0u;  // keys past the last expert are 0 already
    }
  }
  const int id = best_of<VPL>(u, p.top_k, lane, key_sm);  // lane j: the j-th choice
  float w = id >= 0 ? score_sm[id] : 0.0f;
  if (p.renorm) w = w / (warp_sum(w) + 1e-20f);
  if (lane < p.top_k) {
    p.weights[t * p.top_k + lane] = id >= 0 ? p.scale * w : 0.0f;
    p.ids[t * p.top_k + lane] = id;
  }
}

// The logits' gradient of one token per warp; the chosen experts' ds go through shared
// memory to the lanes that hold their logits.
template <int VPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_back_kernel(const RouteBackParams p) {
  extern __shared__ float sm[];
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + warp;
  if (t >= p.tokens) return;
  float* score_sm = sm + warp * 2 * 32 * VPL;
  float* ds_sm = score_sm + 32 * VPL;
  int id = lane < p.top_k ? p.ids[t * p.top_k + lane] : -1;
  if (id >= p.experts) id = -1;
  const bool sigmoid = p.score == MAO_SCORE_SIGMOID;
  float s[VPL];
  float sj = 0.0f, slope = 0.0f;  // score of this lane's chosen expert; sigmoid: s (1 - s)
  if (sigmoid) {  // only the chosen experts' logits matter
    if (id >= 0) {
      const float x = load_elem(p.logits, t * p.ld + id, p.dtype);
      const float q = expf(-fabsf(x)), r = 1.0f / (1.0f + q);
      sj = x >= 0.0f ? r : q * r;
      slope = x == -INFINITY ? 0.0f : q * r * r;
    }
  } else {
    float x[VPL];
    load_logits<VPL>(p.logits, t, p.ld, p.dtype, p.experts, lane, x);
    scores_of<VPL>(x, p.score, s);
#pragma unroll
    for (int i = 0; i < VPL; ++i) score_sm[32 * i + lane] = s[i];
    __syncwarp();
    if (id >= 0) sj = score_sm[id];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) ds_sm[32 * i + lane] = 0.0f;
  __syncwarp();
  float ds = id >= 0 ? p.scale * p.dweights[t * p.top_k + lane] : 0.0f;
  float dot = 0.0f;  // softmax: the sum of ds_j s_j
  if (p.renorm) {
    // divided, not multiplied by a reciprocal: a lone expert's share is then exactly 1, and
    // its gradient exactly 0
    const float sum = warp_sum(sj), total = sum + 1e-20f;
    const float mean = warp_sum(ds * (sj / total));
    ds = id >= 0 ? (ds - mean) / total : 0.0f;
    // sum of ds_j s_j = (mean total - mean sum) / total: nothing where 1e-20 is below the sum's
    // rounding, but not where a bias has chosen experts of tiny scores
    if (total > sum) dot = mean * (1e-20f / total);
  } else if (!sigmoid) {
    dot = warp_sum(ds * sj);
  }
  if (id >= 0) ds_sm[id] = sigmoid ? ds * slope : ds;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    if (e >= p.experts) continue;
    float d = ds_sm[e];
    if (!sigmoid) d = s[i] == 0.0f ? 0.0f : s[i] * (d - dot);  // a masked expert's score is 0
    store_elem(p.dlogits, t * p.dld + e, p.ddtype, d);
  }
}

template <typename P>
using RouteFn = void (*)(const P);

// The instantiation whose lanes hold at least experts / 32 logits each.
template <typename P, template <int> class Pick>
mao_status route_run(const P& p, cudaStream_t stream) {
  if (p.tokens == 0) return MAO_OK;
  const int vpl = int(ceil_div(p.experts, 32));
  RouteFn<P> k;
  int v;
  if (vpl <= 2) k = Pick<2>::fn(), v = 2;
  else if (vpl <= 4) k = Pick<4>::fn(), v = 4;
  else if (vpl <= 8) k = Pick<8>::fn(), v = 8;
  else if (vpl <= 16) k = Pick<16>::fn(), v = 16;
  else k = Pick<32>::fn(), v = 32;
  const size_t smem = size_t(ROUTE_WARPS) * 2 * 32 * v * sizeof(float);
  return launch_dependent(k, unsigned(ceil_div(p.tokens, ROUTE_WARPS)), 32 * ROUTE_WARPS, smem, stream, p);
}
template <int V>
struct PickRoute {
  static RouteFn<RouteParams> fn() { return route_kernel<V>; }
};
template <int V>
struct PickBack {
  static RouteFn<RouteBackParams> fn() { return route_back_kernel<V>; }
};

// ------------------------------------------------------------------ places of the copies
//
// A counting sort of the copies by expert that keeps their order. Each block takes
// PLAN_CHUNK copies: its warps count theirs per expert, 32 at a time (equal experts in a
// warp find each other by ballots), which also ranks every copy within its warp. A copy's row
// is the expert's offset plus the counts of the blocks and warps before it plus its rank.
// Integer sums only: the result does not depend on the order in which blocks run. Latency
// bounds it: 131,072 copies among 256 experts take 7 us to count and 8.3 to place, 10.4 in all in a
// graph of calls; up to 4096 copies one block does both.

constexpr int PLAN_WARPS = 16;
constexpr int PLAN_ROUNDS = 8;
constexpr int PLAN_CHUNK = PLAN_WARPS * 32 * PLAN_ROUNDS;
static_assert(PLAN_CHUNK == kPlanAlone, "copies of one block");
constexpr int PLAN_THREADS = 32 * PLAN_WARPS;
constexpr int PLAN_MAX_EXPERTS = 1024;

// Counts of this block's copies per warp and expert into cnt[PLAN_WARPS][experts] (zeroed
// here), with each copy's expert and rank among its warp's copies of that expert.
__device__ __forceinline__ void plan_count(const int32_t* ids, int64_t n, int experts, int* cnt,
                                           int (&ex)[PLAN_ROUNDS], int (&rank)[PLAN_ROUNDS]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < PLAN_WARPS * experts; i += PLAN_THREADS) cnt[i] = 0;
  __syncthreads();
  const int bits = 32 - __clz(experts - 1);  // 0 for one expert
  const int64_t first = int64_t(blockIdx.x) * PLAN_CHUNK + warp * 32 * PLAN_ROUNDS + lane;
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    const int64_t i = first + 32 * r;
    const int e = i < n ? ids[i] : -1;
    ex[r] = e >= 0 && e < experts ? e : -1;
  }
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    // lanes with this lane's expert: one ballot per bit of the number (dropped copies, -1, only
    // ever meet each other)
    uint32_t same = FULL;
    for (int b = 0; b < bits; ++b) {
      const uint32_t one = __ballot_sync(FULL, (ex[r] >> b) & 1);
      same &= ((ex[r] >> b) & 1) ? one : ~one;
    }
    const uint32_t in = __ballot_sync(FULL, ex[r] >= 0);
    same &= ex[r] >= 0 ? in : ~in;
    int* c = cnt + warp * experts + (ex[r] < 0 ? 0 : ex[r]);
    const int before = ex[r] < 0 ? 0 : *c;
    rank[r] = before + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (ex[r] >= 0 && (__ffs(same) - 1) == lane) *c = before + __popc(same);
    __syncwarp();
  }
  __syncthreads();
}

struct PlanParams {
  const int32_t* ids;
  int64_t n, n_slots;
  int32_t experts, blocks;
  int32_t* block_counts;  // [blocks][experts]
  int32_t* ranks;         // [n]: each copy's rank among its block's copies of its expert
  int32_t* counts;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* slot_of;
};

// cnt[warp][expert] becomes the number of copies of the expert in the warps before; total[expert]
// their sum over all warps.
__device__ __forceinline__ void plan_sum_warps(int experts, int* cnt, int* total) {
  for (int e = threadIdx.x; e < experts; e += PLAN_THREADS) {
    int c[PLAN_WARPS], sum = 0;
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) c[w] = cnt[w * experts + e];
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) {
      cnt[w * experts + e] = sum;
      sum += c[w];
    }
    total[e] = sum;
  }
  __syncthreads();
}

// Offsets of the experts' runs from their counts (thread i owns experts PER i .. of `all`; they
// are written if `write`), and base[e] = offset + before[e].
__device__ __forceinline__ void plan_offsets(const PlanParams& p, const int* all, const int* before,
                                             int* base, bool write) {
  constexpr int PER = (PLAN_MAX_EXPERTS + PLAN_THREADS - 1) / PLAN_THREADS;
  __shared__ int warp_total[PLAN_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.experts + PLAN_THREADS - 1) / PLAN_THREADS;
  int size[PER], own = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = int(threadIdx.x) * per + q;
    size[q] = q < per && e < p.experts ? (all[e] + 127) & ~127 : 0;
    own += size[q];
  }
  int scan = own;  // inclusive over the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  for (int w = 0; w < warp; ++w) scan += warp_total[w];
  int off = scan - own;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int e = int(threadIdx.x) * per + q;
    if (q >= per || e >= p.experts) continue;
    if (write) {
      p.counts[e] = all[e];
      p.offsets[e] = off;
      if (e == p.experts - 1) p.offsets[p.experts] = off + size[q];
    }
    base[e] = off + (before ? before[e] : 0);
    off += size[q];
  }
  __syncthreads();
}

// The first copy of this thread (then every 32nd).
__device__ __forceinline__ int64_t plan_first() {
  return int64_t(blockIdx.x) * PLAN_CHUNK + (threadIdx.x >> 5) * 32 * PLAN_ROUNDS + (threadIdx.x & 31);
}

// Up to PLAN_CHUNK copies: one block does it all.
__global__ void __launch_bounds__(PLAN_THREADS) plan_alone_kernel(const PlanParams p) {
  extern __shared__ int cnt[];
  int* total = cnt + PLAN_WARPS * p.experts;
  int* base = total + p.experts;
  wait_for_previous();
  for (int64_t i = threadIdx.x; i < p.n_slots; i += PLAN_THREADS) p.slot_of[i] = -1;
  int ex[PLAN_ROUNDS], rank[PLAN_ROUNDS];
  plan_count(p.ids, p.n, p.experts, cnt, ex, rank);
  plan_sum_warps(p.experts, cnt, total);
  plan_offsets(p, total, nullptr, base, true);
  const int64_t first = plan_first();
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    const int64_t i = first + 32 * r;
    if (i >= p.n) continue;
    const int e = ex[r];
    const int row = e < 0 ? -1 : base[e] + cnt[(threadIdx.x >> 5) * p.experts + e] + rank[r];
    p.row_of[i] = row;
    if (row >= 0) p.slot_of[row] = int32_t(i);
  }
}

// More: every block counts its copies and ranks them among themselves ..
__global__ void __launch_bounds__(PLAN_THREADS) plan_count_kernel(const PlanParams p) {
  extern __shared__ int cnt[];
  int* total = cnt + PLAN_WARPS * p.experts;
  wait_for_previous();
  int ex[PLAN_ROUNDS], rank[PLAN_ROUNDS];
  plan_count(p.ids, p.n, p.experts, cnt, ex, rank);
  plan_sum_warps(p.experts, cnt, total);
  for (int e = threadIdx.x; e < p.experts; e += PLAN_THREADS)
    p.block_counts[int64_t(blockIdx.x) * p.experts + e] = total[e];
  const int64_t first = plan_first();
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    const int64_t i = first + 32 * r;
    if (i < p.n && ex[r] >= 0) p.ranks[i] = cnt[(threadIdx.x >> 5) * p.experts + ex[r]] + rank[r];
  }
  const int64_t step = int64_t(gridDim.x) * PLAN_THREADS;
  for (int64_t i = int64_t(blockIdx.x) * PLAN_THREADS + threadIdx.x; i < p.n_slots; i += step)
    p.slot_of[i] = -1;
}

// .. and places them after the copies of the blocks before.
__global__ void __launch_bounds__(PLAN_THREADS) plan_place_kernel(const PlanParams p) {
  extern __shared__ int all[];
  int* before = all + p.experts;
  int* base = before + p.experts;
  wait_for_previous();
  for (int e = threadIdx.x; e < p.experts; e += PLAN_THREADS) {
    int sum = 0, mine = 0;
#pragma unroll 16
    for (int b = 0; b < p.blocks; ++b) {
      const int c = p.block_counts[int64_t(b) * p.experts + e];
      sum += c;
      mine += b < int(blockIdx.x) ? c : 0;
    }
    all[e] = sum;
    before[e] = mine;
  }
  const int64_t first = plan_first();
  int ex[PLAN_ROUNDS], rank[PLAN_ROUNDS];
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    const int64_t i = first + 32 * r;
    ex[r] = i < p.n ? p.ids[i] : -1;
    if (ex[r] >= p.experts) ex[r] = -1;
    rank[r] = i < p.n && ex[r] >= 0 ? p.ranks[i] : 0;
  }
  __syncthreads();
  plan_offsets(p, all, before, base, blockIdx.x == 0);
#pragma unroll
  for (int r = 0; r < PLAN_ROUNDS; ++r) {
    const int64_t i = first + 32 * r;
    if (i >= p.n) continue;
    const int row = ex[r] < 0 ? -1 : base[ex[r]] + rank[r];
    p.row_of[i] = row;
    if (row >= 0) p.slot_of[row] = int32_t(i);
  }
}

// ------------------------------------------------------------------ combination

// Stores eight columns from c on (VEC: one 16-byte access for bf16, two for fp32), those below `cols`.
template <bool VEC>
__device__ __forceinline__ void store_cols(void* base, int64_t row, int64_t ld, int dtype,
                                           int64_t c, int64_t cols, const float (&v)[8]) {
  if (VEC) {
    store8(base, row * ld + c, dtype, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) store_elem(base, row * ld + c + i, dtype, v[i]);
  }
}

// Eight columns as they are in memory (!VEC: as fp32, 0 from `cols` on), so that loads can be issued
// ahead of their use. STREAM: the row is read once by this call, and leaves the caches before what
// is read again.
struct RawCols {
  uint4 a, b;  // b: fp32 only
};
template <bool VEC, bool STREAM = false>
__device__ __forceinline__ void load_raw(const void* base, int64_t row, int64_t ld, int dtype,
                                         int64_t c, int64_t cols, RawCols& r) {
  if (VEC) {
    if (dtype == MAO_BF16) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + row * ld + c);
      r.a = STREAM ? __ldcs(q) : *q;
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + row * ld + c);
      r.a = STREAM ? __ldcs(q) : q[0];
      r.b = STREAM ? __ldcs(q + 1) : q[1];
    }
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? load_elem(base, row * ld + c + i, dtype) : 0.0f;
    r.a = *reinterpret_cast<const uint4*>(&v[0]);
    r.b = *reinterpret_cast<const uint4*>(&v[4]);
  }
}
template <bool VEC>
__device__ __forceinline__ void unpack_raw(const RawCols& r, int dtype, float (&v)[8]) {
  if (VEC && dtype == MAO_BF16) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
}

struct CombineParams {
  const void* z;
  void* y;
  const int32_t* row_of;
  const float* weights;
  int64_t zrows, cols, zld, yld, tokens;
  int32_t zdt, ydt, top_k;
};

// Threads of a row own eight columns each; a block holds as many tokens as fit. HBM bounds it:
// 8192 tokens of 8 x 2048 bf16 take 45 us in a row of calls and 58 after others have filled the
// L2 (52 and 62 without the streaming loads, and then 56 and 68 in a row of calls with two and
// eight rows ahead). fp32 takes 88 us. Widths that are no multiple of eight, whose threads read eight
// neighbours one by one, take 114 (2050 columns, bf16) and 149 (fp32).
template <bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  wait_for_previous();
  const int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * 8;
  if (t >= p.tokens || c >= p.cols) return;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int AHEAD = 4;  // rows asked for before the first is used
  for (int j0 = 0; j0 < p.top_k; j0 += AHEAD) {
    int32_t row[AHEAD];
    float w[AHEAD];
    RawCols r[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int64_t i = t * p.top_k + j0 + q;
      const bool in = j0 + q < p.top_k;
      row[q] = in ? p.row_of[i] : -1;
      w[q] = !in ? 0.0f : p.weights ? p.weights[i] : 1.0f;
      if (row[q] >= p.zrows) row[q] = -1;
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      if (row[q] >= 0) load_raw<VEC, true>(p.z, row[q], p.zld, p.zdt, c, p.cols, r[q]);
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      if (row[q] < 0) continue;
      float v[8];
      unpack_raw<VEC>(r[q], p.zdt, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[q], v[e], acc[e]);
    }
  }
  store_cols<VEC>(p.y, t, p.yld, p.ydt, c, p.cols, acc);
}

struct CombineBackParams {
  const void* dy;
  const void* z;
  void* dz;
  const int32_t* row_of;
  const int32_t* slot_of;
  const float* weights;
  float* dweights;
  int64_t rows, cols, dyld, zld, dzld, copies;
  int32_t dydt, zdt, dzdt, top_k;
};

// One warp per row of Z: its copy's token gives dZ's row, and the dot product of the two rows
// the copy's weight's gradient; no sums across warps, and none over copies. AHEAD pieces of Z's
// row (512 bytes each for bf16, from HBM; dY's rows come from L2) are asked for before the first
// is used. HBM bounds it: the gradient of combine_kernel's case takes 110 us (5.7 TB/s) with two
// pieces ahead. Without streaming loads of Z it took 115, and then 127 with one piece ahead, 120
// with four and 131 with eight, which cost resident warps; a block per row instead of a warp
// took 256. Two ahead pay where the types are fixed when compiled, as for bf16 throughout; with types
// looked up, one and two pieces ahead take 125 and 131 us (bf16), 238 and 230 (fp32), 204 and 209 (Z
// fp32, dY bf16), 160 and 144 (Z bf16, dY fp32), so the others have one. Widths that are no multiple
// of eight: 343 to 347 us (2050 columns, bf16) and 480 (fp32), with one piece or two.
template <bool VEC, int AHEAD>
__global__ void __launch_bounds__(256) combine_back_kernel(const CombineBackParams p) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (p.dweights) {  // dropped copies have no row
    const int64_t step = int64_t(gridDim.x) * blockDim.x;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < p.copies; i += step) {
      const int32_t at = p.row_of[i];
      if (at < 0 || at >= p.rows) p.dweights[i] = 0.0f;
    }
  }
  if (r >= p.rows) return;
  const int32_t slot = p.slot_of[r];
  if (slot < 0 || slot >= p.copies) {
    const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t c = lane * 8; c < p.cols; c += 256) store_cols<VEC>(p.dz, r, p.dzld, p.dzdt, c, p.cols, zero);
    return;
  }
  const int64_t t = uint32_t(slot) / uint32_t(p.top_k);
  const float w = p.weights ? p.weights[slot] : 1.0f;
  const int zdt = AHEAD > 1 ? int(MAO_BF16) : p.zdt;  // several ahead: all of it is bf16
  const int dydt = AHEAD > 1 ? int(MAO_BF16) : p.dydt;
  float dot = 0.0f;
#pragma unroll 1
  for (int64_t c0 = lane * 8; c0 < p.cols; c0 += 256 * AHEAD) {
    RawCols z[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (p.dweights && c0 + 256 * a < p.cols) load_raw<VEC, true>(p.z, r, p.zld, zdt, c0 + 256 * a, p.cols, z[a]);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int64_t c = c0 + 256 * a;
      if (c >= p.cols) break;
      float g[8], v[8];
      RawCols y;
      load_raw<VEC>(p.dy, t, p.dyld, dydt, c, p.cols, y);
      unpack_raw<VEC>(y, dydt, g);
      if (p.dweights) {
        unpack_raw<VEC>(z[a], zdt, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) dot = fmaf(g[q], v[q], dot);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) g[q] *= w;
      store_cols<VEC>(p.dz, r, p.dzld, p.dzdt, c, p.cols, g);
    }
  }
  if (!p.dweights) return;
  dot = warp_sum(dot);
  if (lane == 0) p.dweights[slot] = dot;
}

}  // namespace

mao_status route_launch(const RouteParams& p, cudaStream_t stream) {
  return route_run<RouteParams, PickRoute>(p, stream);
}

mao_status route_backward_launch(const RouteBackParams& p, cudaStream_t stream) {
  return route_run<RouteBackParams, PickBack>(p, stream);
}

size_t plan_workspace_size(int64_t n, int32_t experts) {
  const int64_t blocks = ceil_div(n, PLAN_CHUNK);
  return size_t(round_up(blocks > 1 ? blocks * experts * 4 : 0, 256) + round_up(n * 4, 256) + 256);
}

mao_status plan_launch(const int32_t* ids, int64_t n, int32_t experts, int32_t* counts,
                       int32_t* offsets, int32_t* row_of, int32_t* slot_of, int64_t n_slots,
                       void* workspace, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  const mao_status attr = once_per_device(ready, [] {
    const int most = (PLAN_WARPS + 2) * PLAN_MAX_EXPERTS * int(sizeof(int));
    const cudaError_t err = cudaFuncSetAttribute(plan_alone_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return err != cudaSuccess ? err : cudaFuncSetAttribute(plan_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (attr != MAO_OK) return attr;
  const int blocks = int(ceil_div(n, PLAN_CHUNK));
  const size_t row = size_t(experts) * sizeof(int);
  PlanParams p{ids, n, n_slots, experts, blocks, nullptr, nullptr, counts, offsets, row_of, slot_of};
  if (blocks <= 1) return launch_dependent(plan_alone_kernel, 1, PLAN_THREADS, (PLAN_WARPS + 2) * row, stream, p);
  p.block_counts = static_cast<int32_t*>(workspace);
  p.ranks = p.block_counts + round_up(int64_t(blocks) * experts, 64);
  const mao_status st = launch_dependent(plan_count_kernel, blocks, PLAN_THREADS, (PLAN_WARPS + 1) * row, stream, p);
  if (st != MAO_OK) return st;
  return launch_dependent(plan_place_kernel, blocks, PLAN_THREADS, 3 * row, stream, p);
}

mao_status combine_launch(const mao_mat& Z, const int32_t* row_of, const float* weights,
                          int64_t tokens, int32_t top_k, const mao_mat& Y, cudaStream_t stream) {
  if (tokens == 0) return MAO_OK;
  const CombineParams p{Z.data, Y.data, row_of, weights, Z.rows, Y.cols, Z.ld, Y.ld, tokens,
                        Z.dtype, Y.dtype, top_k};
  const bool vec = vec8_ok(Z) && vec8_ok(Y);
  int tx = 1;
  while (tx < 256 && tx * 8 < Y.cols) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const dim3 grid(unsigned(ceil_div(tokens, block.y)), unsigned(ceil_div(Y.cols, tx * 8)));
  return launch_dependent(vec ? combine_kernel<true> : combine_kernel<false>, grid, block, 0, stream, p);
}

mao_status combine_backward_launch(const mao_mat& dY, const mao_mat& Z, const int32_t* row_of,
                                   const int32_t* slot_of, const float* weights, int32_t top_k,
                                   const mao_mat& dZ, float* dweights, cudaStream_t stream) {
  const int64_t copies = dY.rows * top_k;
  if (Z.rows == 0 && (copies == 0 || !dweights)) return MAO_OK;
  const CombineBackParams p{dY.data, Z.data, dZ.data, row_of, slot_of, weights, dweights, Z.rows,
                            Z.cols, dY.ld, Z.ld, dZ.ld, copies, dY.dtype, Z.dtype, dZ.dtype, top_k};
  const bool vec = vec8_ok(dY) && vec8_ok(Z) && vec8_ok(dZ);
  const bool bf = Z.dtype == MAO_BF16 && dY.dtype == MAO_BF16;
  using Kernel = void (*)(const CombineBackParams);
  const Kernel k = !vec ? combine_back_kernel<false, 1> : bf ? combine_back_kernel<true, 2> : combine_back_kernel<true, 1>;
  const unsigned grid = unsigned(ceil_div(Z.rows > 0 ? Z.rows : 1, 8));
  return launch_dependent(k, grid, 256, 0, stream, p);
}

}  // namespace mao
