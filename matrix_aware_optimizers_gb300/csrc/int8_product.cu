// Products of 8-bit integers with a scale per row and per channel on the 5th-generation tensor
// cores, over runs of rows: D[j][i] = sA[j] sB[i] sum_k A[j][k] B[i][k].
//
// This part's tensor cores multiply 16-bit floating point many times faster than 8-bit integers,
// and fp16 holds every code, so codes become fp16 on their way to the tensor core; the products
// are exact in the fp32 sums (below 2^24). The weights B stay 8 bits wide in memory and L2: they
// are converted between shared memory and TMEM, from where tcgen05.mma reads them as its M
// side. The rows A are converted once, by a kernel of their own, into the workspace: done in this
// kernel as well, tile by tile, their way back through shared memory (a fence of the asynchronous
// proxy per stage, some 400 cycles of a stage's 512) held up the tensor cores.
//
// Tiles of 256 x 256 by a pair of CTAs (cta_group::2, M = 256 channels i, N up to 256 rows j).
// Roles per CTA (608 threads):
//   warp 0        TMA producer of A: fp16, a ring of eight slots: 128 deep in one, or 64 with more than 128 rows
//   warp 1        TMEM allocation; in the even CTA it issues the products (converged, one lane)
//   warps 2..9    epilogue: two warps per 32-lane quadrant of TMEM; lane = i
//   warps 10..17  B's rows, one per lane: 64 codes to 32 words of TMEM; four warps for each half of
//                 a stage
//   warp 18       TMA producer of B: 128-deep stages of codes, ring of four
// TMEM: two accumulators in 384 columns, one from the left and one from the right, and two stages of B (64
// columns each). Two tiles of 256 rows share 128 columns; these are read first, and the next tile's
// products wait for that only.
//
// What bounds it: 8192 x 14336 x 4096 takes 500 to 508 us in a graph (1.9 PFLOP/s: cuBLAS's bf16 rate
// alone), more in a long run: the tensor cores, then the power limit. Low tiles do not pay
// less: a product with its M side in TMEM takes some 90 cycles however few the rows, so a stage
// takes 0.43 us from 32 rows on, 0.50 at 128, 0.6 at 160. (Twice the converting warps, or four stages
// of B in TMEM for tiles of up to 128 rows: no difference.) 16,001 rows among 128 x [1536 x 2048]:
// 148 us, 21 of them the rows' conversion; 128 rows for each of them: 116 us.
// What the rings look ahead counts: with A in three 32 KB stages, half empty in tiles of up to 128
// rows, and six stages of B, these two took 168 and 132 us, the prompt 519. Seven slots and five stages: 158
// instead of 156 at that point; nine slots, or five stages beside eight: as now.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "ffn.h"
#include "ffn_few.h"
#include "ffn_tiles.cuh"
#include "internal.h"
#include "ns_plan.h"
#include "tc_ptx.cuh"

namespace mao {
namespace {

using namespace ptx;
using namespace ffn;

constexpr int BK = 128;                   // depth of a stage: rows of 128 bytes of codes
constexpr int RAW_BYTES = HALF * BK;
constexpr int RAW_STAGES = 4;
constexpr int HK = 64;                    // half of it: rows of 128 bytes of fp16
constexpr int A_BYTES = HALF * HK * 2;    // a slot of A
constexpr int A_SLOTS = 8;
constexpr int B_STAGES = 2;
constexpr int EPI_WARPS = 8;
constexpr int CONV_WARPS = 8;
constexpr int THREADS = 32 * (3 + EPI_WARPS + CONV_WARPS);
constexpr int TMEM_COLS = 512;
constexpr int B_COL = 384;                // B's stages; two accumulators in the columns before
constexpr int B_COLS = BK / 2;
constexpr int Q_BOXES = 4;                // heights of boxes of A: 16 << b rows
constexpr size_t SMEM = 1024 + size_t(RAW_STAGES) * RAW_BYTES + size_t(A_SLOTS) * A_BYTES + TABLE_BYTES + 512;
static_assert(SMEM <= 232448, "shared memory budget of one CTA");
static_assert(B_COL + B_STAGES * B_COLS <= TMEM_COLS, "TMEM budget");

struct Int8Params : TileParams {
  CUtensorMap map_p;
  CUtensorMap map_q[Q_BOXES];  // boxes of 16, 32, 64, 128 rows; of one run the last, half a tile's height
  const float* sa;             // scales of A's rows, of B's (null: parts of a sum, not scaled)
  const float* sb;
  void* d;
  int64_t ld;
  int32_t dtype, paired;
};

// The first column of accumulator `acc` with n of them: one from the left, one from the right. Those
// of two tiles meet where their columns together pass B_COL, in columns 128 .. 255 at most.
__device__ __forceinline__ int acc_col(int acc, int n) { return acc ? B_COL - n : 0; }

// Instruction descriptor of kind::f16: fp16 operands, fp32 sums, M = 256.
__device__ __forceinline__ uint32_t instr_desc(int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(TILE >> 4) << 24);
}

// Whether the two halves of a stage's A, each 64 deep, have a slot of their own (tiles of more than
// 128 rows) or share one.
__device__ __forceinline__ bool two_slots(const Int8Params& p, const Tile& t) {
  return (p.offsets ? t.n : p.height) > HALF;
}

// Four 16-deep products: B from TMEM (8 columns each), A from shared memory (32 bytes along its rows
// each).
__device__ __forceinline__ void mma_half(uint32_t elected, uint32_t d, uint32_t b, uint64_t a, uint32_t idesc,
                                         uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm volatile(
        "{\n\t.reg .pred a, e;\n\t"
        "setp.ne.b32 a, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, a;\n\t}\n" ::"r"(d),
        "r"(b + 8 * k), "l"(a + uint64_t(2 * k)), "r"(idesc),
        "r"(k ? 1u : accumulate), "r"(elected)
        : "memory");
  }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// The same of bytes that need not stay in L2.
__device__ __forceinline__ void tma_load_3d_once(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// Four codes as two pairs of fp16: code + 128 into the low byte of 1024, less 1152.
__device__ __forceinline__ void to_half(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = codes ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// 64 codes of row r (from byte 64 h of its 128 swizzled bytes on) as 32 words.
__device__ __forceinline__ void load_row(const uint8_t* raw, int r, int h, uint32_t (&w)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int chunk = (4 * h + q) ^ (r & 7);
    const uint4 c = *reinterpret_cast<const uint4*>(raw + r * BK + 16 * chunk);
    to_half(c.x, w[8 * q], w[8 * q + 1]);
    to_half(c.y, w[8 * q + 2], w[8 * q + 3]);
    to_half(c.z, w[8 * q + 4], w[8 * q + 5]);
    to_half(c.w, w[8 * q + 6], w[8 * q + 7]);
  }
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Sixteen rows of D (from row j on, those below j_end) at column i of this lane.
__device__ __forceinline__ void store16(const Int8Params& p, const Tile& t, int j, int i, float sb,
                                        float (&v)[16], int lane) {
  const bool in = i < p.I;
  const int64_t row = t.row0 + j;
  if (p.sa) {
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] *= (j + c < t.j_end ? __ldg(p.sa + j + c) : 0.0f);
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] *= sb;
  }
  if (p.dtype == MAO_F32) {
    float* d = static_cast<float*>(p.d) + row * p.ld + i;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (in && j + c < t.j_end)
        asm volatile("st.global.L1::no_allocate.f32 [%0], %1;" ::"l"(d + c * p.ld), "f"(v[c]) : "memory");
    return;
  }
  __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + i;
  if (p.paired) {
    const int odd = lane & 1;
    d += odd ? p.ld - 1 : 0;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const uint32_t both = swap_pair(v[c], v[c + 1], odd);
      if (in && j + c + odd < t.j_end) store_word(d, both);
      d += 2 * p.ld;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (in && j + c < t.j_end) d[c * p.ld] = __float2bfloat16_rn(v[c]);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    int8_kernel(const __grid_constant__ Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* raw = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ast = raw + RAW_STAGES * RAW_BYTES;
  int* lo = reinterpret_cast<int*>(ast + A_SLOTS * A_BYTES);
  int* cnt = lo + MAX_GROUPS + 2;
  int* begin = cnt + MAX_GROUPS + 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ast + A_SLOTS * A_BYTES + TABLE_BYTES);
  uint64_t* rfull_bar = bars;                       // [RAW_STAGES]
  uint64_t* rempty_bar = rfull_bar + RAW_STAGES;    // [RAW_STAGES]
  uint64_t* afull_bar = rempty_bar + RAW_STAGES;    // [A_SLOTS]  (used in the even CTA)
  uint64_t* aempty_bar = afull_bar + A_SLOTS;      // [A_SLOTS]
  uint64_t* bfull_bar = aempty_bar + A_SLOTS;      // [B_STAGES]  (used in the even CTA)
  uint64_t* bempty_bar = bfull_bar + B_STAGES;      // [B_STAGES]
  uint64_t* tfull_bar = bempty_bar + B_STAGES;      // [2]
  uint64_t* tempty_bar = tfull_bar + 2;             // [2]  all columns read    (even CTA)
  uint64_t* tshared_bar = tempty_bar + 2;           // [2]  shared columns read (even CTA)
  uint64_t* drain_bar = tshared_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const bool leader = cta == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const uint64_t limit = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < RAW_STAGES; ++s) {
      mbar_init(smem_u32(&rfull_bar[s]), 1);
      mbar_init(smem_u32(&rempty_bar[s]), CONV_WARPS);
    }
    for (int s = 0; s < A_SLOTS; ++s) {
      mbar_init(smem_u32(&afull_bar[s]), 1);
      mbar_init(smem_u32(&aempty_bar[s]), 1);
    }
    for (int s = 0; s < B_STAGES; ++s) {
      mbar_init(smem_u32(&bfull_bar[s]), 2 * CONV_WARPS);
      mbar_init(smem_u32(&bempty_bar[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull_bar[a]), 1);
      mbar_init(smem_u32(&tempty_bar[a]), 2 * EPI_WARPS);
      mbar_init(smem_u32(&tshared_bar[a]), 2 * EPI_WARPS);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane < 2) {
    const CUtensorMap* map = lane ? &p.map_q[Q_BOXES - 1] : &p.map_p;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  // launched as a programmatic dependent: the set-up may overlap the rows' conversion (which began
  // after every kernel before it, so that the offsets are there)
  make_table<THREADS>(p, lo, cnt, begin, reinterpret_cast<int*>(bars + 48));
  tc_fence_before();
  __syncthreads();
  const int total = begin[p.groups] * p.tiles_i * p.splits;
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  wait_for_previous();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer of A (both CTAs)
    // A's rows j0 + n/2 cta .. (each CTA supplies half of the tile's n values of j). The whole
    // warp runs the loop, converged; one lane issues.
    const uint32_t elected = elect_one();
    const uint32_t full0 = mapa_shared(smem_u32(afull_bar), 0);
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      const int j = t.j0 + (t.n >> 1) * int(cta);
      const bool one_box = !p.offsets;
      const int q_rows = one_box ? p.height >> 1 : t.n >> 1;  // a multiple of 16
      const bool two = two_slots(p, t);
      for (int at_k = 0; at_k < t.nkb * BK; at_k += two ? HK : BK) {
        if (!wait_warp<false>(&aempty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        const uint32_t fb = full0 + 8 * stage, dst = smem_u32(ast) + stage * A_BYTES;
        const int k = t.kb0 * BK + at_k;
        if (elected) {
          if (leader) mbar_expect_tx(smem_u32(&afull_bar[stage]), 2 * uint32_t(q_rows) * (two ? HK : BK) * 2);
          if (one_box) {
            tma_load_4d_pair(dst, &p.map_q[Q_BOXES - 1], fb, k, j, 0, 0);
            if (!two) tma_load_4d_pair(dst + A_BYTES / 2, &p.map_q[Q_BOXES - 1], fb, k + HK, j, 0, 0);
          }
          for (int box = Q_BOXES - 1, at = 0; box >= 0 && !one_box; --box)
            if (q_rows & (16 << box)) {
              tma_load_4d_pair(dst + at * (HK * 2), &p.map_q[box], fb, k, j + at, 0, 0);
              if (!two) tma_load_4d_pair(dst + A_BYTES / 2 + at * (HK * 2), &p.map_q[box], fb, k + HK, j + at, 0, 0);
              at += 16 << box;
            }
        }
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == A_SLOTS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // after an abort, the loads already issued land before the CTA leaves
    if (*abort_flag && leader && lane == 0) {
      for (int s = 0; s < A_SLOTS; ++s)
        if ((armed >> s) & 1u) mbar_drain(smem_u32(&afull_bar[s]), (armed_phase >> s) & 1u, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 2 + EPI_WARPS + CONV_WARPS) {
    // ------------------------------------------------------------ TMA producer of B (both CTAs)
    const uint32_t elected = elect_one();
    uint64_t policy;  // runs read their weights once: L2 had better keep the rows in fp16 (1 to 5%)
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      const int i = t.i0 + HALF * int(cta);
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&rempty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        if (elected) {
          const uint32_t fb = smem_u32(&rfull_bar[stage]);
          mbar_expect_tx(fb, RAW_BYTES);
          const uint32_t dst = smem_u32(raw) + stage * RAW_BYTES;
          if (p.offsets) tma_load_3d_once(dst, &p.map_p, fb, kb * BK, i, t.g, policy);
          else tma_load_3d(dst, &p.map_p, fb, (t.kb0 + kb) * BK, i, t.g);
        }
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == RAW_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag && lane == 0) {
      for (int s = 0; s < RAW_STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(smem_u32(&rfull_bar[s]), (armed_phase >> s) & 1u, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      const uint32_t elected = elect_one();
      const uint64_t a_desc = desc_of(smem_u32(ast), 16, 1024, 2);
      int sa = 0, sb = 0, local = 0, before_n = 0;
      uint32_t pa = 0, pb = 0;
      bool ok = true, issued = false, ready = false;
      Tile t;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
        const int acc = local & 1;
        // the accumulator's last tile has been read, and of the tile before this one the
        // columns that the two share
        const bool meet = before_n + t.n > B_COL;
        before_n = t.n;
        if (!wait_warp<true>(&tempty_bar[acc], (uint32_t(local >> 1) & 1u) ^ 1u, abort_flag, limit) ||
            (meet && !wait_warp<true>(&tshared_bar[acc ^ 1], (uint32_t((local + 1) >> 1) & 1u) ^ 1u,
                                      abort_flag, limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc_col(acc, t.n));
        const uint32_t idesc = instr_desc(t.n);
        const bool two = two_slots(p, t);
        for (int kb = 0; kb < t.nkb; ++kb) {
          // the stage was looked at while the products before were issued
          if (!__all_sync(0xFFFFFFFFu, ready) &&
              (!wait_warp<false>(&afull_bar[sa], pa, abort_flag, limit) ||
               !wait_warp<true>(&bfull_bar[sb], pb, abort_flag, limit))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b = tmem_base + uint32_t(B_COL + sb * B_COLS);
          uint64_t a = a_desc + uint64_t(sa * (A_BYTES >> 4));
          uint32_t aempty = smem_u32(&aempty_bar[sa]);
          const uint32_t bempty = smem_u32(&bempty_bar[sb]);
          auto next_slot = [&]() {
            if (++sa == A_SLOTS) {
              sa = 0;
              pa ^= 1u;
            }
          };
          next_slot();
          mma_half(elected, d, b, a, idesc, kb != 0 ? 1u : 0u);
          issued = true;
          if (two) {
            commit_both(elected, aempty);
            if (!wait_warp<false>(&afull_bar[sa], pa, abort_flag, limit)) {
              ok = false;
              break;
            }
            a = a_desc + uint64_t(sa * (A_BYTES >> 4));
            aempty = smem_u32(&aempty_bar[sa]);
            next_slot();
          } else {
            a += A_BYTES / 2 >> 4;
          }
          if (++sb == B_STAGES) {
            sb = 0;
            pb ^= 1u;
          }
          ready = limit != 0 && mbar_test_wait(smem_u32(&afull_bar[sa]), pa) &&
                  mbar_test_wait_cluster(smem_u32(&bfull_bar[sb]), pb);
          mma_half(elected, d, b + B_COLS / 2, a, idesc, 1u);
          commit_both(elected, bempty);
          commit_both(elected, aempty);
        }
        if (!ok) break;
        commit_both(elected, smem_u32(&tfull_bar[acc]));
        ++local;
      }
      if (!ok && issued) {  // wait for everything in flight before TMEM is freed
        if (elected) umma_commit_pair(smem_u32(drain_bar), 1);
        __syncwarp();
        mbar_drain(smem_u32(drain_bar), 0u, 1000000000ull);
      }
    }
    __syncwarp();
  } else if (warp < 2 + EPI_WARPS) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3;         // TMEM lanes 32 quad ..
    const int part = (warp - 2) >> 2;  // which of the quadrant's two warps
    const uint32_t tempty[2] = {mapa_shared(smem_u32(&tempty_bar[0]), 0),
                                mapa_shared(smem_u32(&tempty_bar[1]), 0)};
    const uint32_t tshared[2] = {mapa_shared(smem_u32(&tshared_bar[0]), 0),
                                 mapa_shared(smem_u32(&tshared_bar[1]), 0)};
    // rows that hold no tokens are cleared while the first tiles are multiplied
    if (p.splits == 1) {
      const int es = p.dtype == MAO_F32 ? 4 : 2;
      for_unused_rows(p, lo, cnt, int(blockIdx.x) * EPI_WARPS + warp - 2, int(gridDim.x) * EPI_WARPS,
                      [&](int64_t j0, int64_t j1, int64_t step) {
                        clear_rows(p.d, p.ld * es, int64_t(p.I) * es, j0, j1, step, lane);
                      });
    }
    int local = 0;
    Tile t;
    for (int tile = pair; tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      const int i = t.i0 + HALF * int(cta) + 32 * quad + lane;
      const int acc = local & 1;
      const int n = t.j_end - t.j0;
      const float sb = p.sb && i < p.I ? __ldg(p.sb + int64_t(t.g) * p.I + i) : 0.0f;
      // every lane waits; the warp goes on only if all of them saw the accumulator
      if (!wait_warp<false>(&tfull_bar[acc], uint32_t(local >> 1) & 1u, abort_flag, limit)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t(32 * quad) << 16) + uint32_t(acc_col(acc, t.n));
      // the half with the columns that both accumulators may use, then the other: of each this
      // warp has every second sixteen
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int c0 = ((acc ^ half) ? 0 : HALF) + 16 * part;
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
          const int c = c0 + 32 * q;
          float va[16], vb[16];
          if (c < n) tmem_ld16(trow + uint32_t(c), va);
          if (c + 32 < n) tmem_ld16(trow + uint32_t(c + 32), vb);
          tmem_wait(va);
          tmem_wait(vb);
          if (q == 2) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(half ? tempty[acc] : tshared[acc]);
          }
          if (c < n) store16(p, t, t.j0 + c, i, sb, va, lane);
          if (c + 32 < n) store16(p, t, t.j0 + c + 32, i, sb, vb, lane);
        }
      }
      ++local;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ conversion (both CTAs)
    const int h = (warp - 2 - EPI_WARPS) >> 2;
    const int r = 32 * (warp & 3) + lane;  // TMEM's lane: a warp reaches the quadrant of its number
    const uint32_t full0 = mapa_shared(smem_u32(bfull_bar), 0);
    const uint32_t tcol = tmem_base + (uint32_t(32 * (warp & 3)) << 16) + B_COL;
    int rstage = 0, stage = 0;
    uint32_t rphase = 0, phase = 0;
    bool ok = true;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&rfull_bar[rstage], rphase, abort_flag, limit)) {
          ok = false;
          break;
        }
        uint32_t w[32];
        load_row(raw + rstage * RAW_BYTES, r, h, w);
        __syncwarp();
        if (lane == 0)  // this half of the stage has been read
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&rempty_bar[rstage])) : "memory");
        if (++rstage == RAW_STAGES) {
          rstage = 0;
          rphase ^= 1u;
        }
        if (!wait_warp<false>(&bempty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st32(tcol + uint32_t(stage * B_COLS + h * (B_COLS / 2)), w);
        tc_fence_before();
        __syncwarp();
        // the words are in this SM's TMEM (tcgen05.wait::st, the fence before): as for an
        // accumulator's reads, the arrive only carries that
        if (lane == 0) mbar_arrive_cluster(full0 + 8 * stage);
        if (++stage == B_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // an aborted CTA also gives the peer's copies in flight 50 us to land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 50000ull) {
    }
  }
  cluster_sync_all();  // no CTA leaves while its peer may still touch its shared memory
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

// The splits' parts added up in their order and scaled; four columns per thread.
struct SumParams {
  const float* parts;
  const float* sa;
  const float* sb;
  void* d;
  int64_t rows, cols, pld, ld;
  int32_t splits, dtype;
};
__global__ void __launch_bounds__(256) int8_sum_kernel(const SumParams p) {
  wait_for_previous();
  const int64_t quads = p.pld / 4, all = p.rows * quads;
  for (int64_t x = int64_t(blockIdx.x) * 256 + threadIdx.x; x < all; x += int64_t(gridDim.x) * 256) {
    const int64_t j = x / quads, i = 4 * (x - j * quads);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      const float4 y = *reinterpret_cast<const float4*>(p.parts + (s * p.rows + j) * p.pld + i);
      v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
    }
    const float sa = p.sa[j];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (i + c < p.cols) store_elem(p.d, j * p.ld + i + c, p.dtype, v[c] * sa * p.sb[i + c]);
  }
}

// A's codes in fp16, a row per warp, eight codes per lane and step, up to eight steps under way. With
// counts the rows that hold no tokens are left out: 128 runs of 125 rows, padded to twice that, took
// 41 us with all of them.
struct HalfParams {
  const int8_t* src;
  uint16_t* dst;
  const int32_t* offsets;
  const int32_t* counts;
  int64_t rows, ld, dld;
  int32_t cols, groups;
};
constexpr int AHEAD = 8;  // loads of a lane under way
__global__ void __launch_bounds__(128) to_half_kernel(const HalfParams p) {
  wait_for_previous();
  const int lane = threadIdx.x % 32;
  for (int64_t r = int64_t(blockIdx.x) * 4 + threadIdx.x / 32; r < p.rows; r += int64_t(gridDim.x) * 4) {
    if (p.counts) {
      // offset `end` is the first past the row, and the run before it begins at the largest so far: the
      // product's table raises offsets that fall
      int end = p.groups + 1, first = 0;
#pragma unroll 4
      for (int g0 = 0; g0 <= p.groups; g0 += 32) {
        const int g = g0 + lane, at = g <= p.groups ? __ldg(p.offsets + g) : 0;
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, at > r);
        if (past) end = min(end, g0 + __ffs(past) - 1);
        if (g < end) first = max(first, at);
      }
      first = __reduce_max_sync(0xFFFFFFFFu, first);
      if (end > 0 && end <= p.groups && r >= int64_t(first) + max(__ldg(p.counts + end - 1), 0)) continue;
    }
    const int8_t* s = p.src + r * p.ld;
    uint16_t* d = p.dst + r * p.dld;
    for (int c0 = 8 * lane; c0 < p.cols; c0 += 256 * AHEAD) {
      uint2 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (c0 + 256 * k + 8 <= p.cols) v[k] = *reinterpret_cast<const uint2*>(s + c0 + 256 * k);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int c = c0 + 256 * k;
        if (c + 8 <= p.cols) {
          uint4 h;
          to_half(v[k].x, h.x, h.y);
          to_half(v[k].y, h.z, h.w);
          *reinterpret_cast<uint4*>(d + c) = h;
        } else {
          for (int q = 0; c + q < p.cols; ++q) d[q + c] = __half_as_ushort(__int2half_rn(s[q + c]));
        }
      }
    }
  }
}

std::atomic<bool> g_launched{false};

// A block of 128 takes a pair 0.43 us with 32 rows, 0.65 with 256.
Cut cut_of(const mao_int8& A, const mao_int8& B) {
  return choose_cut(cta_pairs(), ceil_div(B.rows, TILE), A.rows, ceil_div(A.cols, BK), 0.4, 0.25, 0.0, 1.7, A.rows * B.rows, 2);
}

// The workspace: A in fp16, then the parts of split sums.
int64_t half_ld(const mao_int8& A) { return round_up(A.cols, 8); }
size_t half_bytes(const mao_int8& A) { return size_t(round_up(A.rows * half_ld(A) * 2, 256)); }

}  // namespace

size_t int8_product_workspace_size(const mao_int8& A, const mao_int8& B, bool grouped) {
  if (A.rows == 0 || few_rows(A.rows, grouped, false, B.count)) return 0;
  const Cut s = grouped ? Cut{TILE, 1, 0} : cut_of(A, B);
  return half_bytes(A) + (s.splits > 1 ? size_t(round_up(int64_t(s.splits) * A.rows * round_up(B.rows, 4) * 4, 256)) : 0);
}
mao_status int8_product_launch(const mao_int8& A, const mao_int8& B, const mao_mat& D, const Runs& runs,
                               void* workspace, cudaStream_t stream) {
  if (A.rows == 0) return MAO_OK;
  if (few_rows(A.rows, runs.offsets != nullptr, runs.counts != nullptr, runs.groups)) {
    FewParams q = {};
    q.offsets = runs.offsets;
    q.counts = runs.counts;
    q.groups = runs.groups;
    q.rows = int32_t(A.rows);
    q.I = int32_t(B.rows);
    q.depth = int32_t(A.cols);
    q.w = B.codes;
    q.ldw = B.ld;
    q.x = A.codes;
    q.ldx = A.ld;
    q.sa = A.scales;
    q.sb = B.scales;
    q.d = D.data;
    q.ld = D.ld;
    q.dtype = D.dtype;
    return few_launch(q, true, false, 0, stream);
  }
  Int8Params p = {};
  mao_status st = tc_encode_code_map(&p.map_p, B.codes, B.cols, B.rows, B.ld, B.count, HALF);
  const Cut cut = runs.offsets ? Cut{TILE, 1, 0} : cut_of(A, B);
  for (int b = runs.offsets ? 0 : Q_BOXES - 1; b < Q_BOXES && st == MAO_OK; ++b)
    st = tc_encode_bf16_map(&p.map_q[b], workspace, A.cols, A.rows, 1, 1, half_ld(A), A.rows * half_ld(A),
                            A.rows * half_ld(A), runs.offsets ? 16 << b : cut.height / 2);
  if (st != MAO_OK) return st;
  p.offsets = runs.offsets;
  p.counts = runs.offsets ? runs.counts : nullptr;
  p.groups = runs.groups;
  p.rows = int32_t(A.rows);
  p.I = int32_t(B.rows);
  p.J = int32_t(A.rows);
  p.depth = int32_t(A.cols);
  p.halves = 1;
  p.tiles_i = int32_t(ceil_div(B.rows, TILE));
  p.timeout_ns = wait_limit_ns();
  p.sa = A.scales;
  p.sb = B.scales;
  p.d = D.data;
  p.ld = D.ld;
  p.dtype = D.dtype;
  p.paired = D.dtype == MAO_BF16 && D.cols % 2 == 0 && reinterpret_cast<uintptr_t>(D.data) % 4 == 0 && D.ld % 2 == 0;
  void* parts = static_cast<uint8_t*>(workspace) + half_bytes(A);
  p.height = cut.height;
  p.splits = cut.splits;
  p.split_kb = cut.kb;
  const int64_t tiles = (ceil_div(A.rows, p.height) + (runs.offsets ? runs.groups : 0)) * p.tiles_i;
  if (tiles * p.splits > 0x7FFF0000) return MAO_ERR_UNSUPPORTED;
  static std::atomic<bool> ready[64];
  st = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(int8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
  });
  if (st != MAO_OK) return st;
  if (p.splits > 1) {
    p.sa = p.sb = nullptr;
    p.d = parts;
    p.ld = round_up(D.cols, 4);
    p.dtype = MAO_F32;
  }
  const HalfParams half{A.codes, static_cast<uint16_t*>(workspace), p.offsets, p.counts, A.rows, A.ld,
                        half_ld(A), int32_t(A.cols), p.groups};
  const int64_t blocks4 = ceil_div(A.rows, 4);
  using Half = void (*)(const HalfParams);
  st = launch_dependent(static_cast<Half>(to_half_kernel), unsigned(blocks4 < 32 * num_sms() ? blocks4 : 32 * num_sms()),
                        128, 0, stream, half);
  if (st != MAO_OK) return st;
  g_launched.store(true, std::memory_order_release);
  const int64_t units = tiles * p.splits;
  const unsigned grid = unsigned(2 * (units < num_sms() / 2 ? units : num_sms() / 2));
  using Kernel = void (*)(const Int8Params);
  st = launch_dependent(static_cast<Kernel>(int8_kernel), grid, THREADS, SMEM, stream, p);
  if (st != MAO_OK || p.splits == 1) return st;
  const SumParams sum{static_cast<const float*>(parts), A.scales, B.scales, D.data, A.rows, D.cols,
                      p.ld, D.ld, p.splits, D.dtype};
  const int64_t blocks = ceil_div(A.rows * (p.ld / 4), 256);
  using Sum = void (*)(const SumParams);
  return launch_dependent(static_cast<Sum>(int8_sum_kernel), unsigned(blocks < 8 * num_sms() ? blocks : 8 * num_sms()),
                          256, 0, stream, sum);
}

mao_status int8_read_and_clear_error(cudaStream_t stream) {
  return g_launched.load(std::memory_order_acquire) ? read_and_clear_error(stream) : MAO_OK;
}

}  // namespace mao
