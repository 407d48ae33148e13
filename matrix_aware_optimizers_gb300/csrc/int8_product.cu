// Products of 8-bit integers with a scale per row and per channel on the 5th-generation tensor
// cores, over runs of rows: D[j][i] = sA[j] sB[i] sum_k A[j][k] B[i][k].
//
// This part's tensor cores multiply 16-bit floating point many times faster than 8-bit integers,
// and fp16 holds every code, so the codes become fp16 on their way from shared memory to the
// tensor core: memory and L2 move 8 bits per entry, the products are exact in the fp32 sums (below
// 2^24). One operand is converted into TMEM, from where tcgen05.mma reads it as its M side, the
// other into shared memory. (Through shared memory both, a 64-deep block of 256 x 256 moves
// 96 KB of an SM's shared memory in the 512 cycles of its products; so it moves 64 KB.)
//
// Tiles of 256 x 256 by a pair of CTAs (cta_group::2, M = 256 channels i, N up to 256 rows j).
// Roles per CTA (576 threads):
//   warp 0        TMA producer: raw codes, 128-deep stages, ring of four
//   warp 1        TMEM allocation; in the even CTA it issues the products (converged, one lane)
//   warps 2..9    epilogue: two warps per 32-lane quadrant of TMEM; lane = i
//   warps 10..13  B's rows, one per lane: 64 codes to 32 words of TMEM
//   warps 14..17  A's rows: 64 codes to 128 bytes of shared memory, swizzled
// TMEM: two accumulators of 256 columns that share 128 (columns 0..255 and 128..383), and four
// stages of B (32 columns each from 384 on). The shared columns are read into registers first,
// so the next tile's products wait for that only.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "ffn.h"
#include "ffn_tiles.cuh"
#include "internal.h"
#include "ns_plan.h"
#include "tc_ptx.cuh"

namespace mao {
namespace {

using namespace ptx;
using namespace ffn;

constexpr int BK = 128;                   // depth of a raw stage: rows of 128 bytes
constexpr int RAW_OP = HALF * BK;
constexpr int RAW_BYTES = 2 * RAW_OP;
constexpr int RAW_STAGES = 4;
constexpr int HK = 64;                    // depth of a converted stage
constexpr int Q_BYTES = HALF * HK * 2;
constexpr int STAGES = 4;
constexpr int EPI_WARPS = 8;
constexpr int CONV_WARPS = 8;             // of each operand, four for each half of a raw stage
constexpr int THREADS = 64 + 32 * (EPI_WARPS + 2 * CONV_WARPS);
constexpr int TMEM_COLS = 512;
constexpr int ACC1 = 128;                 // first column of the second accumulator
constexpr int B_COL = ACC1 + TILE;        // B's stages
constexpr int B_COLS = HK / 2;
constexpr int Q_BOXES = 4;                // heights of boxes of A: 16 << b rows
constexpr size_t SMEM = 1024 + size_t(RAW_STAGES) * RAW_BYTES + size_t(STAGES) * Q_BYTES + TABLE_BYTES + 512;
static_assert(SMEM <= 232448, "shared memory budget of one CTA");
static_assert(B_COL + STAGES * B_COLS <= TMEM_COLS, "TMEM budget");

struct Int8Params : TileParams {
  CUtensorMap map_p;
  CUtensorMap map_q[Q_BOXES];  // boxes of 16, 32, 64, 128 rows
  const float* sa;             // scales of A's rows, of B's (null: parts of a sum, not scaled)
  const float* sb;
  void* d;
  int64_t ld;
  int32_t dtype, paired;
};

// Instruction descriptor of kind::f16: fp16 operands, fp32 sums, M = 256.
__device__ __forceinline__ uint32_t instr_desc(int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(TILE >> 4) << 24);
}

// The four 16-deep products of a converted stage: B from TMEM (8 columns each), A from shared
// memory (32 bytes along its rows each).
__device__ __forceinline__ void mma_stage(uint32_t elected, uint32_t d, uint32_t b, uint64_t a,
                                          uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm volatile(
        "{\n\t.reg .pred a, e;\n\t"
        "setp.ne.b32 a, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, a;\n\t}\n" ::"r"(d),
        "r"(b + 8 * k), "l"(a + uint64_t(2 * k)), "r"(idesc), "r"(k ? 1u : accumulate), "r"(elected)
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

// Arrive on a barrier of the leader CTA, ordered after this warp's writes to its own shared memory
// at cluster scope. Only shared memory is fenced: a plain cluster-scope release also waits
// for global memory, some 2000 cycles (8192 x 14336 x 4096: 1093 us instead of 647).
__device__ __forceinline__ void mbar_arrive_shared_release(uint32_t cluster_addr) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    int8_kernel(const __grid_constant__ Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* raw = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qst = raw + RAW_STAGES * RAW_BYTES;
  int* lo = reinterpret_cast<int*>(qst + STAGES * Q_BYTES);
  int* cnt = lo + MAX_GROUPS + 2;
  int* begin = cnt + MAX_GROUPS + 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(qst + STAGES * Q_BYTES + TABLE_BYTES);
  uint64_t* rfull_bar = bars;                       // [RAW_STAGES]
  uint64_t* rempty_bar = rfull_bar + RAW_STAGES;    // [RAW_STAGES]
  uint64_t* full_bar = rempty_bar + RAW_STAGES;     // [STAGES]  (used in the even CTA)
  uint64_t* empty_bar = full_bar + STAGES;          // [STAGES]
  uint64_t* tfull_bar = empty_bar + STAGES;         // [2]
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
      mbar_init(smem_u32(&rempty_bar[s]), 2 * CONV_WARPS);
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 2 * CONV_WARPS);
      mbar_init(smem_u32(&empty_bar[s]), 1);
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
  // launched as a programmatic dependent: the set-up so far may overlap the previous kernel
  wait_for_previous();
  make_table<THREADS>(p, lo, cnt, begin, reinterpret_cast<int*>(bars + 32));
  tc_fence_before();
  __syncthreads();
  const int total = begin[p.groups] * p.tiles_i * p.splits;
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    // B's rows i0 + 128 cta .. and A's rows j0 + n/2 cta .. (each CTA supplies half of the
    // tile's n values of j). The whole warp runs the loop, converged; one lane issues.
    const uint32_t elected = elect_one();
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_phase = 0;
    bool ok = true;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      const int i = t.i0 + HALF * int(cta), j = t.j0 + (t.n >> 1) * int(cta);
      const int q_rows = t.n >> 1;  // a multiple of 16
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&rempty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&rfull_bar[stage]), dst = smem_u32(raw) + stage * RAW_BYTES;
        const int k = (t.kb0 + kb) * BK;
        if (elected) {
          mbar_expect_tx(fb, RAW_OP + uint32_t(q_rows) * BK);
          tma_load_3d(dst, &p.map_p, fb, k, i, t.g);
          for (int box = Q_BOXES - 1, at = 0; box >= 0; --box)
            if (q_rows & (16 << box)) {
              tma_load_3d(dst + RAW_OP + at * BK, &p.map_q[box], fb, k, j + at, 0);
              at += 16 << box;
            }
        }
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == RAW_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // after an abort, the loads already issued land before the CTA leaves
    if (*abort_flag && lane == 0) {
      for (int s = 0; s < RAW_STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(smem_u32(&rfull_bar[s]), (armed_phase >> s) & 1u, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      const uint32_t elected = elect_one();
      const uint64_t a_desc = desc_of(smem_u32(qst), 16, 1024, 2);
      int stage = 0, local = 0, before_n = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      Tile t;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
        const int acc = local & 1;
        // the accumulator's last tile has been read, and of the tile before this one the
        // columns that the two share (they do if the first accumulator's tile reaches there)
        const bool meet = (acc ? before_n : t.n) > ACC1;
        before_n = t.n;
        if (!wait_warp<true>(&tempty_bar[acc], (uint32_t(local >> 1) & 1u) ^ 1u, abort_flag, limit) ||
            (meet && !wait_warp<true>(&tshared_bar[acc ^ 1], (uint32_t((local + 1) >> 1) & 1u) ^ 1u,
                                      abort_flag, limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * ACC1);
        const uint32_t idesc = instr_desc(t.n);
        for (int kb = 0; kb < 2 * t.nkb; ++kb) {
          if (!wait_warp<true>(&full_bar[stage], phase, abort_flag, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_stage(elected, d, tmem_base + uint32_t(B_COL + stage * B_COLS),
                    a_desc + uint64_t(stage * (Q_BYTES >> 4)), idesc, kb != 0 ? 1u : 0u);
          issued = true;
          commit_both(elected, smem_u32(&empty_bar[stage]));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
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
      const int64_t turn = int64_t(blockIdx.x) * EPI_WARPS + warp - 2, turns = int64_t(gridDim.x) * EPI_WARPS;
      auto clear = [&](int64_t j0, int64_t j1) {
        clear_rows(p.d, p.ld * es, int64_t(p.I) * es, j0 + turn, j1, turns, lane);
      };
      clear(0, lo[0]);
      if (p.counts)
        for (int g = 0; g < p.groups; ++g) clear(lo[g] + cnt[g], lo[g + 1]);
      clear(lo[p.groups], p.rows);
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
      const uint32_t trow = tmem_base + (uint32_t(32 * quad) << 16) + uint32_t(acc * ACC1);
      // the half of the columns that both accumulators use, then the other: of each this warp
      // has every second sixteen
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int c0 = ((acc ^ half) ? 0 : ACC1) + 16 * part;
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
    // A warp takes the same half of every raw stage (every second converted one), so that its
    // loads, its arithmetic and the hand-over have the time of two stages' products.
    const bool of_b = warp < 2 + EPI_WARPS + CONV_WARPS;
    const int h = ((warp - 2 - EPI_WARPS) >> 2) & 1;
    // B's rows by TMEM's lanes: a warp reaches the quadrant of its number
    const int r = 32 * (of_b ? warp & 3 : (warp - 2 - EPI_WARPS) & 3) + lane;
    const uint32_t full0 = mapa_shared(smem_u32(full_bar), 0);
    const uint32_t tcol = tmem_base + (uint32_t(32 * (warp & 3)) << 16) + B_COL;
    int rstage = 0, stage = h;
    uint32_t rphase = 0, phase = 0;
    bool ok = true;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<NT, TILE, BK>(p, lo, cnt, begin, tile, t);
      const bool mine = of_b || r < (t.n >> 1);
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&rfull_bar[rstage], rphase, abort_flag, limit)) {
          ok = false;
          break;
        }
        uint32_t w[32];
        if (mine) load_row(raw + rstage * RAW_BYTES + (of_b ? 0 : RAW_OP), r, h, w);
        __syncwarp();
        if (lane == 0)  // this half of the raw stage has been read
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&rempty_bar[rstage])) : "memory");
        if (++rstage == RAW_STAGES) {
          rstage = 0;
          rphase ^= 1u;
        }
        if (!wait_warp<false>(&empty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        if (of_b) {
          tc_fence_after();
          tmem_st32(tcol + uint32_t(stage * B_COLS), w);
          tc_fence_before();
        } else {
          if (mine) {
            uint8_t* to = qst + stage * Q_BYTES + r * (HK * 2);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(to + 16 * (q ^ (r & 7))) =
                  make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_shared_release(full0 + 8 * stage);
        stage += 2;
        if (stage >= STAGES) {
          stage -= STAGES;
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

std::atomic<bool> g_launched{false};

// A block of 128 takes a pair 0.6 us, or 0.4 us (the operands' bytes) with few rows.
Split split_of(const mao_int8& A, const mao_int8& B) {
  return choose_split(ceil_div(A.rows, TILE) * ceil_div(B.rows, TILE), ceil_div(A.cols, BK),
                      A.rows < 128 ? 0.4 : 0.6, A.rows * B.rows, 2);
}

}  // namespace

size_t int8_product_workspace_size(const mao_int8& A, const mao_int8& B, bool grouped) {
  if (A.rows == 0 || grouped) return 0;
  const Split s = split_of(A, B);
  return s.splits > 1 ? size_t(round_up(int64_t(s.splits) * A.rows * round_up(B.rows, 4) * 4, 256)) : 0;
}

mao_status int8_product_launch(const mao_int8& A, const mao_int8& B, const mao_mat& D, const Runs& runs,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (A.rows == 0) return MAO_OK;
  Int8Params p = {};
  mao_status st = tc_encode_code_map(&p.map_p, B.codes, B.cols, B.rows, B.ld, B.count, HALF);
  for (int b = 0; b < Q_BOXES && st == MAO_OK; ++b)
    st = tc_encode_code_map(&p.map_q[b], A.codes, A.cols, A.rows, A.ld, 1, 16 << b);
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
  Split split{1, 0};
  const size_t need = int8_product_workspace_size(A, B, runs.offsets != nullptr);
  if (need && workspace && workspace_bytes >= need) split = split_of(A, B);
  p.splits = split.splits;
  p.split_kb = split.kb;
  const int64_t tiles = (ceil_div(A.rows, TILE) + (runs.offsets ? runs.groups : 0)) * p.tiles_i;
  if (tiles * p.splits > 0x7FFF0000) return MAO_ERR_UNSUPPORTED;
  static std::atomic<bool> ready[64];
  st = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(int8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
  });
  if (st != MAO_OK) return st;
  if (p.splits > 1) {
    p.sa = p.sb = nullptr;
    p.d = workspace;
    p.ld = round_up(D.cols, 4);
    p.dtype = MAO_F32;
  }
  g_launched.store(true, std::memory_order_release);
  const int64_t units = tiles * p.splits;
  const unsigned grid = unsigned(2 * (units < num_sms() / 2 ? units : num_sms() / 2));
  using Kernel = void (*)(const Int8Params);
  st = launch_dependent(static_cast<Kernel>(int8_kernel), grid, THREADS, SMEM, stream, p);
  if (st != MAO_OK || p.splits == 1) return st;
  const SumParams sum{static_cast<const float*>(workspace), A.scales, B.scales, D.data, A.rows, D.cols,
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
