// Products of 8-bit matrices with power-of-two block scales on the 5th-generation tensor cores,
// fp32 sums, over groups of rows.
//
// All three forms are one product D[j][i] = sum_k Q[j][k] P[i][k]: i runs along D's rows in
// memory and comes from the second argument (P), j from the first (Q). Only how the operands
// lie in memory differs: an operand whose depth runs along its rows is loaded K-major, one
// whose depth runs down its columns MN-major (the tensor core reads 8-bit codes either way, so
// the weights are quantised once, in 128 x 128 tiles, for the forward product and for the
// gradient of its input).
//
// Tiles of 256 x 256 outputs are computed by a pair of CTAs (tcgen05 cta_group::2, M = 256
// values of i, N up to 256 values of j). The scales enter the tensor core itself
// (kind::mxf8f6f4, one power of two per row and 32-deep slice): the four slices of a 128-deep
// block use the same byte of the scale word in TMEM, whose four bytes cover four blocks.
// So the sums over all of K stay in the fp32 accumulator in TMEM, and nothing is rescaled on
// the way.
//
// Roles per CTA (416 threads):
//   warp 0        TMA producer: a 128 x 128 box of each operand per 128-deep block, into a
//                 ring of 32 KB stages
//   warp 1        TMEM allocation; in the even CTA one thread copies the scale words into TMEM
//                 (tcgen05.cp) and issues the products
//   warps 2..9    epilogue: two warps per 32-lane quadrant of TMEM; lane = i, so a row of D is
//                 written by consecutive lanes
//   warps 10..12  scales: gather the scale bytes of four blocks, from whichever layout they
//                 have, into the words that tcgen05.cp expects
// TMEM (512 columns) holds two accumulators of 256 columns that share 32 of them (columns
// 0..255 and 224..479) and two sets of scale words (480..503). The shared columns are drained
// first: the next tile's products wait for them only, so the rest of a tile's epilogue runs
// under the next tile's products.
// Barriers and their bounded waits are as in the Newton–Schulz product kernel.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <mutex>

#include "common.cuh"
#include "experts.h"
#include "internal.h"
#include "ns_plan.h"
#include "tc_ptx.cuh"

namespace mao {
namespace {

using namespace ptx;

constexpr int TILE = 256;                  // i and j per tile
constexpr int HALF = 128;                  // of each per CTA
constexpr int BK = 128;                    // depth per stage
constexpr int OP_BYTES = HALF * BK;        // one operand of a stage
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int STAGES = 6;
constexpr int SF_SLOTS = 3;                // scale words in shared memory (four blocks each)
constexpr int SF_SETS = 2;                 // and in TMEM
constexpr int SF_BYTES = 3 * 512;          // 128 words of P, 256 of Q
constexpr int MAX_GROUPS = 1024;
constexpr int EPI_WARPS = 8;
constexpr int SF_WARPS = SF_SLOTS;         // each fills its own slot
constexpr int THREADS = 64 + 32 * (EPI_WARPS + SF_WARPS);
constexpr int ACC1 = 224;                  // first column of the second accumulator
constexpr int SHARED = TILE - ACC1;        // columns that both accumulators use
constexpr int SF_COL = ACC1 + TILE;        // scale words: 12 columns per set
constexpr int SF_COLS = 12;
constexpr int TMEM_COLS = 512;
constexpr int BAND = 8;                    // tiles of j that share a pass over i
constexpr size_t TABLE_BYTES = size_t(2) * (MAX_GROUPS + 2) * 4;
// bf16 output is staged: sixteen rows of D at 128 columns, two buffers for each half of the
// epilogue's warps; the rows' pitch puts neighbouring rows in different banks
constexpr int PITCH = 2 * HALF + 64;
constexpr int STAGED = 16 * PITCH;
constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + SF_SLOTS * SF_BYTES + 4 * STAGED +
                        TABLE_BYTES + 256;
static_assert(SMEM <= 232448, "shared memory budget of one CTA");
static_assert(SF_COL + SF_SETS * SF_COLS <= TMEM_COLS, "TMEM budget");

struct ProductParams {
  CUtensorMap map_p, map_q;
  const uint8_t* sp;        // scales of P and Q
  const uint8_t* sq;
  const int32_t* offsets;
  void* d;
  int64_t sp_ld, sq_ld, sp_group;  // sp_group: scale bytes between P's matrices
  int64_t ld;
  int32_t rows;             // t
  int32_t I, J;             // D's columns; D's rows (of a group, for MAO_TN)
  int32_t depth;            // K (MAO_TN: the group's rows)
  int32_t sp_rows;          // rows of scales of one matrix of P
  int32_t tiles_i, groups, form, dtype, accumulate, wide;
  unsigned long long timeout_ns;
};

struct Tile {
  int g;        // group
  int i0, j0;   // first i; first j (a row of D, or of the group's matrix)
  int j_end;    // rows of D in the tile end here
  int n;        // j computed (a multiple of 32), 0: the rows are only cleared
  int k0;       // first row of the depth (MAO_TN)
  int nkb;      // blocks of the depth
};

__device__ __forceinline__ uint64_t desc_of(uint32_t saddr, uint32_t lbo, uint32_t sbo,
                                            uint32_t swizzle) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(lbo >> 4) << 16) |
         (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(swizzle) << 61);
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 operands, scales of type ue8m0, M = 256.
__device__ __forceinline__ uint32_t instr_desc(int p_mn, int q_mn, int n, int byte) {
  return (uint32_t(byte) << 4) | (uint32_t(p_mn) << 15) | (uint32_t(q_mn) << 16) |
         (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(TILE >> 7) << 27) |
         (uint32_t(byte) << 29);
}

// The four 32-deep products of a block, issued by the elected lane of a converged warp: the
// operands' descriptors advance by dp and dq (in 16-byte units) from one to the next.
__device__ __forceinline__ void mma_block(uint32_t elected, uint32_t d, uint64_t p, uint64_t q,
                                          uint32_t dp, uint32_t dq, uint32_t idesc, uint32_t sp,
                                          uint32_t sq, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm volatile(
        "{\n\t.reg .pred a, e;\n\t"
        "setp.ne.b32 a, %6, 0;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
        "[%4], [%5], a;\n\t}\n" ::"r"(d),
        "l"(p + uint64_t(k) * dp), "l"(q + uint64_t(k) * dq), "r"(idesc), "r"(sp), "r"(sq),
        "r"(k ? 1u : accumulate), "r"(elected)
        : "memory");
  }
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e;
}

// 128 scale words (512 bytes of each CTA's shared memory) into four TMEM columns of both.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}

// Arrive that makes this thread's earlier writes visible to the leader CTA's waiter.
__device__ __forceinline__ void mbar_arrive_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// A wait of a whole warp: true once every lane has seen the phase complete.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          uint64_t limit) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_fast<CLUSTER>(smem_u32(bar), parity, abort_flag, limit));
}

// ------------------------------------------------------------------ tiles
//
// lo[g] (g <= groups) is the first row of group g, cut to 0 .. rows and made rising; lo[groups]
// is where the rows without a group begin. begin[g] counts the tiles of j before group g
// (MAO_NT, MAO_NN: of 256 rows each; MAO_TN: the same number for every group), begin[groups]
// those before the rest and begin[groups + 1] all of them.

__device__ __forceinline__ void make_table(const ProductParams& p, int* lo, int* begin) {
  const int tid = threadIdx.x;
  const int n = p.groups;
  if (!p.offsets) {
    if (tid == 0) {
      lo[0] = 0;
      lo[1] = p.rows;
    }
  } else {
    for (int g = tid; g <= n; g += THREADS) lo[g] = max(0, min(p.offsets[g], p.rows));
  }
  __syncthreads();
  if (tid < 32) {
    int high = 0, sum = 0;  // the largest offset and the tiles so far
    for (int base = 0; base <= n; base += 32) {
      const int g = base + tid;
      int v = g <= n ? lo[g] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (tid >= o) v = max(v, u);
      }
      v = max(v, high);
      if (g <= n) lo[g] = v;
      high = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    __syncwarp();
    for (int base = 0; base <= n; base += 32) {
      const int g = base + tid;
      int c = 0;
      if (p.form == MAO_TN) {
        c = g < n ? (p.J + TILE - 1) / TILE : 0;
      } else if (g < n) {
        c = (lo[g + 1] - lo[g] + TILE - 1) / TILE;
      } else if (g == n && !p.accumulate) {
        c = (p.rows - lo[n] + TILE - 1) / TILE;
      }
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (tid >= o) s += u;
      }
      if (g <= n) begin[g] = sum + s - c;
      sum += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (tid == 0) begin[n + 1] = sum;
  }
  __syncthreads();
}

__device__ __forceinline__ void decode(const ProductParams& p, const int* lo, const int* begin,
                                       int tile, Tile& t) {
  // the group whose tiles hold this one: the last with begin * tiles_i <= tile
  int a = 0, b = p.groups;
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (begin[m] * p.tiles_i <= tile) a = m;
    else b = m - 1;
  }
  t.g = a;
  const int count = begin[a + 1] - begin[a];
  int local = tile - begin[a] * p.tiles_i;
  // bands of BAND tiles of j: within a band j runs fastest, then i, so that the pairs at work
  // at one time share operand rows in both directions
  const int band = local / (BAND * p.tiles_i);
  local -= band * BAND * p.tiles_i;
  const int nb = min(BAND, count - band * BAND);
  const int jt = band * BAND + local % nb;
  t.i0 = (local / nb) * TILE;
  t.k0 = 0;
  if (p.form == MAO_TN) {
    t.j0 = jt * TILE;
    t.j_end = min(t.j0 + TILE, p.J);
    t.k0 = lo[a];
    t.nkb = (lo[a + 1] - lo[a] + BK - 1) / BK;
  } else {
    const int end = a < p.groups ? lo[a + 1] : p.rows;
    t.j0 = lo[a] + jt * TILE;
    t.j_end = min(t.j0 + TILE, end);
    t.nkb = a < p.groups ? (p.depth + BK - 1) / BK : 0;
  }
  t.n = t.nkb ? (t.j_end - t.j0 + 31) & ~31 : 0;
}

// The first tile from `tile` on (in steps) that multiplies anything.
__device__ __forceinline__ int next_tile(const ProductParams& p, const int* lo, const int* begin,
                                         int tile, int step, int total, Tile& t) {
  for (; tile < total; tile += step) {
    decode(p, lo, begin, tile, t);
    if (t.nkb) break;
  }
  return tile;
}

// ------------------------------------------------------------------ scales

// Four scale bytes down a column (stride ld), from block kb on; 1.0 past the last block.
__device__ __forceinline__ uint32_t bytes_down(const uint8_t* s, int64_t ld, int kb, int nkb) {
  uint32_t w = 0x7F7F7F7Fu;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (kb + q < nkb) w = (w & ~(0xFFu << (8 * q))) | (uint32_t(s[(kb + q) * ld]) << (8 * q));
  return w;
}
// Four consecutive scale bytes of a row.
__device__ __forceinline__ uint32_t bytes_along(const uint8_t* s, int kb, int nkb) {
  if (kb + 4 <= nkb && (reinterpret_cast<uintptr_t>(s + kb) & 3) == 0)
    return *reinterpret_cast<const uint32_t*>(s + kb);
  return bytes_down(s, 1, kb, nkb);
}

// Words of thread r: row r of this CTA's half of P, rows r and r + 128 of Q.
__device__ __forceinline__ void load_scales(const ProductParams& p, const Tile& t, int cta, int kb,
                                            int r, uint32_t (&w)[3]) {
  const int i = t.i0 + HALF * cta + r;
  const int row0 = t.k0 / BK;  // MAO_TN: the group's first row of scales
  if (p.form == MAO_TN) {
    w[0] = i < p.I ? bytes_down(p.sp + int64_t(row0) * p.sp_ld + i, p.sp_ld, kb, t.nkb) : 0x7F7F7F7Fu;
  } else {
    const uint8_t* s = p.sp + int64_t(t.g) * p.sp_group;
    w[0] = i >= p.I ? 0x7F7F7F7Fu
           : p.form == MAO_NT ? bytes_along(s + int64_t(i / BK) * p.sp_ld, kb, t.nkb)
                              : bytes_down(s + i / BK, p.sp_ld, kb, t.nkb);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = t.j0 + HALF * h + r;
    w[1 + h] = j >= t.j_end ? 0x7F7F7F7Fu
               : p.form == MAO_TN ? bytes_down(p.sq + int64_t(row0) * p.sq_ld + j, p.sq_ld, kb, t.nkb)
                                  : bytes_along(p.sq + int64_t(j) * p.sq_ld, kb, t.nkb);
  }
}

// ------------------------------------------------------------------ output

// Sixteen rows of D (from row j on, those below j_end) at column i of this lane.
__device__ __forceinline__ void store16(const ProductParams& p, const Tile& t, int j, int i,
                                        const float (&v)[16], int lane) {
  const bool in = i < p.I;
  int64_t row = j;
  if (p.form == MAO_TN) row += int64_t(t.g) * p.J;
  if (p.dtype == MAO_F32) {
    float* d = static_cast<float*>(p.d) + row * p.ld + i;
    if (p.accumulate) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (in && j + c < t.j_end) d[c * p.ld] += v[c];
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (in && j + c < t.j_end) d[c * p.ld] = v[c];
    }
    return;
  }
  __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + i;
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (in && j + c < t.j_end)
      d[c * p.ld] = __float2bfloat16_rn(p.accumulate ? __bfloat162float(d[c * p.ld]) + v[c] : v[c]);
}

// The same for bf16 rows that take 16-byte stores, by the four warps that hold 128 columns i
// (i0 is the first): they transpose their sixteen rows in `buf` and write whole 256-byte
// pieces of rows. Between two uses of a buffer lies the other buffer's barrier.
__device__ __forceinline__ void store16_wide(const ProductParams& p, const Tile& t, int j, int i0,
                                             const float (&v)[16], uint8_t* buf, int quad, int part,
                                             int lane) {
  // rows c and c + 1 of lanes 2 l and 2 l + 1: the even lane writes both columns of row c, the
  // odd lane both of row c + 1
  const int odd = lane & 1;
  uint8_t* s = buf + odd * PITCH + 2 * (32 * quad + lane - odd);
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[c], v[c + 1]);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
    const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    *reinterpret_cast<uint32_t*>(s + c * PITCH) = odd ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
  }
  asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
  const int i = i0 + 8 * (lane & 15);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = 4 * quad + 2 * h + (lane >> 4);
    if (j + c >= t.j_end || i >= p.I) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(buf + c * PITCH + 16 * (lane & 15));
    int64_t row = j + c;
    if (p.form == MAO_TN) row += int64_t(t.g) * p.J;
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + i;
    if (i + 8 <= p.I) {
      *reinterpret_cast<uint4*>(d) = x;
    } else {
      const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&x);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i + q < p.I) d[q] = e[q];
    }
  }
}

// ------------------------------------------------------------------ the kernel

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* sf = ring + STAGES * STAGE_BYTES;
  uint8_t* staging = sf + SF_SLOTS * SF_BYTES;
  int* lo = reinterpret_cast<int*>(staging + 4 * STAGED);
  int* begin = lo + MAX_GROUPS + 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 4 * STAGED + TABLE_BYTES);
  uint64_t* full_bar = bars;                    // [STAGES]    (used in the even CTA)
  uint64_t* empty_bar = full_bar + STAGES;      // [STAGES]
  uint64_t* sf_full_bar = empty_bar + STAGES;   // [SF_SLOTS]  (used in the even CTA)
  uint64_t* sf_empty_bar = sf_full_bar + SF_SLOTS;  // [SF_SLOTS]
  uint64_t* tfull_bar = sf_empty_bar + SF_SLOTS;    // [2]
  uint64_t* tempty_bar = tfull_bar + 2;         // [2]  all columns read   (even CTA)
  uint64_t* tshared_bar = tempty_bar + 2;       // [2]  shared columns read (even CTA)
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
  const int p_mn = p.form != MAO_NT, q_mn = p.form == MAO_TN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int s = 0; s < SF_SLOTS; ++s) {
      mbar_init(smem_u32(&sf_full_bar[s]), 2);
      mbar_init(smem_u32(&sf_empty_bar[s]), 1);
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
    const CUtensorMap* map = lane ? &p.map_q : &p.map_p;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  make_table(p, lo, begin);
  const int total = begin[p.groups + 1] * p.tiles_i;
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    // lane 0 loads this CTA's half of P, lane 1 its half of Q: P's rows i0 + 128 cta .., and
    // Q's rows j0 + n/2 cta .. (each CTA supplies half of the tile's n values of j)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t armed = 0, armed_phase = 0;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      Tile t;
      decode(p, lo, begin, tile, t);
      const int mn = lane == 0 ? t.i0 + HALF * int(cta) : t.j0 + (t.n >> 1) * int(cta);
      const int z = lane == 0 && p.form != MAO_TN ? t.g : 0;
      const bool mn_major = lane == 0 ? p_mn : q_mn;
      const CUtensorMap* map = lane == 0 ? &p.map_p : &p.map_q;
      for (int kb = 0; kb < t.nkb; ++kb) {
        int okw = 1;
        if (lane == 0) {
          if (!mbar_wait_fast(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, limit)) {
            okw = 0;
          } else if (leader) {
            mbar_expect_tx(smem_u32(&full_bar[stage]), 2 * STAGE_BYTES);
            armed |= 1u << stage;
            armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          }
        }
        okw = __shfl_sync(0xFFFFFFFFu, okw, 0);
        if (!okw) {
          ok = false;
          break;
        }
        if (lane < 2) {
          const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
          const uint32_t dst = smem_u32(ring + stage * STAGE_BYTES) + (lane ? OP_BYTES : 0);
          const int k = t.k0 + kb * BK;
          if (mn_major) tma_load_3d_pair(dst, map, fb, mn, k, z);
          else tma_load_3d_pair(dst, map, fb, k, mn, z);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // after an abort, the loads already issued land before the CTA leaves
    if (*abort_flag && leader && lane == 0) {
      for (int s = 0; s < STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(smem_u32(&full_bar[s]), (armed_phase >> s) & 1u, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp runs the loop, converged, so that descriptors stay in uniform registers;
    // one lane issues.
    if (leader) {
      const uint32_t elected = elect_one();
      const uint64_t p_desc = desc_of(smem_u32(ring), 16, 1024, 2);
      const uint64_t q_desc = desc_of(smem_u32(ring) + OP_BYTES, 16, 1024, 2);
      const uint64_t sf_desc = desc_of(smem_u32(sf), 16, 128, 0);
      // per 32-deep slice: 32 bytes along the swizzled rows (K-major), or four 1024-byte atoms
      // of eight k rows (MN-major)
      const uint32_t dp = p_mn ? 4096 >> 4 : 32 >> 4, dq = q_mn ? 4096 >> 4 : 32 >> 4;
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false, started = false;
      // Scale words: the slot of the blocks being multiplied (every three groups of blocks the
      // phase flips), the set of TMEM columns that holds them, and the slot copied next.
      int slot = 0, set = 0, copied = 0;
      uint32_t copied_phase = 0, before_phase = 1;
      int before = SF_SLOTS - 2;  // slot of the group two before the one copied next
      auto copy_next = [&]() {
        // the set's columns were last used two groups ago
        if (!wait_warp<false>(&sf_empty_bar[before], before_phase, abort_flag, limit) ||
            !wait_warp<true>(&sf_full_bar[copied], copied_phase, abort_flag, limit))
          return false;
        tc_fence_after();
        const uint32_t dst = tmem_base + uint32_t(SF_COL + SF_COLS * (set ^ (started ? 1 : 0)));
        const uint64_t src = sf_desc + uint64_t(copied * (SF_BYTES >> 4));
        if (elected) {
          copy_scales(dst, src);
          copy_scales(dst + 4, src + (512 >> 4));
          copy_scales(dst + 8, src + (1024 >> 4));
        }
        started = issued = true;
        if (++copied == SF_SLOTS) {
          copied = 0;
          copied_phase ^= 1u;
        }
        if (++before == SF_SLOTS) {
          before = 0;
          before_phase ^= 1u;
        }
        return true;
      };
      Tile t, next;
      int tile = next_tile(p, lo, begin, pair, npairs, total, t);
      if (tile < total) ok = copy_next();
      while (ok && tile < total) {
        const int after = next_tile(p, lo, begin, tile + npairs, npairs, total, next);
        const int acc = local & 1;
        // the accumulator's last tile has been read, and of the tile before this one the
        // columns that the two share
        if (!wait_warp<true>(&tempty_bar[acc], (uint32_t(local >> 1) & 1u) ^ 1u, abort_flag, limit) ||
            !wait_warp<true>(&tshared_bar[acc ^ 1], (uint32_t((local + 1) >> 1) & 1u) ^ 1u, abort_flag,
                             limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * ACC1);
        const uint32_t idesc0 = instr_desc(p_mn, q_mn, t.n, 0);
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!wait_warp<false>(&full_bar[stage], phase, abort_flag, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tsf = tmem_base + uint32_t(SF_COL + SF_COLS * set);
          const uint64_t at = uint64_t(stage * (STAGE_BYTES >> 4));
          mma_block(elected, d, p_desc + at, q_desc + at, dp, dq,
                    idesc0 | uint32_t(kb & 3) << 4 | uint32_t(kb & 3) << 29, tsf, tsf + 4,
                    kb != 0 ? 1u : 0u);
          issued = true;
          if (elected) umma_commit_pair(smem_u32(&empty_bar[stage]), 3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          const bool last = (kb & 3) == 3 || kb + 1 == t.nkb;
          // the next scale words follow two or three blocks behind the current ones: by then
          // the slot's last products are done, and the copy is done before it is needed
          if (((kb & 3) == 2 || (last && (kb & 3) < 2)) && ((kb | 3) + 1 < t.nkb || after < total)) {
            if (!copy_next()) {
              ok = false;
              break;
            }
          }
          if (last) {
            if (elected) umma_commit_pair(smem_u32(&sf_empty_bar[slot]), 3);
            if (++slot == SF_SLOTS) slot = 0;
            set ^= 1;
          }
        }
        if (!ok) break;
        if (elected) umma_commit_pair(smem_u32(&tfull_bar[acc]), 3);
        ++local;
        tile = after;
        t = next;
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
    int local = 0;
    for (int tile = pair; tile < total; tile += npairs) {
      Tile t;
      decode(p, lo, begin, tile, t);
      const int i = t.i0 + HALF * int(cta) + 32 * quad + lane;
      float v[16];
      if (t.nkb == 0) {  // nothing was multiplied: D is cleared (or stays, when added to)
        if (p.accumulate) continue;
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = 0.0f;
        for (int c = 16 * part; c < t.j_end - t.j0; c += 32) store16(p, t, t.j0 + c, i, v, lane);
        continue;
      }
      const int acc = local & 1;
      // every lane waits; the warp goes on only if all of them saw the accumulator
      if (!wait_warp<false>(&tfull_bar[acc], uint32_t(local >> 1) & 1u, abort_flag, limit)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t(32 * quad) << 16) + uint32_t(acc * ACC1);
      // this warp's 128 columns in eight steps: its half of the shared ones, then the others
      const int shared0 = (acc ? 0 : ACC1) + 16 * part;
      const int rest0 = (acc ? SHARED : 0) + (ACC1 / 2) * part;
#pragma unroll 1
      for (int s = 0; s < 8; ++s) {
        const int c = s == 0 ? shared0 : rest0 + 16 * (s - 1);
        const bool any = c < t.j_end - t.j0;
        if (any) tmem_ld16(trow + uint32_t(c), v);
        if (s == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tshared[acc]);
        } else if (s == 7) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty[acc]);
        }
        if (!any) continue;
        if (p.wide) store16_wide(p, t, t.j0 + c, i - 32 * quad - lane, v, staging + (2 * part + (s & 1)) * STAGED, quad, part, lane);
        else store16(p, t, t.j0 + c, i, v, lane);
      }
      ++local;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scales (both CTAs)
    // The warps take the groups of four blocks in turn, each into its own slot, so that one
    // group's loads and its hand-over (a release to the other CTA) have the time of three
    // groups' products.
    const int slot = warp - 2 - EPI_WARPS;
    Tile t;
    int tile = next_tile(p, lo, begin, pair, npairs, total, t);
    int kb = 0, turn = 0;
    uint32_t phase = 0;
    while (tile < total) {
      if (turn == slot) {
        uint32_t w[4][3];
#pragma unroll
        for (int q = 0; q < 4; ++q) load_scales(p, t, int(cta), kb, 32 * q + lane, w[q]);
        if (!wait_warp<false>(&sf_empty_bar[slot], phase ^ 1u, abort_flag, limit)) break;
        // word r of 128: row r % 32 of 16 bytes, column r / 32
        uint8_t* dst = sf + slot * SF_BYTES + 16 * lane;
#pragma unroll
        for (int h = 0; h < 3; ++h)
          *reinterpret_cast<uint4*>(dst + 512 * h) = make_uint4(w[0][h], w[1][h], w[2][h], w[3][h]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_release(mapa_shared(smem_u32(&sf_full_bar[slot]), 0));
      }
      if (++turn == SF_WARPS) {
        turn = 0;
        phase ^= 1u;
      }
      kb += 4;
      if (kb >= t.nkb) {
        kb = 0;
        tile = next_tile(p, lo, begin, tile + npairs, npairs, total, t);
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

}  // namespace

mao_status product_launch(const mao_fp8& A, const mao_fp8& B, const mao_mat& D, int32_t form,
                          const int32_t* offsets, int32_t groups, int32_t accumulate,
                          cudaStream_t stream) {
  const bool tn = form == MAO_TN;
  const int es = elem_size(D.dtype);
  if (A.rows == 0) {  // no rows of D, or sums over nothing
    if (!tn || accumulate) return MAO_OK;
    return cuda_status(cudaMemset2DAsync(D.data, size_t(D.ld) * es, 0, size_t(D.cols) * es,
                                         size_t(D.rows), stream));
  }
  ProductParams p = {};
  mao_status st = tc_encode_code_map(&p.map_p, B.codes, B.cols, B.rows, B.ld, B.count, HALF);
  if (st == MAO_OK) st = tc_encode_code_map(&p.map_q, A.codes, A.cols, A.rows, A.ld, 1, HALF);
  if (st != MAO_OK) return st;
  p.sp = B.scales;
  p.sq = A.scales;
  p.sp_ld = B.scale_ld;
  p.sq_ld = A.scale_ld;
  p.sp_group = tn ? 0 : ceil_div(B.rows, 128) * B.scale_ld;
  p.offsets = offsets;
  p.d = D.data;
  p.ld = D.ld;
  p.rows = int32_t(A.rows);
  p.I = int32_t(D.cols);
  p.J = int32_t(tn ? A.cols : A.rows);
  p.depth = int32_t(A.cols);
  p.tiles_i = int32_t(ceil_div(D.cols, TILE));
  p.groups = groups;
  p.form = form;
  p.dtype = D.dtype;
  p.accumulate = accumulate != 0;
  p.wide = D.dtype == MAO_BF16 && !accumulate && reinterpret_cast<uintptr_t>(D.data) % 16 == 0 && D.ld % 8 == 0;
  p.timeout_ns = wait_limit_ns();
  // tiles at most: every group may end in a part of one
  const int64_t tiles = (tn ? ceil_div(p.J, TILE) * groups : ceil_div(A.rows, TILE) + groups + 1) * p.tiles_i;
  if (tiles > 0x7FFFFFFF || A.cols > 0x7FFFFFFF || B.cols > 0x7FFFFFFF) return MAO_ERR_UNSUPPORTED;
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MAO_ERR_CUDA;
  cudaError_t attr = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    attr = cudaFuncSetAttribute(product_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
  });
  if (attr != cudaSuccess) return MAO_ERR_CUDA;
  const int64_t pairs = tiles < num_sms() / 2 ? tiles : num_sms() / 2;
  product_kernel<<<unsigned(2 * pairs), THREADS, SMEM, stream>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

mao_status product_read_and_clear_error(cudaStream_t stream) { return read_and_clear_error(stream); }

}  // namespace mao
