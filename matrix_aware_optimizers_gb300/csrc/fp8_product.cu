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
//   warp 0        TMA producer: a 128 x 128 box of P and the tile's rows of Q per 128-deep
//                 block, into a ring of six 32 KB stages
//   warp 1        TMEM allocation; in the even CTA the whole warp runs the loop, converged, and
//                 one lane copies the scale words into TMEM (tcgen05.cp) and issues the products
//                 (issued from a divergent lane, the descriptors' arithmetic cost more than the
//                 products: 387 us against 338 on the dense forward below)
//   warps 2..9    epilogue: two warps per 32-lane quadrant of TMEM; lane = i, so a warp
//                 stores rows as they come: 128 bytes of an fp32 row, or, by pairs of lanes
//                 that swap halves, 64 bytes of two bf16 rows; past L1 (no_allocate: the fp32
//                 gradient below went from 358 to 326 us by that alone). Transposing bf16 rows in
//                 shared memory for wider stores or bulk copies made no difference (335, 334
//                 and 333 us dense, each in a run); fp32 rows got slower (423 and 468 us)
//   warps 10..12  scales: gather the scale bytes of four blocks, from whichever layout they
//                 have, into the words that tcgen05.cp expects
// TMEM (512 columns) holds two accumulators of 256 columns that share 32 of them (columns
// 0..255 and 224..479) and two sets of scale words (480..503). The shared columns are drained
// first: the next tile's products wait for them only, so the rest of a tile's epilogue runs
// under the next tile's products. Without sharing, tiles of 224 columns fit twice; they were
// slower (320 against 301 us dense), as every block of P then serves fewer columns.
//
// What bounds it: a pair's block of 256 x 256 x 128 takes 512 cycles of the tensor cores and
// brings 32 KB into each SM. Dense products that run back to back meet the power limit. Over groups,
// forward, the tensor cores' cycles are 106 us at 1.76 GHz and 12.6 MB come into each SM (41 bytes per
// cycle over the kernel's time); what fills the rest of its 175 us is known in part only. Parts of the
// work taken out (of 174 us): no stores 156, no loads of Q 165, all loads from the same L2 lines 154;
// the tensor pipe is active 58% of the time. Measured in a graph of ten calls and in a run of
// 0.15 s (ranges: on different cards), on experts 128 x [1536 x 2048], 65,536 rows:
//   dense 8192 x 14336 x 4096, bf16 out     288 to 293 us (3.3 PFLOP/s), 329 to 344 us in a run
//   forward (nt), bf16 out                  175 us (2.3 PFLOP/s), 193 to 206 us in a run
//   input gradient (nn, 128 x [2048 x 768], 60,007 rows)  92 us, 99 to 103 us in a run
//   weight gradient (tn), fp32 out          316 us, 324 to 330 in a run (5.7 TB/s: its 1.6 GB of outputs)
// Dense nn and tn of the same sizes take 307 and (fp32) 313 us. Adding to D reads and writes it entry
// by entry, each after the one before: 760 us for that tn, 4.7 ms for the experts'.
// Barriers and their bounded waits are as in the Newton–Schulz product kernel.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <atomic>

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
constexpr int Q_BOXES = 4;                 // heights of boxes of Q: 16 << b rows
constexpr int BAND = 8;                    // tiles of j that share a pass over i
constexpr size_t TABLE_BYTES = size_t(2) * (MAX_GROUPS + 2) * 4;
constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + SF_SLOTS * SF_BYTES + TABLE_BYTES + 256;
static_assert(SMEM <= 232448, "shared memory budget of one CTA");
static_assert(SF_COL + SF_SETS * SF_COLS <= TMEM_COLS, "TMEM budget");

struct ProductParams {
  CUtensorMap map_p;
  CUtensorMap map_q[Q_BOXES];  // boxes of 16, 32, 64, 128 rows (MAO_TN: the last only)
  const uint8_t* sp;        // scales of P and Q
  const uint8_t* sq;
  const int32_t* offsets;
  void* d;
  int64_t sp_ld, sq_ld, sp_group;  // sp_group: scale bytes between P's matrices
  int64_t ld;
  int32_t rows;             // t
  int32_t I, J;             // D's columns; D's rows (of a group, for MAO_TN)
  int32_t depth;            // K (MAO_TN: the group's rows)
  int32_t tiles_i, groups, dtype, accumulate, paired;
  int32_t sp_words, sq_words;  // scales allow 4-byte loads
  int32_t splits, split_kb;    // parts of the depth (one group), blocks of each
  unsigned long long timeout_ns;
};

struct Tile {
  int g = 0;    // group
  int i0, j0;   // first i; first j (a row of D, or of the group's matrix)
  int j_end;    // rows of D in the tile end here
  int n;        // j computed (a multiple of 32), 0: the rows are only cleared
  int k0;       // first row of the depth (MAO_TN)
  int kb0;      // first block of the depth (of a split)
  int nkb;      // blocks of the depth
  int64_t row0; // row of the output that j counts from
};

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

// 128 scale words (512 bytes of each CTA's shared memory) into four TMEM columns of both, for
// the three sets of words of a slot.
__device__ __forceinline__ void copy_scales(uint32_t elected, uint32_t taddr, uint64_t desc) {
#pragma unroll
  for (int h = 0; h < 3; ++h)
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}\n" ::"r"(taddr + 4 * h),
        "l"(desc + uint64_t(h * (512 >> 4))), "r"(elected)
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

// ------------------------------------------------------------------ tiles
//
// lo[g] (g <= groups) is the first row of group g, cut to 0 .. rows and made rising; the rows before
// lo[0] and from lo[groups] on have no group. begin[g] counts the tiles of j before group g
// (MAO_NT, MAO_NN: of its rows; MAO_TN: the same number for every group), begin[groups] all.

template <int FORM>
__device__ __forceinline__ void make_table(const ProductParams& p, int* lo, int* begin, int* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  bool falls = false;
  for (int g = tid; g < n; g += THREADS) falls = falls || lo[g + 1] < lo[g];
  if (__syncthreads_or(falls)) {  // offsets that fall are raised to the largest before them
    if (tid == 0)
      for (int g = 0; g < n; ++g) lo[g + 1] = max(lo[g + 1], lo[g]);
    __syncthreads();
  }
  // thread i (of 256) sums the tiles of groups 4 i .. 4 i + 3
  int c[4], own = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int g = 4 * tid + q;
    c[q] = g >= n ? 0 : FORM == MAO_TN ? (p.J + TILE - 1) / TILE : (lo[g + 1] - lo[g] + TILE - 1) / TILE;
    own += c[q];
  }
  int s = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  for (int w = 0; w < warp; ++w) s += sums[w];
  s -= own;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int g = 4 * tid + q;
    if (g <= n) begin[g] = s;
    s += c[q];
  }
}

// A split's share of the depth, and its rows of the partial sums.
__device__ __forceinline__ void take_split(const ProductParams& p, int split, Tile& t) {
  t.kb0 = 0;
  if (p.splits > 1) {
    t.kb0 = split * p.split_kb;
    t.nkb = min(p.split_kb, t.nkb - t.kb0);
    t.row0 = int64_t(split) * p.J;
  }
}

// The whole warp decodes: t.g is a group at or before the tile's (tiles come in rising order).
template <int FORM>
__device__ __forceinline__ void decode(const ProductParams& p, const int* lo, const int* begin,
                                       int tile, Tile& t) {
  int split = 0;
  if (p.splits > 1) {
    const int tiles = begin[1] * p.tiles_i;
    split = tile / tiles;
    tile -= split * tiles;
  }
  // the last group with begin * tiles_i <= tile: the one whose tiles hold this one
  const int lane = threadIdx.x & 31;
  int a = t.g;
  while (true) {
    const int g = a + 1 + lane;
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, g >= p.groups || begin[g] * p.tiles_i > tile);
    if (past) {
      a += __ffs(past) - 1;
      break;
    }
    a += 32;
  }
  t.g = a;
  const int count = begin[a + 1] - begin[a];
  int local = tile - begin[a] * p.tiles_i;
  if (FORM == MAO_TN) {
    // i runs fastest: the pairs at work at one time write whole rows of a matrix
    const int jt = local / p.tiles_i;
    t.i0 = (local - jt * p.tiles_i) * TILE;
    t.j0 = jt * TILE;
    t.j_end = min(t.j0 + TILE, p.J);
    t.k0 = lo[a];
    t.nkb = (lo[a + 1] - lo[a] + BK - 1) / BK;
    t.row0 = int64_t(a) * p.J;
    take_split(p, split, t);
    t.n = t.nkb ? (t.j_end - t.j0 + 31) & ~31 : 0;
    return;
  }
  // bands of BAND tiles of j: within a band j runs fastest, then i, so that the pairs at work
  // at one time share operand rows in both directions
  const int band = count > BAND ? local / (BAND * p.tiles_i) : 0;
  local -= band * BAND * p.tiles_i;
  const int nb = min(BAND, count - band * BAND);
  // local / nb by a float product: exact below 2^21 (half a unit is kept to either side)
  const int it = int((float(local) + 0.5f) * (1.0f / float(nb)));
  const int jt = band * BAND + local - it * nb;
  t.i0 = it * TILE;
  t.k0 = 0;
  // a group's tiles are of even height: those of up to 224 rows do not share TMEM columns
  const int rows = lo[a + 1] - lo[a];
  // ((rows - 1) / count + 1 is the quotient rounded up: rows + count may pass 2^31)
  const int height = count > 1 ? ((rows - 1) / count + 32) & ~31 : TILE;
  t.j0 = lo[a] + jt * height;
  t.j_end = min(t.j0 + height, lo[a + 1]);
  t.nkb = (p.depth + BK - 1) / BK;
  t.row0 = 0;
  take_split(p, split, t);
  t.n = t.nkb ? (t.j_end - t.j0 + 31) & ~31 : 0;
}

// The first tile from `tile` on (in steps) that multiplies anything.
template <int FORM>
__device__ __forceinline__ int next_tile(const ProductParams& p, const int* lo, const int* begin,
                                         int tile, int step, int total, Tile& t) {
  for (; tile < total; tile += step) {
    decode<FORM>(p, lo, begin, tile, t);
    if (t.nkb) break;
  }
  return tile;
}

// ------------------------------------------------------------------ scales

// Where the scales come from takes a path of their own, since their bytes lie in the order of
// the quantised tensor: a byte per row and block, or per block and column, or per tile. A lane
// issues all of a group's loads before it uses one (done byte by byte, each waiting for the one
// before, the weight gradient took 394 us instead of 369).
//
// The scale words of four blocks (from kb on) for 128 rows, row r as tcgen05.cp expects it: at
// 16 (r % 32) + 4 (r / 32). Each lane of a warp gathers four words; the loads of a group are
// all issued before the first is used. Blocks past the last and rows past `n` get 1.0 (they
// meet zeros, or outputs that are not stored).
constexpr uint32_t ONES = 0x7F7F7F7Fu;

// Scales that run along the rows (one row of scales per row): row r's at s + r * ld. Lane l
// holds rows l + 32 q.
struct Along {
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint8_t* s, int64_t ld, int n, int kb, int nkb,
                                       bool words, int lane) {
    if (words && kb + 4 <= nkb) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = lane + 32 * q;
        w[q] = r < n ? *reinterpret_cast<const uint32_t*>(s + r * ld + kb) : ONES;
      }
    } else {
      uint32_t b[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = lane + 32 * q;
          b[q][k] = r < n && kb + k < nkb ? s[r * ld + kb + k] : 0x7Fu;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = b[q][0] | b[q][1] << 8 | b[q][2] << 16 | b[q][3] << 24;
    }
  }
  __device__ __forceinline__ void store(uint8_t* dst, int lane) const {
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Scales that run across them (one row of scales per block): block k's at s + k * ld. Lane l
// holds rows 4 l .. 4 l + 3, loaded four bytes of one block at a time and transposed.
struct Across {
  uint32_t w[4];  // by block until store
  __device__ __forceinline__ void load(const uint8_t* s, int64_t ld, int n, int kb, int nkb,
                                       bool words, int lane) {
    const int r = 4 * lane;
    if (words && r + 4 <= n) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = kb + k < nkb ? *reinterpret_cast<const uint32_t*>(s + (kb + k) * ld + r) : ONES;
    } else {
      uint32_t b[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          b[k][q] = r + q < n && kb + k < nkb ? s[(kb + k) * ld + r + q] : 0x7Fu;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = b[k][0] | b[k][1] << 8 | b[k][2] << 16 | b[k][3] << 24;
    }
  }
  __device__ __forceinline__ void store(uint8_t* dst, int lane) const {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
    const uint32_t o[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                           __byte_perm(c, d, 0x5410), __byte_perm(c, d, 0x7632)};
    // rows 4 l + q: 16-byte rows (4 l + q) % 32, column l / 8
    uint8_t* at = dst + 64 * (lane & 7) + 4 * (lane >> 3);
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint32_t*>(at + 16 * q) = o[q];
  }
};

// Scales of 128 x 128 tiles: the same word for all rows; block k's byte at s + k * step.
struct Same {
  uint32_t w;
  __device__ __forceinline__ void load(const uint8_t* s, int64_t step, int n, int kb, int nkb, int lane) {
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = n > 0 && kb + k < nkb ? s[(kb + k) * step] : 0x7Fu;
    w = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
  }
  __device__ __forceinline__ void store(uint8_t* dst, int lane) const {
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w, w, w, w);
  }
};

// Scale words of a group of blocks: 128 rows of this CTA's half of P, 256 of Q.
template <int FORM>
struct Scales;
template <>
struct Scales<MAO_TN> {
  Across p0, q0, q1;
  __device__ __forceinline__ void load(const ProductParams& p, const Tile& t, int cta, int kb, int lane) {
    const int end = t.kb0 + t.nkb;
    const int row0 = t.k0 / BK, i = t.i0 + HALF * cta;  // the group's first row of scales
    const uint8_t* sp = p.sp + row0 * p.sp_ld + i;
    const uint8_t* sq = p.sq + row0 * p.sq_ld + t.j0;
    p0.load(sp, p.sp_ld, p.I - i, kb, end, p.sp_words, lane);
    q0.load(sq, p.sq_ld, t.j_end - t.j0, kb, end, p.sq_words, lane);
    q1.load(sq + HALF, p.sq_ld, t.j_end - t.j0 - HALF, kb, end, p.sq_words, lane);
  }
};
template <int FORM>
struct Scales {
  Same p0;
  Along q0, q1;
  __device__ __forceinline__ void load(const ProductParams& p, const Tile& t, int cta, int kb, int lane) {
    const int end = t.kb0 + t.nkb;
    const int i = t.i0 + HALF * cta;
    const uint8_t* sp = p.sp + int64_t(t.g) * p.sp_group;
    if (FORM == MAO_NT) p0.load(sp + int64_t(i / BK) * p.sp_ld, 1, p.I - i, kb, end, lane);
    else p0.load(sp + i / BK, p.sp_ld, p.I - i, kb, end, lane);
    const uint8_t* sq = p.sq + int64_t(t.j0) * p.sq_ld;
    q0.load(sq, p.sq_ld, t.j_end - t.j0, kb, end, p.sq_words, lane);
    q1.load(sq + HALF * p.sq_ld, p.sq_ld, t.j_end - t.j0 - HALF, kb, end, p.sq_words, lane);
  }
};

// ------------------------------------------------------------------ output

// Sixteen rows of D (from row j on, those below j_end) at column i of this lane.
__device__ __forceinline__ void store16(const ProductParams& p, const Tile& t, int j, int i,
                                        const float (&v)[16], int lane) {
  const bool in = i < p.I;
  const int64_t row = t.row0 + j;
  if (p.dtype == MAO_F32) {
    float* d = static_cast<float*>(p.d) + row * p.ld + i;
    if (p.accumulate) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (in && j + c < t.j_end) d[c * p.ld] += v[c];
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (in && j + c < t.j_end)
          asm volatile("st.global.L1::no_allocate.f32 [%0], %1;" ::"l"(d + c * p.ld), "f"(v[c]) : "memory");
    }
    return;
  }
  __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + i;
  if (p.paired) {
    // rows c and c + 1 of lanes 2 l and 2 l + 1: the even lane writes both columns of row c, the
    // odd lane both of row c + 1
    const int odd = lane & 1;
    d += odd ? p.ld - 1 : 0;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[c], v[c + 1]);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      const uint32_t both = odd ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
      if (in && j + c + odd < t.j_end)  // an even number of columns: both or none are there
        asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(d), "r"(both) : "memory");
      d += 2 * p.ld;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (in && j + c < t.j_end)
      d[c * p.ld] = __float2bfloat16_rn(p.accumulate ? __bfloat162float(d[c * p.ld]) + v[c] : v[c]);
}

// Clears columns i0 .. i0 + ni of rows j0 .. j1 of D, one row per turn of a warp.
__device__ __forceinline__ void clear_rows(const ProductParams& p, int64_t j0, int64_t j1, int64_t step,
                                           int i0, int ni, int lane) {
  const int es = p.dtype == MAO_F32 ? 4 : 2;
  uint8_t* base = static_cast<uint8_t*>(p.d) + int64_t(i0) * es;
  const int bytes = ni * es;
  const bool vec = reinterpret_cast<uintptr_t>(base) % 16 == 0 && p.ld * es % 16 == 0;
  for (int64_t j = j0; j < j1; j += step) {
    uint8_t* d = base + j * p.ld * es;
    int done = 0;
    if (vec) {
      for (int b = 16 * lane; b + 16 <= bytes; b += 512) *reinterpret_cast<uint4*>(d + b) = make_uint4(0u, 0u, 0u, 0u);
      done = bytes & ~15;
    }
    for (int b = done + 2 * lane; b < bytes; b += 64) *reinterpret_cast<uint16_t*>(d + b) = 0;
  }
}

// ------------------------------------------------------------------ the kernel

template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* sf = ring + STAGES * STAGE_BYTES;
  int* lo = reinterpret_cast<int*>(sf + SF_SLOTS * SF_BYTES);
  int* begin = lo + MAX_GROUPS + 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf + SF_SLOTS * SF_BYTES + TABLE_BYTES);
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
  constexpr int p_mn = FORM != MAO_NT, q_mn = FORM == MAO_TN;

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
    const CUtensorMap* map = lane ? &p.map_q[Q_BOXES - 1] : &p.map_p;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  // launched as a programmatic dependent: the set-up so far may overlap the previous kernel
  wait_for_previous();
  make_table<FORM>(p, lo, begin, reinterpret_cast<int*>(sf));
  tc_fence_before();
  __syncthreads();
  const int total = begin[p.groups] * p.tiles_i * p.splits;
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    // P's rows i0 + 128 cta .. and Q's rows j0 + n/2 cta .. (each CTA supplies half of the
    // tile's n values of j). The whole warp runs the loop, converged; one lane issues.
    const uint32_t elected = elect_one();
    const uint32_t full0 = mapa_shared(smem_u32(full_bar), 0);
    const uint32_t ring0 = smem_u32(ring);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t armed = 0, armed_phase = 0;
    Tile t;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      decode<FORM>(p, lo, begin, tile, t);
      const int i = t.i0 + HALF * int(cta), j = t.j0 + (t.n >> 1) * int(cta);
      const int z = FORM != MAO_TN ? t.g : 0;
      // this CTA's n / 2 rows of Q, a multiple of 16: one box each for its bits
      const int q_rows = q_mn ? HALF : t.n >> 1;
      const uint32_t q_bytes = uint32_t(q_rows) * BK;
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&empty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        const uint32_t fb = full0 + 8 * stage, dst = ring0 + stage * STAGE_BYTES;
        const int k = t.k0 + (t.kb0 + kb) * BK;
        if (elected) {
          if (leader) mbar_expect_tx(smem_u32(&full_bar[stage]), 2 * (OP_BYTES + q_bytes));
          if (p_mn) tma_load_3d_pair(dst, &p.map_p, fb, i, k, z);
          else tma_load_3d_pair(dst, &p.map_p, fb, k, i, z);
          if (q_mn) tma_load_3d_pair(dst + OP_BYTES, &p.map_q[Q_BOXES - 1], fb, j, k, 0);
          else if (q_rows == HALF) tma_load_3d_pair(dst + OP_BYTES, &p.map_q[Q_BOXES - 1], fb, k, j, 0);
          else
            for (int b = Q_BOXES - 2, at = 0; b >= 0; --b)
              if (q_rows & (16 << b)) {
                tma_load_3d_pair(dst + OP_BYTES + at * BK, &p.map_q[b], fb, k, j + at, 0);
                at += 16 << b;
              }
        }
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
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
      int stage = 0, local = 0, before_n = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false, ready = false;
      // Scale words: the slot of the blocks being multiplied, the set of TMEM columns that holds
      // them, and the slot copied next (copied just before its products; earlier copies, one to
      // three blocks ahead, were up to 3% slower).
      int slot = 0, set = 0, copied = 0;
      uint32_t copied_phase = 0, before_phase = 1;
      int before = SF_SLOTS - 2;  // slot of the group two before the one copied next
      auto copy_next = [&]() {
        // the set's columns were last used two groups ago
        if (!wait_warp<false>(&sf_empty_bar[before], before_phase, abort_flag, limit) ||
            !wait_warp<true>(&sf_full_bar[copied], copied_phase, abort_flag, limit))
          return false;
        copy_scales(elected, tmem_base + uint32_t(SF_COL + SF_COLS * set),
                    sf_desc + uint64_t(copied * (SF_BYTES >> 4)));
        issued = true;
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
      int tile = next_tile<FORM>(p, lo, begin, pair, npairs, total, t);
      if (tile < total) ok = copy_next();
      while (ok && tile < total) {
        const int after = next_tile<FORM>(p, lo, begin, tile + npairs, npairs, total, next);
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
        const uint32_t idesc0 = instr_desc(p_mn, q_mn, t.n, 0);
        for (int kb = 0; kb < t.nkb; ++kb) {
          // the stage was looked at while the products before were issued
          if (!__all_sync(0xFFFFFFFFu, ready) && !wait_warp<false>(&full_bar[stage], phase, abort_flag, limit)) {
            ok = false;
            break;
          }
          const uint32_t empty = smem_u32(&empty_bar[stage]);
          const uint64_t at = uint64_t(stage * (STAGE_BYTES >> 4));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ready = limit != 0 && mbar_test_wait(smem_u32(&full_bar[stage]), phase);
          const uint32_t tsf = tmem_base + uint32_t(SF_COL + SF_COLS * set);
          mma_block(elected, d, p_desc + at, q_desc + at, dp, dq,
                    idesc0 | uint32_t(kb & 3) << 4 | uint32_t(kb & 3) << 29, tsf, tsf + 4,
                    kb != 0 ? 1u : 0u);
          issued = true;
          commit_both(elected, empty);
          if ((kb & 3) == 3 || kb + 1 == t.nkb) {  // the last block of its scale words
            commit_both(elected, smem_u32(&sf_empty_bar[slot]));
            if (++slot == SF_SLOTS) slot = 0;
            set ^= 1;
            if (kb + 1 < t.nkb && !copy_next()) {
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        commit_both(elected, smem_u32(&tfull_bar[acc]));
        if (after < total) ok = copy_next();
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
    // rows before the first group and past the last are cleared while the first tiles are multiplied
    if (FORM != MAO_TN && !p.accumulate) {
      const int64_t turn = int64_t(blockIdx.x) * EPI_WARPS + warp - 2, turns = int64_t(gridDim.x) * EPI_WARPS;
      clear_rows(p, turn, lo[0], turns, 0, p.I, lane);
      clear_rows(p, lo[p.groups] + turn, p.rows, turns, 0, p.I, lane);
    }
    int local = 0;
    Tile t;
    for (int tile = pair; tile < total; tile += npairs) {
      decode<FORM>(p, lo, begin, tile, t);
      const int i = t.i0 + HALF * int(cta) + 32 * quad + lane;
      if (t.nkb == 0) {  // MAO_TN: an empty group's matrix is cleared (or stays, when added to)
        const int i0 = t.i0 + HALF * int(cta);
        if (!p.accumulate)
          clear_rows(p, t.row0 + t.j0 + warp - 2, t.row0 + t.j_end, EPI_WARPS, i0, min(HALF, p.I - i0), lane);
        continue;
      }
      const int acc = local & 1;
      // every lane waits; the warp goes on only if all of them saw the accumulator
      if (!wait_warp<false>(&tfull_bar[acc], uint32_t(local >> 1) & 1u, abort_flag, limit)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t(32 * quad) << 16) + uint32_t(acc * ACC1);
      // this warp's 128 columns in eight steps: its half of the shared ones, then of the others
      // (every second sixteen, so that both warps have work in small tiles)
      const int shared0 = (acc ? 0 : ACC1) + 16 * part;
      const int rest0 = (acc ? SHARED : 0) + 16 * part;
      const int n = t.j_end - t.j0;
      auto column = [&](int s) { return s == 0 ? shared0 : rest0 + 32 * (s - 1); };
      auto out = [&](int s, const float(&v)[16]) {
        const int c = column(s);
        if (c >= n) return;
        store16(p, t, t.j0 + c, i, v, lane);
      };
      // a step's columns are loaded while the step before is stored
      float va[16], vb[16];
      if (column(0) < n) tmem_ld16(trow + uint32_t(column(0)), va);
#pragma unroll 1
      for (int s = 0; s < 8; s += 2) {
        tmem_wait(va);
        if (s == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tshared[acc]);
        }
        if (column(s + 1) < n) tmem_ld16(trow + uint32_t(column(s + 1)), vb);
        out(s, va);
        tmem_wait(vb);
        if (s == 6) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty[acc]);
        } else if (column(s + 2) < n) {
          tmem_ld16(trow + uint32_t(column(s + 2)), va);
        }
        out(s + 1, vb);
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
    uint8_t* dst = sf + slot * SF_BYTES;
    const uint32_t full = mapa_shared(smem_u32(&sf_full_bar[slot]), 0);
    Tile t;
    int tile = next_tile<FORM>(p, lo, begin, pair, npairs, total, t);
    int kb = 0;
    auto skip = [&](int groups) {
      for (int q = 0; q < groups && tile < total; ++q) {
        kb += 4;
        if (kb >= t.nkb) {
          kb = 0;
          tile = next_tile<FORM>(p, lo, begin, tile + npairs, npairs, total, t);
        }
      }
    };
    skip(slot);
    Scales<FORM> w;
    if (tile < total) w.load(p, t, int(cta), t.kb0 + kb, lane);
    uint32_t phase = 0;
    while (tile < total) {
      if (!wait_warp<false>(&sf_empty_bar[slot], phase ^ 1u, abort_flag, limit)) break;
      w.p0.store(dst, lane);
      w.q0.store(dst + 512, lane);
      w.q1.store(dst + 1024, lane);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_release(full);
      phase ^= 1u;
      skip(SF_WARPS);
      if (tile < total) w.load(p, t, int(cta), t.kb0 + kb, lane);
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

// D = (D +) the sum of the splits' partial sums, in their order; four columns per thread.
struct SumParams {
  const float* parts;
  void* d;
  int64_t rows, cols, pld, ld;
  int32_t splits, dtype, accumulate, vec;
};

__global__ void __launch_bounds__(256) split_sum_kernel(const SumParams p) {
  wait_for_previous();
  const int64_t quads = p.pld / 4, all = p.rows * quads;
  for (int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x; q < all; q += int64_t(gridDim.x) * 256) {
    const int64_t j = q / quads, i = 4 * (q - j * quads);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(p.parts + (s * p.rows + j) * p.pld + i);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    const int64_t at = j * p.ld + i;
    if (p.accumulate) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < p.cols) v[c] += load_elem(p.d, at + c, p.dtype);
    }
    if (p.vec && i + 4 <= p.cols) {
      if (p.dtype == MAO_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.d) + at) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.d) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < p.cols) store_elem(p.d, at + c, p.dtype, v[c]);
    }
  }
}

// How many parts the depth of a product without groups is split into when its tiles leave
// pairs of SMs idle: the number with the least time by a model of the two kernels (about
// 0.25 us per block of the depth; 2.5 us for the second kernel and 3 TB/s for the partial
// sums, which stay in L2), parts of whole scale words. In parts and whole (us, fp32 out): 768 x 768
// over 32,768 rows 26.5 and 75.7, over 8192 16.2 and 25.2; 256 x 256 over 4096 11.9 and 16.0; 2048 x
// 768 over 131,072 129 and 280; 1 x 4096 over 14,336 18.0 and 35.3, 16 rows 16.2 and 31.0; 128 x 768
// over 4096 11.1 and 13.5; 1 x 768 over 2048 8.7 and 9.2.
struct Split {
  int splits, kb;
};
Split choose_split(int64_t tiles, int64_t nkb, int64_t outputs) {
  Split best{1, int(nkb)};
  const int64_t pairs = num_sms() / 2;
  double least = 0.25 * double(nkb);
  for (int64_t s = 2; s <= 32 && s * tiles <= pairs && 4 * s <= nkb; ++s) {
    const int64_t kb = round_up(ceil_div(nkb, s), 4), parts = ceil_div(nkb, kb);
    const double t = 0.25 * double(kb) + 2.5 + double(parts) * double(outputs) * 8.0 / 3e6;
    if (parts > 1 && t < least) {
      least = t;
      best = Split{int(parts), int(kb)};
    }
  }
  return best;
}

// Set for good by the first product, captured ones included: from then on the error word is read.
std::atomic<bool> g_launched{false};

struct Shape {
  int64_t rows, cols, depth;  // of D (one group) and the product
};
Shape shape_of(const mao_fp8& A, const mao_fp8& B, int32_t form) {
  return form == MAO_NT   ? Shape{A.rows, B.rows, A.cols}
         : form == MAO_NN ? Shape{A.rows, B.cols, A.cols}
                          : Shape{A.cols, B.cols, A.rows};
}
Split split_of(const Shape& d) {
  return choose_split(ceil_div(d.rows, TILE) * ceil_div(d.cols, TILE), ceil_div(d.depth, BK), d.rows * d.cols);
}
size_t parts_bytes(const Shape& d, const Split& s) {
  return s.splits > 1 ? size_t(round_up(int64_t(s.splits) * d.rows * round_up(d.cols, 4) * 4, 256)) : 0;
}

}  // namespace

size_t product_workspace_size(const mao_fp8& A, const mao_fp8& B, int32_t form) {
  const Shape d = shape_of(A, B, form);
  return A.rows == 0 ? 0 : parts_bytes(d, split_of(d));
}

mao_status product_launch(const mao_fp8& A, const mao_fp8& B, const mao_mat& D, int32_t form,
                          const int32_t* offsets, int32_t groups, int32_t accumulate,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const bool tn = form == MAO_TN;
  const int es = elem_size(D.dtype);
  if (A.rows == 0) {  // no rows of D, or sums over nothing
    if (!tn || accumulate) return MAO_OK;
    return cuda_status(cudaMemset2DAsync(D.data, size_t(D.ld) * es, 0, size_t(D.cols) * es,
                                         size_t(D.rows), stream));
  }
  ProductParams p = {};
  mao_status st = tc_encode_code_map(&p.map_p, B.codes, B.cols, B.rows, B.ld, B.count, HALF);
  for (int b = tn ? Q_BOXES - 1 : 0; b < Q_BOXES && st == MAO_OK; ++b)
    st = tc_encode_code_map(&p.map_q[b], A.codes, A.cols, A.rows, A.ld, 1, 16 << b);
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
  p.dtype = D.dtype;
  p.accumulate = accumulate != 0;
  p.paired = D.dtype == MAO_BF16 && !accumulate && D.cols % 2 == 0 && reinterpret_cast<uintptr_t>(D.data) % 4 == 0 && D.ld % 2 == 0;
  p.sp_words = reinterpret_cast<uintptr_t>(B.scales) % 4 == 0 && B.scale_ld % 4 == 0;
  p.sq_words = reinterpret_cast<uintptr_t>(A.scales) % 4 == 0 && A.scale_ld % 4 == 0;
  p.timeout_ns = wait_limit_ns();
  // tiles at most: every group may end in a part of one
  const int64_t tiles = (tn ? ceil_div(p.J, TILE) * groups : ceil_div(A.rows, TILE) + groups) * p.tiles_i;
  if (tiles > 0x7FFF0000 || p.tiles_i > (1 << 17)) return MAO_ERR_UNSUPPORTED;
  using Kernel = void (*)(const ProductParams);
  const Kernel kernels[3] = {product_kernel<MAO_NT>, product_kernel<MAO_NN>, product_kernel<MAO_TN>};
  static std::atomic<bool> ready[64];
  st = once_per_device(ready, [&] {
    cudaError_t err = cudaSuccess;
    for (int f = 0; f < 3 && err == cudaSuccess; ++f)
      err = cudaFuncSetAttribute(kernels[f], cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
    return err;
  });
  if (st != MAO_OK) return st;
  p.splits = 1;
  const Shape shape = shape_of(A, B, form);
  Split split{1, 0};
  if (!offsets && workspace) {
    split = split_of(shape);
    if (workspace_bytes < parts_bytes(shape, split)) split = Split{1, 0};
  }
  if (split.splits > 1) {  // fp32 partial sums in the workspace, then their sum
    p.splits = split.splits;
    p.split_kb = split.kb;
    p.J = int32_t(shape.rows);
    p.d = workspace;
    p.ld = round_up(D.cols, 4);
    p.dtype = MAO_F32;
    p.accumulate = p.paired = 0;
  }
  g_launched.store(true, std::memory_order_release);
  const int64_t units = tiles * p.splits;
  const int64_t pairs = units < num_sms() / 2 ? units : num_sms() / 2;
  st = launch_dependent(kernels[form], unsigned(2 * pairs), THREADS, SMEM, stream, p);
  if (st != MAO_OK || split.splits == 1) return st;
  const SumParams sum{static_cast<const float*>(workspace), D.data, shape.rows, D.cols, p.ld, D.ld,
                      split.splits, D.dtype, accumulate,
                      reinterpret_cast<uintptr_t>(D.data) % 16 == 0 && D.ld % 4 == 0};
  const int64_t blocks = ceil_div(shape.rows * (p.ld / 4), 256);
  return launch_dependent(split_sum_kernel, unsigned(blocks < 4 * num_sms() ? blocks : 4 * num_sms()),
                          256, 0, stream, sum);
}

mao_status product_read_and_clear_error(cudaStream_t stream) {
  // a copy and a synchronisation that programs without 8-bit products do not wait for
  return g_launched.load(std::memory_order_acquire) ? read_and_clear_error(stream) : MAO_OK;
}

}  // namespace mao
