// Products of the gated feed-forward block in bf16 on the 5th-generation tensor cores, fp32 sums,
// over runs of rows.
//
// Every product is D[j][i] = sum_k Q[j][k] P[i][k]: i runs along D's rows in memory. An operand
// whose depth runs along its rows is loaded K-major, one whose depth runs down its columns
// MN-major, so no operand is transposed in memory:
//   GATE       H = act(X Wg^T) * (X Wu^T)        P = [Wg; Wu], Q = X               nt
//   down       Y = H Wd^T                        P = Wd, Q = H                     nt
//   GATE_BACK  dG, dU, H from dH = dY Wd, G, U   P = Wd, Q = dY                    nn
//   dX         dG Wg + dU Wu                     P = [Wg; Wu], Q = [dG, dU]        nn, depth 2 N
//   dup        dG^T X, dU^T X                    P = X, Q = dG or dU               tn
//   ddown      dY^T H                            P = H, Q = dY                     tn
// dH never reaches memory: the epilogue of its product turns it into dG, dU and H. For GATE each
// 32 lanes of the accumulator hold 16 rows of Wg and the same 16 of Wu (sixteen-row boxes, loaded
// that way), so that a channel's G and U meet by one exchange within a warp.
//
// Tiles of 256 x 256 (GATE: 128 channels, twice) by a pair of CTAs (tcgen05 cta_group::2, M = 256
// values of i, N up to 256 values of j). Roles per CTA (576 threads):
//   warp 0      TMA producer: 64-deep stages, 128 rows of P and the tile's half of Q, ring of six
//   warp 1      TMEM allocation; in the even CTA it issues the products (converged, one lane)
//   warps 2..17 epilogue: four warps per 32-lane quadrant of TMEM; lane = i. Its loops are kept
//               short: unrolled over two steps the code left the instruction cache
// TMEM holds two accumulators of 256 columns: a tile's epilogue runs under the next one's products.
//
// What bounds it. Dense, at 8192 x 4096 x 14336 (one launch alone): GATE 1.05 ms, down 0.50, dX 1.02,
// dup 1.01, ddown 0.57: the tensor cores, 1.7 to 1.92 PFLOP/s, cuBLAS's own rate here; in a run of
// steps the power limit. GATE_BACK 0.67 ms: its epilogue's reads and writes (13.7 bytes per cycle and
// SM) come on top of the operands' 62.5, and what the SMs take in together stops at about 18 TB/s.
// Over 128 runs of 512 rows on average (2048 x 768) the same bound comes first, as a tile of some
// 205 rows brings more bytes to a product: GATE 324 us, down 164, GATE_BACK 295, dX 290, dup 308,
// ddown 168 (4.1 to 4.9 TB/s of HBM traffic, 61 to 72% of a copy's; tensor cores 42 to 56% busy).
// A stage of 128 instead of 64 (half the waits) made dense steps 4% and experts' 5% slower.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "ffn_few.h"
#include "ffn_tiles.cuh"
#include "internal.h"
#include "ns_plan.h"
#include "tc_ptx.cuh"

namespace mao {
namespace {

using namespace ptx;
using namespace ffn;

constexpr int BK = 64;                // depth per stage: rows of 128 bytes
constexpr int OP_BYTES = HALF * BK * 2;
constexpr int RING_BYTES = 12 * OP_BYTES;  // six stages; more of them where few rows make Q's part small
constexpr int CHUNK_BYTES = 64 * BK * 2;  // 64 values of i or j of an MN-major operand
constexpr int MAX_STAGES = 11;
constexpr int EPI_WARPS = 16;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 512;
constexpr int Q_BOXES = 4;            // heights of boxes of a K-major Q: 16 << b rows
constexpr size_t SMEM = 1024 + RING_BYTES + TABLE_BYTES + 512;
static_assert(SMEM <= 232448, "shared memory budget of one CTA");

enum Epilogue { PLAIN, GATE, GATE_BACK };

struct alignas(64) FfnParams : TileParams {
  CUtensorMap map_p;
  // Boxes of 16, 32, 64, 128 rows. The last only for products of one run (half a tile's height) and
  // TN (64 x 64)
  CUtensorMap map_q[Q_BOXES];
  void* d;                     // PLAIN: D; GATE, GATE_BACK: H
  void* z;                     // G and U, fp32 or bf16: GATE writes them (null: not wanted), GATE_BACK reads them
  __nv_bfloat16* dz;           // GATE_BACK: dG and dU
  int64_t ld, ldz, lddz;
  int32_t early;               // the offsets are older than the kernel before this one
  int32_t dz_half;             // columns from dG to dU
  int32_t dtype;
  int32_t z_dtype;
  int32_t paired, paired_z;  // entries 2 i, 2 i + 1 of a row are one word (D: of bf16; Z: of its type)
  int32_t part_half;           // GATE: columns from G's parts to U's
  int32_t stages, stage_bytes; // of the ring
};

// GRADS: dX, dup, ddown, those that are not wanted without tiles.
template <int N>
struct FfnArgs {
  FfnParams p[N];
};

// Instruction descriptor of kind::f16: bf16 operands, fp32 sums, M = 256.
__device__ __forceinline__ uint32_t instr_desc(int p_mn, int q_mn, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(p_mn) << 15) | (uint32_t(q_mn) << 16) |
         (uint32_t(n >> 3) << 17) | (uint32_t(TILE >> 4) << 24);
}

// The four 16-deep products of a block, issued by the elected lane of a converged warp: the
// operands' descriptors advance by dp and dq (in 16-byte units) from one to the next.
__device__ __forceinline__ void mma_block(uint32_t elected, uint32_t d, uint64_t p, uint64_t q,
                                          uint32_t dp, uint32_t dq, uint32_t idesc,
                                          uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    asm volatile(
        "{\n\t.reg .pred a, e;\n\t"
        "setp.ne.b32 a, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, a;\n\t}\n" ::"r"(d),
        "l"(p + uint64_t(k) * dp), "l"(q + uint64_t(k) * dq), "r"(idesc),
        "r"(k ? 1u : accumulate), "r"(elected)
        : "memory");
  }
}

// ------------------------------------------------------------------ output

__device__ __forceinline__ uint32_t pack2(uint64_t p) {
  float a, b;
  split_pair(p, a, b);
  return pack(a, b);
}

// Sixteen rows of D (from row j on, those below j_end) at column i of this lane.
__device__ __forceinline__ void store16(const FfnParams& p, const Tile& t, int j, int i,
                                        const float (&v)[16], int lane) {
  const bool in = i < p.I;
  const int64_t row = t.row0 + j;
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
      if (in && j + c + odd < t.j_end)  // an even number of columns: both or none are there
        store_word(d, both);
      d += 2 * p.ld;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (in && j + c < t.j_end) d[c * p.ld] = __float2bfloat16_rn(v[c]);
}

// The same of a split of GATE: lanes 0 .. 15 hold G, lanes 16 .. 31 U, of channel i.
__device__ __forceinline__ void store16_gate_parts(const FfnParams& p, const Tile& t, int j, int i,
                                                   const float (&v)[16], int lane) {
  float* d = static_cast<float*>(p.d) + (t.row0 + j) * p.ld + i + (lane & 16 ? p.part_half : 0);
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (i < p.I && j + c < t.j_end)
      asm volatile("st.global.L1::no_allocate.f32 [%0], %1;" ::"l"(d + c * p.ld), "f"(v[c]) : "memory");
}

// GATE: lanes 0 .. 15 hold G and lanes 16 .. 31 U of sixteen rows at channel i (the same for l and
// l + 16). Of each four rows the lower lanes take two and the upper ones two; then the lanes of
// a pair take one row each.
template <int ACT>
__device__ __forceinline__ void gate16(const FfnParams& p, const Tile& t, int j, int i,
                                       const float (&v)[16], int lane) {
  const int up = lane >> 4, odd = lane & 1, col = i - odd;
  const bool in = col < p.I;
  const int left = t.j_end - j - 2 * up - odd;  // rows from this lane's first on
  const int64_t row = j + 2 * up + odd;
  // H's rows are padded to whole words
  __nv_bfloat16* h = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + col;
  __nv_bfloat16* z = static_cast<__nv_bfloat16*>(p.z) + row * p.ldz + col;
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const float s0 = up ? v[c] : v[c + 2], s1 = up ? v[c + 1] : v[c + 3];
    const float r0 = __shfl_xor_sync(0xFFFFFFFFu, s0, 16), r1 = __shfl_xor_sync(0xFFFFFFFFu, s1, 16);
    const float g0 = up ? r0 : v[c], g1 = up ? r1 : v[c + 1];
    const float u0 = up ? v[c + 2] : r0, u1 = up ? v[c + 3] : r1;
    const uint32_t wh = swap_pair(activate<ACT>(g0) * u0, activate<ACT>(g1) * u1, odd);
    const bool ok = in && c < left;
    if (ok) store_word(h, wh);
    h += 4 * p.ld;
    if (p.z && p.z_dtype == MAO_F32) {  // this lane's channel of its two rows
      float* zf = static_cast<float*>(p.z) + int64_t(j + c + 2 * up) * p.ldz + i;
      const int rows = t.j_end - (j + c + 2 * up);
      if (i < p.I && rows > 0) {
        zf[0] = g0;
        zf[p.I] = u0;
      }
      if (i < p.I && rows > 1) {
        zf[p.ldz] = g1;
        zf[p.ldz + p.I] = u1;
      }
    } else if (p.z) {
      const uint32_t wg = swap_pair(g0, g1, odd), wu = swap_pair(u0, u1, odd);
      if (p.paired_z) {
        if (ok) {
          store_word(z, wg);
          store_word(z + p.I, wu);
        }
      } else if (ok) {
        uint16_t* z16 = reinterpret_cast<uint16_t*>(z);
        z16[0] = uint16_t(wg);
        z16[p.I] = uint16_t(wu);
        if (col + 1 < p.I) {
          z16[1] = uint16_t(wg >> 16);
          z16[p.I + 1] = uint16_t(wu >> 16);
        }
      }
      z += 4 * p.ldz;
    }
  }
}

// GATE_BACK: G and U of eight rows at column i and its neighbour: even lanes have those of rows j,
// j + 2, ..., odd lanes of the others.
template <bool F32>
struct Saved;
template <>
struct Saved<false> {
  uint32_t g[4], u[4];
  __device__ __forceinline__ void load(const FfnParams& p, const Tile& t, int j, int i, int lane) {
    const int odd = lane & 1, col = i - odd;
    const uint16_t* z = static_cast<const uint16_t*>(p.z) + int64_t(j + odd) * p.ldz + col;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool a = col < p.I && j + 2 * c + odd < t.j_end, b = a && col + 1 < p.I;
      if (p.paired_z) {
        g[c] = a ? __ldg(reinterpret_cast<const uint32_t*>(z)) : 0u;
        u[c] = a ? __ldg(reinterpret_cast<const uint32_t*>(z + p.I)) : 0u;
      } else {
        g[c] = (a ? uint32_t(z[0]) : 0u) | (b ? uint32_t(z[1]) << 16 : 0u);
        u[c] = (a ? uint32_t(z[p.I]) : 0u) | (b ? uint32_t(z[p.I + 1]) << 16 : 0u);
      }
      z += 2 * p.ldz;
    }
  }
  static __device__ __forceinline__ uint64_t wide(uint32_t w) { return pair_of(low_half(w), high_half(w)); }
  __device__ __forceinline__ uint64_t gate(int c) const { return wide(g[c]); }
  __device__ __forceinline__ uint64_t linear(int c) const { return wide(u[c]); }
};
template <>
struct Saved<true> {
  uint64_t g[4], u[4];
  __device__ __forceinline__ void load(const FfnParams& p, const Tile& t, int j, int i, int lane) {
    const int odd = lane & 1, col = i - odd;
    const float* z = static_cast<const float*>(p.z) + int64_t(j + odd) * p.ldz + col;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool a = col < p.I && j + 2 * c + odd < t.j_end, b = a && col + 1 < p.I;
      if (p.paired_z) {
        g[c] = a ? __ldg(reinterpret_cast<const unsigned long long*>(z)) : 0ull;
        u[c] = a ? __ldg(reinterpret_cast<const unsigned long long*>(z + p.I)) : 0ull;
      } else {
        g[c] = pair_of(a ? z[0] : 0.0f, b ? z[1] : 0.0f);
        u[c] = pair_of(a ? z[p.I] : 0.0f, b ? z[p.I + 1] : 0.0f);
      }
      z += 2 * p.ldz;
    }
  }
  __device__ __forceinline__ uint64_t gate(int c) const { return g[c]; }
  __device__ __forceinline__ uint64_t linear(int c) const { return u[c]; }
};

// Asks L2 for a tile's G and U (this CTA's columns), two threads per row.
__device__ __forceinline__ void prefetch_saved(const FfnParams& p, const Tile& t, int cta, int thread) {
  const int i = t.i0 + HALF * cta, row = t.j0 + (thread >> 1);
  if (row >= t.j_end) return;
  const int es = p.z_dtype == MAO_F32 ? 4 : 2;
  const uint8_t* z = static_cast<const uint8_t*>(p.z) + (int64_t(row) * p.ldz + (thread & 1 ? p.I : 0) + i) * es;
  const int bytes = min(HALF, p.I - i) * es;
  for (int b = 0; b < bytes; b += 128) prefetch_l2(z + b);
}

// dG, dU and H of eight rows of dH, those from FROM on of the sixteen in v. The buffers' rows are padded to whole words.
template <int ACT, bool F32, int FROM>
__device__ __forceinline__ void gate_back8(const FfnParams& p, const Tile& t, int j, int i,
                                            const float (&v)[16], const Saved<F32>& s, int lane) {
  const int odd = lane & 1, col = i - odd;
  const int left = col < p.I ? t.j_end - j - odd : 0;  // rows from this lane's first on
  const int64_t row = j + odd;
  __nv_bfloat16* h = static_cast<__nv_bfloat16*>(p.d) + row * p.ld + col;
  __nv_bfloat16* dg = p.dz + row * p.lddz + col;
  __nv_bfloat16* du = dg + p.dz_half;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[FROM + 2 * c] : v[FROM + 2 * c + 1], 1);
    const uint64_t d = odd ? pair_of(o, v[FROM + 2 * c + 1]) : pair_of(v[FROM + 2 * c], o), u = s.linear(c);
    uint64_t a, slope;
    activate2<ACT>(s.gate(c), a, slope);
    if (2 * c < left) {
      store_word(dg, pack2(mul2(mul2(d, u), slope)));
      store_word(du, pack2(mul2(d, a)));
      store_word(h, pack2(mul2(a, u)));
    }
    dg += 2 * p.lddz;
    du += 2 * p.lddz;
    h += 2 * p.ld;
  }
}

// Rows j0, j0 + step, ... below j1 of the outputs hold no tokens.
template <int EPI>
__device__ __forceinline__ void clear_unused(const FfnParams& p, int64_t j0, int64_t j1, int64_t step, int lane) {
  const int es = p.dtype == MAO_F32 ? 4 : 2;
  if (EPI != GATE) clear_rows(p.d, p.ld * es, int64_t(p.I) * es, j0, j1, step, lane);
  const int ez = p.z_dtype == MAO_F32 ? 4 : 2;
  if (EPI == GATE && p.z) clear_rows(p.z, p.ldz * ez, int64_t(p.I) * 2 * ez, j0, j1, step, lane);
  if (EPI == GATE_BACK) {
    clear_rows(p.dz, p.lddz * 2, int64_t(p.I) * 2, j0, j1, step, lane);
    clear_rows(p.dz + p.dz_half, p.lddz * 2, int64_t(p.I) * 2, j0, j1, step, lane);
  }
}

// ------------------------------------------------------------------ the kernel

template <int FORM, int EPI, int ACT, bool ZF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    ffn_kernel(const __grid_constant__ FfnArgs<FORM == GRADS ? 3 : 1> args) {
  const FfnParams& p0 = args.p[0];  // the runs, the ring and the waits are the same for all
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* lo = reinterpret_cast<int*>(ring + RING_BYTES);
  int* cnt = lo + MAX_GROUPS + 2;
  int* begin = cnt + MAX_GROUPS + 2;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + RING_BYTES + TABLE_BYTES);
  uint64_t* full_bar = bars;                  // [stages]  (used in the even CTA)
  uint64_t* empty_bar = full_bar + MAX_STAGES;  // [stages]
  uint64_t* tfull_bar = empty_bar + MAX_STAGES; // [2]
  uint64_t* tempty_bar = tfull_bar + 2;       // [2]       (even CTA)
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const bool leader = cta == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const uint64_t limit = p0.timeout_ns;
  const int stages = p0.stages, stage_bytes = p0.stage_bytes;
  constexpr int PRODUCTS = FORM == GRADS ? 3 : 1, p_mn = FORM != NT;
  constexpr int STEP_I = EPI == GATE ? HALF : TILE;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull_bar[a]), 1);
      mbar_init(smem_u32(&tempty_bar[a]), 2 * EPI_WARPS);
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
  if (warp == 0 && lane < 2 * PRODUCTS) {
    const FfnParams& p = args.p[lane >> 1];
    const CUtensorMap* map = lane & 1 ? &p.map_q[Q_BOXES - 1] : &p.map_p;
    if (p.tiles_i > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  // launched as a programmatic dependent: the set-up may overlap the previous kernel's end (1.5 us; all
  // of it unless it reads offsets that that kernel may have written). First loads of down's P as early
  // made 48 rows 1.4 us slower.
  const bool early = !p0.offsets || p0.early;
  if (!early) wait_for_previous();
  make_table<THREADS>(p0, lo, cnt, begin, reinterpret_cast<int*>(bars + 40));
  tc_fence_before();
  __syncthreads();
  // tiles of the first product, of the first two, of all
  auto tn_tiles = [](const FfnParams& p) {
    return (p.J + p.height - 1) / p.height * p.tiles_i * p.groups * p.halves * p.splits;
  };
  const int tiles0 = FORM == TN ? tn_tiles(p0) : begin[p0.groups] * p0.tiles_i * p0.splits;
  const int tiles1 = FORM == GRADS ? tiles0 + tn_tiles(args.p[PRODUCTS / 2]) : tiles0;
  const int total = FORM == GRADS ? tiles1 + tn_tiles(args.p[PRODUCTS - 1]) : tiles0;
  // The tile's product, and the tile.
  auto take = [&](int tile, Tile& t) {
    if (FORM != GRADS) {
      decode<FORM == GRADS ? NN : FORM, STEP_I, BK>(p0, lo, cnt, begin, tile, t);
      return 0;
    }
    const int q = (tile >= tiles0) + (tile >= tiles1);
    if (q) decode<TN, TILE, BK>(args.p[q], lo, cnt, begin, tile - (q > 1 ? tiles1 : tiles0), t);
    else decode<NN, TILE, BK>(p0, lo, cnt, begin, tile, t);
    return q;
  };
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  if (early) wait_for_previous();

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
      const int product = take(tile, t);
      const FfnParams& p = args.p[product];
      const bool q_mn = FORM == TN || product > 0, nn = FORM == NN || (FORM == GRADS && !q_mn);
      const int half_kb = (p.depth + BK - 1) / BK;  // NN: blocks of a half of the depth
      const int i = t.i0 + (EPI == GATE ? HALF / 2 : HALF) * int(cta);
      const int j = t.j0 + (t.n >> 1) * int(cta);
      const int z = q_mn ? 0 : t.g;
      const bool one_box = !p.offsets;
      const int q_rows = one_box && !q_mn ? p.height >> 1 : t.n >> 1;  // a multiple of 16
      const int q_chunks = (q_rows + 63) >> 6;
      const uint32_t q_bytes = q_mn ? uint32_t(q_chunks) * CHUNK_BYTES : uint32_t(q_rows) * BK * 2;
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_warp<false>(&empty_bar[stage], phase ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        const uint32_t fb = full0 + 8 * stage, dst = ring0 + stage * stage_bytes;
        const int b = t.kb0 + kb;
        const int second = nn && b >= half_kb;  // half of the depth
        const int k = t.k0 + (second ? b - half_kb : b) * BK;
        if (elected) {
          if (leader) mbar_expect_tx(smem_u32(&full_bar[stage]), 2 * (OP_BYTES + q_bytes));
          if (EPI == GATE) {
#pragma unroll
            for (int r = 0; r < 8; ++r)  // 16 rows of Wg, the same 16 of Wu, ...
              tma_load_4d_pair(dst + r * (16 * BK * 2), &p.map_p, fb, k, i + 16 * (r >> 1), r & 1, z);
          } else if (p_mn) {
            tma_load_4d_pair(dst, &p.map_p, fb, i, k, second, z);
            tma_load_4d_pair(dst + CHUNK_BYTES, &p.map_p, fb, i + 64, k, second, z);
          } else {
            tma_load_4d_pair(dst, &p.map_p, fb, k, i, 0, z);
          }
          if (q_mn) {
            for (int c = 0; c < q_chunks; ++c)
              tma_load_4d_pair(dst + OP_BYTES + c * CHUNK_BYTES, &p.map_q[Q_BOXES - 1], fb, j + 64 * c, k, t.half, 0);
          } else if (one_box || q_rows == HALF) {
            tma_load_4d_pair(dst + OP_BYTES, &p.map_q[Q_BOXES - 1], fb, k, j, second, 0);
          } else {
            for (int box = Q_BOXES - 2, at = 0; box >= 0; --box)
              if (q_rows & (16 << box)) {
                tma_load_4d_pair(dst + OP_BYTES + at * (BK * 2), &p.map_q[box], fb, k, j + at, second, 0);
                at += 16 << box;
              }
          }
        }
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // after an abort, the loads already issued land before the CTA leaves
    if (*abort_flag && leader && lane == 0) {
      for (int s = 0; s < stages; ++s)
        if ((armed >> s) & 1u) mbar_drain(smem_u32(&full_bar[s]), (armed_phase >> s) & 1u, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader) {
      const uint32_t elected = elect_one();
      // K-major: rows of 128 bytes, 1024 between groups of eight; 32 bytes along them per product.
      // MN-major: eight rows of the depth per 1024 bytes, 64 values of i or j per chunk; two
      // groups of eight per product.
      const uint64_t p_desc = desc_of(smem_u32(ring), p_mn ? CHUNK_BYTES : 16, 1024, 2);
      const uint32_t dp = p_mn ? 2048 >> 4 : 32 >> 4;
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false, ready = false;
      Tile t;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        const int product = take(tile, t);
        if (t.nkb == 0) continue;
        const bool q_mn = FORM == TN || product > 0;
        const uint64_t q_desc = desc_of(smem_u32(ring) + OP_BYTES, q_mn ? CHUNK_BYTES : 16, 1024, 2);
        const uint32_t dq = q_mn ? 2048 >> 4 : 32 >> 4;
        const int acc = local & 1;
        if (!wait_warp<true>(&tempty_bar[acc], (uint32_t(local >> 1) & 1u) ^ 1u, abort_flag, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * TILE);
        const uint32_t idesc = instr_desc(p_mn, q_mn, t.n);
        for (int kb = 0; kb < t.nkb; ++kb) {
          // the stage was looked at while the products before were issued
          if (!__all_sync(0xFFFFFFFFu, ready) && !wait_warp<false>(&full_bar[stage], phase, abort_flag, limit)) {
            ok = false;
            break;
          }
          const uint32_t empty = smem_u32(&empty_bar[stage]);
          const uint64_t at = uint64_t(stage * (stage_bytes >> 4));
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
          ready = limit != 0 && mbar_test_wait(smem_u32(&full_bar[stage]), phase);
          mma_block(elected, d, p_desc + at, q_desc + at, dp, dq, idesc, kb != 0 ? 1u : 0u);
          issued = true;
          commit_both(elected, empty);
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
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3;         // TMEM lanes 32 quad ..
    const int part = (warp - 2) >> 2;  // which of the quadrant's four warps
    const bool saved = EPI == GATE_BACK && p0.splits == 1;
    const uint32_t tempty[2] = {mapa_shared(smem_u32(&tempty_bar[0]), 0),
                                mapa_shared(smem_u32(&tempty_bar[1]), 0)};
    // rows that hold no tokens are cleared while the first tiles are multiplied
    if (FORM != TN && p0.splits == 1 && p0.tiles_i > 0) {
      for_unused_rows(p0, lo, cnt, int(blockIdx.x) * EPI_WARPS + warp - 2, int(gridDim.x) * EPI_WARPS,
                      [&](int64_t j0, int64_t j1, int64_t step) { clear_unused<EPI>(p0, j0, j1, step, lane); });
    }
    int local = 0;
    Tile t;
    for (int tile = pair; tile < total; tile += npairs) {
      const FfnParams& p = args.p[take(tile, t)];
      if (saved) {
        // this tile's G and U if it is the first, and the next one's: they have a tile's time
        if (tile == pair) prefetch_saved(p, t, int(cta), int(threadIdx.x) - 64);
        if (tile + npairs < total) {
          Tile u = t;
          take(tile + npairs, u);
          prefetch_saved(p, u, int(cta), int(threadIdx.x) - 64);
        }
      }
      const int i = EPI == GATE ? t.i0 + HALF / 2 * int(cta) + 16 * quad + (lane & 15)
                                : t.i0 + HALF * int(cta) + 32 * quad + lane;
      if (t.nkb == 0) {  // TN: an empty run's matrix is zero
        const int es = p.dtype == MAO_F32 ? 4 : 2, i0 = t.i0 + HALF * int(cta);
        clear_rows(static_cast<uint8_t*>(p.d) + int64_t(i0) * es, p.ld * es, int64_t(min(HALF, p.I - i0)) * es,
                   t.row0 + t.j0 + warp - 2, t.row0 + t.j_end, EPI_WARPS, lane);
        continue;
      }
      const int acc = local & 1;
      const int n = t.j_end - t.j0;
      // this warp's 64 columns in four steps, every fourth sixteen
      // every lane waits; the warp goes on only if all of them saw the accumulator
      if (!wait_warp<false>(&tfull_bar[acc], uint32_t(local >> 1) & 1u, abort_flag, limit)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t(32 * quad) << 16) + uint32_t(acc * TILE);
      // G and U of eight rows are on their way while eight others are worked on
      Saved<ZF32> za, zb;
      if (saved && 16 * part < n) za.load(p, t, t.j0 + 16 * part, i, lane);
#pragma unroll 1
      for (int c = 16 * part; c < n; c += 64) {
        float v[16];
        if (saved) zb.load(p, t, t.j0 + c + 8, i, lane);
        tmem_ld16(trow + uint32_t(c), v);
        tmem_wait(v);
        if (EPI == GATE && p.splits > 1) {
          store16_gate_parts(p, t, t.j0 + c, i, v, lane);
        } else if (EPI == GATE) {
          gate16<ACT>(p, t, t.j0 + c, i, v, lane);
        } else if (saved) {
          gate_back8<ACT, ZF32, 0>(p, t, t.j0 + c, i, v, za, lane);
          if (c + 64 < n) za.load(p, t, t.j0 + c + 64, i, lane);
          gate_back8<ACT, ZF32, 8>(p, t, t.j0 + c + 8, i, v, zb, lane);
        } else {
          store16(p, t, t.j0 + c, i, v, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty[acc]);
      ++local;
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

// ------------------------------------------------------------------ sums of the splits' parts

// The splits' parts added up in their order, then what the product's epilogue does; four columns
// per thread. q.d, q.dtype, q.ld, q.paired are those of the whole product.
struct SumParams {
  FfnParams q;
  const float* parts;
  int64_t prows, pld;  // rows and row stride of one part
};

__device__ __forceinline__ void add_parts(const SumParams& p, int64_t j, int64_t i, float (&v)[4]) {
  v[0] = v[1] = v[2] = v[3] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < p.q.splits; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(p.parts + (s * p.prows + j) * p.pld + i);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
  }
}

// Four bf16 columns, those below n, of a row that starts at d.
__device__ __forceinline__ void store4(__nv_bfloat16* d, int64_t i, int n, bool words, const float (&v)[4]) {
  if (words && i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(d + i) = pack(v[0], v[1]);
    *reinterpret_cast<uint32_t*>(d + i + 2) = pack(v[2], v[3]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (i + c < n) d[i + c] = __float2bfloat16_rn(v[c]);
  }
}

template <int EPI, int ACT>
__global__ void __launch_bounds__(256) ffn_sum_kernel(const __grid_constant__ SumParams p) {
  wait_for_previous();
  const FfnParams& q = p.q;
  const int64_t quads = (q.I + 3) / 4, all = p.prows * quads;
  for (int64_t x = int64_t(blockIdx.x) * 256 + threadIdx.x; x < all; x += int64_t(gridDim.x) * 256) {
    const int64_t j = x / quads, i = 4 * (x - j * quads);
    float v[4];
    add_parts(p, j, i, v);
    if (EPI == PLAIN) {
      if (q.dtype == MAO_F32) {
        float* d = static_cast<float*>(q.d) + j * q.ld + i;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (i + c < q.I) d[c] = v[c];
      } else {
        store4(static_cast<__nv_bfloat16*>(q.d) + j * q.ld, i, q.I, q.paired, v);
      }
    } else if (EPI == GATE) {
      float u[4], h[4];
      add_parts(p, j, q.part_half + i, u);
#pragma unroll
      for (int c = 0; c < 4; ++c) h[c] = activate<ACT>(v[c]) * u[c];
      store4(static_cast<__nv_bfloat16*>(q.d) + j * q.ld, i, q.I, q.paired, h);
      if (q.z) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (i + c < q.I) {
            store_elem(q.z, j * q.ldz + i + c, q.z_dtype, v[c]);
            store_elem(q.z, j * q.ldz + q.I + i + c, q.z_dtype, u[c]);
          }
      }
    } else {
      float h[4], dg[4], du[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = i + c < q.I;
        const float g = in ? load_elem(q.z, j * q.ldz + i + c, q.z_dtype) : 0.0f;
        const float u = in ? load_elem(q.z, j * q.ldz + q.I + i + c, q.z_dtype) : 0.0f;
        float a, slope;
        activate<ACT>(g, a, slope);
        h[c] = a * u;
        dg[c] = v[c] * u * slope;
        du[c] = v[c] * a;
      }
      store4(static_cast<__nv_bfloat16*>(q.d) + j * q.ld, i, q.I, true, h);
      store4(q.dz + j * q.lddz, i, q.I, true, dg);
      store4(q.dz + j * q.lddz + q.dz_half, i, q.I, true, du);
    }
  }
}

// ------------------------------------------------------------------ copies of unaligned operands

// Up to four operands to rows that start at multiples of 16 bytes, in one launch: eight entries per
// thread and step.
struct CopyParams {
  struct Part {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld, dld, first, groups;  // first of all groups of eight, their number
    int32_t cols, per_row;
  } part[4];
  int32_t n;
};
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p) {
  wait_for_previous();
  int64_t all = 0;
  for (int q = 0; q < p.n; ++q) all += p.part[q].groups;
  for (int64_t x = int64_t(blockIdx.x) * 256 + threadIdx.x; x < all; x += int64_t(gridDim.x) * 256) {
    int q = 0;
    while (q + 1 < p.n && x >= p.part[q + 1].first) ++q;
    const CopyParams::Part& c = p.part[q];
    const int64_t y = x - c.first, r = y / c.per_row;
    const int col = 8 * int(y - r * c.per_row);
    const uint16_t* s = c.src + r * c.ld + col;
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = col + k < c.cols ? uint32_t(s[k]) : 0u;
    *reinterpret_cast<uint4*>(c.dst + r * c.dld + col) =
        make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
}

// ------------------------------------------------------------------ host

std::atomic<bool> g_launched{false};

// A bf16 operand as the kernels see it: rows that start at multiples of 16 bytes.
struct Operand {
  const void* data;
  int64_t rows, cols, ld;
  bool copied;
  size_t bytes() const { return copied ? size_t(round_up(rows * ld * 2, 256)) : 0; }
};
Operand operand(const mao_mat& m) {
  const bool whole = reinterpret_cast<uintptr_t>(m.data) % 16 == 0 && (m.ld % 8 == 0 || m.rows <= 1);
  // a single row's stride may be anything, but a map wants a multiple of 16 bytes
  if (whole) return Operand{m.data, m.rows, m.cols, round_up(m.rows <= 1 ? m.cols : m.ld, 8), false};
  return Operand{nullptr, m.rows, m.cols, round_up(m.cols, 8), true};
}
// Copies of operands, in one launch; at: the workspace from there on.
struct Copies {
  CopyParams p = {};
  int64_t all = 0;
  void add(Operand& o, const mao_mat& m, uint8_t*& at) {
    if (!o.copied || o.rows == 0) return;
    o.data = at;
    const int64_t per_row = o.ld / 8;
    p.part[p.n++] = {static_cast<const uint16_t*>(m.data), reinterpret_cast<uint16_t*>(at), m.ld, o.ld, all,
                     m.rows * per_row, int32_t(m.cols), int32_t(per_row)};
    all += m.rows * per_row;
    at += o.bytes();
  }
  mao_status launch(cudaStream_t stream) const {
    if (p.n == 0) return MAO_OK;
    const int64_t blocks = ceil_div(all, 256);
    return launch_dependent(copy_kernel, unsigned(blocks < 16 * num_sms() ? blocks : 16 * num_sms()), 256, 0, stream, p);
  }
};

// The products of a call, with the sizes that their splits and parts go by.
struct Plan {
  int form, epi;
  int64_t I, J, depth;  // of D: columns (GATE: channels), rows (one matrix's for TN); depth per half
  int32_t halves;
  Cut split{TILE, 1, 0};
  int64_t prows = 0, pld = 0;

  int64_t tiles_i() const { return ceil_div(I, epi == GATE ? HALF : TILE); }
  int64_t matrices() const { return form == TN ? halves : 1; }
  // share: of the GPU, while other products run beside this one
  void choose(bool grouped, double share = 1.0) {
    if (grouped) return;
    const int64_t all = cta_pairs(), part = int64_t(share * double(all) + 0.5), pairs = part < 1 ? 1 : part;
    const int64_t nkb = ceil_div(depth, BK) * (form == NN ? halves : 1);
    const int64_t outputs = J * matrices() * I * (epi == GATE ? 2 : 1);
    // A block takes a pair 0.27 us (the tensor cores), at least 0.14 (its copies and their waits),
    // or 0.37 where few rows leave the operands' bytes to bound it.
    split = choose_cut(pairs, tiles_i() * matrices(), J, nkb, 0.0, 0.27, form != TN && J < 128 ? 0.37 : 0.14,
                       epi == GATE_BACK ? 9.5 : epi == GATE ? 3.5 : 1.7, outputs, 4);
    prows = J * matrices();
    pld = round_up(I, 4) * (epi == GATE ? 2 : 1);
  }
  size_t bytes() const { return split.splits > 1 ? size_t(round_up(split.splits * prows * pld * 4, 256)) : 0; }
};

template <int N>
using Kernel = void (*)(const FfnArgs<N>);
using SumKernel = void (*)(const SumParams);

// Fills in what the plan and the runs say; the tiles there may be, or -1: too many.
int64_t describe(const Plan& plan, FfnParams& p, const Runs& runs, int64_t rows) {
  p.offsets = runs.offsets;
  p.counts = runs.offsets ? runs.counts : nullptr;
  p.groups = runs.groups;
  p.rows = int32_t(rows);
  p.I = int32_t(plan.I);
  p.J = int32_t(plan.J);
  p.depth = int32_t(plan.depth);
  p.halves = plan.halves;
  p.tiles_i = int32_t(plan.tiles_i());
  p.timeout_ns = wait_limit_ns();
  p.height = plan.split.height;
  p.splits = plan.split.splits;
  p.split_kb = plan.split.kb;
  p.part_half = int32_t(round_up(plan.I, 4));
  const bool tn = plan.form == TN;
  const int64_t tiles = (tn ? ceil_div(plan.J, p.height) * runs.groups * plan.halves
                            : ceil_div(rows, p.height) + (runs.offsets ? runs.groups : 0)) * plan.tiles_i();
  const bool small_q = !runs.offsets && !tn;
  p.stage_bytes = OP_BYTES + (small_q ? int32_t(round_up(p.height / 2 * BK * 2, 1024)) : OP_BYTES);
  p.stages = RING_BYTES / p.stage_bytes < MAX_STAGES ? RING_BYTES / p.stage_bytes : MAX_STAGES;
  return tiles * p.splits > 0x3FFF0000 ? -1 : tiles * p.splits;
}

// Lets the product write its parts; the sum to launch after it.
SumParams split_sum(const Plan& plan, FfnParams& p, void* parts) {
  SumParams sum;
  sum.q = p;
  sum.parts = static_cast<const float*>(parts);
  sum.prows = plan.prows;
  sum.pld = plan.pld;
  p.d = parts;
  p.ld = plan.pld;
  p.dtype = MAO_F32;
  return sum;
}
mao_status launch_sum(const Plan& plan, int32_t act, const SumParams& sum, cudaStream_t stream) {
  static const SumKernel sums[7] = {
      ffn_sum_kernel<PLAIN, 0>,
      ffn_sum_kernel<GATE, MAO_SILU>, ffn_sum_kernel<GATE, MAO_GELU>, ffn_sum_kernel<GATE, MAO_GELU_TANH>,
      ffn_sum_kernel<GATE_BACK, MAO_SILU>, ffn_sum_kernel<GATE_BACK, MAO_GELU>, ffn_sum_kernel<GATE_BACK, MAO_GELU_TANH>};
  const int k = plan.epi == GATE ? 1 + act : plan.epi == GATE_BACK ? 4 + act : 0;
  const int64_t blocks = ceil_div(plan.prows * ceil_div(plan.I, 4), 256);
  return launch_dependent(sums[k], unsigned(blocks < 8 * num_sms() ? blocks : 8 * num_sms()), 256, 0, stream, sum);
}

unsigned grid_of(int64_t units) { return unsigned(2 * (units < cta_pairs() ? units : cta_pairs())); }

mao_status run(const Plan& plan, int32_t act, FfnArgs<1>& args, const Runs& runs, int64_t rows, void* parts,
               cudaStream_t stream) {
  FfnParams& p = args.p[0];
  const int64_t units = describe(plan, p, runs, rows);
  if (units < 0) return MAO_ERR_UNSUPPORTED;
  // the plain products, then those of each activation (GATE_BACK: from a bf16, then a fp32 Z)
  static const Kernel<1> kernels[12] = {
      ffn_kernel<NT, PLAIN, 0, false>, ffn_kernel<NN, PLAIN, 0, false>, ffn_kernel<TN, PLAIN, 0, false>,
      ffn_kernel<NT, GATE, MAO_SILU, false>, ffn_kernel<NT, GATE, MAO_GELU, false>,
      ffn_kernel<NT, GATE, MAO_GELU_TANH, false>,
      ffn_kernel<NN, GATE_BACK, MAO_SILU, false>, ffn_kernel<NN, GATE_BACK, MAO_SILU, true>,
      ffn_kernel<NN, GATE_BACK, MAO_GELU, false>, ffn_kernel<NN, GATE_BACK, MAO_GELU, true>,
      ffn_kernel<NN, GATE_BACK, MAO_GELU_TANH, false>, ffn_kernel<NN, GATE_BACK, MAO_GELU_TANH, true>};
  const int k = plan.epi == GATE        ? 3 + act
                : plan.epi == GATE_BACK ? 6 + 2 * act + (p.z_dtype == MAO_F32)
                                        : plan.form;
  static std::atomic<bool> ready[64];
  mao_status st = once_per_device(ready, [&] {
    cudaError_t err = cudaSuccess;
    for (int f = 0; f < 12 && err == cudaSuccess; ++f)
      err = cudaFuncSetAttribute(kernels[f], cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
    return err;
  });
  if (st != MAO_OK) return st;
  g_launched.store(true, std::memory_order_release);
  if (p.splits == 1) return launch_dependent(kernels[k], grid_of(units), THREADS, SMEM, stream, args);
  const SumParams sum = split_sum(plan, p, parts);
  st = launch_dependent(kernels[k], grid_of(units), THREADS, SMEM, stream, args);
  return st == MAO_OK ? launch_sum(plan, act, sum, stream) : st;
}

// dX, dup and ddown, those that are wanted. Nothing of them depends on another, so where they have few
// tiles they go in one launch: 18 us less for a training step of 1000 rows, 1037 x 515 (now 54). With
// many tiles one launch each is faster, their forms known to the compiler: 1.58 ms instead of 1.61
// for the step of 128 experts, 5.32 instead of 5.41 for the dense one.
mao_status run_grads(const Plan* const (&plans)[3], const bool (&wanted)[3], FfnArgs<3>& args, const Runs& runs,
                     int64_t rows, uint8_t* parts, cudaStream_t stream) {
  int64_t units = 0;
  for (int q = 0; q < 3; ++q) {
    FfnParams& p = args.p[q];
    const int64_t tiles = describe(*plans[q], p, runs, rows);
    if (tiles < 0) return MAO_ERR_UNSUPPORTED;
    p.stage_bytes = 2 * OP_BYTES;
    p.stages = RING_BYTES / p.stage_bytes;
    if (wanted[q]) units += tiles;
    else p.tiles_i = 0;
  }
  if (units == 0) return MAO_OK;
  if (units > 8 * cta_pairs()) {
    mao_status st = MAO_OK;
    for (int q = 0; q < 3 && st == MAO_OK; ++q) {
      if (!wanted[q]) continue;
      FfnArgs<1> one;
      one.p[0] = args.p[q];
      st = run(*plans[q], 0, one, runs, rows, parts, stream);
    }
    return st;
  }
  SumParams sums[3];
  for (int q = 0; q < 3; ++q) {
    if (!wanted[q] || args.p[q].splits == 1) continue;
    sums[q] = split_sum(*plans[q], args.p[q], parts);
    parts += plans[q]->bytes();
  }
  const Kernel<3> kernel = ffn_kernel<GRADS, PLAIN, 0, false>;
  static std::atomic<bool> ready[64];
  mao_status st = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM));
  });
  if (st != MAO_OK) return st;
  g_launched.store(true, std::memory_order_release);
  st = launch_dependent(kernel, grid_of(units), THREADS, SMEM, stream, args);
  for (int q = 0; q < 3 && st == MAO_OK; ++q)
    if (wanted[q] && args.p[q].splits > 1) st = launch_sum(*plans[q], 0, sums[q], stream);
  return st;
}

void set_saved(FfnParams& p, const mao_mat& Z) {
  p.z = Z.data;
  p.ldz = Z.ld;
  p.z_dtype = Z.dtype;
  p.paired_z = reinterpret_cast<uintptr_t>(Z.data) % (2 * elem_size(Z.dtype)) == 0 && Z.ld % 2 == 0 && Z.cols % 4 == 0;
}
bool words(const void* data, int64_t ld, int64_t cols) {
  return reinterpret_cast<uintptr_t>(data) % 4 == 0 && ld % 2 == 0 && cols % 2 == 0;
}
void set_out(FfnParams& p, const mao_mat& D) {
  p.d = D.data;
  p.ld = D.ld;
  p.dtype = D.dtype;
  p.paired = words(D.data, D.ld, D.cols);
}

struct Sizes {
  int64_t R, K, N, C;
};

// Buffers of the workspace, in order: the intermediate rows, copies of operands, parts.
struct Forward {
  Sizes s;
  int64_t ldh;
  Operand x, up, down;
  Plan gate, out;
  Forward(const mao_mat& X, const mao_mat& Up, const mao_mat& Down, int32_t groups, bool grouped)
      : s{X.rows, X.cols, Down.cols, Down.rows / groups}, ldh(round_up(s.N, 8)), x(operand(X)), up(operand(Up)),
        down(operand(Down)), gate{NT, GATE, s.N, s.R, s.K, 1}, out{NT, PLAIN, s.C, s.R, s.N, 1} {
    if (few_rows(s.R, grouped, false, groups)) return;  // these products are not cut
    gate.choose(grouped);
    out.choose(grouped);
  }
  size_t h_bytes() const { return size_t(round_up(s.R * ldh * 2, 256)); }
  size_t parts_bytes() const { return gate.bytes() > out.bytes() ? gate.bytes() : out.bytes(); }
  size_t bytes() const { return h_bytes() + x.bytes() + up.bytes() + down.bytes() + parts_bytes(); }
};

struct Backward {
  Sizes s;
  int64_t ldh;
  Operand dy, x, up, down;
  Plan back, dx, dup, ddown;
  Backward(const mao_mat& dY, const mao_mat& X, const mao_mat& Up, const mao_mat& Down, int32_t groups, bool grouped)
      : s{X.rows, X.cols, Down.cols, Down.rows / groups}, ldh(round_up(s.N, 8)), dy(operand(dY)), x(operand(X)),
        up(operand(Up)), down(operand(Down)), back{NN, GATE_BACK, s.N, s.R, s.C, 1}, dx{NN, PLAIN, s.K, s.R, s.N, 2},
        dup{TN, PLAIN, s.K, s.N, s.R, 2}, ddown{TN, PLAIN, s.N, s.C, s.R, 1} {
    back.choose(grouped);
    // the three run side by side: each has its share of the work's pairs of SMs
    const double width = double(4 * s.K + s.C);
    dx.choose(grouped, 2 * s.K / width);
    dup.choose(grouped, 2 * s.K / width);
    ddown.choose(grouped, s.C / width);
  }
  size_t h_bytes() const { return size_t(round_up(s.R * ldh * 2, 256)); }
  size_t dz_bytes() const { return size_t(round_up(s.R * ldh * 4, 256)); }
  size_t parts_bytes() const {
    const size_t grads = dx.bytes() + dup.bytes() + ddown.bytes();
    return back.bytes() > grads ? back.bytes() : grads;
  }
  size_t bytes() const {
    return h_bytes() + dz_bytes() + dy.bytes() + x.bytes() + up.bytes() + down.bytes() + parts_bytes();
  }
};

// Maps of a K-major Q.
mao_status encode_q(FfnParams& p, const Plan& plan, bool grouped, const void* base, int64_t cols, int64_t rows,
                    int64_t halves, int64_t ld, int64_t half_stride) {
  mao_status st = MAO_OK;
  for (int b = grouped ? 0 : Q_BOXES - 1; b < Q_BOXES && st == MAO_OK; ++b)
    st = tc_encode_bf16_map(&p.map_q[b], base, cols, rows, halves, 1, ld, half_stride, rows * ld,
                            grouped ? 16 << b : plan.split.height / 2);
  return st;
}

}  // namespace

size_t gated_ffn_workspace_size(const mao_mat& X, const mao_mat& up, const mao_mat& down, int32_t groups,
                                bool grouped) {
  return X.rows == 0 ? 0 : Forward(X, up, down, groups, grouped).bytes();
}

mao_status gated_ffn_launch(const mao_mat& X, const mao_mat& up, const mao_mat& down, int32_t act,
                            const Runs& runs, const mao_mat* Z, const mao_mat& Y, void* workspace,
                            cudaStream_t stream) {
  if (X.rows == 0) return MAO_OK;
  Forward f(X, up, down, runs.groups, runs.offsets != nullptr);
  const Sizes& s = f.s;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  uint8_t* h = at;
  at += f.h_bytes();
  Copies copies;
  copies.add(f.x, X, at);
  copies.add(f.up, up, at);
  copies.add(f.down, down, at);
  mao_status st = copies.launch(stream);
  if (st != MAO_OK) return st;

  if (few_rows(s.R, runs.offsets != nullptr, runs.counts != nullptr, runs.groups)) {
    FewParams q = {};
    q.offsets = runs.offsets;
    q.counts = runs.counts;
    q.groups = runs.groups;
    q.rows = int32_t(s.R);
    q.I = int32_t(s.N);
    q.depth = int32_t(s.K);
    q.w = f.up.data;
    q.ldw = f.up.ld;
    q.x = f.x.data;
    q.ldx = f.x.ld;
    q.d = h;
    q.ld = f.ldh;
    q.dtype = MAO_BF16;
    if (Z) {
      q.z = Z->data;
      q.ldz = Z->ld;
      q.z_dtype = Z->dtype;
    }
    st = few_launch(q, false, true, act, stream);
    if (st != MAO_OK) return st;
    q.I = int32_t(s.C);
    q.depth = int32_t(s.N);
    q.w = f.down.data;
    q.ldw = f.down.ld;
    q.x = h;
    q.ldx = f.ldh;
    q.d = Y.data;
    q.ld = Y.ld;
    q.dtype = Y.dtype;
    q.early = 1;  // the kernel before it wrote H and Z only, and began after all others
    return few_launch(q, false, false, act, stream);
  }
  FfnArgs<1> gate = {};
  FfnParams& p = gate.p[0];
  st = tc_encode_bf16_map(&p.map_p, f.up.data, s.K, s.N, 2, runs.groups, f.up.ld, s.N * f.up.ld, 2 * s.N * f.up.ld, 16);
  if (st == MAO_OK) st = encode_q(p, f.gate, runs.offsets != nullptr, f.x.data, s.K, s.R, 1, f.x.ld, s.R * f.x.ld);
  if (st != MAO_OK) return st;
  p.d = h;
  p.ld = f.ldh;
  p.dtype = MAO_BF16;
  p.paired = 1;
  if (Z) set_saved(p, *Z);
  st = run(f.gate, act, gate, runs, s.R, at, stream);
  if (st != MAO_OK) return st;

  FfnArgs<1> out = {};
  FfnParams& q = out.p[0];
  st = tc_encode_bf16_map(&q.map_p, f.down.data, s.N, s.C, 1, runs.groups, f.down.ld, s.C * f.down.ld, s.C * f.down.ld, HALF);
  if (st == MAO_OK) st = encode_q(q, f.out, runs.offsets != nullptr, h, s.N, s.R, 1, f.ldh, s.R * f.ldh);
  if (st != MAO_OK) return st;
  set_out(q, Y);
  q.early = 1;
  return run(f.out, act, out, runs, s.R, at, stream);
}

size_t gated_ffn_backward_workspace_size(const mao_mat& dY, const mao_mat& X, const mao_mat& up,
                                         const mao_mat& down, int32_t groups, bool grouped) {
  return X.rows == 0 ? 0 : Backward(dY, X, up, down, groups, grouped).bytes();
}

mao_status gated_ffn_backward_launch(const mao_mat& dY, const mao_mat& X, const mao_mat& up,
                                     const mao_mat& down, const mao_mat& Z, int32_t act, const Runs& runs,
                                     const mao_mat* dX, const mao_mat* dup, const mao_mat* ddown,
                                     void* workspace, cudaStream_t stream) {
  if (X.rows == 0) {  // sums over nothing
    for (const mao_mat* D : {dup, ddown}) {
      if (!D) continue;
      const int es = elem_size(D->dtype);
      const cudaError_t err = cudaMemset2DAsync(D->data, size_t(D->ld) * es, 0, size_t(D->cols) * es,
                                                size_t(D->rows), stream);
      if (err != cudaSuccess) return MAO_ERR_CUDA;
    }
    return MAO_OK;
  }
  Backward b(dY, X, up, down, runs.groups, runs.offsets != nullptr);
  const Sizes& s = b.s;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  uint8_t* h = at;
  at += b.h_bytes();
  uint8_t* dz = at;
  at += b.dz_bytes();
  Copies copies;
  copies.add(b.dy, dY, at);
  copies.add(b.x, X, at);
  copies.add(b.up, up, at);
  copies.add(b.down, down, at);
  mao_status st = copies.launch(stream);
  if (st != MAO_OK) return st;

  {
    FfnArgs<1> back = {};
    FfnParams& p = back.p[0];
    st = tc_encode_bf16_map(&p.map_p, b.down.data, s.N, s.C, 1, runs.groups, b.down.ld, s.C * b.down.ld, s.C * b.down.ld, BK);
    if (st == MAO_OK) st = encode_q(p, b.back, runs.offsets != nullptr, b.dy.data, s.C, s.R, 1, b.dy.ld, s.R * b.dy.ld);
    if (st != MAO_OK) return st;
    p.d = h;
    p.ld = b.ldh;
    p.dtype = MAO_BF16;
    p.paired = 1;
    set_saved(p, Z);
    p.dz = reinterpret_cast<__nv_bfloat16*>(dz);
    p.lddz = 2 * b.ldh;
    p.dz_half = int32_t(b.ldh);
    st = run(b.back, act, back, runs, s.R, at, stream);
    if (st != MAO_OK) return st;
  }
  FfnArgs<3> grads = {};
  if (dX) {
    FfnParams& p = grads.p[0];
    st = tc_encode_bf16_map(&p.map_p, b.up.data, s.K, s.N, 2, runs.groups, b.up.ld, s.N * b.up.ld, 2 * s.N * b.up.ld, BK);
    if (st == MAO_OK) st = encode_q(p, b.dx, runs.offsets != nullptr, dz, s.N, s.R, 2, 2 * b.ldh, b.ldh);
    if (st != MAO_OK) return st;
    set_out(p, *dX);
  }
  if (dup) {
    FfnParams& p = grads.p[1];
    st = tc_encode_bf16_map(&p.map_p, b.x.data, s.K, s.R, 1, 1, b.x.ld, s.R * b.x.ld, s.R * b.x.ld, BK);
    if (st == MAO_OK)
      st = tc_encode_bf16_map(&p.map_q[Q_BOXES - 1], dz, s.N, s.R, 2, 1, 2 * b.ldh, b.ldh, s.R * 2 * b.ldh, BK);
    if (st != MAO_OK) return st;
    set_out(p, *dup);
  }
  if (ddown) {
    FfnParams& p = grads.p[2];
    st = tc_encode_bf16_map(&p.map_p, h, s.N, s.R, 1, 1, b.ldh, s.R * b.ldh, s.R * b.ldh, BK);
    if (st == MAO_OK)
      st = tc_encode_bf16_map(&p.map_q[Q_BOXES - 1], b.dy.data, s.C, s.R, 1, 1, b.dy.ld, s.R * b.dy.ld, s.R * b.dy.ld, BK);
    if (st != MAO_OK) return st;
    set_out(p, *ddown);
  }
  for (FfnParams& p : grads.p) p.early = 1;
  return run_grads({&b.dx, &b.dup, &b.ddown}, {dX != nullptr, dup != nullptr, ddown != nullptr}, grads, runs, s.R, at, stream);
}

mao_status ffn_read_and_clear_error(cudaStream_t stream) {
  // a copy and a synchronisation that programs without these products do not wait for
  return g_launched.load(std::memory_order_acquire) ? read_and_clear_error(stream) : MAO_OK;
}

}  // namespace mao
