// The feed-forward products for few rows: Y = X W^T (W's rows are channels), the gated pair of them,
// and the same of 8-bit integers. Reading W bounds them: each weight is read once, and nothing
// may hold the reads up. A block per SM works on sixteen channels at a time, whose sums' length its
// eight warps share, 128 bytes of each row at a time (short sums: as many teams of four or two
// warps, each with channels of its own); every warp has a ring of its own in shared
// memory that its TMA loads keep full across the ends of sums (24 KB per warp: 192 KB under way
// per SM), so no warp waits for another but where a sum ends.
//
// Up to sixteen rows of X meet the weights in mma.sync m16n8k16 with fp32 sums: with so few rows the
// tensor cores' rate does not count, and the fragments come straight from the ring. Any order of the
// products within a sum does, so a lane takes 32 bytes in a row of W's row and the same 32 of X's and
// hands out eight of them per product. 8-bit codes are multiplied as whole numbers (m16n8k32): slower
// products than fp16's, but no conversion; one row or two by dot products instead. The warps' sums are added in their order.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// What bounds it: HBM, at 6.1 TB/s over both products of one row of the 4096-wide block (gated 37 us,
// 235 MB; down 24 us, 117 MB); a launch and its first loads (5 us) in the shorter calls: an 8-bit
// product of 14336 x 4096, 59 MB, 13 us; eight of 128 experts' blocks of 2048 x 768, 75 MB, 24 us.
// Weights loaded straight to registers instead, two batches in turn: 46 and 33 us.
// 8-bit rows that are multiplied by dot products of four codes: the whole numbers' tensor products take
// as long for one row as for eight, and hold up the stream (14336 x 4096, one row and two: 12.9 and 14.0 us
// against 15.8; three: 15.8 either way). Two or four stages at a time, or X's codes straight to
// registers: 14.6 to 15.7.
constexpr int DOT_ROWS = 2;
constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int CHANNELS = 16;           // per unit
constexpr int BOX_BYTES = 16 * 128;    // sixteen rows of 128 bytes
// A warp's ring; the gated sums of sixteen rows need more room elsewhere.
constexpr int ring_bytes(bool gate, int nt) { return gate && nt == 2 ? 20 * 1024 : 24 * 1024; }

struct FewKernelParams : FewParams {
  CUtensorMap map_w;
  CUtensorMap map_x;
  int32_t x_rows;  // rows of an X box
  int32_t team;    // warps that share a unit: 8, 4 or 2
};

// A lane's 32 bytes of a row.
struct Entries {
  uint32_t w[8];
};

// Bytes 32 (lane % 4) .. + 31 of row r of a box (128-byte rows, swizzled).
__device__ __forceinline__ Entries entries(const uint8_t* box, int r, int lane) {
  const int c = 2 * (lane & 3);
  const uint4 a = *reinterpret_cast<const uint4*>(box + r * 128 + 16 * (c ^ (r & 7)));
  const uint4 b = *reinterpret_cast<const uint4*>(box + r * 128 + 16 * ((c + 1) ^ (r & 7)));
  return Entries{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The sums of a lane: fp32, or whole numbers.
template <bool INT8>
struct Sums {
  using T = float;
};
template <>
struct Sums<true> {
  using T = int;
};
// Two parts of a lane's sum, and the sum in fp32. A warp sums up to 2^17 products of codes (an eighth of
// a depth of 2^20): more than -2^31, and 2^31 itself where all codes are -128, whose word is that of -2^31.
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ int add(int a, int b) { return int(uint32_t(a) + uint32_t(b)); }
__device__ __forceinline__ float sum_of(float v) { return v; }
__device__ __forceinline__ float sum_of(int v) { return v == INT32_MIN ? 0x1p31f : float(v); }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load(bool codes, uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                         int32_t y, int32_t z, int32_t w) {
  if (codes)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(w), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Unit number `unit`: sixteen channels for up to 8 NT rows of a run. The whole warp decodes.
struct Unit {
  int run = 0;  // at or before the unit's (units come in rising order)
  int i0, n;
  int64_t j0;
};
template <int NT>
__device__ __forceinline__ void decode_unit(const FewParams& p, const int* lo, const int* cnt, const int* begin,
                                            int unit, Unit& u) {
  int local = unit, count = (p.rows + 8 * NT - 1) / (8 * NT);
  int64_t first = 0;
  int rows = p.rows;
  if (p.offsets) {
    // (by the whole warp: run after run took 7 us of a call with 128 runs)
    while (true) {
      const int g = u.run + 1 + (threadIdx.x & 31);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, g >= p.groups || begin[g] * p.tiles_i > unit);
      if (past) {
        u.run += __ffs(past) - 1;
        break;
      }
      u.run += 32;
    }
    local = unit - begin[u.run] * p.tiles_i;
    count = begin[u.run + 1] - begin[u.run];
    first = lo[u.run];
    rows = cnt[u.run];
  }
  const int it = local / count, jt = local - it * count;
  u.i0 = it * CHANNELS;
  u.j0 = first + int64_t(jt) * (8 * NT);
  u.n = int(min(int64_t(8 * NT), rows - int64_t(jt) * (8 * NT)));
}

template <bool INT8, bool GATE, int ACT, int NT>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ FewKernelParams p) {
  constexpr int MATS = GATE ? 2 : 1;
  constexpr int CHAINS = MATS * NT == 1 ? 2 : 1;  // sums in turn, so that products do not wait for one another
  constexpr int STAGE = MATS * BOX_BYTES + NT * 1024;  // a multiple of 1024
  constexpr int RING = ring_bytes(GATE, NT), STAGES = RING / STAGE;
  static_assert(RING % 1024 == 0 && STAGE % 1024 == 0, "swizzled boxes");
  extern __shared__ uint8_t smem_raw[];
  __shared__ float parts[2][WARPS][MATS][NT][32][4];
  __shared__ int table[3 * (MAX_GROUPS + 2)];
  __shared__ int scratch[WARPS];
  __shared__ uint64_t bars[WARPS][STAGES];
  __shared__ int abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &abort_word;
  int* lo = table;
  int* cnt = lo + MAX_GROUPS + 2;
  int* begin = cnt + MAX_GROUPS + 2;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
                  warp * RING;
  if (threadIdx.x == 0) abort_word = 0;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&bars[warp][s]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  // launched as a programmatic dependent: the set-up so far may overlap the previous kernel, with
  // `early` the first loads of W too
  if (!p.early) wait_for_previous();
  int units = p.tiles_i * ((p.rows + 8 * NT - 1) / (8 * NT));
  if (p.offsets) {
    make_table<THREADS>(p, lo, cnt, begin, scratch);
    __syncthreads();
    units = begin[p.groups] * p.tiles_i;
  }
  const int chunks = (p.depth * (INT8 ? 1 : 2) + 127) / 128;
  const int step = INT8 ? 128 : 64;  // entries of a chunk

  // The warp's items: every team-th chunk of each of its team's units. The next one to load:
  const int team = p.team, member = warp % team;
  const int unit0 = int(blockIdx.x) * (WARPS / team) + warp / team, unit_step = int(gridDim.x) * (WARPS / team);
  Unit next;
  int next_unit = unit0, next_chunk = member, loaded = 0;
  if (next_chunk >= chunks) next_unit = units;  // no chunk of any sum is this warp's
  if (next_unit < units) decode_unit<NT>(p, lo, cnt, begin, next_unit, next);
  int first_k = 0, first_j = 0;  // lane s: where the first load into stage s has its rows of X
  auto load_next = [&](bool with_x) {
    if (next_unit >= units) return;
    const int stage = loaded % STAGES;
    const int k = next_chunk * step;
    if (lane == stage && !with_x) {
      first_k = k;
      first_j = int(next.j0);
    }
    if (lane == 0) {
      const uint32_t bar = smem_u32(&bars[warp][stage]), dst = smem_u32(ring) + stage * STAGE;
      mbar_expect_tx(bar, MATS * BOX_BYTES + p.x_rows * 128);
#pragma unroll
      for (int m = 0; m < MATS; ++m) tma_load(INT8, dst + m * BOX_BYTES, &p.map_w, bar, k, next.i0, m, next.run);
      if (with_x) tma_load(INT8, dst + MATS * BOX_BYTES, &p.map_x, bar, k, int(next.j0), 0, 0);
    }
    ++loaded;
    next_chunk += team;
    if (next_chunk >= chunks) {
      next_chunk = member;
      next_unit += unit_step;
      if (next_unit < units) decode_unit<NT>(p, lo, cnt, begin, next_unit, next);
    }
  };
  for (int s = 0; s < STAGES; ++s) load_next(!p.early);
  if (p.early) {
    wait_for_previous();
    if (lane < loaded)
      tma_load(INT8, smem_u32(ring) + lane * STAGE + MATS * BOX_BYTES, &p.map_x, smem_u32(&bars[warp][lane]), first_k,
               first_j, 0, 0);
    __syncwarp();
  }

  if (p.offsets) {  // rows that hold no tokens, while the first loads are under way
    const int turn = int(blockIdx.x) * WARPS + warp, turns = int(gridDim.x) * WARPS;
    const int es = p.dtype == MAO_F32 ? 4 : 2, ez = p.z_dtype == MAO_F32 ? 4 : 2;
    for_unused_rows(p, lo, cnt, turn, turns, [&](int64_t j0, int64_t j1, int64_t every) {
      if (!GATE) clear_rows(p.d, p.ld * es, int64_t(p.I) * es, j0, j1, every, lane);
      else if (p.z) clear_rows(p.z, p.ldz * ez, int64_t(p.I) * 2 * ez, j0, j1, every, lane);
    });
  }

  Unit u;
  int used = 0, flip = 0;
  bool ok = true;
  for (int unit = unit0; unit < units; unit += unit_step, flip ^= 1) {
    decode_unit<NT>(p, lo, cnt, begin, unit, u);
    typename Sums<INT8>::T acc[CHAINS][MATS][NT][4] = {};
    int dots[DOT_ROWS][2] = {};  // of up to DOT_ROWS rows: of row j of X with W's rows r and r + 8
    for (int c = member; c < chunks; c += team) {
      const int stage = used % STAGES;
      ok = ok && wait_warp<false>(&bars[warp][stage], uint32_t(used / STAGES) & 1u, abort_flag, p.timeout_ns);
      if (!ok) break;
      const uint8_t* box = ring + stage * STAGE;
      const int r = lane >> 2;
      if (INT8 && NT == 1 && u.n <= DOT_ROWS) {
        const Entries a = entries(box, r, lane), b = entries(box, r + 8, lane);
#pragma unroll
        for (int j = 0; j < DOT_ROWS; ++j) {
          if (j >= u.n) break;
          const Entries x = entries(box + BOX_BYTES, j, lane);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            dots[j][0] = __dp4a(int(a.w[s]), int(x.w[s]), dots[j][0]);
            dots[j][1] = __dp4a(int(b.w[s]), int(x.w[s]), dots[j][1]);
          }
        }
        ++used;
        __syncwarp();  // every lane has read the stage
        load_next(true);
        continue;
      }
      Entries x[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) x[q] = entries(box + MATS * BOX_BYTES, r + 8 * q, lane);
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const Entries a = entries(box + m * BOX_BYTES, r, lane);
        const Entries b = entries(box + m * BOX_BYTES, r + 8, lane);
#pragma unroll
        for (int s = 0; s < 8; s += 2)
#pragma unroll
          for (int q = 0; q < NT; ++q) mma(acc[(s / 2) % CHAINS][m][q], a.w[s], b.w[s], a.w[s + 1], b.w[s + 1], x[q].w[s], x[q].w[s + 1]);
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      load_next(true);
    }
    if (INT8 && NT == 1 && u.n <= DOT_ROWS) {
      // a lane's sums are over a quarter of the columns; lane 4 c + j / 2 hands over row j's, channels c, c + 8
#pragma unroll
      for (int j = 0; j < DOT_ROWS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int v = dots[j][h];
          v = add(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
          v = add(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
          if ((lane & 3) == j >> 1) acc[0][0][0][2 * h + (j & 1)] = v;
        }
    }
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          parts[flip][warp][m][q][lane][e] =
              sum_of(CHAINS == 1 ? acc[0][m][q][e] : add(acc[0][m][q][e], acc[CHAINS - 1][m][q][e]));
    // (the other half of `parts` was read before this barrier's last use but one)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / team), "r"(32 * team) : "memory");
    // row j0 + r of X, channel i0 + c
    for (int x = threadIdx.x % (32 * team); x < CHANNELS * u.n; x += 32 * team) {
      const int c = x % CHANNELS, r = x / CHANNELS, i = u.i0 + c;
      if (i >= p.I) continue;
      float v[MATS] = {};
      const int from = (c & 7) * 4 + ((r & 7) >> 1), e = (c >> 3) * 2 + (r & 1);
      float part[WARPS][MATS];  // all on their way before the first is added
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
#pragma unroll
        for (int m = 0; m < MATS; ++m)
          part[w][m] = w < team ? parts[flip][warp - member + w][m][NT == 1 ? 0 : r >> 3][from][e] : 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
#pragma unroll
        for (int m = 0; m < MATS; ++m) v[m] += part[w][m];
      const int64_t j = u.j0 + r;
      if (GATE) {
        static_cast<__nv_bfloat16*>(p.d)[j * p.ld + i] = __float2bfloat16_rn(activate<ACT>(v[0]) * v[MATS - 1]);
        if (p.z) {
          store_elem(p.z, j * p.ldz + i, p.z_dtype, v[0]);
          store_elem(p.z, j * p.ldz + p.I + i, p.z_dtype, v[MATS - 1]);
        }
      } else {
        if (INT8) v[0] = v[0] * __ldg(p.sa + j) * __ldg(p.sb + int64_t(u.run) * p.I + i);
        store_elem(p.d, j * p.ld + i, p.dtype, v[0]);
      }
    }
  }
  // after an abort, the loads already issued land before the block leaves
  if (*abort_flag && lane == 0)
    for (; used < loaded; ++used)
      mbar_drain(smem_u32(&bars[warp][used % STAGES]), uint32_t(used / STAGES) & 1u, 20000000ull);
}

using Kernel = void (*)(const FewKernelParams);

std::atomic<bool> g_launched{false};

}  // namespace

mao_status few_launch(const FewParams& params, bool int8, bool gate, int32_t act, cudaStream_t stream) {
  FewKernelParams p = {};
  static_cast<FewParams&>(p) = params;
  p.tiles_i = int32_t(ceil_div(p.I, CHANNELS));
  p.timeout_ns = wait_limit_ns();
  const int two = !p.offsets && p.rows > 8;
  p.height = two ? 16 : 8;
  p.x_rows = p.rows < p.height ? p.rows : p.height;
  const int64_t chunks = ceil_div(int64_t(p.depth) * (int8 ? 1 : 2), 128);
  const int64_t least = int8 ? 8 : 4;  // chunks of a warp (14336 x 4096 8-bit, one row: 12.9 us; four 15.2, sixteen 14.8)
  p.team = chunks >= 8 * least ? 8 : chunks >= 4 * least ? 4 : 2;
  const int64_t mats = gate ? 2 : 1, w_rows = int64_t(p.I);
  mao_status st = int8 ? tc_encode_code_map(&p.map_w, p.w, p.depth, w_rows, p.ldw, p.groups, CHANNELS)
                       : tc_encode_bf16_map(&p.map_w, p.w, p.depth, w_rows, mats, p.groups, p.ldw, w_rows * p.ldw,
                                            mats * w_rows * p.ldw, CHANNELS);
  if (st == MAO_OK)
    st = int8 ? tc_encode_code_map(&p.map_x, p.x, p.depth, p.rows, p.ldx, 1, p.x_rows)
              : tc_encode_bf16_map(&p.map_x, p.x, p.depth, p.rows, 1, 1, p.ldx, p.rows * p.ldx, p.rows * p.ldx, p.x_rows);
  if (st != MAO_OK) return st;
  static const Kernel kernels[10] = {
      few_kernel<true, false, 0, 1>,          few_kernel<true, false, 0, 2>,
      few_kernel<false, false, 0, 1>,         few_kernel<false, false, 0, 2>,
      few_kernel<false, true, MAO_SILU, 1>,   few_kernel<false, true, MAO_SILU, 2>,
      few_kernel<false, true, MAO_GELU, 1>,   few_kernel<false, true, MAO_GELU, 2>,
      few_kernel<false, true, MAO_GELU_TANH, 1>, few_kernel<false, true, MAO_GELU_TANH, 2>};
  static std::atomic<bool> ready[64];
  st = once_per_device(ready, [&] {
    cudaError_t err = cudaSuccess;
    for (int f = 0; f < 10 && err == cudaSuccess; ++f)
      err = cudaFuncSetAttribute(kernels[f], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 1024 + WARPS * ring_bytes(f >= 4, 1 + f % 2));
    return err;
  });
  if (st != MAO_OK) return st;
  g_launched.store(true, std::memory_order_release);
  const int64_t units = p.offsets ? int64_t(num_sms()) * WARPS : int64_t(p.tiles_i) * ceil_div(p.rows, p.height);
  const int64_t blocks = ceil_div(units, WARPS / p.team);
  return launch_dependent(kernels[(int8 ? 0 : gate ? 4 + 2 * act : 2) + two], unsigned(blocks < num_sms() ? blocks : num_sms()),
                          THREADS, size_t(1024 + WARPS * ring_bytes(gate, 1 + two)), stream, p);
}

mao_status few_read_and_clear_error(cudaStream_t stream) {
  return g_launched.load(std::memory_order_acquire) ? read_and_clear_error(stream) : MAO_OK;
}

}  // namespace mao
