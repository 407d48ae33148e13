// Quantisation to 8-bit floating point (e4m3) with a power-of-two scale for each block of 128.
//
// A thread block takes one 128 x 128 tile of the matrix into registers (256 threads, eight
// rows of eight columns each, 16-byte loads), finds the largest magnitudes of the tile's row
// blocks, column blocks or of the whole tile, and writes the codes: one pass over the input
// whatever the blocks, both directions included.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "experts.h"
#include "internal.h"

namespace mao {
namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr uint32_t INF_BITS = 0x7F800000u;
constexpr int TABLE = 64;  // matrices of a descriptor array per launch

struct Out {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, scale_ld;
};

struct QuantParams {
  const void* base;           // matrix 0 (stride > 0)
  int64_t stride;             // elements between matrices; 0: ptr and lds below
  int64_t ld;
  int64_t rows, cols;         // of the result
  int64_t src_rows;           // of X
  const int32_t* index;       // source rows (times copies), or null
  int32_t copies;
  int32_t row_tiles, col_tiles;
  int64_t first;              // number of matrix 0 among the results
  Out row, col, tile;
  const void* ptr[TABLE];
  int64_t lds[TABLE];
};

// The scale byte of a block from the bits of its largest magnitude a = m 2^q, m in [1, 2):
// 448 = 1.75 * 2^8, so a <= 448 * 2^e holds from e = q - 8 on if m <= 1.75 and from q - 7
// on if not. Adding 0x1FFFFF carries into the exponent just when m > 1.75.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  return max(int((amax_bits + 0x1FFFFFu) >> 23) - 8, 0);
}
// 2^-(byte - 127): a normal number for every byte that scale_byte gives (0 .. 247).
__device__ __forceinline__ float scale_inverse(int byte) {
  return __uint_as_float(uint32_t(254 - byte) << 23);
}

// Eight consecutive entries of a row as they are in memory.
template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
  uint4 q;
  __device__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ void load(const void* base, int64_t at) {
    q = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + at);
  }
  __device__ void load_some(const void* base, int64_t at, int n) {
    zero();
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= uint32_t(s[i]) << (16 * (i & 1));
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ uint32_t word(int i) const { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }
  __device__ float value(int i) const {
    const uint32_t w = word(i >> 1);
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <>
struct Raw<false> {
  uint4 q[2];
  __device__ void zero() { q[0] = q[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ void load(const void* base, int64_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(base) + at);
    q[0] = s[0];
    q[1] = s[1];
  }
  __device__ void load_some(const void* base, int64_t at, int n) {
    uint32_t w[8];
    const uint32_t* s = reinterpret_cast<const uint32_t*>(base) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? s[i] : 0u;
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ float value(int i) const {
    const uint4& u = q[i >> 2];
    return __uint_as_float((i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w);
  }
};

// Magnitudes as ordered integers: NaN and infinities are the largest, or count as 0 with
// FINITE. bf16 works on two values per word.
__device__ __forceinline__ uint32_t mag(uint32_t bits, bool finite) {
  const uint32_t a = bits & 0x7FFFFFFFu;
  return finite && a >= INF_BITS ? 0u : a;
}
__device__ __forceinline__ uint32_t mag2(uint32_t w, bool finite) {
  const uint32_t a = w & 0x7FFF7FFFu;
  return finite ? a & ~__vcmpgeu2(a, 0x7F807F80u) : a;
}

template <bool BF16, bool ROW, bool COL, bool TILE>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t part[8][128];
  __shared__ __align__(8) uint8_t col_byte[128];
  wait_for_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rr = tid >> 4;  // columns 8 cg .., rows rr + 16 it
  const int tiles = p.row_tiles * p.col_tiles;
  const int z = int(blockIdx.x / unsigned(tiles));
  const int in = int(blockIdx.x - unsigned(z) * unsigned(tiles));
  const int rb = in / p.col_tiles, cb = in - rb * p.col_tiles;
  const int64_t es = BF16 ? 2 : 4;
  const void* base = p.stride ? static_cast<const uint8_t*>(p.base) + int64_t(z) * p.stride * es : p.ptr[z];
  const int64_t ld = p.stride ? p.ld : p.lds[z];
  const int64_t c0 = int64_t(cb) * 128 + 8 * cg;
  const int nc = int(min(int64_t(8), p.cols - c0));  // columns of this thread (may be <= 0)
  const bool vec = nc == 8 && (reinterpret_cast<uintptr_t>(base) % 16 == 0) && (ld * es) % 16 == 0;

  Raw<BF16> x[8];
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    int64_t r = int64_t(rb) * 128 + 16 * it + rr;
    bool have = r < p.rows && nc > 0;
    if (have && p.index) {
      const int32_t i = p.index[r];
      r = i < 0 ? -1 : i / p.copies;
      have = r >= 0 && r < p.src_rows;
    }
    if (!have) x[it].zero();
    else if (vec) x[it].load(base, r * ld + c0);
    else x[it].load_some(base, r * ld + c0, nc);
  }

  uint32_t rmax[8];             // the thread's share of each row
  uint32_t cmax[BF16 ? 4 : 8];  // and of each column (bf16: two per word)
  auto largest = [&](bool finite) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) cmax[i] = 0u;
    uint32_t all = 0u;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      if constexpr (BF16) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = mag2(x[it].word(i), finite);
          m = __vmaxu2(m, a);
          if (COL) cmax[i] = __vmaxu2(cmax[i], a);
        }
        rmax[it] = max(m & 0xFFFF0000u, m << 16);
      } else {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t a = mag(__float_as_uint(x[it].value(i)), finite);
          m = max(m, a);
          if (COL) cmax[i] = max(cmax[i], a);
        }
        rmax[it] = m;
      }
      all = max(all, rmax[it]);
    }
    return all;
  };
  uint32_t all = largest(false);
  const bool bad = __syncthreads_or(all >= INF_BITS) != 0;  // a NaN or infinity in the tile
  if (bad) all = largest(true);

  auto write = [&](const Out& o, int it, const float (&inv)[8]) {
    const int64_t r = int64_t(rb) * 128 + 16 * it + rr;
    if (r >= p.rows || nc <= 0) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[it].value(i) * inv[i];
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(fabsf(x[it].value(i)) < INFINITY)) v[i] = __uint_as_float(0x7FC00000u);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(v[4 * h], v[4 * h + 1]), __NV_SATFINITE, __NV_E4M3)) |
             uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2], v[4 * h + 3]), __NV_SATFINITE, __NV_E4M3)) << 16;
    uint8_t* d = o.codes + ((p.first + z) * p.rows + r) * o.ld + c0;
    if (nc == 8) {
      *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nc) d[i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
    }
  };

  if constexpr (ROW) {
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      uint32_t m = rmax[it];
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(FULL, m, o));
      const int byte = scale_byte(m);
      const float s = scale_inverse(byte);
      const float inv[8] = {s, s, s, s, s, s, s, s};
      write(p.row, it, inv);
      const int64_t r = int64_t(rb) * 128 + 16 * it + rr;
      if (cg == 0 && r < p.rows)
        p.row.scales[((p.first + z) * p.rows + r) * p.row.scale_ld + cb] = uint8_t(byte);
    }
  }
  if constexpr (COL) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
      if constexpr (BF16) {
        const uint32_t m = __vmaxu2(cmax[i], __shfl_xor_sync(FULL, cmax[i], 16));
        if (lane < 16) {
          part[warp][8 * cg + 2 * i] = m << 16;
          part[warp][8 * cg + 2 * i + 1] = m & 0xFFFF0000u;
        }
      } else {
        const uint32_t m = max(cmax[i], __shfl_xor_sync(FULL, cmax[i], 16));
        if (lane < 16) part[warp][8 * cg + i] = m;
      }
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t m = 0u;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, part[w][tid]);
      const int byte = scale_byte(m);
      col_byte[tid] = uint8_t(byte);
      const int64_t c = int64_t(cb) * 128 + tid;
      if (c < p.cols)
        p.col.scales[((p.first + z) * p.row_tiles + rb) * p.col.scale_ld + c] = uint8_t(byte);
    }
    __syncthreads();
    const uint2 b = *reinterpret_cast<const uint2*>(&col_byte[8 * cg]);
    float inv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = scale_inverse(((i < 4 ? b.x : b.y) >> (8 * (i & 3))) & 255u);
#pragma unroll
    for (int it = 0; it < 8; ++it) write(p.col, it, inv);
  }
  if constexpr (TILE) {
    const uint32_t m = __reduce_max_sync(FULL, all);
    if (lane == 0) part[warp][0] = m;
    __syncthreads();
    uint32_t t = 0u;
#pragma unroll
    for (int w = 0; w < 8; ++w) t = max(t, part[w][0]);
    const int byte = scale_byte(t);
    const float s = scale_inverse(byte);
    const float inv[8] = {s, s, s, s, s, s, s, s};
#pragma unroll
    for (int it = 0; it < 8; ++it) write(p.tile, it, inv);
    if (tid == 0) p.tile.scales[((p.first + z) * p.row_tiles + rb) * p.tile.scale_ld + cb] = uint8_t(byte);
  }
}

Out out_of(const mao_fp8* m) {
  return m ? Out{m->codes, m->scales, m->ld, m->scale_ld} : Out{nullptr, nullptr, 0, 0};
}

}  // namespace

mao_status quantize_launch(const mao_mat* X, int32_t batch, int64_t batch_stride,
                           const int32_t* index, int64_t n_index, int32_t copies,
                           const mao_fp8* row, const mao_fp8* col, const mao_fp8* tile,
                           cudaStream_t stream) {
  QuantParams p = {};
  p.rows = copies > 0 ? n_index : X[0].rows;
  p.cols = X[0].cols;
  p.src_rows = X[0].rows;
  if (p.rows == 0) return MAO_OK;
  p.index = copies > 0 ? index : nullptr;
  p.copies = copies;
  const int64_t rt = ceil_div(p.rows, 128), ct = ceil_div(p.cols, 128);
  p.row = out_of(row);
  p.col = out_of(col);
  p.tile = out_of(tile);
  const int64_t most = 0x7FFFFFFF;
  if (rt * ct > most) return MAO_ERR_UNSUPPORTED;
  p.row_tiles = int32_t(rt);
  p.col_tiles = int32_t(ct);
  const bool bf = X[0].dtype == MAO_BF16;
  using Kernel = void (*)(const QuantParams);
  const Kernel k =
      tile ? (bf ? quantize_kernel<true, false, false, true> : quantize_kernel<false, false, false, true>)
      : row && col ? (bf ? quantize_kernel<true, true, true, false> : quantize_kernel<false, true, true, false>)
      : row ? (bf ? quantize_kernel<true, true, false, false> : quantize_kernel<false, true, false, false>)
            : (bf ? quantize_kernel<true, false, true, false> : quantize_kernel<false, false, true, false>);
  int32_t per = batch_stride > 0 || batch == 1 ? int32_t(most / (rt * ct)) : TABLE;
  if (int64_t(per) * rt * ct > most) per = int32_t(most / (rt * ct));
  for (int32_t b = 0; b < batch; b += per) {
    const int32_t n = batch - b < per ? batch - b : per;
    p.first = b;
    if (batch_stride > 0) {
      const int64_t es = elem_size(X[0].dtype);
      p.base = static_cast<const uint8_t*>(X[0].data) + int64_t(b) * batch_stride * es;
      p.stride = batch_stride;
      p.ld = X[0].ld;
    } else {
      p.stride = 0;
      for (int32_t i = 0; i < n; ++i) {
        p.ptr[i] = X[b + i].data;
        p.lds[i] = X[b + i].ld;
      }
    }
    const mao_status st = launch_dependent(k, unsigned(int64_t(n) * rt * ct), 256, 0, stream, p);
    if (st != MAO_OK) return st;
  }
  return MAO_OK;
}

}  // namespace mao
