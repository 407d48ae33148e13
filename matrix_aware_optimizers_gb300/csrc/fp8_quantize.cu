// Quantisation to 8-bit floating point (e4m3) with a power-of-two scale for each block of 128.
//
// A thread block takes one 128 x 128 tile of the matrix into registers (256 threads, eight
// rows of eight columns each, 16-byte loads), finds the largest magnitudes of the tile's row
// blocks, column blocks or of the whole tile, and writes the codes: one pass over the input
// whatever the blocks, both directions included.
//
// With y = x 2^-e exact, the only rounding is that of the code, and the code and scale do not
// depend on how or where they are computed.
//
// HBM bounds it, except for gathered rows, which instructions and latency bound (bf16: eight per
// entry in one direction and eleven in both, 58% of the issue slots). So bf16 maxima and the
// rows' scales are taken two to a register and products two to an instruction, an entry is
// unpacked once for both directions, places are divided by multiplications, tiles that reach
// over an edge or hold NaN or infinities take a path out of line, and registers are kept to 64
// for four blocks per SM (bf16; two for fp32): with 121 registers the gathered both-direction
// pass took 133 us instead of 84. Blocks of 512 and 1024 threads were slower everywhere (80 and
// 150 us against 61 for bf16 rows). Measured, 65,536 x 2048: bf16 row 59 us (6.8 TB/s), column
// 59, tile 58, both 80 (6.7 TB/s); fp32 row 100 us (6.7 TB/s), both 124; 81,792 rows gathered
// from 8192, bf16: row 59 us, both 84 (fp32: 104, 141); 128 matrices of 1536 x 2048, bf16, tile:
// 166 us (7.3 TB/s). For gathered rows, a block that copies its next tile's rows into shared
// memory while it encodes (98 us), or takes several tiles in a row (119), was slower: registers
// spill.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "experts.h"
#include "internal.h"

namespace mao {
namespace {

constexpr uint32_t FULL_MASK = 0xFFFFFFFFu;
constexpr uint32_t INF_BITS = 0x7F800000u;
constexpr int THREADS = 256;
constexpr int IT = 2048 / THREADS;    // rows of a thread
constexpr int STEP = THREADS / 16;    // apart
constexpr int WARPS = THREADS / 32;
constexpr int TABLE = 64;  // matrices of a descriptor array per launch

struct Out {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, scale_ld;
};

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery): with 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d), m d - 2^(31+s) < 2^s, so n m / 2^(31+s) stays below the next integer.
struct Divisor {
  uint32_t m, s;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return uint32_t((uint64_t(n) * m) >> s);
  }
};
Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {uint32_t(((uint64_t(1) << (31 + s)) + d - 1) / d), 31 + s};
}

struct QuantParams {
  const void* base;           // matrix 0 (stride > 0)
  int64_t stride;             // elements between matrices; 0: ptr and lds below
  int64_t ld;
  int64_t rows, cols;         // of the result
  int64_t src_rows;           // of X
  const int32_t* index;       // source rows (times copies), or null
  int32_t row_tiles, col_tiles;
  Divisor by_copies, by_tiles, by_cols;  // copies, tiles of a matrix, col_tiles
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
  uint32_t w[4];
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const void* at) {
    const uint4 q = *reinterpret_cast<const uint4*>(at);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  }
  __device__ __forceinline__ void load_some(const void* at, int n) {
    zero();
    const uint16_t* s = reinterpret_cast<const uint16_t*>(at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= uint32_t(s[i]) << (16 * (i & 1));
  }
  __device__ __forceinline__ float value(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Raw<false> {
  uint32_t w[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* at) {
    const uint4 a = reinterpret_cast<const uint4*>(at)[0], b = reinterpret_cast<const uint4*>(at)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void load_some(const void* at, int n) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(at);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? s[i] : 0u;
  }
  __device__ __forceinline__ float value(int i) const { return __uint_as_float(w[i]); }
};

// Magnitudes: fp32 as ordered integers; bf16 two to a word. NaN is above infinity, and both
// above all numbers; with `finite` they count as 0 instead.
__device__ __forceinline__ uint32_t mag(uint32_t bits, bool finite) {
  const uint32_t a = bits & 0x7FFFFFFFu;
  return finite && a >= INF_BITS ? 0u : a;
}
__device__ __forceinline__ uint32_t mag2(uint32_t w, bool finite) {
  const uint32_t a = w & 0x7FFF7FFFu;
  return finite ? a & ~__vcmpgeu2(a, 0x7F807F80u) : a;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Two products at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}

// The codes of eight entries scaled by inv; `bad`: some may not be finite.
template <bool BF16>
__device__ __forceinline__ uint2 encode(const Raw<BF16>& x, const float2 (&inv)[4], bool bad) {
  float2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(make_float2(x.value(2 * i), x.value(2 * i + 1)), inv[i]);
  if (bad) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(fabsf(x.value(2 * i)) < INFINITY)) v[i].x = __uint_as_float(0x7FC00000u);
      if (!(fabsf(x.value(2 * i + 1)) < INFINITY)) v[i].y = __uint_as_float(0x7FC00000u);
    }
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __nv_cvt_float2_to_fp8x2(v[i], __NV_SATFINITE, __NV_E4M3);
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// A tile wherever it lies and whatever it holds; out of line, so that the common path keeps
// its registers.
template <bool BF16, bool ROW, bool COL, bool TILE>
__device__ __noinline__ void quantize_tile(const QuantParams& p, int64_t matrix, int rb, int cb,
                                              const uint8_t* base, int64_t ld, bool vec,
                                              uint32_t (*part)[128], uint8_t* col_byte,
                                              const int64_t* src) {
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rr = tid >> 4;  // columns 8 cg .., rows rr + STEP it
  const int64_t c0 = int64_t(cb) * 128 + 8 * cg;
  const int nc = int(min(int64_t(8), p.cols - c0));  // columns here (may be <= 0)
  const int nr = int(min(int64_t(128), p.rows - int64_t(rb) * 128));

  Raw<BF16> x[IT];
  const uint8_t* at = base + (int64_t(rb) * 128 * ld + c0) * ES;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int r = STEP * it + rr;
    const uint8_t* a;
    bool have = r < nr && nc > 0;
    if (src) {
      const int64_t from = src[r];
      have = have && from >= 0;
      a = base + from + c0 * ES;
    } else {
      a = at + r * ld * ES;
    }
    if (!have) x[it].zero();
    else if (vec && nc == 8) x[it].load(a);
    else x[it].load_some(a, nc);
  }

  // the thread's share of each row's and column's largest magnitude (bf16: of two rows or
  // columns per word)
  constexpr int NR = BF16 ? IT / 2 : IT, NC = BF16 ? 4 : 8;
  uint32_t rmax[NR], cmax[NC];
  auto largest = [&](bool finite) {
    uint32_t all = 0u;
#pragma unroll
    for (int i = 0; i < NC; ++i) cmax[i] = 0u;
    if constexpr (BF16) {
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        uint32_t m[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t a[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = mag2(x[2 * h + q].w[i], finite);
            if (COL) cmax[i] = max2(cmax[i], a[i]);
          }
          m[q] = max2(max2(a[0], a[1]), max2(a[2], a[3]));
        }
        rmax[h] = max2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
        all = max2(all, rmax[h]);
      }
      return max(all & 0xFFFF0000u, all << 16);
    } else {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t a = mag(x[it].w[i], finite);
          m = max(m, a);
          if (COL) cmax[i] = max(cmax[i], a);
        }
        rmax[it] = m;
        all = max(all, m);
      }
      return all;
    }
  };
  uint32_t all = largest(false);
  const bool bad = __syncthreads_or(all >= INF_BITS) != 0;  // a NaN or infinity in the tile
  if (bad) all = largest(true);

  const int64_t row0 = matrix * p.rows + int64_t(rb) * 128 + rr;  // of the stacked results
  auto put = [&](uint8_t* d, uint2 c) {
    if (nc == 8) {
      *reinterpret_cast<uint2*>(d) = c;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nc) d[i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
  };

  float2 col_inv[4];
  if constexpr (COL) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t other = __shfl_xor_sync(FULL_MASK, cmax[i], 16);
      if constexpr (BF16) {
        const uint32_t m = max2(cmax[i], other);
        if (lane < 16) {
          part[warp][8 * cg + 2 * i] = m << 16;
          part[warp][8 * cg + 2 * i + 1] = m & 0xFFFF0000u;
        }
      } else {
        if (lane < 16) part[warp][8 * cg + i] = max(cmax[i], other);
      }
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t m = 0u;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) m = max(m, part[w][tid]);
      const int byte = scale_byte(m);
      col_byte[tid] = uint8_t(byte);
      const int64_t c = int64_t(cb) * 128 + tid;
      if (c < p.cols) p.col.scales[(matrix * p.row_tiles + rb) * p.col.scale_ld + c] = uint8_t(byte);
    }
    __syncthreads();
    const uint2 b = *reinterpret_cast<const uint2*>(&col_byte[8 * cg]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = (i < 2 ? b.x : b.y) >> (16 * (i & 1));
      col_inv[i] = make_float2(scale_inverse(h & 255u), scale_inverse((h >> 8) & 255u));
    }
  }
  if constexpr (ROW) {
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int o = 8; o; o >>= 1) {
        const uint32_t other = __shfl_xor_sync(FULL_MASK, rmax[h], o);
        rmax[h] = BF16 ? max2(rmax[h], other) : max(rmax[h], other);
      }
  }
  if constexpr (ROW || COL) {
    uint8_t* dr = p.row.codes + row0 * p.row.ld + c0;
    uint8_t* dc = p.col.codes + row0 * p.col.ld + c0;
    uint8_t* sc = p.row.scales + row0 * p.row.scale_ld + cb;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (STEP * it + rr < nr && nc > 0) {
        if (ROW) {
          const uint32_t m = !BF16 ? rmax[it % NR] : (it & 1) ? rmax[it / 2] & 0xFFFF0000u : rmax[it / 2] << 16;
          const int byte = scale_byte(m);
          const float s = scale_inverse(byte);
          const float2 inv[4] = {{s, s}, {s, s}, {s, s}, {s, s}};
          put(dr, encode<BF16>(x[it], inv, bad));
          if (cg == 0) *sc = uint8_t(byte);
        }
        if (COL) put(dc, encode<BF16>(x[it], col_inv, bad));
      }
      dr += STEP * p.row.ld;
      dc += STEP * p.col.ld;
      sc += STEP * p.row.scale_ld;
    }
  }
  if constexpr (TILE) {
    const uint32_t m = __reduce_max_sync(FULL_MASK, all);
    if (lane == 0) part[warp][0] = m;
    __syncthreads();
    uint32_t t = 0u;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) t = max(t, part[w][0]);
    const int byte = scale_byte(t);
    const float s = scale_inverse(byte);
    const float2 inv[4] = {{s, s}, {s, s}, {s, s}, {s, s}};
    uint8_t* d = p.tile.codes + row0 * p.tile.ld + c0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (STEP * it + rr < nr && nc > 0) put(d, encode<BF16>(x[it], inv, bad));
      d += STEP * p.tile.ld;
    }
    if (tid == 0) p.tile.scales[(matrix * p.row_tiles + rb) * p.tile.scale_ld + cb] = uint8_t(byte);
  }
}

// The codes of four entries, the first in the lowest byte.
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
  uint32_t c;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(c)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return c;
}

// A tile inside the matrix whose rows take 16-byte loads and that holds finite numbers only:
// returns false, with nothing written, if there are others.
template <bool BF16, bool ROW, bool COL, bool TILE>
__device__ __forceinline__ bool quantize_full(const QuantParams& p, int64_t matrix, int rb, int cb,
                                              const uint8_t* base, int64_t ld, uint32_t (*part)[128],
                                              uint8_t* byte_of, const int64_t* src, bool gaps) {
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rr = tid >> 4;  // columns 8 cg .., rows rr + STEP it
  Raw<BF16> x[IT];
  const uint8_t* at = base + (int64_t(cb) * 128 + 8 * cg) * ES;
  if (src && gaps) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t from = src[STEP * it + rr];
      x[it].zero();
      if (from >= 0) x[it].load(at + from);
    }
  } else if (src) {
#pragma unroll
    for (int it = 0; it < IT; ++it) x[it].load(at + src[STEP * it + rr]);
  } else {
    at += (int64_t(rb) * 128 + rr) * ld * ES;
#pragma unroll
    for (int it = 0; it < IT; ++it) x[it].load(at + int64_t(STEP * it) * ld * ES);
  }
  // largest magnitudes of the thread's share of rows and columns (bf16: two to a word)
  constexpr int NR = BF16 ? IT / 2 : IT, NC = BF16 ? 4 : 8;
  uint32_t rmax[NR], cmax[NC], all = 0u;
#pragma unroll
  for (int i = 0; i < NC; ++i) cmax[i] = 0u;
#pragma unroll
  for (int h = 0; h < NR; ++h) {
    if constexpr (BF16) {
      uint32_t m[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = x[2 * h + q].w[i] & 0x7FFF7FFFu;
          if (COL) cmax[i] = max2(cmax[i], a[i]);
        }
        m[q] = max2(max2(a[0], a[1]), max2(a[2], a[3]));
      }
      rmax[h] = max2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
      all = max2(all, rmax[h]);
    } else {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = x[h].w[i] & 0x7FFFFFFFu;
        m = max(m, a);
        if (COL) cmax[i] = max(cmax[i], a);
      }
      rmax[h] = m;
      all = max(all, m);
    }
  }
  if (BF16) all = max(all & 0xFFFF0000u, all << 16);
  if constexpr (COL) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t other = __shfl_xor_sync(FULL_MASK, cmax[i], 16);
      if constexpr (BF16) {
        const uint32_t m = max2(cmax[i], other);
        if (lane < 16) *reinterpret_cast<uint2*>(&part[warp][8 * cg + 2 * i]) = make_uint2(m << 16, m & 0xFFFF0000u);
      } else {
        if (lane < 16) part[warp][8 * cg + i] = max(cmax[i], other);
      }
    }
  }
  if constexpr (TILE) {
    const uint32_t m = __reduce_max_sync(FULL_MASK, all);
    if (lane == 0) part[warp][0] = m;
  }
  if (__syncthreads_or(all >= INF_BITS)) return false;
  const int64_t row0 = matrix * p.rows + int64_t(rb) * 128;  // of the stacked results
  if (COL && tid < 128) {
    uint32_t m = 0u;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = max(m, part[w][tid]);
    byte_of[tid] = uint8_t(scale_byte(m));
    p.col.scales[(matrix * p.row_tiles + rb) * p.col.scale_ld + int64_t(cb) * 128 + tid] = byte_of[tid];
  }
  if constexpr (ROW) {
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int o = 8; o; o >>= 1) {
        const uint32_t other = __shfl_xor_sync(FULL_MASK, rmax[h], o);
        rmax[h] = BF16 ? max2(rmax[h], other) : max(rmax[h], other);
      }
  }
  uint32_t row_inv[NR];  // bf16: of two rows; fp32: see below
  if constexpr (ROW && BF16) {
    // scale_byte and scale_inverse on the upper halves of two maxima at once: 15 bits each, and
    // (262 - exponent) << 7 is the upper half of 2^-(byte - 127)
#pragma unroll
    for (int h = 0; h < NR; ++h)
      row_inv[h] = 0x83008300u - __vmaxu2((rmax[h] + 0x001F001Fu) & 0xFF80FF80u, 0x04000400u);
  }
  float2 inv[4];  // of the columns, or of the tile
  if constexpr (COL) {
    __syncthreads();
    const uint2 b = *reinterpret_cast<const uint2*>(&byte_of[8 * cg]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = (i < 2 ? b.x : b.y) >> (16 * (i & 1));
      inv[i] = make_float2(scale_inverse(h & 255u), scale_inverse((h >> 8) & 255u));
    }
  }
  if constexpr (TILE) {
    uint32_t m = 0u;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = max(m, part[w][0]);
    const int byte = scale_byte(m);
    inv[0] = inv[1] = inv[2] = inv[3] = make_float2(scale_inverse(byte), scale_inverse(byte));
    if (tid == 0) p.tile.scales[(matrix * p.row_tiles + rb) * p.tile.scale_ld + cb] = uint8_t(byte);
  }
  const Out& o = TILE ? p.tile : p.col;
  uint8_t* dr = p.row.codes + (row0 + rr) * p.row.ld + int64_t(cb) * 128 + 8 * cg;
  uint8_t* d = o.codes + (row0 + rr) * o.ld + int64_t(cb) * 128 + 8 * cg;
  uint8_t* row_byte = byte_of + 128;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(x[it].value(2 * i), x[it].value(2 * i + 1));
    if constexpr (ROW) {
      float si;
      if constexpr (BF16) si = __uint_as_float((it & 1) ? row_inv[it / 2] & 0xFFFF0000u : row_inv[it / 2] << 16);
      else si = scale_inverse(scale_byte(rmax[it]));
      const float2 s = make_float2(si, si);
      *reinterpret_cast<uint2*>(dr + int64_t(STEP * it) * p.row.ld) =
          make_uint2(codes4(mul2(v[0], s), mul2(v[1], s)), codes4(mul2(v[2], s), mul2(v[3], s)));
      if (cg == 0) row_byte[STEP * it + rr] = uint8_t(254u - (__float_as_uint(si) >> 23));
    }
    if constexpr (COL || TILE)
      *reinterpret_cast<uint2*>(d + int64_t(STEP * it) * o.ld) =
          make_uint2(codes4(mul2(v[0], inv[0]), mul2(v[1], inv[1])), codes4(mul2(v[2], inv[2]), mul2(v[3], inv[3])));
  }
  if constexpr (ROW) {
    __syncthreads();
    if (tid < 128) p.row.scales[(row0 + tid) * p.row.scale_ld + cb] = row_byte[tid];
  }
  return true;
}

template <bool BF16, bool ROW, bool COL, bool TILE>
__global__ void __launch_bounds__(THREADS, BF16 ? 4 : 2) quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t part[WARPS][128];
  __shared__ __align__(8) uint8_t byte_of[256];  // scale bytes of the columns, of the rows
  __shared__ int64_t src[128];  // where the tile's source rows begin (bytes), -1: zeros
  wait_for_previous();
  const unsigned tiles = unsigned(p.row_tiles) * unsigned(p.col_tiles);
  const unsigned z = p.by_tiles(blockIdx.x), in = blockIdx.x - z * tiles;
  const int rb = int(p.by_cols(in)), cb = int(in - unsigned(rb) * unsigned(p.col_tiles));
  constexpr int ES = BF16 ? 2 : 4;
  const uint8_t* base = static_cast<const uint8_t*>(p.stride ? p.base : p.ptr[z]);
  if (p.stride) base += int64_t(z) * p.stride * ES;
  const int64_t ld = p.stride ? p.ld : p.lds[z];
  const bool vec = reinterpret_cast<uintptr_t>(base) % 16 == 0 && (ld * ES) % 16 == 0;
  const bool full = vec && int64_t(rb + 1) * 128 <= p.rows && int64_t(cb + 1) * 128 <= p.cols;
  bool gaps = false;
  if (p.index) {
    const int64_t r = int64_t(rb) * 128 + threadIdx.x;
    if (threadIdx.x < 128) {
      const int32_t i = r < p.rows ? p.index[r] : -1;
      const int64_t row = p.by_copies(uint32_t(i));
      gaps = i < 0 || row >= p.src_rows;
      src[threadIdx.x] = gaps ? -1 : row * ld * ES;
    }
    gaps = __syncthreads_or(gaps) != 0;
  }
  const int64_t matrix = p.first + z;
  const int64_t* rows = p.index ? src : nullptr;
  if (full && quantize_full<BF16, ROW, COL, TILE>(p, matrix, rb, cb, base, ld, part, byte_of, rows, gaps)) return;
  __syncthreads();  // the shared memory is used again
  quantize_tile<BF16, ROW, COL, TILE>(p, matrix, rb, cb, base, ld, vec, part, byte_of, rows);
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
  p.by_copies = divisor(copies > 0 ? copies : 1);
  const int64_t rt = ceil_div(p.rows, 128), ct = ceil_div(p.cols, 128);
  p.row = out_of(row);
  p.col = out_of(col);
  p.tile = out_of(tile);
  const int64_t most = 0x7FFFFFFF;
  if (rt * ct > most) return MAO_ERR_UNSUPPORTED;
  p.row_tiles = int32_t(rt);
  p.col_tiles = int32_t(ct);
  p.by_tiles = divisor(uint32_t(rt * ct));
  p.by_cols = divisor(uint32_t(ct));
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
    const mao_status st = launch_dependent(k, unsigned(int64_t(n) * rt * ct), THREADS, 0, stream, p);
    if (st != MAO_OK) return st;
  }
  return MAO_OK;
}

}  // namespace mao
