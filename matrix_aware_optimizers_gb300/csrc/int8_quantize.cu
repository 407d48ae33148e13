// Rows to 8-bit integers with a scale each, or gated rows act(a) * b of [a | b].
//
// One pass: a row's values stay in the registers of the threads that share it (those past
// 8 CACHED per thread are read again), between the largest magnitude and the codes. Instructions
// bound it: at 22 per value 8192 x 4096 bf16 took 37 us, now 22 to 27 (on different cards; 100 MB: up to
// 4.6 TB/s, 68% of the issue slots). 3001 gated rows of 2053 fp32, gelu_tanh: 20 to 25 us (103
// instructions per value, most of them tanhf's).
//
// code = 127 x / a rounded to nearest even, as if computed exactly: x (127 / a) with a rounded
// quotient is off by less than 2^-15, so only products that near to a border between two codes
// need the exact comparison of 127 x with (m + 1/2) a, by products in two words each. The rounding
// is that of the sum with 1.5 * 2^23, which leaves the code in its low bits.
#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"

namespace mao {
namespace {

constexpr int kMany = 64;  // matrices of a list per launch

struct QuantParams {
  const void* x[kMany];  // stride < 0: matrix b is x[b], with rows of ld[b]
  int64_t ld[kMany];
  int64_t stride;        // elements from one matrix to the next
  int64_t rows, total;   // of one matrix, of all
  int64_t out_ld, first;    // first: row of out where x[0] starts
  int8_t* codes;
  float* scales;
  int32_t cols, act;
};

// act(g) * u with each operation rounded as it stands (no contraction).
__device__ __forceinline__ float gated(float g, float u, int act) {
  float a;
  if (act == MAO_SILU) {
    a = __fdiv_rn(g, __fadd_rn(1.0f, expf(-g)));
  } else if (act == MAO_GELU) {
    a = __fmul_rn(__fmul_rn(0.5f, g), __fadd_rn(1.0f, erff(__fmul_rn(g, 0.7071067811865476f))));
  } else {
    const float cube = __fmul_rn(__fmul_rn(__fmul_rn(kTanhA, g), g), g);
    a = __fmul_rn(__fmul_rn(0.5f, g), __fadd_rn(1.0f, tanhf(__fmul_rn(kTanhC, __fadd_rn(g, cube)))));
  }
  return __fmul_rn(a, u);
}

// The thread's values number 8 k .. 8 k + 7 of a row: eight columns in a row (VEC), or every TEAM-th
// column, where rows do not start at multiples of 16 bytes. Zeros past the last column.
template <bool VEC, int TEAM>
__device__ __forceinline__ int column(int t, int k, int q) {
  return VEC ? 8 * (t + k * TEAM) + q : (8 * k + q) * TEAM + t;
}

// Magnitudes order as their bits do, NaN above infinity.
__device__ __forceinline__ uint32_t top_of(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7FFFFFFFu);
  return top;
}

__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// Eight values as they lie in memory.
template <typename T, bool VEC, int TEAM>
struct Raw {
  static constexpr int WORDS = sizeof(T) / 2;  // 16-byte words of eight values
  uint4 w[VEC ? WORDS : 1];
  T e[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const T* x, int cols, int t, int k) {
    if (VEC) {
      const int c = column<VEC, TEAM>(t, k, 0);
      if (c + 8 <= cols) {
#pragma unroll
        for (int q = 0; q < WORDS; ++q) w[q] = reinterpret_cast<const uint4*>(x + c)[q];
      } else {  // the last columns of a row
        uint32_t* to = &w[0].x;
#pragma unroll
        for (int q = 0; q < 4 * WORDS; ++q) to[q] = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (c + q < cols) to[q * WORDS / 2] |= bits(x[c + q]) << (WORDS == 1 ? 16 * (q & 1) : 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int c = column<VEC, TEAM>(t, k, q);
        e[q] = c < cols ? x[c] : T(0.0f);
      }
    }
  }
  // The largest magnitude's bits (as those of fp32).
  __device__ __forceinline__ uint32_t top() const {
    if (VEC && WORDS == 1) {
      const uint32_t m = 0x7FFF7FFFu;
      const uint32_t t = __vmaxu2(__vmaxu2(w[0].x & m, w[0].y & m), __vmaxu2(w[0].z & m, w[0].w & m));
      return max(t << 16, t & 0xFFFF0000u);
    }
    float v[8];
    get(v);
    return top_of(v);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if (!VEC) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = float(e[q]);
    } else if (WORDS == 2) {
#pragma unroll
      for (int q = 0; q < WORDS; ++q) {
        v[4 * q] = __uint_as_float(w[q].x), v[4 * q + 1] = __uint_as_float(w[q].y);
        v[4 * q + 2] = __uint_as_float(w[q].z), v[4 * q + 3] = __uint_as_float(w[q].w);
      }
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(u[q] << 16);
        v[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
      }
    }
  }
};

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
constexpr float kBorder = 0.5f - 1.0f / 32768.0f;

// The code of x next to a border, for a row whose largest magnitude is a (both times a power of two
// that keeps the products in range), q = x * (127 / a).
__device__ __noinline__ int border_code(float x, float a, float q) {
  const float below = floorf(q), h = below + 0.5f;
  const float s = __fmul_rn(127.0f, x), t = __fmul_rn(h, a);
  const float diff = (s - t) + (__fmaf_rn(127.0f, x, -s) - __fmaf_rn(h, a, -t));
  const int lower = int(below);
  return diff > 0.0f ? lower + 1 : diff < 0.0f ? lower : lower + (lower & 1);
}

// The codes of eight values, a byte each in the low bits; r = 127 / a.
__device__ __forceinline__ void codes_of(const float (&x)[8], float a, float r, uint32_t (&code)[8]) {
  float far = 0.0f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float m = __fmaf_rn(x[q], r, kRound);
    code[q] = __float_as_uint(m);
    far = fmaxf(far, fabsf(__fmaf_rn(x[q], r, kRound - m)));  // from the product to the code
  }
  if (far >= kBorder) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float m = __fmaf_rn(x[q], r, kRound);
      if (fabsf(__fmaf_rn(x[q], r, kRound - m)) >= kBorder) code[q] = uint32_t(border_code(x[q], a, x[q] * r));
    }
  }
}

// TEAM threads share a row and keep CACHED times eight values each; blocks of BLOCK threads.
template <bool GATED, bool VEC, typename T, int TEAM, int BLOCK, int CACHED>
__global__ void __launch_bounds__(BLOCK) quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t tops[2][BLOCK / 32];
  wait_for_previous();
  const int t = threadIdx.x % TEAM;
  const int64_t turn = int64_t(blockIdx.x) * (BLOCK / TEAM) + threadIdx.x / TEAM;
  const int64_t turns = int64_t(gridDim.x) * (BLOCK / TEAM);
  const int steps = (p.cols + 8 * TEAM - 1) / (8 * TEAM);
  using Values = Raw<T, VEC, TEAM>;
  // values number 8 k ..: the row's, or gated ones
  auto gated_values = [&](const T* x, int k, float(&v)[8]) {
    Values g, u;
    float w[8];
    g.load(x, p.cols, t, k);
    u.load(x + p.cols, p.cols, t, k);
    g.get(v);
    u.get(w);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = gated(v[q], w[q], p.act);
  };
  int flip = 0;
  for (int64_t row = turn; row < p.total; row += turns) {
    int64_t b = 0, i = row;
    if (p.rows != p.total) {
      b = row / p.rows;
      i = row - b * p.rows;
    }
    const T* x = static_cast<const T*>(p.stride < 0 ? p.x[b] : p.x[0]) +
                 (p.stride < 0 ? i * p.ld[b] : i * p.ld[0] + b * p.stride);
    Values raw[GATED ? 1 : CACHED];
    float v[GATED ? CACHED : 1][8];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < CACHED; ++k) {
      if (k >= steps) break;
      if (GATED) gated_values(x, k, v[GATED ? k : 0]);
      else raw[GATED ? 0 : k].load(x, p.cols, t, k);
    }
#pragma unroll
    for (int k = 0; k < CACHED; ++k) {
      if (k >= steps) break;
      top = max(top, GATED ? top_of(v[GATED ? k : 0]) : raw[GATED ? 0 : k].top());
    }
    for (int k = CACHED; k < steps; ++k) {
      if (GATED) {
        float w[8];
        gated_values(x, k, w);
        top = max(top, top_of(w));
      } else {
        Values w;
        w.load(x, p.cols, t, k);
        top = max(top, w.top());
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (TEAM > 32) {
      if ((threadIdx.x & 31) == 0) tops[flip][threadIdx.x / 32] = top;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x) / TEAM), "n"(TEAM) : "memory");  // the team's own
      const int first = threadIdx.x / TEAM * (TEAM / 32);
      top = __reduce_max_sync(0xFFFFFFFFu, (threadIdx.x & 31) < TEAM / 32 ? tops[flip][first + (threadIdx.x & 31)] : 0u);
      flip ^= 1;
    }
    const bool bad = top >= 0x7F800000u;
    const float a = __uint_as_float(top);
    const int64_t out = p.first + row;
    if (t == 0) p.scales[out] = bad ? __uint_as_float(0x7FFFFFFFu) : a / 127.0f;
    const float lift = a < 0x1p-60f ? 0x1p80f : a > 0x1p100f ? 0x1p-40f : 1.0f;
    const float al = a * lift, r = top == 0 || bad ? 0.0f : 127.0f / al;
    int8_t* codes = p.codes + out * p.out_ld;
    auto store = [&](int k, float (&w)[8]) {
      uint32_t code[8];
      if (lift != 1.0f) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] *= lift;
      }
      if (r != 0.0f) {
        codes_of(w, al, r, code);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) code[q] = 0;
      }
      const int c0 = column<VEC, TEAM>(t, k, 0);
      if (VEC && c0 + 8 <= p.cols) {
        const uint32_t a0 = __byte_perm(code[0], code[1], 0x0040), a1 = __byte_perm(code[2], code[3], 0x0040);
        const uint32_t b0 = __byte_perm(code[4], code[5], 0x0040), b1 = __byte_perm(code[6], code[7], 0x0040);
        *reinterpret_cast<uint2*>(codes + c0) = make_uint2(__byte_perm(a0, a1, 0x5410), __byte_perm(b0, b1, 0x5410));
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = column<VEC, TEAM>(t, k, q);
          if (c < p.cols) codes[c] = int8_t(code[q] & 0xFFu);
        }
      }
    };
#pragma unroll
    for (int k = 0; k < CACHED; ++k) {
      if (k >= steps) break;
      if (GATED) {
        store(k, v[GATED ? k : 0]);
      } else {
        float w[8];
        raw[GATED ? 0 : k].get(w);
        store(k, w);
      }
    }
    for (int k = CACHED; k < steps; ++k) {
      float w[8];
      if (GATED) {
        gated_values(x, k, w);
      } else {
        Values y;
        y.load(x, p.cols, t, k);
        y.get(w);
      }
      store(k, w);
    }
  }
}

// Teams by row length. Rows as they are in bf16 take half the registers: twice the values each.
constexpr int TEAMS = 6;
#define QUANT_KERNELS(GATED, VEC, T, CACHED)                                                                   \
  {                                                                                                            \
    quantize_kernel<GATED, VEC, T, 32, 128, CACHED>, quantize_kernel<GATED, VEC, T, 64, 128, CACHED>,          \
        quantize_kernel<GATED, VEC, T, 128, 128, CACHED>, quantize_kernel<GATED, VEC, T, 256, 256, CACHED>,    \
        quantize_kernel<GATED, VEC, T, 512, 512, CACHED>, quantize_kernel<GATED, VEC, T, 1024, 1024, CACHED>   \
  }

}  // namespace

mao_status int8_quantize_launch(const mao_mat* X, int32_t batch, int64_t batch_stride, int32_t act,
                                bool gated_rows, const mao_int8& out, cudaStream_t stream) {
  if (out.rows == 0) return MAO_OK;
  const bool list = batch_stride == 0 && batch > 1;
  for (int32_t b0 = 0; b0 < batch; b0 += list ? kMany : batch) {
    QuantParams p = {};
    const int32_t n = !list ? batch : batch - b0 < kMany ? batch - b0 : kMany;
    const int es = elem_size(X[0].dtype);
    p.stride = list ? -1 : batch_stride;
    p.rows = out.rows;
    p.total = out.rows * n;
    p.out_ld = out.ld;
    p.first = int64_t(b0) * out.rows;
    p.codes = out.codes;
    p.scales = out.scales;
    p.cols = int32_t(out.cols);
    p.act = act;
    bool vec = (!gated_rows || out.cols * es % 16 == 0) && (list || p.stride * es % 16 == 0);
    for (int32_t b = 0; b < (list ? n : 1); ++b) {
      p.x[b] = X[b0 + b].data;
      p.ld[b] = X[b0 + b].ld;
      vec = vec && reinterpret_cast<uintptr_t>(p.x[b]) % 16 == 0 && p.ld[b] * es % 16 == 0;
    }
    // The smallest team of threads that keeps a row in its registers; with few rows a larger one,
    // whose threads then have less to do each.
    const bool bf16 = X[0].dtype == MAO_BF16;
    const int each = p.total <= num_sms() ? 8 : bf16 && vec && !gated_rows ? 32 : 16;  // values per thread
    int kind = 0;
    while (kind < TEAMS - 1 && out.cols > each * (32 << kind)) ++kind;
    using Kernel = void (*)(const QuantParams);
    static const Kernel kernels[2][2][2][TEAMS] = {
        {{QUANT_KERNELS(false, false, float, 2), QUANT_KERNELS(false, false, __nv_bfloat16, 2)},
         {QUANT_KERNELS(false, true, float, 2), QUANT_KERNELS(false, true, __nv_bfloat16, 4)}},
        {{QUANT_KERNELS(true, false, float, 2), QUANT_KERNELS(true, false, __nv_bfloat16, 2)},
         {QUANT_KERNELS(true, true, float, 2), QUANT_KERNELS(true, true, __nv_bfloat16, 2)}}};
    const int team = 32 << kind, threads = team < 128 ? 128 : team;
    const int64_t blocks = ceil_div(p.total, threads / team), most = int64_t(1) << 30;
    const mao_status st = launch_dependent(kernels[gated_rows][vec][bf16][kind],
                                           unsigned(blocks < most ? blocks : most), threads, 0, stream, p);
    if (st != MAO_OK) return st;
  }
  return MAO_OK;
}

}  // namespace mao
