// Rows to 8-bit integers with a scale each, or gated rows act(a) * b of [a | b].
//
// One pass: a row's values stay in the registers of the threads that share it (those past
// 8 CACHED per thread are read again), between the largest magnitude and the codes. Memory bounds the
// rows as they are, the gate's arithmetic (a division, e^x) the gated ones.
//
// code = 127 x / a rounded to nearest even, as if computed exactly: x * (127 / a) in fp32 is
// off by less than 2^-15, so only quotients that near to a border between two codes need the
// exact comparison of 127 x with (m + 1/2) a, by products in two words each.
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
  int32_t cols, dtype, act, vec;
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

// Eight values from column c on, zeros past the last.
__device__ __forceinline__ void load_values(const QuantParams& p, const void* x, int64_t at, int c,
                                            float (&v)[8]) {
  if (p.vec && c + 8 <= p.cols) {
    load8(x, at + c, p.dtype, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < p.cols ? load_elem(x, at + c + q, p.dtype) : 0.0f;
  }
}

template <bool GATED>
__device__ __forceinline__ void load_row(const QuantParams& p, const void* x, int64_t at, int c, float (&v)[8]) {
  load_values(p, x, at, c, v);
  if (GATED) {
    float u[8];
    load_values(p, x, at + p.cols, c, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = gated(v[q], u[q], p.act);
  }
}

// The code of x for a row whose largest magnitude is a (both times a power of two that keeps the
// products in range), r = 127 / a.
__device__ __forceinline__ int code_of(float x, float a, float r) {
  const float q = x * r;
  const float m = rintf(q);
  if (fabsf(q - m) < 0.5f - 1.0f / 32768.0f) return int(m);
  const float below = floorf(q), h = below + 0.5f;
  const float s = __fmul_rn(127.0f, x), t = __fmul_rn(h, a);
  const float diff = (s - t) + (__fmaf_rn(127.0f, x, -s) - __fmaf_rn(h, a, -t));
  const int lower = int(below);
  return diff > 0.0f ? lower + 1 : diff < 0.0f ? lower : lower + (lower & 1);
}

// TEAM threads share a row and keep CACHED vectors of eight values each; blocks of BLOCK threads.
template <bool GATED, int TEAM, int BLOCK, int CACHED>
__global__ void __launch_bounds__(BLOCK) quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ uint32_t tops[2][BLOCK / 32];
  wait_for_previous();
  const int t = threadIdx.x % TEAM;
  const int64_t turn = int64_t(blockIdx.x) * (BLOCK / TEAM) + threadIdx.x / TEAM;
  const int64_t turns = int64_t(gridDim.x) * (BLOCK / TEAM);
  int flip = 0;
  for (int64_t row = turn; row < p.total; row += turns) {
    const int64_t b = row / p.rows, i = row - b * p.rows;
    const void* x = p.stride < 0 ? p.x[b] : p.x[0];
    const int64_t at = p.stride < 0 ? i * p.ld[b] : i * p.ld[0] + b * p.stride;
    float v[CACHED][8];
    uint32_t top = 0;  // magnitudes order as their bits do, NaN above infinity
#pragma unroll
    for (int k = 0; k < CACHED; ++k) {
      const int c = 8 * (t + k * TEAM);
      if (c >= p.cols) break;
      load_row<GATED>(p, x, at, c, v[k]);
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[k][q]) & 0x7FFFFFFFu);
    }
    for (int c = 8 * (t + CACHED * TEAM); c < p.cols; c += 8 * TEAM) {
      float w[8];
      load_row<GATED>(p, x, at, c, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(w[q]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (TEAM > 32) {
      if ((threadIdx.x & 31) == 0) tops[flip][threadIdx.x / 32] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TEAM / 32; ++w) top = max(top, tops[flip][w]);
      flip ^= 1;
    }
    const bool bad = top >= 0x7F800000u;
    const float a = __uint_as_float(top);
    const int64_t out = p.first + row;
    if (t == 0) p.scales[out] = bad ? __uint_as_float(0x7FFFFFFFu) : a / 127.0f;
    const float lift = a < 0x1p-60f ? 0x1p80f : a > 0x1p100f ? 0x1p-40f : 1.0f;
    const float al = a * lift, r = top == 0 || bad ? 0.0f : 127.0f / al;
    int8_t* codes = p.codes + out * p.out_ld;
    auto store = [&](int c, const float(&w)[8]) {
      uint32_t lo = 0, hi = 0;
      if (r != 0.0f) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          lo |= uint32_t(code_of(w[q] * lift, al, r) & 0xFF) << (8 * q);
          hi |= uint32_t(code_of(w[q + 4] * lift, al, r) & 0xFF) << (8 * q);
        }
      }
      if (c + 8 <= p.cols) {
        *reinterpret_cast<uint2*>(codes + c) = make_uint2(lo, hi);
      } else {
        for (int q = 0; c + q < p.cols; ++q) codes[c + q] = int8_t((q < 4 ? lo >> (8 * q) : hi >> (8 * q - 32)) & 0xFF);
      }
    };
#pragma unroll
    for (int k = 0; k < CACHED; ++k) {
      const int c = 8 * (t + k * TEAM);
      if (c >= p.cols) break;
      store(c, v[k]);
    }
    for (int c = 8 * (t + CACHED * TEAM); c < p.cols; c += 8 * TEAM) {
      float w[8];
      load_row<GATED>(p, x, at, c, w);
      store(c, w);
    }
  }
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
    p.dtype = X[0].dtype;
    p.act = act;
    bool vec = (!gated_rows || out.cols * es % 16 == 0) && (list || p.stride * es % 16 == 0);
    for (int32_t b = 0; b < (list ? n : 1); ++b) {
      p.x[b] = X[b0 + b].data;
      p.ld[b] = X[b0 + b].ld;
      vec = vec && reinterpret_cast<uintptr_t>(p.x[b]) % 16 == 0 && p.ld[b] * es % 16 == 0;
    }
    p.vec = vec;
    // A warp for short rows, a block for longer ones; with few rows a larger block, whose threads
    // then have little to do each.
    using Kernel = void (*)(const QuantParams);
    static const Kernel kernels[2][3] = {
        {quantize_kernel<false, 32, 256, 4>, quantize_kernel<false, 256, 256, 4>, quantize_kernel<false, 1024, 1024, 2>},
        {quantize_kernel<true, 32, 256, 4>, quantize_kernel<true, 256, 256, 4>, quantize_kernel<true, 1024, 1024, 2>}};
    const int kind = out.cols <= 1024 ? 0 : out.cols > 4096 && p.total <= 2 * num_sms() ? 2 : 1;
    const int threads = kind == 2 ? 1024 : 256;
    const int64_t blocks = ceil_div(p.total, kind == 0 ? 8 : 1), most = int64_t(num_sms()) * (kind == 2 ? 2 : 64);
    const mao_status st = launch_dependent(kernels[gated_rows][kind], unsigned(blocks < most ? blocks : most), threads,
                                           0, stream, p);
    if (st != MAO_OK) return st;
  }
  return MAO_OK;
}

}  // namespace mao
