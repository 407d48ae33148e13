// Products of 8-bit matrices with power-of-two block scales, fp32 sums, over groups of rows.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "experts.h"
#include "internal.h"

namespace mao {
namespace {

struct ProductParams {
  const uint8_t* a;
  const uint8_t* as;
  const uint8_t* b;
  const uint8_t* bs;
  void* d;
  const int32_t* offsets;
  int64_t ald, asld, bld, bsld, dld, brows;  // brows: rows of one matrix of B
  int64_t rows;                              // t
  int64_t I, J, K;  // D rows (of a group), D columns, depth of the product
  int32_t ddt, groups, accumulate, form;
};

__device__ __forceinline__ float value(uint8_t code, uint8_t scale) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
  return __half2float(__half(h)) * exp2f(float(int(scale) - 127));
}

constexpr int T = 64;   // outputs per block, each way
constexpr int KB = 16;  // depth per step

// D[i][j] = sum_k P(i, k) Q(k, j): 64 x 64 outputs per block, 4 x 4 per thread.
__global__ void __launch_bounds__(256) product_kernel(const ProductParams p) {
  __shared__ float ps[KB][T + 4], qs[KB][T + 4];
  const bool tn = p.form == MAO_TN;
  int g = 0;
  int64_t i0 = int64_t(blockIdx.y) * T, lo = 0, hi = p.rows;
  bool outside = false;
  if (tn) {
    g = blockIdx.z;
    if (p.offsets) {
      lo = max(int64_t(0), min(int64_t(p.offsets[g]), p.rows));
      hi = max(lo, min(int64_t(p.offsets[g + 1]), p.rows));
    }
  } else if (p.offsets) {
    // blockIdx.y counts the groups' tiles of 64 rows, then those of the rest
    int64_t y = blockIdx.y;
    for (g = 0; g <= p.groups; ++g) {
      lo = max(int64_t(0), min(int64_t(p.offsets[g]), p.rows));
      hi = g < p.groups ? max(lo, min(int64_t(p.offsets[g + 1]), p.rows)) : p.rows;
      const int64_t tiles = (hi - lo + T - 1) / T;
      if (y < tiles) break;
      y -= tiles;
    }
    if (g > p.groups) return;
    outside = g == p.groups;
    i0 = lo + y * T;
  }
  const int64_t i_end = tn ? p.I : hi;
  const int64_t j0 = int64_t(blockIdx.x) * T;
  const int64_t k0 = tn ? lo : 0, k1 = outside ? k0 : tn ? hi : p.K;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k = k0; k < k1; k += KB) {
    for (int q = threadIdx.x; q < T * KB; q += 256) {
      const int kk = tn || p.form == MAO_NN ? q / T : q % KB;
      const int jj = tn || p.form == MAO_NN ? q % T : q / KB;
      float v = 0.0f;
      if (k + kk < k1 && j0 + jj < p.J) {
        const int64_t r = p.form == MAO_NT ? j0 + jj : k + kk, c = p.form == MAO_NT ? k + kk : j0 + jj;
        if (tn) {
          v = value(p.b[r * p.bld + c], p.bs[(r / 128) * p.bsld + c]);
        } else {
          const int64_t sr = (p.brows + 127) / 128;
          v = value(p.b[(g * p.brows + r) * p.bld + c], p.bs[(g * sr + r / 128) * p.bsld + c / 128]);
        }
      }
      qs[kk][jj] = v;
    }
    for (int q = threadIdx.x; q < T * KB; q += 256) {
      const int kk = tn ? q / T : q % KB, ii = tn ? q % T : q / KB;
      float v = 0.0f;
      if (k + kk < k1 && i0 + ii < i_end) {
        const int64_t i = i0 + ii, kx = k + kk;
        v = tn ? value(p.a[kx * p.ald + i], p.as[(kx / 128) * p.asld + i])
               : value(p.a[i * p.ald + kx], p.as[i * p.asld + kx / 128]);
      }
      ps[kk][ii] = v;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < KB; ++kk)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(ps[kk][4 * ty + a], qs[kk][4 * tx + b], acc[a][b]);
    __syncthreads();
  }
  for (int a = 0; a < 4; ++a)
    for (int b = 0; b < 4; ++b) {
      const int64_t i = i0 + 4 * ty + a, j = j0 + 4 * tx + b;
      if (i >= i_end || j >= p.J) continue;
      const int64_t at = (tn ? g * p.I + i : i) * p.dld + j;
      if (p.accumulate) {
        if (!outside) store_elem(p.d, at, p.ddt, load_elem(p.d, at, p.ddt) + acc[a][b]);
      } else {
        store_elem(p.d, at, p.ddt, acc[a][b]);
      }
    }
}

}  // namespace

mao_status product_launch(const mao_fp8& A, const mao_fp8& B, const mao_mat& D, int32_t form,
                          const int32_t* offsets, int32_t groups, int32_t accumulate,
                          cudaStream_t stream) {
  const bool tn = form == MAO_TN;
  if (A.rows == 0 && !tn) return MAO_OK;
  ProductParams p = {A.codes, A.scales, B.codes, B.scales, D.data, offsets, A.ld, A.scale_ld,
                     B.ld, B.scale_ld, D.ld, B.rows, A.rows, tn ? A.cols : A.rows, D.cols,
                     form == MAO_NT ? A.cols : form == MAO_NN ? B.rows : A.rows,
                     D.dtype, groups, accumulate, form};
  const int64_t ti = tn ? ceil_div(A.cols, T) : ceil_div(A.rows, T) + (offsets ? groups + 1 : 0);
  const dim3 grid(unsigned(ceil_div(D.cols, T)), unsigned(ti), tn ? unsigned(groups) : 1u);
  if (ti > 65535) return MAO_ERR_UNSUPPORTED;
  product_kernel<<<grid, 256, 0, stream>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace mao
