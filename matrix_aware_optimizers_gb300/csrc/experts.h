// Internal launchers of the expert-layer calls (arguments validated by experts_abi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mao.h"

namespace mao {

struct RouteParams {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  int64_t ld;
  int64_t tokens;
  int32_t dtype, experts, top_k, score, groups, keep, group_score, renorm;
  float scale;
};
mao_status route_launch(const RouteParams& p, cudaStream_t stream);

struct RouteBackParams {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t ld, dld;
  int64_t tokens;
  int32_t dtype, ddtype, experts, top_k, score, renorm;
  float scale;
};
mao_status route_backward_launch(const RouteBackParams& p, cudaStream_t stream);

constexpr int64_t kPlanAlone = 4096;  // copies that one block places, without a workspace
size_t plan_workspace_size(int64_t n, int32_t experts);
mao_status plan_launch(const int32_t* ids, int64_t n, int32_t experts, int32_t* counts,
                       int32_t* offsets, int32_t* row_of, int32_t* slot_of, int64_t n_slots,
                       void* workspace, cudaStream_t stream);

mao_status combine_launch(const mao_mat& Z, const int32_t* row_of, const float* weights,
                          int64_t tokens, int32_t top_k, const mao_mat& Y, cudaStream_t stream);
mao_status combine_backward_launch(const mao_mat& dY, const mao_mat& Z, const int32_t* row_of,
                                   const int32_t* slot_of, const float* weights, int32_t top_k,
                                   const mao_mat& dZ, float* dweights, cudaStream_t stream);

mao_status quantize_launch(const mao_mat* X, int32_t batch, int64_t batch_stride,
                           const int32_t* index, int64_t n_index, int32_t copies,
                           const mao_fp8* row, const mao_fp8* col, const mao_fp8* tile,
                           cudaStream_t stream);

mao_status product_launch(const mao_fp8& A, const mao_fp8& B, const mao_mat& D, int32_t form,
                          const int32_t* offsets, int32_t groups, int32_t accumulate,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream);
size_t product_workspace_size(const mao_fp8& A, const mao_fp8& B, int32_t form);
// Reads and clears the device error word of the product kernel (after a stream sync).
mao_status product_read_and_clear_error(cudaStream_t stream);

}  // namespace mao
