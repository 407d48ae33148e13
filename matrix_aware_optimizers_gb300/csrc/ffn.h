// Internal launchers of the feed-forward calls (arguments validated by ffn_abi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mao.h"

namespace mao {

// Rows of a call: one run (offsets null), or groups of them, the first counts[g] rows of each in use.
struct Runs {
  const int32_t* offsets;
  const int32_t* counts;
  int32_t groups;
};

size_t gated_ffn_workspace_size(const mao_mat& X, const mao_mat& up, const mao_mat& down, int32_t groups,
                                bool grouped);
mao_status gated_ffn_launch(const mao_mat& X, const mao_mat& up, const mao_mat& down, int32_t act,
                            const Runs& runs, const mao_mat* Z, const mao_mat& Y, void* workspace,
                            cudaStream_t stream);
size_t gated_ffn_backward_workspace_size(const mao_mat& dY, const mao_mat& X, const mao_mat& up,
                                         const mao_mat& down, int32_t groups, bool grouped);
mao_status gated_ffn_backward_launch(const mao_mat& dY, const mao_mat& X, const mao_mat& up,
                                     const mao_mat& down, const mao_mat& Z, int32_t act, const Runs& runs,
                                     const mao_mat* dX, const mao_mat* dup, const mao_mat* ddown,
                                     void* workspace, cudaStream_t stream);

mao_status int8_quantize_launch(const mao_mat* X, int32_t batch, int64_t batch_stride, int32_t act,
                                bool gated, const mao_int8& out, cudaStream_t stream);
size_t int8_product_workspace_size(const mao_int8& A, const mao_int8& B, bool grouped);
mao_status int8_product_launch(const mao_int8& A, const mao_int8& B, const mao_mat& D, const Runs& runs,
                               void* workspace, cudaStream_t stream);
// Read and clear the device error words of the products (after a stream sync).
mao_status ffn_read_and_clear_error(cudaStream_t stream);
mao_status int8_read_and_clear_error(cudaStream_t stream);

}  // namespace mao
