// C ABI entry points of the feed-forward blocks: argument validation (synchronous, nothing enqueued
// on error) and dispatch to the launchers. No exception crosses this boundary.
#include "common.cuh"
#include "ffn.h"
#include "internal.h"

using namespace mao;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;  // tile ends fit 32 bits
constexpr int64_t kMaxCols = int64_t(1) << 20;

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// A matrix that may have no rows (its data is then not looked at).
mao_status check_rows(const mao_mat* m, bool bf16_only) {
  if (!m || !valid_dtype(m->dtype) || (bf16_only && m->dtype != MAO_BF16)) return MAO_ERR_INVALID_ARG;
  if (m->reserved != 0 || m->rows < 0 || m->cols < 1 || m->ld < m->cols) return MAO_ERR_INVALID_ARG;
  if (m->rows > kMaxRows || m->cols > 2 * kMaxCols || m->ld > (int64_t(1) << 39) / (m->rows + 1))
    return MAO_ERR_UNSUPPORTED;
  if (m->rows == 0) return MAO_OK;
  if (!m->data) return MAO_ERR_INVALID_ARG;
  return aligned(m->data, elem_size(m->dtype)) ? MAO_OK : MAO_ERR_MISALIGNED;
}

mao_status check_runs(const int32_t* offsets, const int32_t* counts, int32_t groups) {
  if (groups < 1 || (!offsets && (groups != 1 || counts))) return MAO_ERR_INVALID_ARG;
  if (groups > 1024) return MAO_ERR_UNSUPPORTED;
  return aligned(offsets, 4) && aligned(counts, 4) ? MAO_OK : MAO_ERR_MISALIGNED;
}

// X, up and down of a block.
mao_status check_block(const mao_mat* X, const mao_mat* up, const mao_mat* down, int32_t groups) {
  mao_status st = check_rows(X, true);
  if (st == MAO_OK) st = check_rows(up, true);
  if (st == MAO_OK) st = check_rows(down, true);
  if (st != MAO_OK) return st;
  const int64_t N = down->cols;
  if (up->cols != X->cols || up->rows != 2 * N * groups || down->rows < 1 || down->rows % groups != 0)
    return MAO_ERR_INVALID_ARG;
  if (X->cols > kMaxCols || N > kMaxCols || down->rows / groups > kMaxCols) return MAO_ERR_UNSUPPORTED;
  return MAO_OK;
}

mao_status check_act(int32_t act) { return act < MAO_SILU || act > MAO_GELU_TANH ? MAO_ERR_INVALID_ARG : MAO_OK; }

mao_status check_ws(const void* workspace, size_t have, size_t need) {
  if (need == 0) return MAO_OK;
  if (!workspace) return MAO_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MAO_ERR_MISALIGNED;
  return have < need ? MAO_ERR_WORKSPACE : MAO_OK;
}

bool shaped(const mao_mat* m, int64_t rows, int64_t cols) { return m->rows == rows && m->cols == cols; }

mao_status check_int8(const mao_int8* m) {
  if (!m || m->reserved != 0 || m->count < 1 || m->rows < 0 || m->cols < 1 || m->ld < m->cols || m->ld % 16 != 0)
    return MAO_ERR_INVALID_ARG;
  if (m->rows > kMaxRows / m->count || m->cols > kMaxCols || m->ld > (int64_t(1) << 39) / (m->rows * m->count + 1))
    return MAO_ERR_UNSUPPORTED;
  if (m->rows == 0) return MAO_OK;
  if (!m->codes || !m->scales) return MAO_ERR_INVALID_ARG;
  return aligned(m->codes, 16) && aligned(m->scales, 4) ? MAO_OK : MAO_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

mao_status gated_ffn(const mao_mat* X, const mao_mat* up, const mao_mat* down, int32_t act,
                     const int32_t* offsets, const int32_t* counts, int32_t groups, const mao_mat* Z,
                     const mao_mat* Y, void* workspace, size_t workspace_bytes, void* stream) {
  mao_status st = check_runs(offsets, counts, groups);
  if (st == MAO_OK) st = check_act(act);
  if (st == MAO_OK) st = check_block(X, up, down, groups);
  if (st == MAO_OK && Z) st = check_rows(Z, false);
  if (st == MAO_OK) st = check_rows(Y, false);
  if (st != MAO_OK) return st;
  if (!shaped(Y, X->rows, down->rows / groups) || (Z && !shaped(Z, X->rows, 2 * down->cols)))
    return MAO_ERR_INVALID_ARG;
  if (device_cc() / 10 != 10) return MAO_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, gated_ffn_workspace_size(*X, *up, *down, groups, offsets != nullptr));
  if (st != MAO_OK) return st;
  return gated_ffn_launch(*X, *up, *down, act, Runs{offsets, counts, groups}, Z, *Y, workspace,
                          static_cast<cudaStream_t>(stream));
}

size_t gated_ffn_workspace_bytes(const mao_mat* X, const mao_mat* up, const mao_mat* down,
                                 int32_t groups, int32_t grouped) {
  if (groups < 1 || check_block(X, up, down, groups) != MAO_OK) return 0;
  return gated_ffn_workspace_size(*X, *up, *down, groups, grouped != 0);
}

mao_status gated_ffn_backward(const mao_mat* dY, const mao_mat* X, const mao_mat* up,
                              const mao_mat* down, const mao_mat* Z, int32_t act,
                              const int32_t* offsets, const int32_t* counts, int32_t groups,
                              const mao_mat* dX, const mao_mat* dup, const mao_mat* ddown,
                              void* workspace, size_t workspace_bytes, void* stream) {
  mao_status st = check_runs(offsets, counts, groups);
  if (st == MAO_OK) st = check_act(act);
  if (st == MAO_OK) st = check_block(X, up, down, groups);
  if (st == MAO_OK) st = check_rows(dY, true);
  if (st == MAO_OK) st = check_rows(Z, false);
  for (const mao_mat* D : {dX, dup, ddown})
    if (st == MAO_OK && D) st = check_rows(D, false);
  if (st != MAO_OK) return st;
  if (!shaped(dY, X->rows, down->rows / groups) || !shaped(Z, X->rows, 2 * down->cols) ||
      (dX && !shaped(dX, X->rows, X->cols)) || (dup && !shaped(dup, up->rows, up->cols)) ||
      (ddown && !shaped(ddown, down->rows, down->cols)))
    return MAO_ERR_INVALID_ARG;
  if (device_cc() / 10 != 10) return MAO_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes,
                gated_ffn_backward_workspace_size(*dY, *X, *up, *down, groups, offsets != nullptr));
  if (st != MAO_OK) return st;
  return gated_ffn_backward_launch(*dY, *X, *up, *down, *Z, act, Runs{offsets, counts, groups}, dX, dup, ddown,
                                   workspace, static_cast<cudaStream_t>(stream));
}

size_t gated_ffn_backward_workspace_bytes(const mao_mat* dY, const mao_mat* X, const mao_mat* up,
                                          const mao_mat* down, int32_t groups, int32_t grouped) {
  if (groups < 1 || check_block(X, up, down, groups) != MAO_OK || check_rows(dY, true) != MAO_OK) return 0;
  return gated_ffn_backward_workspace_size(*dY, *X, *up, *down, groups, grouped != 0);
}

mao_status int8_quantize(const mao_mat* X, int32_t batch, int64_t batch_stride, int32_t gated,
                         int32_t act, const mao_int8* out, void* stream) {
  if (!X || batch < 1 || batch_stride < 0) return MAO_ERR_INVALID_ARG;
  mao_status st = check_int8(out);
  if (st == MAO_OK && gated) st = check_act(act);
  if (st != MAO_OK) return st;
  for (int32_t b = 0; b < (batch_stride > 0 ? 1 : batch); ++b) {
    st = check_rows(&X[b], false);
    if (st != MAO_OK) return st;
    if (!shaped(&X[b], out->rows, gated ? 2 * out->cols : out->cols) || X[b].dtype != X[0].dtype)
      return MAO_ERR_INVALID_ARG;
  }
  if (out->count != batch) return MAO_ERR_INVALID_ARG;
  return int8_quantize_launch(X, batch, batch_stride, act, gated != 0, *out, static_cast<cudaStream_t>(stream));
}

mao_status int8_product(const mao_int8* A, const mao_int8* B, const mao_mat* D,
                        const int32_t* offsets, const int32_t* counts, int32_t groups,
                        void* workspace, size_t workspace_bytes, void* stream) {
  mao_status st = check_runs(offsets, counts, groups);
  if (st == MAO_OK) st = check_int8(A);
  if (st == MAO_OK) st = check_int8(B);
  if (st == MAO_OK) st = check_rows(D, false);
  if (st != MAO_OK) return st;
  if (A->count != 1 || B->count != groups || B->rows < 1 || B->cols != A->cols || !shaped(D, A->rows, B->rows))
    return MAO_ERR_INVALID_ARG;
  if (B->rows > kMaxCols) return MAO_ERR_UNSUPPORTED;
  if (device_cc() / 10 != 10) return MAO_ERR_UNSUPPORTED;
  st = check_ws(workspace, workspace_bytes, int8_product_workspace_size(*A, *B, offsets != nullptr));
  if (st != MAO_OK) return st;
  return int8_product_launch(*A, *B, *D, Runs{offsets, counts, groups}, workspace,
                             static_cast<cudaStream_t>(stream));
}

size_t int8_product_workspace_bytes(const mao_int8* A, const mao_int8* B, int32_t grouped) {
  if (!A || !B || A->rows < 0 || A->cols < 1 || B->rows < 1 || B->cols < 1) return 0;
  return int8_product_workspace_size(*A, *B, grouped != 0);
}

}  // extern "C"
