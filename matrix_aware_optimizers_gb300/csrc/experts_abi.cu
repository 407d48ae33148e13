// C ABI entry points of the expert-layer operators: argument validation (synchronous, nothing
// enqueued on error) and dispatch to the launchers. No exception crosses this boundary.
#include <cmath>

#include "common.cuh"
#include "experts.h"
#include "internal.h"

using namespace mao;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxCodes = kMaxRows - 1024;  // rows or columns of codes: tile ends fit 32 bits

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// A matrix that may have no rows (its data is then not looked at).
mao_status check_rows(const mao_mat* m) {
  if (!m) return MAO_ERR_INVALID_ARG;
  if (m->rows != 0) return check_mat(*m);
  if (!valid_dtype(m->dtype) || m->reserved != 0 || m->cols < 1 || m->ld < m->cols)
    return MAO_ERR_INVALID_ARG;
  return m->cols > kMaxRows ? MAO_ERR_UNSUPPORTED : MAO_OK;
}

mao_status check_fp8(const mao_fp8* m, int32_t blocks) {
  if (!m || m->blocks != blocks || m->count < 1 || m->rows < 0 || m->cols < 1 ||
      m->ld < m->cols || m->ld % 16 != 0)
    return MAO_ERR_INVALID_ARG;
  if (m->scale_ld < (blocks == MAO_BLOCKS_COL ? m->cols : ceil_div(m->cols, 128)))
    return MAO_ERR_INVALID_ARG;
  if (m->rows > kMaxCodes || m->cols > kMaxCodes || m->rows * m->count > kMaxCodes)
    return MAO_ERR_UNSUPPORTED;
  if (m->rows == 0) return MAO_OK;
  if (!m->codes || !m->scales) return MAO_ERR_INVALID_ARG;
  return aligned(m->codes, 16) ? MAO_OK : MAO_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

mao_status fp8_quantize(const mao_mat* X, int32_t batch, int64_t batch_stride,
                        const int32_t* index, int64_t n_index, int32_t copies,
                        const mao_fp8* row, const mao_fp8* col, const mao_fp8* tile,
                        void* stream) {
  if (!X || batch < 1 || batch_stride < 0) return MAO_ERR_INVALID_ARG;
  if ((!row && !col && !tile) || (tile && (row || col))) return MAO_ERR_INVALID_ARG;
  if (copies < 0 || (copies > 0 && (batch != 1 || n_index < 0 || (n_index > 0 && !index))))
    return MAO_ERR_INVALID_ARG;
  if (copies > 0 && !aligned(index, 4)) return MAO_ERR_MISALIGNED;
  for (int32_t b = 0; b < (batch_stride > 0 ? 1 : batch); ++b) {
    const mao_status st = check_rows(&X[b]);
    if (st != MAO_OK) return st;
    if (X[b].rows != X[0].rows || X[b].cols != X[0].cols || X[b].dtype != X[0].dtype)
      return MAO_ERR_INVALID_ARG;
  }
  const int64_t rows = copies > 0 ? n_index : X[0].rows;
  const mao_fp8* outs[3] = {row, col, tile};
  const int32_t kinds[3] = {MAO_BLOCKS_ROW, MAO_BLOCKS_COL, MAO_BLOCKS_TILE};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i]) continue;
    const mao_status st = check_fp8(outs[i], kinds[i]);
    if (st != MAO_OK) return st;
    if (outs[i]->rows != rows || outs[i]->cols != X[0].cols || outs[i]->count != batch)
      return MAO_ERR_INVALID_ARG;
  }
  return quantize_launch(X, batch, batch_stride, index, n_index, copies, row, col, tile,
                         static_cast<cudaStream_t>(stream));
}

mao_status fp8_product(const mao_fp8* A, const mao_fp8* B, const mao_mat* D, int32_t form,
                       const int32_t* offsets, int32_t groups, int32_t accumulate,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (form < MAO_NT || form > MAO_TN || groups < 1) return MAO_ERR_INVALID_ARG;
  if (groups > 1024) return MAO_ERR_UNSUPPORTED;
  if (!offsets && groups != 1) return MAO_ERR_INVALID_ARG;
  if (offsets && !aligned(offsets, 4)) return MAO_ERR_MISALIGNED;
  if (!aligned(workspace, 256)) return MAO_ERR_MISALIGNED;
  const bool tn = form == MAO_TN;
  mao_status st = check_fp8(A, tn ? MAO_BLOCKS_COL : MAO_BLOCKS_ROW);
  if (st == MAO_OK) st = check_fp8(B, tn ? MAO_BLOCKS_COL : MAO_BLOCKS_TILE);
  if (st == MAO_OK) st = check_rows(D);
  if (st != MAO_OK) return st;
  if (A->count != 1 || B->count != (tn ? 1 : groups)) return MAO_ERR_INVALID_ARG;
  if (!tn && B->rows < 1) return MAO_ERR_INVALID_ARG;
  const bool fits = form == MAO_NT   ? B->cols == A->cols && D->rows == A->rows && D->cols == B->rows
                    : form == MAO_NN ? B->rows == A->cols && D->rows == A->rows && D->cols == B->cols
                                     : B->rows == A->rows && D->cols == B->cols &&
                                           D->rows == A->cols * groups;
  if (!fits) return MAO_ERR_INVALID_ARG;
  if (device_cc() / 10 != 10) return MAO_ERR_UNSUPPORTED;
  return product_launch(*A, *B, *D, form, offsets, groups, accumulate, workspace, workspace_bytes,
                        static_cast<cudaStream_t>(stream));
}

size_t fp8_product_workspace_bytes(const mao_fp8* A, const mao_fp8* B, int32_t form) {
  if (!A || !B || form < MAO_NT || form > MAO_TN || A->rows < 0 || A->cols < 1 || B->rows < 0 ||
      B->cols < 1)
    return 0;
  return product_workspace_size(*A, *B, form);
}

mao_status expert_route(const mao_mat* logits, const float* bias, int32_t top_k, int32_t score,
                        int32_t groups, int32_t keep_groups, int32_t group_score,
                        int32_t renorm, float scale, float* weights, int32_t* ids,
                        void* stream) {
  const mao_status st = check_rows(logits);
  if (st != MAO_OK) return st;
  const int64_t E = logits->cols;
  if (E > 1024) return MAO_ERR_UNSUPPORTED;
  if (top_k < 1 || top_k > E || groups < 1 || E % groups != 0 || keep_groups < 1 ||
      keep_groups > groups || top_k > E / groups * keep_groups)
    return MAO_ERR_INVALID_ARG;
  if (top_k > 32 || groups > 32) return MAO_ERR_UNSUPPORTED;
  if ((score != MAO_SCORE_SOFTMAX && score != MAO_SCORE_SIGMOID) ||
      (group_score != MAO_GROUP_MAX && group_score != MAO_GROUP_TOP2) || !std::isfinite(scale))
    return MAO_ERR_INVALID_ARG;
  if (logits->rows == 0) return MAO_OK;
  if (!weights || !ids) return MAO_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(bias, 4)) return MAO_ERR_MISALIGNED;
  const RouteParams p{logits->data, bias, weights, ids, logits->ld, logits->rows, logits->dtype,
                      int32_t(E), top_k, score, groups, keep_groups, group_score, renorm, scale};
  return route_launch(p, static_cast<cudaStream_t>(stream));
}

mao_status expert_route_backward(const mao_mat* logits, const int32_t* ids,
                                 const float* dweights, int32_t top_k, int32_t score,
                                 int32_t renorm, float scale, const mao_mat* dlogits,
                                 void* stream) {
  mao_status st = check_rows(logits);
  if (st == MAO_OK) st = check_rows(dlogits);
  if (st != MAO_OK) return st;
  if (logits->cols > 1024 || top_k > 32) return MAO_ERR_UNSUPPORTED;
  if (dlogits->rows != logits->rows || dlogits->cols != logits->cols || top_k < 1 ||
      top_k > logits->cols || (score != MAO_SCORE_SOFTMAX && score != MAO_SCORE_SIGMOID) ||
      !std::isfinite(scale))
    return MAO_ERR_INVALID_ARG;
  if (logits->rows == 0) return MAO_OK;
  if (!ids || !dweights) return MAO_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(dweights, 4)) return MAO_ERR_MISALIGNED;
  const RouteBackParams p{logits->data, ids, dweights, dlogits->data, logits->ld, dlogits->ld,
                          logits->rows, logits->dtype, dlogits->dtype, int32_t(logits->cols),
                          top_k, score, renorm, scale};
  return route_backward_launch(p, static_cast<cudaStream_t>(stream));
}

int64_t expert_rows(int64_t n, int32_t experts) {
  if (n < 0 || experts < 1) return 0;
  return (n + 127 * (n < experts ? n : experts)) / 128 * 128;
}

size_t expert_plan_workspace_bytes(int64_t n, int32_t experts) {
  if (n < 0 || n > (int64_t(1) << 24) || experts < 1 || experts > 1024) return 0;
  return plan_workspace_size(n, experts);
}

mao_status expert_plan(const int32_t* ids, int64_t n, int32_t experts, int32_t* counts,
                       int32_t* offsets, int32_t* row_of, int32_t* slot_of, int64_t n_slots,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || experts < 1 || !counts || !offsets) return MAO_ERR_INVALID_ARG;
  if (n > (int64_t(1) << 24) || experts > 1024) return MAO_ERR_UNSUPPORTED;
  if ((n > 0 && (!ids || !row_of)) || (n_slots > 0 && !slot_of)) return MAO_ERR_INVALID_ARG;
  if (n_slots < expert_rows(n, experts)) return MAO_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(row_of, 4) ||
      !aligned(slot_of, 4) || !aligned(workspace, 256))
    return MAO_ERR_MISALIGNED;
  if (n > kPlanAlone) {
    if (!workspace) return MAO_ERR_INVALID_ARG;
    if (workspace_bytes < plan_workspace_size(n, experts)) return MAO_ERR_WORKSPACE;
  }
  return plan_launch(ids, n, experts, counts, offsets, row_of, slot_of, n_slots, workspace,
                     static_cast<cudaStream_t>(stream));
}

mao_status expert_combine(const mao_mat* Z, const int32_t* row_of, const float* weights,
                          int64_t tokens, int32_t top_k, const mao_mat* Y, void* stream) {
  mao_status st = check_rows(Z);
  if (st == MAO_OK) st = check_rows(Y);
  if (st != MAO_OK) return st;
  if (top_k < 1 || Y->rows != tokens || Y->cols != Z->cols) return MAO_ERR_INVALID_ARG;
  if (top_k > 32 || ceil_div(Y->cols, 8) > 65535 * int64_t(256)) return MAO_ERR_UNSUPPORTED;
  if (tokens == 0) return MAO_OK;
  if (!row_of) return MAO_ERR_INVALID_ARG;
  if (!aligned(row_of, 4) || !aligned(weights, 4)) return MAO_ERR_MISALIGNED;
  return combine_launch(*Z, row_of, weights, tokens, top_k, *Y, static_cast<cudaStream_t>(stream));
}

mao_status expert_combine_backward(const mao_mat* dY, const mao_mat* Z, const int32_t* row_of,
                                   const int32_t* slot_of, const float* weights, int32_t top_k,
                                   const mao_mat* dZ, float* dweights, void* stream) {
  mao_status st = check_rows(dY);
  if (st == MAO_OK) st = check_rows(Z);
  if (st == MAO_OK) st = check_rows(dZ);
  if (st != MAO_OK) return st;
  if (top_k < 1 || dY->cols != Z->cols || dZ->cols != Z->cols || dZ->rows != Z->rows)
    return MAO_ERR_INVALID_ARG;
  if (top_k > 32) return MAO_ERR_UNSUPPORTED;
  if ((Z->rows > 0 && !slot_of) || (dweights && dY->rows > 0 && !row_of)) return MAO_ERR_INVALID_ARG;
  if (!aligned(row_of, 4) || !aligned(slot_of, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return MAO_ERR_MISALIGNED;
  return combine_backward_launch(*dY, *Z, row_of, slot_of, weights, top_k, *dZ, dweights,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"
