// Launcher of the feed-forward products for few rows.
#pragma once

#include "ffn_tiles.cuh"

namespace mao {

struct FewParams : ffn::TileParams {  // rows, I, depth, offsets, counts, groups (the rest is set here)
  const void* w;    // bf16 or codes: rows of I channels (gated: of Wg, then of Wu) for each run
  const void* x;    // bf16 or codes
  const float* sa;  // 8-bit integers: scales of X's rows and of W's
  const float* sb;
  void* d;          // H (gated), D
  void* z;          // gated: G and U, fp32 or bf16, or null
  int64_t ldw, ldx, ld, ldz;  // in entries
  int32_t dtype, z_dtype;
};
mao_status few_launch(const FewParams& params, bool int8, bool gate, int32_t act, cudaStream_t stream);

// Reads and clears its device error word (after a stream sync).
mao_status few_read_and_clear_error(cudaStream_t stream);

// Whether a call's rows are few: its products read each weight once then, whatever the tile. A call
// with counts may hold a few rows in each of a few runs of 128.
inline bool few_rows(int64_t rows, bool grouped, bool counts) {
  return grouped ? counts && rows <= 16 * 128 : rows <= 16;
}

}  // namespace mao
