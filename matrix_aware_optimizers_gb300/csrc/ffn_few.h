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
  int32_t early;    // all but X is older than the kernel before this one
};
mao_status few_launch(const FewParams& params, bool int8, bool gate, int32_t act, cudaStream_t stream);

// Reads and clears its device error word (after a stream sync).
mao_status few_read_and_clear_error(cudaStream_t stream);

// Whether a call's rows are few: up to sixteen; or, with counts, up to sixteen blocks of 128 rows and
// less than one for each run, which is how expert_plan lays out that many tokens of different runs (with
// a block per run it may be any number up to 128 a run, and only the device knows; a run of more
// rows than a pass takes reads its weights again). One row of the 4096-wide block: 56 us against
// 66 by tiles, 16 rows 63 against 68; 8 and 16 tokens of 128 experts of 2048 x 768: 24 and 40 against
// 30 and 43, but 130 of 8 experts 36 against 24, and where 8 of 17 hold 32 tokens each or 125, in rows
// cut to those in use, 55 and 192 against 23 and 25 (the header says so); an 8-bit product of 14336 x 4096, one row, eight and 16: 13,
// 16 and 22 against 22, 20 and 20.
inline bool few_rows(int64_t rows, bool grouped, bool counts, int32_t groups) {
  return grouped ? counts && rows <= 16 * 128 && rows < int64_t(128) * groups : rows <= 16;
}

}  // namespace mao
