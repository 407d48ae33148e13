// Tiles of products over runs of rows, their outputs' helpers and the split of long sums: shared
// by the feed-forward products in bf16 and in 8-bit integers.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace mao {
namespace ffn {

constexpr int TILE = 256;  // i and (at most) j per tile
constexpr int HALF = 128;  // of each per CTA
constexpr int MAX_GROUPS = 1024;
constexpr int BAND = 8;    // tiles of j that share a pass over i
constexpr size_t TABLE_BYTES = size_t(3) * (MAX_GROUPS + 2) * 4;

enum Form { NT, NN, TN, GRADS };  // GRADS: a product NN and two TN in one launch

struct TileParams {
  const int32_t* offsets;
  const int32_t* counts;
  int32_t rows;              // t
  int32_t I, J;              // D's columns (or channels); rows of D or, for TN, of one matrix
  int32_t depth;             // per half of the depth (TN: the run's rows)
  int32_t halves;            // NN: halves of the depth; TN: matrices per run
  int32_t tiles_i, groups;
  int32_t height;            // j per tile, at most: a multiple of 32
  int32_t splits, split_kb;  // parts of the depth (one run), blocks of each: D are fp32 parts
  unsigned long long timeout_ns;
};

struct Tile {
  int g = 0;    // run
  int half = 0; // TN: which of the run's matrices
  int i0, j0;   // first i; first j (a row of D, or of the run's matrix)
  int j_end;    // rows of D in the tile end here
  int n;        // j computed (a multiple of 32)
  int k0;       // TN: first row of the depth
  int kb0;      // first block of the depth (of a split)
  int nkb;      // blocks of the depth, 0: the tile is only cleared
  int64_t row0; // row of the output that j counts from
};

// lo[g] (g <= groups) is the first row of run g, cut to 0 .. rows and made rising; cnt[g] its rows
// in use. begin[g] counts the tiles of j before run g (NT, NN), begin[groups] all of them.

template <int THREADS>
__device__ __forceinline__ void make_table(const TileParams& p, int* lo, int* cnt, int* begin, int* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.groups;
  if (!p.offsets) {
    if (tid == 0) {
      lo[0] = 0;
      lo[1] = p.rows;
    }
  } else {
    for (int g = tid; g <= n; g += THREADS) lo[g] = max(0, min(p.offsets[g], p.rows));
  }
  __syncthreads();
  bool falls = false;
  for (int g = tid; g < n; g += THREADS) falls = falls || lo[g + 1] < lo[g];
  if (__syncthreads_or(falls)) {  // offsets that fall are raised to the largest before them
    if (tid == 0)
      for (int g = 0; g < n; ++g) lo[g + 1] = max(lo[g + 1], lo[g]);
    __syncthreads();
  }
  // thread i sums the tiles of groups 4 i .. 4 i + 3
  static_assert(4 * THREADS >= MAX_GROUPS, "a thread for every four groups");
  int c[4], own = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int g = 4 * tid + q;
    c[q] = 0;
    if (g < n) {
      const int all = lo[g + 1] - lo[g];
      const int used = p.counts ? max(0, min(p.counts[g], all)) : all;
      cnt[g] = used;
      c[q] = (used - 1) / p.height + (used > 0);  // (used + height may pass 2^31)
    }
    own += c[q];
  }
  int s = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  for (int w = 0; w < warp; ++w) s += sums[w];
  s -= own;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int g = 4 * tid + q;
    if (g <= n) begin[g] = s;
    s += c[q];
  }
  if (tid == THREADS - 1 && 4 * THREADS <= n) begin[n] = s;  // no thread's four reach that entry
}

// A split's share of the depth, and its rows of the partial sums.
template <int FORM>
__device__ __forceinline__ void take_split(const TileParams& p, int split, Tile& t) {
  t.kb0 = 0;
  if (p.splits > 1) {
    t.kb0 = split * p.split_kb;
    t.nkb = min(p.split_kb, t.nkb - t.kb0);
    t.row0 += int64_t(split) * p.J * (FORM == TN ? p.halves : 1);
  }
}

// STEP_I: values of i per tile; BK: the depth's blocks. The whole warp decodes: t.g is a run at or before the tile's (tiles come in rising order; with
// splits there is one run).
template <int FORM, int STEP_I, int BK>
__device__ __forceinline__ void decode(const TileParams& p, const int* lo, const int* cnt,
                                       const int* begin, int tile, Tile& t) {
  if (FORM == TN) {
    // i runs fastest: the pairs at work at one time write whole rows of a matrix
    const int tiles_j = (p.J + p.height - 1) / p.height, each = tiles_j * p.tiles_i;
    int m = tile / each;  // split, run, half
    const int local = tile - m * each;
    const int jt = local / p.tiles_i;
    const int matrices = p.groups * p.halves, split = m / matrices;
    m -= split * matrices;
    t.g = m / p.halves;
    t.half = m - t.g * p.halves;
    t.i0 = (local - jt * p.tiles_i) * TILE;
    t.j0 = jt * p.height;
    t.j_end = min(t.j0 + p.height, p.J);
    t.k0 = lo[t.g];
    t.nkb = (cnt[t.g] + BK - 1) / BK;
    t.row0 = int64_t(m) * p.J;
    take_split<FORM>(p, split, t);
    t.n = (t.j_end - t.j0 + 31) & ~31;
    return;
  }
  int split = 0;
  if (p.splits > 1) {
    const int tiles = begin[1] * p.tiles_i;
    split = tile / tiles;
    tile -= split * tiles;
  }
  // the last run with begin * tiles_i <= tile: the one whose tiles hold this one
  const int lane = threadIdx.x & 31;
  int a = t.g;
  while (true) {
    const int g = a + 1 + lane;
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, g >= p.groups || begin[g] * p.tiles_i > tile);
    if (past) {
      a += __ffs(past) - 1;
      break;
    }
    a += 32;
  }
  t.g = a;
  const int count = begin[a + 1] - begin[a];
  int local = tile - begin[a] * p.tiles_i;
  // bands of BAND tiles of j: within a band j runs fastest, then i, so that the pairs at work
  // at one time share operand rows in both directions
  const int band = count > BAND ? local / (BAND * p.tiles_i) : 0;
  local -= band * BAND * p.tiles_i;
  const int nb = min(BAND, count - band * BAND);
  const int it = local / nb;
  const int jt = band * BAND + local - it * nb;
  t.i0 = it * STEP_I;
  t.half = 0;
  t.k0 = 0;
  // a run's tiles are of even height
  const int rows = cnt[a];
  const int height = count > 1 ? ((rows - 1) / count + 32) & ~31 : p.height;
  t.j0 = lo[a] + jt * height;
  t.j_end = min(t.j0 + height, lo[a] + rows);
  t.nkb = (p.depth + BK - 1) / BK * (FORM == NN ? p.halves : 1);
  t.row0 = 0;
  take_split<FORM>(p, split, t);
  t.n = (t.j_end - t.j0 + 31) & ~31;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void store_word(void* at, uint32_t w) {
  asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(at), "r"(w) : "memory");
}

// Entries a of row c and b of row c + 1, both of this lane's column, as words of two columns:
// the even lane of a pair gets both columns of row c, the odd lane both of row c + 1.
__device__ __forceinline__ uint32_t swap_pair(float a, float b, int odd) {
  const uint32_t w = pack(a, b);
  const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
  return odd ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
}

// Clears `bytes` (a multiple of 2) of rows j0, j0 + step, ... below j1, a row per turn of a warp.
__device__ __forceinline__ void clear_rows(void* base, int64_t ld_bytes, int64_t bytes, int64_t j0, int64_t j1,
                                           int64_t step, int lane) {
  uint8_t* b0 = static_cast<uint8_t*>(base);
  const bool vec = reinterpret_cast<uintptr_t>(b0) % 16 == 0 && ld_bytes % 16 == 0;
  for (int64_t j = j0; j < j1; j += step) {
    uint8_t* d = b0 + j * ld_bytes;
    int64_t done = 0;
    if (vec) {
      for (int64_t b = 16 * lane; b + 16 <= bytes; b += 512) *reinterpret_cast<uint4*>(d + b) = make_uint4(0u, 0u, 0u, 0u);
      done = bytes & ~int64_t(15);
    }
    for (int64_t b = done + 2 * lane; b < bytes; b += 64) *reinterpret_cast<uint16_t*>(d + b) = 0;
  }
}

// Calls clear(first, end, step) with this turn's share of the rows that hold no tokens: each run's
// padding is shared by every groups-th turn (dealt to all turns range by range, short paddings all
// fell to the first few blocks: 192 us instead of 174 for a product of 128 runs of 125 rows; dealt
// evenly by a count over all ranges, the count took 5 us).
template <typename Clear>
__device__ __forceinline__ void for_unused_rows(const TileParams& p, const int* lo, const int* cnt, int turn,
                                                int turns, Clear&& clear) {
  const int n = p.groups;
  clear(int64_t(turn), int64_t(lo[0]), int64_t(turns));
  clear(int64_t(lo[n]) + turn, int64_t(p.rows), int64_t(turns));
  if (!p.counts) return;
  const int parts = (turns + n - 1) / n;  // those with a turn of their own below `turns`
  for (int g = turn % n, part = turn / n; g < n; g += turns) {
    const int of = turns < n ? 1 : parts - (g + (parts - 1) * n >= turns);
    clear(int64_t(lo[g]) + cnt[g] + (turns < n ? 0 : part), int64_t(lo[g + 1]), int64_t(of));
  }
}

// Pairs of CTAs that fit the GPU (sizes are asked for without one, too).
inline int64_t cta_pairs() { return num_sms() > 1 ? num_sms() / 2 : 1; }

// How a product of one run is cut: the height of its tiles, and the parts of its depth with their
// blocks.
struct Cut {
  int height, splits, kb;
};
// The cut with the least time by a model of the kernels, in us: per block of the depth `fixed` and
// `block` for a tile of 256, of which less for a lower one, at least `least_block`; `epilogue` for a tile
// of 256; 2.5 us and 3 TB/s for the sum of the fp32 parts, which stay in L2. tiles_i: tiles of i (of all
// matrices); pairs: pairs of CTAs at work on it. Heights go by 32: with 256, 128, 64 and 32 only 5000 rows of a
// 2048 x 2048 block took 109 us instead of 79, their gradients 241 instead of 192.
inline Cut choose_cut(int64_t pairs, int64_t tiles_i, int64_t J, int64_t nkb, double fixed, double block, double least_block,
                      double epilogue, int64_t outputs, int64_t least_kb) {
  Cut best{TILE, 1, int(nkb)};
  double least = 1e30;
  for (int h = TILE; h >= 32; h -= 32) {
    if (h - 32 >= J) continue;  // (one tile either way)
    const int64_t tiles = tiles_i * ceil_div(J, h);
    const double part = double(J < h ? round_up(J, 32) : h) / TILE;
    const double by_rows = fixed + block * part, each = by_rows > least_block ? by_rows : least_block;
    for (int64_t s = 1; s <= 32 && (s == 1 || least_kb * s <= nkb); ++s) {
      const int64_t kb = ceil_div(nkb, s), parts = ceil_div(nkb, kb);
      double t = each * double(kb * ceil_div(tiles * parts, pairs)) + epilogue * part;
      if (parts > 1) t += 2.5 + double(parts) * double(outputs) * 8.0 / 3e6;
      if (t < 0.95 * least) {
        least = t;
        best = Cut{h, int(parts), int(kb)};
      }
    }
  }
  if (J < best.height) best.height = int(round_up(J, 32));
  return best;
}

}  // namespace ffn
}  // namespace mao
