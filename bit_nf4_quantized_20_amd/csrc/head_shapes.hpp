// head_shapes.hpp -- which tiles the products of k_head.hip take, by sizes and the weight's
// format alone.  Host code without the runtime, so that a test asks the rule itself
// which kernels its sizes reach.
#pragma once

#include "sizes.hpp"

namespace qlora {

constexpr int kHeadTile = 256;  // a piece's columns are a multiple of it (the last piece's may not be)
constexpr int kHeadStep = 64;   // columns (logits: of a row, E W: of the vocabulary) of one step
constexpr int64_t kHeadCus = 256;  // of the part; fixed, so that sizes depend on shapes only

// Rows of a tile of 256 columns.  A round of tiles (one a CU) of 64, 128, 192 and 256
// rows takes 53, 68, 95 and 107 us at 4096 columns, about 36 + 0.28 rows: the shorter ones
// read more weights a product, so which is best goes by how they fill the rounds.
// Measured with one height throughout (64 / 128 / 192 / 256), gradient calls: 40 x 50021 x
// 2304 136 / 140 / 146 / 150 us, 200 x 32000 x 4096 203 / 174 / 192 / 200, 301 x 50021 x
// 2304 350 / 285 / 226 / 250, 1024 x 32000 x 4096 722 / 495 / 508 / 440.  (Of 4- and
// 8-bit weights 64 rows have the tiles below.  224 are left out: their kernels have up to
// 118 vector registers too few, E W of 8 bits, and 24 to 43 in the logits.  Those of 256 have
// 31 to 67 too few in the logits' epilogue, once a tile, and 7 in E W; the cost does not count
// that, and the two have not been timed against each other.)
constexpr int kHeights[] = {64, 96, 128, 160, 192, 224, 256};
constexpr int64_t height_cost(int rows) { return 128 + rows; }
constexpr bool height_fits(int rows, bool codes) { return !codes || (rows != 64 && rows != 224); }

// Few rows: tiles of 128 columns, two workgroups a CU, so that one works while the
// other waits for its LDS reads and turns codes into bf16 (128 rows of an 8-bit
// weight 32000 x 4096: 82 us with 256 columns, 64 with 128, gradient 143 and 125).  A bf16
// weight's tiles wait for HBM instead; there the logits of up to 64 rows take them where
// tiles of 256 columns would fill no more than half of the CUs (16 x 32000 x 4096: 69
// us, 77 with 256 columns; 16 x 128000 x 4096: 223 and 213), with a CU to themselves.
inline bool half_tiles(int64_t T, int64_t n, bool codes) {
  return codes ? T <= 128 : T <= 64 && ceil_div(n, int64_t(256)) <= kHeadCus / 2;
}
// (of codes also 32 rows: 16 x 32000 x 4096 in NF4 52 us instead of 56, in 8 bits 49 and 51)
inline int half_rows(int64_t T, bool codes) { return codes && T <= 32 ? 32 : T <= 64 ? 64 : 128; }

struct TileShape {
  int rows, cols;
};
inline TileShape logits_shape(int64_t T, int64_t n, bool codes) {
  if (half_tiles(T, n, codes)) return {half_rows(T, codes), 128};
  int best = 0;
  int64_t least = 0;
  for (int rows : kHeights) {
    if (!height_fits(rows, codes)) continue;
    const int64_t cost = ceil_div(ceil_div(T, rows) * ceil_div(n, int64_t(256)), kHeadCus) * height_cost(rows);
    if (best == 0 || cost < least) best = rows, least = cost;
  }
  return {best, 256};
}

// The tiles of E W and the ranges of the vocabulary, each of 1024 columns or more: as
// many as give every CU its workgroups.
struct GradShape {
  TileShape tile;
  int splits;
};
inline GradShape grad_shape(int64_t T, int64_t H, int64_t n, bool codes) {
  const int64_t steps = round_up(n, kHeadTile) / kHeadStep;
  const auto splits = [&](int64_t workgroups, int64_t tiles) {
    int64_t S = workgroups / tiles;
    if (S > steps / 16) S = steps / 16;
    return S < 1 ? int64_t(1) : S;
  };
  if (codes && half_tiles(T, n, codes))
    return {{half_rows(T, codes), 128}, static_cast<int>(splits(2 * kHeadCus, ceil_div(H, int64_t(128))))};
  GradShape best{{0, 256}, 1};
  int64_t least = 0;
  for (int rows : kHeights) {
    if (!height_fits(rows, codes)) continue;
    const int64_t tiles = ceil_div(T, rows) * ceil_div(H, int64_t(256)), S = splits(kHeadCus, tiles);
    const int64_t cost = ceil_div(tiles * S, kHeadCus) * ceil_div(steps, S) * height_cost(rows);
    if (best.tile.rows == 0 || cost < least) best = GradShape{{rows, 256}, static_cast<int>(S)}, least = cost;
  }
  return best;
}

// columns that one wave of the logits reduces, and ranges of the vocabulary of E W
inline int head_cols(int64_t T, int64_t n, bool codes) { return logits_shape(T, n, codes).cols / 2; }
inline int head_splits(int64_t T, int64_t H, int64_t n, bool codes) { return grad_shape(T, H, n, codes).splits; }

}  // namespace qlora
