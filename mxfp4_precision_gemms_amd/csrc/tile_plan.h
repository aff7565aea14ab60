// Which tiles a product of bf16 operands takes (bf16_tiles.h): plain C++, so that
// the host can evaluate it without a GPU.
#pragma once

#include <cstdint>

#include "linear_plan.h"

namespace adahop {
namespace tiles {

// Tiles of 256 x 256, or of 128 or 64 rows by 128 columns (an operand A across K:
// 256 or 128 rows).
constexpr int tile_rows(TileShape s) { return 256 >> s; }
constexpr int tile_cols(TileShape s) { return s == kTile256 ? 256 : 128; }

// Tiles 0 .. full - 1 are whole, the `split` after them are each formed in `parts`
// parts of K.
struct ProductPlan {
  TileShape shape;
  int64_t full, split;
  int parts;
  double us;                 // estimate
};

inline ProductPlan product_plan(int64_t m, int64_t n, int64_t K, bool along, bool splits, int64_t cus) {
  ProductPlan best{};
  best.us = 1e30;
  const int64_t units = (K + 127) / 128;
  for (const TileShape shape : {kTile256, kTile128, kTile64}) {
    if (!along && shape > kTile128) break;
    const int64_t bm = tile_rows(shape), bn = tile_cols(shape);
    const int64_t all = ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
    const double stage = shape == kTile256 ? 1.0 : shape == kTile128 ? 0.4 : 0.35;
    const int64_t rem = all % cus;
    int64_t parts = splits && rem > 0 ? cus / rem : 1;
    if (parts > units / 4) parts = units / 4;
    if (parts > 32) parts = 32;
    ProductPlan p{shape, all, 0, 1, 0};
    if (parts >= 2) p = {shape, all - rem, rem, (int)parts, 0};
    const int64_t rounds = (p.full + cus - 1) / cus;
    p.us = 5 + stage * 2 * (double)units * (double)rounds;
    if (p.split) p.us += 5 + stage * 2 * (double)((units + p.parts - 1) / p.parts);
    if (p.us < best.us) best = p;
  }
  return best;
}

}  // namespace tiles
}  // namespace adahop
