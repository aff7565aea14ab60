// Which tiles a product of bf16 operands takes (bf16_tiles.h), and the pieces of the
// vocabulary in the cross entropy's gradient (xent.hip): plain C++, so that the host
// can evaluate it without a GPU.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace adahop {
namespace tiles {

// How an operand lies: along K, across it, or across it in MXFP8 (B alone).
enum Kind { kAlong = 0, kAcross = 1, kCodes = 2 };

// Rows x columns. An operand A across K takes the first and the third alone.
enum Tile { k256x256 = 0, k192x256 = 1, k128x128 = 2, k64x128 = 3 };
constexpr int tile_rows(Tile s) { return s == k256x256 ? 256 : s == k192x256 ? 192 : s == k128x128 ? 128 : 64; }
constexpr int tile_cols(Tile s) { return s == k256x256 || s == k192x256 ? 256 : 128; }

// Tiles 0 .. full - 1 are whole, the `split` after them are each formed in `parts`
// parts of K.
struct ProductPlan {
  Tile tile;
  int64_t full, split;
  int parts;
  double us;                 // estimate
};

// Columns of B of one row of small tiles: a launch of one tile a workgroup stays
// far below 2^32 threads.
constexpr int64_t kMostSmall = int64_t{1} << 28;

// Estimates in microseconds, to rank the tiles by: constants set to products of one
// to a few rounds of tiles on the whole device (256 CUs), a launch and a tile's first
// loads and epilogue 5, a stage of K as below; parts of K a second launch and their
// sums written and read at 4.5 TB/s. They are no times of large tiles in many
// rounds, nor of epilogues longer than a store (333 x 50021 x 2080 with the cross
// entropy's statistics: estimate 64, measured 100; 1531 x 50021 x 2048 with its
// gradient: 181 and 273; 1531 x 2048 x 50021 in parts: 200 and 270; 8192 x 4096 x
// 65536: 2258 and 2860), and so rank those before smaller ones by up to a half too
// much. An A of two terms takes the tiles of one. The last round
// of tiles may be split where it leaves half of the compute units or more without
// one (dh of 1000 x 1024 x 3000: 128 tiles of 64 x 128 whole 18 us, in two parts
// 19; 37 x 1032 x 8191: 9 tiles of it 39 us, in 16 parts 11). Up to 128 rows the
// small tiles alone: what binds there is B's way from memory, which four slots
// keep busier than two (1 x 131072 x 4096: 179 us with 64 x 128 tiles, 188 with
// 128 x 128, 245 with 256 x 256).
inline ProductPlan product_plan(int64_t m, int64_t n, int64_t K, Kind a, Kind b, bool splits, int64_t cus) {
  ProductPlan best{};
  best.us = 1e30;
  const int64_t units = (K + 127) / 128;
  for (const Tile tile : {k256x256, k192x256, k128x128, k64x128}) {
    if (a != kAlong && (tile == k192x256 || tile == k64x128)) continue;
    const bool small = tile >= k128x128;
    if (a == kAlong && m <= 128 && !small && n <= kMostSmall) continue;
    const int64_t bm = tile_rows(tile), bn = tile_cols(tile);
    const int64_t all = ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
    if (small && all > kMostSmall / 128) continue;
    const int64_t rem = all % cus;
    int64_t parts = splits && rem > 0 ? cus / rem : 1;
    if (parts > units / 4) parts = units / 4;
    if (parts > 32) parts = 32;
    for (const bool split : {false, true}) {
      if (split && parts < 2) continue;
      // The smallest tiles on half of the compute units are not yet held up by the
      // way of their operands.
      const double stage = tile == k256x256   ? (b == kCodes ? 1.4 : 1.1)
                           : tile == k192x256 ? 0.86
                           : tile == k64x128  ? (!split && 2 * all <= cus ? 0.3 : 0.4)
                           : a == kAcross     ? 0.6
                                              : 0.46;
      ProductPlan p{tile, all, 0, 1, 0};
      if (split) p = {tile, all - rem, rem, (int)parts, 0};
      const int64_t rounds = (p.full + cus - 1) / cus;
      p.us = 5 + stage * 2 * (double)units * (double)rounds;
      if (split)
        p.us += 4 + stage * 2 * (double)((units + p.parts - 1) / p.parts) +
                p.parts * ((double)p.split / (double)all) * (double)m * (double)n * 8 / 4.5e6;
      if (p.us < best.us) best = p;
    }
  }
  return best;
}

// Whole columns of 256, which every tile's columns divide.
inline int64_t whole_tiles(int64_t n) { return (n + 255) / 256 * 256; }
// Rows that g is held in.
inline int64_t padded_rows(int64_t T) { return (T + 63) / 64 * 64; }

// Pieces of V entries: their columns, a multiple of 256, and how many there are.
struct XentPieces {
  int64_t size, count;
};
// piece: columns that the caller asks for, 0: as many as keep g, `terms` bf16
// numbers an element, within 1 GiB, but 256 at least; pieces of about the same size.
inline XentPieces xent_pieces(int64_t T, int64_t V, int64_t piece, int terms) {
  if (piece == 0) {
    const int64_t all = whole_tiles(V);
    piece = (int64_t{1} << 29) / terms / padded_rows(T > 0 ? T : 1) / 256 * 256;
    if (piece < 256) piece = 256;
    if (piece > all) piece = all;
    const int64_t count = (all + piece - 1) / piece;
    piece = (all + count - 1) / count;
  }
  piece = whole_tiles(piece < V ? piece : V);
  return {piece, (V + piece - 1) / piece};
}

}  // namespace tiles
}  // namespace adahop
