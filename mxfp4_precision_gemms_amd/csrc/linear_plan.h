// Which of the linear layer's kernels a product takes, and the workspace that
// goes with it: plain C++, so that the host can evaluate it without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace adahop {

// Rows of a gated layer's B: its output columns make less than 2^24 groups of 32,
// whose launch it takes at once.
constexpr int64_t kMaxGatedN = (int64_t{1} << 30) - 64;

// Whether the products are formed exactly (products: adahop_products). AUTO goes
// by the output alone, so that a caller can tell, and a device's or an
// estimate's change moves no result. Up to 32768 MXFP8 values come mostly from
// few rows, where loads bind and exact products cost little (microseconds exact
// and scaled: 1 x 4096 x 14336, E2M1 16.0 and 13.7, 1 x 14336 gated x 4096 20.7
// and 16.9, 8 x 4096 x 4096, E4M3 10.4 and 9.6); the most where few columns
// meet a long K (32 x 960 x 14336: 26.0 and 10.4). Above, tiles are faster by
// 1.6 times at 32 rows and 4 at 100 (14336 gated x 4096, E4M3: 45 and 28, 130
// and 33), 11 at 4096 rows (4096 x 4096, E4M3: 733 and 65).
constexpr bool exact_products(int products, bool mx8_out, int64_t m, int64_t n) {
  return products == 2 || (products == 0 && mx8_out && m * n <= 32768);
}

// Tile kernel of a product (linear_tiles.hip) and its workspace: scale words
// by stage, then the K parts' sums.
enum TileShape { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile32 = 3 };   // 256 rows >> shape
struct TilePlan {
  TileShape shape;
  int parts;
  size_t scale_bytes, part_bytes;
  double us;                 // estimate
};

// Estimates in microseconds, from measurements on the whole device (256 CUs):
// a launch and a tile's first loads and epilogue 5, a stage 0.1 and its bytes
// at 55 KB / us a compute unit (32 x 128 tiles 0.33 and 0.45, 64 x 128 0.4 and
// 0.53, 128 x 128 0.57 and 0.65, E2M1 and E4M3 weights), of 256 x 256 tiles
// 1.45 and 1.55 with 4 for ordering the scales; K parts 3 for the second
// kernel and their sums written and read at 4 TB/s. On 36 cases (m = 40 ..
// 3000, six weights) the choice was within 6 % of the fastest of all shapes
// and parts on 33, at worst 16 % off.
inline TilePlan linear_tile_plan(int64_t m, int64_t n, int64_t K, int b_fp4, int gated, int64_t cus) {
  const int64_t N = gated ? 2 * n : n, nk = (K + 127) / 128;
  TilePlan best{};
  best.us = 1e30;
  for (int shape = kTile256; shape <= kTile32; ++shape) {
    const int lm = 8 - shape, ln = shape == kTile256 ? 8 : 7;     // log2 of the tile's rows and columns
    const int lu = shape == kTile256 ? 1 : 2;                     // and of the stages that parts are made of
    const double kb = (double)((128 << lm) + ((b_fp4 ? 64 : 128) << ln)) / 1024;
    const double stage = shape == kTile256 ? (b_fp4 ? 1.45 : 1.55) : 0.1 + kb / 55;
    // The smaller tiles of E2M1 weights run two to a compute unit.
    const bool two = b_fp4 && lm <= 6;
    const int64_t tiles = ((m + (1 << lm) - 1) >> lm) * ((N + (1 << ln) - 1) >> ln);
    const uint32_t units = (uint32_t)((nk + (1 << lu) - 1) >> lu);
    for (const uint32_t parts : {1u, 2u, 3u, 4u, 6u, 8u, 12u, 16u}) {
      if (parts > units || (parts > 1 && tiles * parts > 2 * cus)) break;
      const double rounds = parts == 1 ? (double)((tiles + cus - 1) / cus) : tiles * parts > cus ? 2 : 1;
      double us = 5 + rounds * (double)((units + parts - 1) / parts << lu) * stage;
      if (shape == kTile256) us += 4;
      else us += (K % 512 ? 3 : 0) + (two ? 0 : 1.5 * (rounds - 1));
      if (parts > 1) us += 3 + (double)parts * (double)m * (double)N * 8 / 4e6;
      if (us < best.us) {
        best = {(TileShape)shape, (int)parts, 0, 0, us};
        if (parts > 1) best.part_bytes = (size_t)tiles * 4 * parts << (lm + ln);
      }
    }
  }
  // Whole groups of 64 rows, gated 32 columns' gate and up rows, and 4 stages.
  best.scale_bytes = (size_t)((nk + 3) / 4 * 16 * (m + N + 256));
  return best;
}

// 16 columns and 8 waves a workgroup while that makes at most two for each
// compute unit (1 x 4096 x 14336, E2M1: 10.6 us, with 32 columns and 4 waves
// 17.1), else 32 columns and 4 waves, which read A half as often (16 x 14336
// gated x 4096: 21.0, with 16 columns 23.9). An MXFP8 block needs 32 (1 x 4096 x
// 14336: 13.7, exact 16.0).
constexpr bool few_narrow(int64_t n) { return n <= 16 * 512; }
// Output columns of a launch of more than those: with 256 threads for 32
// columns, 2^31 threads. (A gated layer's go at once.)
constexpr int64_t kFewLaunchCols = int64_t{1} << 28;
constexpr int64_t few_wide_threads(int64_t n) { return (n + 31) / 32 * 256; }
static_assert(few_wide_threads(kFewLaunchCols) < int64_t{1} << 32 &&
              few_wide_threads(kMaxGatedN / 2) < int64_t{1} << 32, "");

// Estimate in microseconds, as linear_tile_plan's, for scaled products: a launch
// 3.5, all of B at 5 TB/s, and what a compute unit reads of A and B (again for
// every 32 rows) at 28 KB / us with 8 waves (24 where workgroups of 32 columns
// share one) and 20 with 4. On 162 cases of each type (m = 1 .. 100, nine
// weights in both formats) the choice against the tiles was within 6 % of the
// faster on 154 (MXFP8 out) and 158 (bf16), at worst 24 % and 27 % off.
inline double few_us(int64_t m, int64_t n, int64_t K, int b_fp4, int gated, bool mx8_out, int64_t cus) {
  const double kb = (double)K / 1024, b = b_fp4 ? 17.0 / 32 : 33.0 / 32, a = 33.0 / 32;
  const int cols = few_narrow(n) && !mx8_out ? 16 : 32;
  const bool eight = few_narrow(n) && !(mx8_out && gated);
  const double down = (double)((m + 31) / 32), rows = (double)m / down;
  const double groups = down * (double)((n + cols - 1) / cols) / (double)cus;
  const double group_kb = kb * (cols * (gated ? 2 : 1) * b + rows * a);
  const double cu = (groups < 1 ? 1 : groups) * group_kb / (!eight ? 20 : mx8_out && groups > 1 ? 24 : 28);
  const double hbm = (double)n * (gated ? 2 : 1) * kb * b / 4883;
  return 3.5 + (cu > hbm ? cu : hbm);
}

inline bool take_few(int64_t m, const TilePlan& p, int64_t n, int64_t K, int b_fp4, int gated, bool mx8_out,
                     int64_t cus) {
  return few_us(m, n, K, b_fp4, gated, mx8_out, cus) <= p.us;
}

}  // namespace adahop
