// Launch shapes of the norm and linear layer's kernels: plain C++, so that the
// host can check them without a GPU. A launch's grid times its workgroup, in
// each dimension, has to stay below 2^32 threads.
#pragma once

#include <cstdint>

namespace adahop {

// RMS norm. Up to 2048 columns a wave holds a row; above, 4 waves, then 16,
// share it: at most 4 groups of 8 columns a thread.
struct NormShape {
  int waves, groups;
};
constexpr NormShape norm_shape(int64_t cols) {
  return cols <= 512 ? NormShape{1, 1} : cols <= 1024 ? NormShape{1, 2} : cols <= 2048 ? NormShape{1, 4}
       : cols <= 4096 ? NormShape{4, 2} : cols <= 8192 ? NormShape{4, 4}
       : cols <= 16384 ? NormShape{16, 2} : NormShape{16, 4};
}
// With one wave a row, a workgroup takes 4 rows.
constexpr int64_t norm_grid(int64_t rows, int waves) { return waves == 1 ? (rows + 3) / 4 : rows; }
constexpr int norm_block(int waves) { return waves == 1 ? 256 : 64 * waves; }
// Rows of a launch: 2^31 threads where 16 waves share a row.
constexpr int64_t kNormLaunchRows = int64_t{1} << 21;

// Column sums over workgroups' parts: 16 columns a workgroup.
constexpr int kReduceBlock = 1024;
constexpr int64_t reduce_grid(int64_t cols) { return (cols + 15) / 16; }
constexpr int64_t kReduceLaunchCols = int64_t{1} << 24;   // 2^30 threads

}  // namespace adahop
