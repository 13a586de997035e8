// fp4q_ffn_sizes.h -- which sizes the kernels' 32-bit arithmetic holds: plain
// host arithmetic without HIP, so that a test can compile it by itself.
#pragma once

#include <stdint.h>

namespace fp4q {

// The tile kernel with the LDS ring has 128 rows of either factor of a gated call
// in a tile, and adds up the offset of a row's scales in 32 bits from the tile's
// first row of the first factor on: to row n / 2 + 127 from there.  (n rows of both
// factors; k / 16 bytes of scales a row, MXFP4's half as many.)
constexpr int64_t kRingFactorRows = 128;
inline bool ring_scales_fit(bool gated, int64_t n, int64_t k) {
  return !gated || (n / 2 + kRingFactorRows) * (k / 16) <= (int64_t)INT32_MAX;
}

// The kernel of few rows has offsets of 32 bits into 8-bit rows, which are dense.
inline bool few_eight_fits(int64_t rows, int64_t k) { return rows * k <= (int64_t)INT32_MAX; }

// A launch takes fewer than 2^32 threads in a dimension of its grid, and workgroups
// here have at most 1024.  More workgroups than kGridRow make rows of so many: number
// y kGridRow + x; the last row's may be past the end.
constexpr int64_t kGridRow = 1 << 21;
inline unsigned grid_x(int64_t groups) { return (unsigned)(groups < kGridRow ? groups : kGridRow); }
inline unsigned grid_y(int64_t groups) { return (unsigned)((groups + kGridRow - 1) / kGridRow); }

// The kernels of many rows have a workgroup for each tile, of 512 threads at most, in
// one dimension, their number rounded up to a multiple of 8.
inline bool tiles_fit(int64_t tiles) { return (tiles + 7) / 8 * 8 * 512 < (int64_t)1 << 32; }

}  // namespace fp4q
