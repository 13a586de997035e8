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

}  // namespace fp4q
