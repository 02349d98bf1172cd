// How a group's rows are cut into tiles and in which order the tiles come: the integer
// arithmetic of the products over groups (gemm_grouped.cu), for host and device, so
// that it is tested without a GPU.
#pragma once
#include <cstdint>

#include "intmath.h"

namespace lgt {

constexpr uint32_t kGgBand = 8;  // tiles of a band

// recip[d] for d from 2 to kGgBand: 2^32 / d, rounded up.
inline void band_reciprocals(uint32_t (&recip)[kGgBand + 1]) {
  for (uint32_t d = 0; d <= kGgBand; ++d) recip[d] = d < 2 ? 0u : static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d);
}

// n / d for d from 1 to kGgBand and n below 2^29.
LGT_HD uint32_t divide_few(const uint32_t* recip, uint32_t n, uint32_t d) {
  return d == 1 ? n : static_cast<uint32_t>(static_cast<uint64_t>(n) * recip[d] >> 32);
}

// Rows of each of a group's `tiles` tiles (the last one has what is left): as even as
// multiples of `step` allow.
LGT_HD uint32_t even_width(const uint32_t* recip, uint32_t rows, uint32_t tiles, uint32_t step) {
  const uint32_t each = tiles <= kGgBand ? divide_few(recip, rows + tiles - 1, tiles) : (rows + tiles - 1) / tiles;
  return (each + step - 1) / step * step;
}

// Tile r of a group's p_tiles x q_tiles: in bands of the N side, so that those that run
// at once read no more of either operand than they have to.
LGT_HD void tile_in_bands(const uint32_t* recip, uint32_t r, uint32_t p_tiles, uint32_t q_tiles, uint32_t& p, uint32_t& q) {
  uint32_t band = 0, high = q_tiles;
  if (q_tiles > kGgBand) {
    band = r / (p_tiles * kGgBand);
    r -= band * (p_tiles * kGgBand);
    high = kGgBand < q_tiles - band * kGgBand ? kGgBand : q_tiles - band * kGgBand;
  }
  p = divide_few(recip, r, high);
  q = band * kGgBand + r - p * high;
}

}  // namespace lgt
