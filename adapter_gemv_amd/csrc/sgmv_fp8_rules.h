// Which kernel form a product with 8-bit weights takes.  Nothing here needs a GPU.
#pragma once

#include "sgmv_rules.h"

namespace sgmv_host {

struct BlockLaunch : Launch {
  int buffers;  // stages that the tiled form holds; 0: streaming
};

// Streaming: 32 columns and 4 wavefronts to a workgroup, or 16 and 8 where that leaves CUs without work
// (whole kernel, one row, the first and the second: 4096 x 4096, 12.1 and 9.6 us; 5120 x 13824, 17.4 and
// 22.8; 16 rows, 8 experts of 5120 x 13824, 100 and 143).  64 columns read x half as often, but a ring of
// its own for each of 4 wavefronts then fills a CU: 5120 x 13824, 16 rows, 21.9 us to 21.8.
inline BlockLaunch fp8_skinny_launch(int32_t n, int32_t G, bool grouped, int32_t h_out) {
  const int64_t row_tiles = max_row_tiles(n, G, grouped, kSkinnyRows);
  const int cols = row_tiles * (h_out / 32) >= 256 ? 32 : 16;
  return {{kSkinnyRows, cols, cols == 32 ? 4 : 8, row_tiles * tiles_of(h_out, cols)}, 0};
}

// The smallest of four estimates in microseconds of a call (with the quantiser's kernel, which streaming
// does without), fitted to 1 to 64 groups of 1 to 1024 rows of weights 1024 x 8192 to 5120 x 13824.  Of
// groups only the mean size is known: each is taken to end in half a tile.
// A step is 128 contracted elements.  Tiles of 64 take 0.52 us for a step while they leave CUs free, and
// 0.0014 us a tile beyond; of 128, 0.95 and 0.0037; of 256, 1.9 us a round of the card.  All of them, 8 to 12 us
// and the weights at 4.8 TB/s.  Streaming takes 0.2 to 0.4 us, by rows, for a million weights and row
// tile of 32, and 5 us and 1.1 to 1.9 for 1024 contracted elements at least.
// Measured, us:                          streaming   64 x 64   128 x 128   256 x 256
//   2048 x 2048, 32 rows                  9.4         12.2      16.1
//   4096 x 4096, 64 rows                  20.3        22.8      29.9
//   4096 x 4096, 256 rows                 44.8        23.7      34.9
//   4096 x 4096, 1024 rows                152         50.7      38.1
//   5120 x 13824, 16 rows                 26.1        31.1      43.4
//   5120 x 13824, 64 rows                 56.9        32.4      40.0
//   5120 x 13824, 256 rows                168         70.2      45.0
//   8192 x 1024, 128 rows                 21.4        32.9      55.7
//   64 of 4096 x 1024, 4 rows each        64.6        68.6      73.3
//   64 of 4096 x 1024, 32 rows each       116         78.8      85.6
//   8 of 5120 x 13824, 64 rows each       359         190       152
//   8192 x 8192, 8192 rows (8 bits)                   1090                  541
inline BlockLaunch fp8_launch(bool dx, int32_t n, int32_t G, bool grouped, int32_t h_in, int32_t h_out) {
  const double met = std::max(1, std::min(n, G)), million = 1e-6 * h_in * h_out, rows = n, mean = rows / met;
  const int32_t out = dx ? h_in : h_out, depth = dx ? h_out : h_in;
  const double steps = std::ceil(depth / 128.0);
  const auto row_tiles = [&](int B) { return grouped ? std::max(met, rows / B + met / 2) : std::ceil(rows / B); };
  const auto tiles = [&](int B) { return row_tiles(B) * static_cast<double>(tiles_of(out, B)); };
  const double t64 = steps * std::max(0.52, 0.0014 * tiles(64)), t128 = steps * std::max(0.95, 0.0037 * tiles(128)),
               t256 = steps * 1.9 * std::max(1.0, std::ceil(tiles(256) / kCus - 0.1));
  const double tiled = std::max(5 + std::min({t64, t128, t256}), 8 + std::min(4.0, 0.06 * met * million) + met * million / 4.8);
  if (!dx) {
    const double one = mean <= 32 ? 0.2 + 0.0065 * mean : 0.36;
    if (5 + std::max((mean <= 16 ? 0.0011 : 0.0019) * h_in, row_tiles(32) * million * one) < tiled)
      return fp8_skinny_launch(n, G, grouped, h_out);
  }
  const int B = t64 <= std::min(t128, t256) ? 64 : t128 <= t256 ? 128 : 256;
  const int64_t workgroups = tiles_of(max_row_tiles(n, G, grouped, B) * tiles_of(out, B), kTileXcds) * kTileXcds;
  // as many stages as LDS holds for the workgroups of a CU
  const bool one_each = tiles(B) <= kCus;
  return {{B, B, B == 256 ? 8 : 4, workgroups}, B == 256 ? 2 : B == 128 ? (one_each ? 4 : 2) : (one_each ? 8 : 4)};
}

}  // namespace sgmv_host
