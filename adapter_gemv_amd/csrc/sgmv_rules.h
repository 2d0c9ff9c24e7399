// Host checks of the grouped and 4-bit products, and which kernel form each call takes.  Nothing
// here needs a GPU.
#pragma once

#include <algorithm>
#include <cmath>

#include "sgmv_checks.h"

namespace sgmv_dev {

// What the tiled kernel computes: x W^T, dy W, dy^T x, and x W^T with W or both sides in 4 bits
enum Mode { kForward, kDx, kDw, kMxW, kMxBoth };

}  // namespace sgmv_dev

namespace sgmv_host {

constexpr int kMaxGroups = SGMV_MAX_GROUPS;
constexpr int32_t kMaxGroupRows = 1 << 30;  // row numbers plus a workgroup's stride stay int32

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// tables and group count of a grouped call; 0 when fine (n may be 0)
inline int check_groups(int32_t n, int32_t G, int32_t share, const int32_t* starts,
                        const int32_t* perm) {
  if (n < 0 || n > kMaxGroupRows || G < 1 || share < 1) return SGMV_ERR_SHAPE;
  if (G > kMaxGroups) return SGMV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n) * share > INT32_MAX) return SGMV_ERR_SHAPE;
  if (!starts && G != 1) return SGMV_ERR_NULL;
  if (n > 0 && (starts == nullptr) != (perm == nullptr)) return SGMV_ERR_NULL;
  return SGMV_OK;
}

// whether an output lies over the tables of its call (rows are looked up until the last is written)
inline bool over_tables(const void* out, size_t bytes, const int32_t* starts, const int32_t* perm,
                        int32_t n, int32_t G) {
  return (starts && ranges_overlap(out, bytes, starts, sizeof(int32_t) * (static_cast<size_t>(G) + 1))) ||
         (perm && ranges_overlap(out, bytes, perm, sizeof(int32_t) * static_cast<size_t>(n)));
}

// rows of x that n rows sharing it read
inline int32_t shared_rows(int32_t n, int32_t share) { return (n + share - 1) / share; }

// at most this many row tiles of BM rows in the groups and behind them
inline int64_t max_row_tiles(int32_t n, int32_t G, bool grouped, int BM) {
  const int64_t most = n / BM + (grouped ? G + 1 : n % BM != 0);
  return most < n ? most : n;
}

inline size_t pool_bytes16(int32_t G, int64_t stride, int64_t elems) {
  return 2 * (static_cast<size_t>(G - 1) * static_cast<size_t>(stride) + static_cast<size_t>(elems));
}

// A launch: output rows, output columns and wavefronts of a workgroup, and the workgroups.  Row
// tiles of kSkinnyRows are the streaming form's, larger ones the tiled form's.
constexpr int kSkinnyRows = 32;
constexpr int kTileXcds = 8;  // workgroups of tiles come in whole rounds of the XCDs
struct Launch {
  int rows, cols, waves;
  int64_t workgroups;
  bool fits() const { return workgroups * 64 * waves <= UINT32_MAX; }  // the threads of a grid
};

inline int64_t tiles_of(int64_t n, int size) { return (n + size - 1) / size; }

// Columns and wavefronts of a workgroup.  16-bit weights: 16 columns, 4 wavefronts (64 experts of
// 4096 x 1024, 32 rows: 38 us; 40 with 8 wavefronts, 44 with 32 columns).
// 4-bit weights, of whose rows a wavefront has a quarter of the bytes: 32 columns, 2 wavefronts
// (8 experts of 5120 x 13824, 32 rows, in the first form: 93 us; 104 with 4 wavefronts, 124 with 16
// columns; the call is now at 85 to 92), or 16 columns and 8 wavefronts where that leaves CUs without work
// (now, the first and the second: 4096 x 4096, 32 rows, 17.5 and 12.1 us; 64 rows 17.9 and 22.2;
// 4096 x 8192, 32 rows, 17.7 and 22.1; 5120 x 13824, 16 rows, 18.7 and 37.5).
inline Launch skinny_launch(int32_t n, int32_t G, bool grouped, int32_t h_out, bool mx) {
  const int64_t row_tiles = max_row_tiles(n, G, grouped, kSkinnyRows);
  const int cols = mx && row_tiles * (h_out / 32) >= 256 ? 32 : 16;
  return {kSkinnyRows, cols, !mx ? 4 : cols == 32 ? 2 : 8, row_tiles * tiles_of(h_out, cols)};
}

// Whether few rows meet each weight, so that streaming beats tiles: the smaller of two estimates,
// in microseconds, fitted to 1 to 64 groups of 1 to 512 rows (weights 4096 x 1024 to 5120 x 13824, and
// with both sides in 4 bits from 1024 x 1024).  Of groups only the mean size is known: each is taken
// to end in half a tile.
// Streaming takes 0.38 to 0.5 us (16-bit) or 0.17 to 0.26 us (4-bit weights) for a million weights
// and row tile, the less where the rows are at most 16.  Tiles of 128 x 128 take 0.56 us (4-bit
// weights: 0.8 us) for 64 contracted elements and round of the card, and for 16-bit weights no less
// than the stream at 4.3 TB/s.
// With both sides in 4 bits tiles take 0.64 us for 256 contracted elements and round, and no less
// than the stream at 4.3 TB/s: a fifth of what tiles with converted weights take, so that streaming
// pays only while it is short of workgroups as well.  It then takes 1.15 to 3.8 us for 1024
// contracted elements, by rows and form, or 0.12 to 0.18 us for a million weights.
// Measured, streaming against tiles, us:     16-bit         4-bit weights   both sides in 4 bits
//   2048 x 2048, 16 rows                                                    7.6   8.2
//   4096 x 4096, 16 rows                     8.9   36.9     9.5   44.4      10.0  13.0
//   4096 x 4096, 64 rows                     20.6  38.3     17.7  44.4      20.1  13.3
//   4096 x 4096, 256 rows                    68.4  38.6     37.9  44.5      39.7  13.8
//   8192 x 1024, 128 rows                    26.9  68.5     20.1  84.7      21.5  22.9
//   5120 x 13824, 64 rows                    75.4  49.2     46.0  55.4      49.5  18.1
//   8 of 5120 x 13824, 16 rows each          261   266      113   246       107   92
//   64 of 4096 x 1024, 16 rows each          108   128      55.6  71.5      55.0  27.9
inline bool few_rows(sgmv_dev::Mode M, int32_t n, int32_t G, bool grouped, int32_t h_in, int32_t h_out) {
  const double met = std::min(n, G), weights = 1e-6 * h_in * h_out;
  const auto tiles = [&](double B) { return G == 1 ? std::ceil(n / B) : std::max(met, n / B + met / 2); };
  const bool small = n <= 16 * met;
  const double tiles128 = tiles(128) * std::ceil(h_out / 128.0), steps = h_in / 64.0;
  if (M == sgmv_dev::kMxBoth) {
    const Launch L = skinny_launch(n, G, grouped, h_out, true);
    const double length = L.waves == 8 ? (small ? 1.15 : 2.0) * std::max(1.0, L.workgroups / 256.0)
                                       : (small ? 1.6 : 3.8);
    const double million = small ? 0.12 + 0.004 * n / met : 0.26;
    return 4.5 + std::max(length * h_in / 1024, tiles(32) * weights * million) <
           std::max(3.5 + 0.16 * steps * std::max(1.0, tiles128 / 320), met * weights * 0.53 / 4.3);
  }
  const bool mx = M == sgmv_dev::kMxW;
  const double stream = 8 + tiles(32) * weights * (mx ? (small ? 0.17 : 0.26) : (small ? 0.38 : 0.5));
  const double tiled = mx ? 0.8 * steps * std::max(1.0, tiles128 / 320)
                          : std::max(0.56 * steps * std::max(1.0, tiles128 / 512), met * weights * 2 / 4.3);
  return stream < tiled;
}

// Tile size.  256 x 256 (one workgroup to a CU) runs full tiles at 1.3 times the rate of
// 128 x 128 (two to a CU; 8192^3, bfloat16: 1470 and 1150 TFLOP/s), but wastes more where groups
// or columns end and needs four times the tiles' room to fill the card.  What counts is rounds of
// the 256 CUs: a round of 128 x 128 tiles takes 0.64 to 0.75 of one of 256 x 256 (measured at
// 8 groups of 256 to 1024 rows).  A group's last tile is taken to be half full.
constexpr int kCus = 256;

inline bool big_tiles(double tiles256, double tiles128) {
  return std::ceil(tiles256 / kCus) <= 0.7 * std::ceil(tiles128 / (2 * kCus));
}

// With 4-bit weights there is room for 128 rows x 256 columns, two workgroups to a CU: half as much
// of a group's last tile is empty, and each weight is still turned into 16 bits only once for 128
// rows.  For 64 stages (4096 contracted elements) a CU takes 118 us for a tile of 256 x 256, 67 us
// for one of 128 x 256 and 54 us for one of 128 x 128, whether one or two of the latter run
// together.  Measured with each: 8 groups of 192 rows, 4096 x 8192, 126 us against 165 with
// 128 x 128; of 256 rows, 133 against 127 with 256 x 256; 64 groups of 384 rows, 4096 x 1024, 225
// against 257; one of 1024 rows, 4096 x 4096, 69 against 57 with 128 x 128, of 2048 rows 77
// against 106.
template <typename F>
int mx_tile(F tiles) {
  const auto time = [](double one, double n) { return one * std::ceil(n / kCus); };
  const double big = time(1, tiles(256, 256)), half = time(0.57, tiles(128, 256)),
               small = time(0.46, tiles(128, 128));
  return big <= std::min(half, small) ? 0 : half < small ? 1 : 2;
}

// The product of rows with weights of their group (not kDw): row tiles of every group, and of the
// rows of none, times column tiles.
inline Launch rows_launch(sgmv_dev::Mode M, int32_t n, int32_t G, bool grouped, int32_t h_in, int32_t h_out) {
  const bool mx = M == sgmv_dev::kMxW || M == sgmv_dev::kMxBoth;
  if (M != sgmv_dev::kDx && few_rows(M, n, G, grouped, h_in, h_out)) return skinny_launch(n, G, grouped, h_out, mx);
  const int32_t out = M == sgmv_dev::kDx ? h_in : h_out;
  const auto expected = [&](int BR, int BC) {
    const double rows = n;
    return (grouped ? rows / BR + 0.5 * std::min(n, G) : std::ceil(rows / BR)) * tiles_of(out, BC);
  };
  int rows = 128, cols = 128;
  if (M == sgmv_dev::kMxW) {
    const int tile = mx_tile(expected);
    rows = tile == 0 ? 256 : 128;
    cols = tile == 2 ? 128 : 256;
  } else if (big_tiles(expected(256, 256), expected(128, 128))) {
    rows = cols = 256;
  }
  const int64_t tiles = max_row_tiles(n, G, grouped, rows) * tiles_of(out, cols);
  return {rows, cols, rows == 256 ? 8 : 4, tiles_of(tiles, kTileXcds) * kTileXcds};
}

// The gradient of the weights: every XCD takes an eighth of each group's tiles.
inline Launch dw_launch(int32_t G, int32_t h_in, int32_t h_out) {
  const auto tiles = [&](int B) { return static_cast<double>(G) * tiles_of(h_out, B) * tiles_of(h_in, B); };
  const int B = big_tiles(tiles(256), tiles(128)) ? 256 : 128;
  return {B, B, B == 256 ? 8 : 4, tiles_of(tiles_of(h_out, B) * tiles_of(h_in, B), kTileXcds) * kTileXcds * G};
}

}  // namespace sgmv_host
