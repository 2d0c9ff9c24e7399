// Group tables on the device, shared by the grouped products (sgmv_group.hip) and the products
// with microscaled 4-bit weights (sgmv_mx.hip).
#pragma once

#include "sgmv_device.h"
#include "sgmv_rules.h"

namespace sgmv_dev {

// Rows of a batch by group: rows perm[starts[g] .. starts[g+1]) belong to group g, rows
// perm[starts[G] .. n) to none.  starts == nullptr: one group of n rows in caller order.
struct RowTab {
  const int32_t* starts;
  const int32_t* perm;
  int32_t n, G;
  __device__ int row(int j) const { return perm ? perm[j] : j; }
};

// i / share for 0 <= i < 2^31 / share by a multiplication: m = ceil(2^32 / share) is off by
// less than share / 2^32, so the product's high word is exact below 2^32 / share (the host
// checks n * share)
struct Share {
  uint32_t m;    // 0 for share == 1
  uint32_t one;  // all bits for share == 1
  __device__ int div(int i) const { return m ? static_cast<int>(__umulhi(i, m)) : i; }
  // the same without a branch
  __device__ int div_any(int i) const { return static_cast<int>(__umulhi(i, m) | (i & one)); }
};

// `rows` positions of the tables from `row0` on, all of group g (G: of no group)
struct RowTile {
  int g, row0, rows;
};

// inclusive sum over the lanes of a wavefront
__device__ inline int wave_scan(int v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(v, d);
    if ((threadIdx.x & 63) >= d) v += u;
  }
  return v;
}

// The row tiles of all groups, at most BM rows each, counted and found by one wavefront: 64
// groups at a time, one to a lane.  A group's tiles stand together, the rows of no group behind
// them all.  Everything returned is uniform.
struct TileList {
  RowTab T;
  int BM;
  int count;
  int first, len, incl;  // this lane's group of the first 64, and its inclusive tile count

  // tiles of group g (G: the rows of none)
  __device__ int tiles(int g, int* f, int* l) const {
    int a = 0, b = 0;
    if (g <= T.G) {
      a = T.starts[g];
      b = g < T.G ? T.starts[g + 1] : T.n;
    }
    *f = a;
    *l = b - a;
    return (b - a + BM - 1) / BM;
  }

  __device__ TileList(const RowTab& t, int bm) : T(t), BM(bm) {
    if (!T.starts) {
      count = (T.n + BM - 1) / BM;
      return;
    }
    const int lane = threadIdx.x & 63;
    incl = wave_scan(tiles(lane, &first, &len));
    count = __builtin_amdgcn_readlane(incl, 63);
    for (int g0 = 64; g0 <= T.G; g0 += 64) {
      int f, l;
      count += __builtin_amdgcn_readlane(wave_scan(tiles(g0 + lane, &f, &l)), 63);
    }
  }

  __device__ RowTile find(int m) const {
    if (!T.starts) return {0, m * BM, min(BM, T.n - m * BM)};
    const int lane = threadIdx.x & 63;
    int f = first, l = len, in = incl, before = 0;
    for (int g0 = 0; g0 <= T.G; g0 += 64) {
      if (g0) in = wave_scan(tiles(g0 + lane, &f, &l));
      const uint64_t past = __ballot(before + in > m);
      if (past) {
        const int who = __builtin_ctzll(past);
        const int gf = __builtin_amdgcn_readlane(f, who), gl = __builtin_amdgcn_readlane(l, who);
        const int at = m - (before + __builtin_amdgcn_readlane(in, who) - (gl + BM - 1) / BM);
        return {g0 + who, gf + at * BM, min(BM, gl - at * BM)};
      }
      before += __builtin_amdgcn_readlane(in, 63);
    }
    return {T.G, 0, 0};
  }
};

}  // namespace sgmv_dev

namespace sgmv_host {

inline sgmv_dev::Share share_of(int32_t share) {
  if (share == 1) return {0u, ~0u};
  return {static_cast<uint32_t>(((uint64_t(1) << 32) + share - 1) / static_cast<uint64_t>(share)), 0u};
}

}  // namespace sgmv_host
