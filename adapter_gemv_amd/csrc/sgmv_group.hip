// Rows grouped by an id, and the products of each group's rows with its own weight: forward,
// gradient of the rows, gradient of the weights.
#include <type_traits>

#include "sgmv_skinny.h"
#include "sgmv_tile.h"

using namespace sgmv_dev;
using namespace sgmv_host;

namespace {

// ------------------------------------------------------------------------------------
// group tables: a stable counting sort in one launch
// ------------------------------------------------------------------------------------
// Bin G takes the rows of no group.  A workgroup places a contiguous run of rows, each of its
// wavefronts a contiguous part of it (a multiple of 64).  It counts them per bin in LDS, and the
// rows before and behind its run (by itself, so that nothing is exchanged between workgroups);
// sums over (bin, wavefront) in that order, behind the rows before the run, give each wavefront
// its places.  It then places its rows 64 at a time: a row's place is its bin's next free one
// plus the number of lower lanes of the same bin, found by one ballot per bit of the bin number.
// All counts are integers, so the tables do not depend on timing.  What takes time is the
// placing, one memory access for each row.  Whole calls with 32768 rows of 64 groups: 32 us by one
// workgroup, 27 with its ids fetched eight at a time, 12 with one workgroup for 4096 rows.
constexpr int kBinSlots = 8 * (kMaxGroups + 1) + 8;  // 16 wavefronts up to 512 groups, 8 above
constexpr int kGroupRun = 4096;                      // rows of a workgroup, at least
constexpr int kGroupMost = 64;                       // workgroups
inline int group_waves(int G) { return 16 * (G + 1) <= kBinSlots ? 16 : 8; }

__global__ __launch_bounds__(1024) void group_rows_kernel(const int32_t* __restrict__ ids, int32_t n,
                                                          int32_t G, int32_t* __restrict__ perm,
                                                          int32_t* __restrict__ starts) {
  __shared__ int bins[kBinSlots];  // [wavefront][G + 1]
  __shared__ int before[kMaxGroups + 1], behind[kMaxGroups + 1];
  __shared__ int sums[16];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, waves = blockDim.x >> 6;
  const int B = G + 1;
  for (int i = tid; i < waves * B; i += blockDim.x) bins[i] = 0;
  for (int i = tid; i < B; i += blockDim.x) before[i] = behind[i] = 0;
  __syncthreads();
  // 64-bit: the last workgroups' runs may start past n
  const int run = ((n + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x) + 1023) & ~1023;
  const int first = static_cast<int>(min<int64_t>(n, static_cast<int64_t>(blockIdx.x) * run));
  const int last = static_cast<int>(min<int64_t>(n, static_cast<int64_t>(first) + run));
  const int part = run / waves;  // a multiple of 64
  const int lo = min(last, first + w * part), hi = min(last, lo + part);
  int* mine = bins + w * B;
  auto bin_of = [&](int id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(G) ? id : G; };
  // ids come eight at a time: one trip to memory for 512 rows of the wavefront
  constexpr int U = 8;
  int id[U];
  auto fetch = [&](int i0, int step, int end) {
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = ids[min(i0 + step * u, end - 1)];
  };
  for (int i0 = lo; i0 < hi; i0 += 64 * U) {
    fetch(i0 + lane, 64, hi);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 64 * u + lane < hi) atomicAdd(&mine[bin_of(id[u])], 1);
  }
  auto count = [&](int* where, int from, int to) {  // by the whole workgroup
    const int step = blockDim.x;
    for (int64_t i0 = from; i0 < to; i0 += step * U) {
      fetch(static_cast<int>(i0) + tid, step, to);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + step * u + tid < to) atomicAdd(&where[bin_of(id[u])], 1);
    }
  };
  count(before, 0, first);
  count(behind, last, n);
  __syncthreads();
  // exclusive sums over bins, then over a bin's wavefronts
  int carry = 0;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int total = 0;
    if (b < B) {
      total = before[b] + behind[b];
      for (int v = 0; v < waves; ++v) total += bins[v * B + b];
    }
    const int incl = wave_scan(total);
    if (lane == 63) sums[w] = incl;
    __syncthreads();
    int at = carry + incl - total;
    for (int v = 0; v < w; ++v) at += sums[v];
    for (int v = 0; v < waves; ++v) carry += sums[v];
    if (b < B) {
      if (blockIdx.x == 0) starts[b] = at;
      at += before[b];
      for (int v = 0; v < waves; ++v) {
        const int c = bins[v * B + b];
        bins[v * B + b] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(static_cast<uint32_t>(G));
  volatile int* next = mine;
  for (int i0 = lo; i0 < hi; i0 += 64 * U) {
    fetch(i0 + lane, 64, hi);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 64 * u + lane;
      const bool in = i < hi;
      const int b = bin_of(id[u]);
      uint64_t same = __ballot(in);
      for (int k = 0; k < bits; ++k) {
        const uint64_t set = __ballot((b >> k) & 1);
        same &= (b >> k) & 1 ? set : ~set;
      }
      if (in) {
        const int below = __popcll(same & ((uint64_t(1) << lane) - 1));
        const int base = next[b];
        perm[base + below] = i;
        // the bin's last lane moves its next free place on, after every lane read it (LDS
        // accesses of one wavefront keep their order)
        if ((same >> lane) == 1) next[b] = base + below + 1;
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

inline int check_weights(int64_t stride, int32_t h_in, int32_t h_out) {
  if (stride < static_cast<int64_t>(h_in) * h_out) return SGMV_ERR_SHAPE;
  return stride % 8 != 0 ? SGMV_ERR_ALIGNMENT : SGMV_OK;
}

}  // namespace

extern "C" int sgmv_group_rows(hipStream_t stream, const int32_t* ids, int32_t n, int32_t n_groups,
                               int32_t* perm, int32_t* starts) {
  if (n < 0 || n > kMaxGroupRows || n_groups < 1) return SGMV_ERR_SHAPE;
  if (n_groups > kMaxGroups) return SGMV_ERR_UNSUPPORTED;
  if (!starts || (n > 0 && (!ids || !perm))) return SGMV_ERR_NULL;
  const size_t row_bytes = sizeof(int32_t) * static_cast<size_t>(n);
  const size_t starts_bytes = sizeof(int32_t) * (static_cast<size_t>(n_groups) + 1);
  if (n > 0 && (ranges_overlap(perm, row_bytes, ids, row_bytes) ||
                ranges_overlap(starts, starts_bytes, ids, row_bytes) ||
                ranges_overlap(starts, starts_bytes, perm, row_bytes)))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const int grid = std::min(kGroupMost, std::max(1, n / kGroupRun));
  group_rows_kernel<<<grid, 64 * group_waves(n_groups), 0, stream>>>(ids, n, n_groups, perm, starts);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_group_matmul(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y,
                                 const void* x, int64_t ld_x, int32_t share, const void* W,
                                 int64_t W_stride, const int32_t* starts, const int32_t* perm,
                                 int32_t n, int32_t n_groups, int32_t h_in, int32_t h_out) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  int st;
  if ((st = check_groups(n, n_groups, share, starts, perm)) || (st = check_dim(h_in, ld_x)) ||
      (st = check_dim(h_out, ld_y)) || (st = check_weights(W_stride, h_in, h_out)))
    return st;
  if (n == 0) return SGMV_OK;
  if (!y || !x || !W) return SGMV_ERR_NULL;
  if (!aligned16(y) || !aligned16(x) || !aligned16(W)) return SGMV_ERR_ALIGNMENT;
  const size_t y_bytes = matrix_bytes(n, ld_y, h_out);
  if (over_tables(y, y_bytes, starts, perm, n, n_groups) ||
      ranges_overlap(y, y_bytes, x, matrix_bytes(shared_rows(n, share), ld_x, h_in)) ||
      ranges_overlap(y, y_bytes, W, pool_bytes16(n_groups, W_stride, int64_t(h_in) * h_out)))
    return SGMV_ERR_ALIAS;
  const Launch L = rows_launch(kForward, n, n_groups, starts, h_in, h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if ((st = check_device())) return st;
  if (L.rows == kSkinnyRows) {
    SkinnyArgs S{};
    S.T = {starts, perm, n, n_groups};
    S.share = share_of(share);
    S.x = static_cast<const uint16_t*>(x);
    S.w = static_cast<const char*>(W);
    S.y = static_cast<uint16_t*>(y);
    S.ld_x = ld_x, S.ld_y = ld_y, S.w_group = 2 * W_stride, S.h_in = h_in, S.h_out = h_out;
    return hip_status(launch_skinny<false, false>(dtype, stream, S));
  }
  TileArgs A{};
  A.T = {starts, perm, n, n_groups};
  A.share = share_of(share);
  A.r = static_cast<const char*>(x);
  A.c = static_cast<const char*>(W);
  A.out = static_cast<uint16_t*>(y);
  A.ld_r = 2 * ld_x, A.ld_c = 2 * static_cast<int64_t>(h_in), A.ld_out = ld_y, A.c_group = 2 * W_stride;
  A.cols = h_out, A.depth = 2 * h_in;
  return hip_status(launch_tiles<kForward>(dtype, stream, A, L));
}

extern "C" int sgmv_group_matmul_dx(hipStream_t stream, int32_t dtype, void* dx, int64_t ld_dx,
                                    const void* dy, int64_t ld_dy, const void* W, int64_t W_stride,
                                    const int32_t* starts, const int32_t* perm, int32_t n,
                                    int32_t n_groups, int32_t h_in, int32_t h_out) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  int st;
  if ((st = check_groups(n, n_groups, 1, starts, perm)) || (st = check_dim(h_in, ld_dx)) ||
      (st = check_dim(h_out, ld_dy)) || (st = check_weights(W_stride, h_in, h_out)))
    return st;
  if (n == 0) return SGMV_OK;
  if (!dx || !dy || !W) return SGMV_ERR_NULL;
  if (!aligned16(dx) || !aligned16(dy) || !aligned16(W)) return SGMV_ERR_ALIGNMENT;
  const size_t dx_bytes = matrix_bytes(n, ld_dx, h_in);
  if (over_tables(dx, dx_bytes, starts, perm, n, n_groups) ||
      ranges_overlap(dx, dx_bytes, dy, matrix_bytes(n, ld_dy, h_out)) ||
      ranges_overlap(dx, dx_bytes, W, pool_bytes16(n_groups, W_stride, int64_t(h_in) * h_out)))
    return SGMV_ERR_ALIAS;
  const Launch L = rows_launch(kDx, n, n_groups, starts, h_in, h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if ((st = check_device())) return st;
  TileArgs A{};
  A.T = {starts, perm, n, n_groups};
  A.r = static_cast<const char*>(dy);
  A.c = static_cast<const char*>(W);
  A.out = static_cast<uint16_t*>(dx);
  A.ld_r = 2 * ld_dy, A.ld_c = 2 * static_cast<int64_t>(h_in), A.ld_out = ld_dx, A.c_group = 2 * W_stride;
  A.cols = h_in, A.depth = h_out;
  return hip_status(launch_tiles<kDx>(dtype, stream, A, L));
}

extern "C" int sgmv_group_matmul_dw(hipStream_t stream, int32_t dtype, void* dW, int64_t dW_stride,
                                    const void* x, int64_t ld_x, int32_t share, const void* dy,
                                    int64_t ld_dy, const int32_t* starts, const int32_t* perm,
                                    int32_t n, int32_t n_groups, int32_t h_in, int32_t h_out) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  int st;
  if ((st = check_groups(n, n_groups, share, starts, perm)) || (st = check_dim(h_in, ld_x)) ||
      (st = check_dim(h_out, ld_dy)) || (st = check_weights(dW_stride, h_in, h_out)))
    return st;
  if (!dW || (n > 0 && (!x || !dy))) return SGMV_ERR_NULL;
  if (!aligned16(dW) || (n > 0 && (!aligned16(x) || !aligned16(dy)))) return SGMV_ERR_ALIGNMENT;
  const size_t dw_bytes = pool_bytes16(n_groups, dW_stride, int64_t(h_in) * h_out);
  if (over_tables(dW, dw_bytes, starts, perm, n, n_groups) ||
      (n > 0 && (ranges_overlap(dW, dw_bytes, x, matrix_bytes(shared_rows(n, share), ld_x, h_in)) ||
                 ranges_overlap(dW, dw_bytes, dy, matrix_bytes(n, ld_dy, h_out)))))
    return SGMV_ERR_ALIAS;
  const Launch L = dw_launch(n_groups, h_in, h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if ((st = check_device())) return st;
  TileArgs A{};
  A.T = {starts, perm, n, n_groups};
  A.share = share_of(share);
  A.r = static_cast<const char*>(dy);
  A.c = static_cast<const char*>(x);
  A.out = static_cast<uint16_t*>(dW);
  A.ld_r = 2 * ld_dy, A.ld_c = 2 * ld_x, A.ld_out = h_in, A.out_group = dW_stride;
  A.rows = h_out, A.cols = h_in;
  return hip_status(perm ? launch_tiles<kDw, true>(dtype, stream, A, L) : launch_tiles<kDw, false>(dtype, stream, A, L));
}
