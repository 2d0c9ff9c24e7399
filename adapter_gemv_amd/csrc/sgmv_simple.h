// A plain tiled product that serves every operand form of the grouped calls: 64 x 64 tiles,
// operands staged through registers into LDS 32 contracted elements at a time.
#pragma once

#include "sgmv_skinny.h"

namespace sgmv_dev {

// how an operand lies in memory: contracted dimension contiguous, contracted dimension across
// rows, or 4-bit codes with the contracted dimension contiguous
enum Form { kAlong, kAcross, kCodes };

static __constant__ uint16_t kFp4F16[8] = {0x0000, 0x3800, 0x3c00, 0x3e00, 0x4000, 0x4200, 0x4400, 0x4600};
static __constant__ uint16_t kFp4Bf16[8] = {0x0000, 0x3f00, 0x3f80, 0x3fc0, 0x4000, 0x4040, 0x4080, 0x40c0};

struct SimpleArgs {
  RowTab T;
  Share share;
  const uint16_t *r, *c;           // row and column operands
  const uint8_t *r_scale, *c_scale;
  uint16_t* out;
  int64_t ld_r, ld_c, ld_out, c_stride, out_stride;
  int32_t rows, cols, depth;       // dW only: rows; columns of the output; contracted length
};

// MODE 0: y / dx (rows gathered; a column operand per group); MODE 1: dW (contracted over rows)
template <int DT, Form RF, Form CF, int MODE>
__global__ __launch_bounds__(256) void simple_kernel(SimpleArgs A) {
  using E = Elem<DT>;
  __shared__ uint16_t rs[64][40], cs[64][40];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
  const int nt = (A.cols + 63) / 64;
  RowTile t;
  int c0, r0 = 0;
  if (MODE == 0) {
    const TileList list(A.T, 64, true);
    const int m = blockIdx.x / nt;
    if (m >= list.count) return;
    t = list.find(m);
    c0 = (blockIdx.x % nt) * 64;
  } else {
    const int rt = (A.rows + 63) / 64;
    const int g = blockIdx.x / (nt * rt), in = blockIdx.x % (nt * rt);
    t.g = g;
    if (A.T.n == 0) { t.row0 = 0; t.rows = 0; }
    else if (!A.T.starts) { t.row0 = 0; t.rows = A.T.n; }
    else { t.row0 = A.T.starts[g]; t.rows = A.T.starts[g + 1] - t.row0; }
    c0 = (in % nt) * 64;
    r0 = (in / nt) * 64;
  }
  const bool none = MODE == 0 && t.g == A.T.G;
  const int depth = none ? 0 : (MODE == 0 ? A.depth : t.rows);
  f32x4_t acc[4];
  for (int f = 0; f < 4; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int64_t cbase = MODE == 0 ? static_cast<int64_t>(t.g) * A.c_stride : 0;
  for (int k0 = 0; k0 < depth; k0 += 32) {
    __syncthreads();
    auto stage = [&](auto form, uint16_t (*dst)[40], const uint16_t* p, int64_t ld, int64_t base,
                     bool is_row) {
      constexpr Form F = decltype(form)::value;
      if constexpr (F == kAcross) {
        const int k = k0 + tid / 8, e0 = (tid & 7) * 8;
        uint4 v = zero4();
        const int first = is_row ? r0 : c0, lim = is_row ? A.rows : A.cols;
        if (k < depth && first + e0 < lim) {
          int64_t row = k;
          if (MODE == 1) {
            const int j = A.T.row(t.row0 + k);
            row = is_row ? j : A.share.div(j);
          }
          v = ld16(p + base + row * ld + first + e0);
        }
        for (int e = 0; e < 8; ++e)
          dst[e0 + e][tid / 8] = static_cast<uint16_t>(word(v, e >> 1) >> (16 * (e & 1)));
      } else {
        const int q = tid / 4, k = k0 + (tid & 3) * 8;
        int64_t row = -1;
        if (is_row) {
          if (q < t.rows) row = A.share.div(A.T.row(t.row0 + q));
        } else if (c0 + q < A.cols) {
          row = c0 + q;
        }
        uint16_t e8[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (row >= 0 && k < depth) {
          if constexpr (F == kAlong) {
            const uint4 v = ld16(p + base + row * ld + k);
            for (int e = 0; e < 8; ++e) e8[e] = static_cast<uint16_t>(word(v, e >> 1) >> (16 * (e & 1)));
          } else {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(
                reinterpret_cast<const uint8_t*>(p) + (base + row * ld + k) / 2);
            for (int e = 0; e < 8; ++e) {
              const int code = (v >> (4 * e)) & 15;
              e8[e] = (DT == SGMV_F16 ? kFp4F16 : kFp4Bf16)[code & 7] | ((code & 8) << 12);
            }
          }
        }
        for (int e = 0; e < 8; ++e) dst[q][(tid & 3) * 8 + e] = e8[e];
      }
    };
    stage(std::integral_constant<Form, RF>{}, rs, A.r, A.ld_r, 0, true);
    stage(std::integral_constant<Form, CF>{}, cs, A.c, A.ld_c, cbase, false);
    __syncthreads();
    const uint4 rv = *reinterpret_cast<const uint4*>(&rs[16 * w + l16][8 * kq]);
    float srow = 1.f;
    if (RF == kCodes) {
      const int q = 16 * w + l16;
      if (q < t.rows)
        srow = mx_scale(A.r_scale[(A.share.div(A.T.row(t.row0 + q)) * A.ld_r + k0) / 32]);
    }
    for (int f = 0; f < 4; ++f) {
      const uint4 cv = *reinterpret_cast<const uint4*>(&cs[16 * f + l16][8 * kq]);
      if constexpr (CF == kCodes) {
        const f32x4_t d = E::mfma(cv, rv, f32x4_t{0.f, 0.f, 0.f, 0.f});
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 16 * f + 4 * kq + i;
          const float s = c < A.cols ? mx_scale(A.c_scale[(cbase + c * A.ld_c + k0) / 32]) : 0.f;
          acc[f][i] += d[i] * srow * s;
        }
      } else {
        acc[f] = E::mfma(cv, rv, acc[f]);
      }
    }
  }
  const int q = 16 * w + l16;
  uint16_t* to;
  if (MODE == 0) {
    if (q >= t.rows) return;
    to = A.out + static_cast<int64_t>(A.T.row(t.row0 + q)) * A.ld_out;
  } else {
    if (r0 + q >= A.rows) return;
    to = A.out + static_cast<int64_t>(t.g) * A.out_stride + static_cast<int64_t>(r0 + q) * A.ld_out;
  }
  for (int f = 0; f < 4; ++f) {
    const int c = c0 + 16 * f + 4 * kq;
    if (c < A.cols) {
      const uint32_t o[2] = {E::pack(acc[f][0], acc[f][1]), E::pack(acc[f][2], acc[f][3])};
      store_words<2>(to + c, o);
    }
  }
}

}  // namespace sgmv_dev
