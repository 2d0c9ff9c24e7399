// Products of a few rows per group: the form for decode batches, bound by streaming the weight.
//
// One workgroup makes 16 * CT output columns for at most 64 rows of one group.  Its 8
// wavefronts take turns along the contracted dimension (128 bytes of every weight row at a
// time, so the workgroup walks each row in whole lines), load weight pieces straight into
// registers as first MFMA operands and the rows of x, which stay in the L2, as second ones, and
// add their sums in LDS at the end, always in the same order.  No tile is staged: a weight
// element is used once per row tile, so the LDS would only add a trip.
//
// 4-bit weights: a lane loads one block (16 bytes) of a weight row and its scale.  The block's
// four groups of 8 elements are four MFMA operands, with x taken at the same positions.
// bfloat16 holds every element times its scale exactly, so the scale goes in with the
// conversion.  float16 does for scales 2^-23 .. 2^13; where a wavefront meets another one it
// takes x apart into two bfloat16 (8 + 3 of its 11 bits) and runs that block as two exact
// bfloat16 products.
#pragma once

#include "sgmv_rows.h"

namespace sgmv_dev {

struct SkinnyArgs {
  RowTab T;
  Share share;
  const uint16_t* x;
  const char* w;             // 16-bit weights or codes
  const uint8_t* scales;
  uint16_t* y;
  int64_t ld_x, ld_y;        // elements
  int64_t w_group;           // bytes between groups of w
  int32_t h_in, h_out;
};

constexpr int kSkinnyRows = 64, kSkinnyWaves = 8;

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;

// 2^(b - 127); NaN for 255
__device__ inline float mx_scale(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7fc00000u : (b ? b << 23 : 1u << 22));
}

// 8 codes of a word times a scale, as 16-bit elements (exact in bfloat16; in float16 for scales
// in its window)
template <int DT>
__device__ inline uint4 mx_eight(uint32_t codes, float scale) {
  uint4 v;
  if constexpr (DT == SGMV_BF16) {
    v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  } else {
    v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0));
    v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1));
    v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2));
    v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3));
  }
  return v;
}

// float16 holds 0.5 .. 6 times the scale exactly
__device__ inline bool f16_holds(uint32_t b) { return b - 104u <= 36u; }

// 8 float16 values as the sum of two bfloat16 each: the upper 8 bits and what is left of them
__device__ inline void f16_split(const uint4& v, uint4* hi, uint4* lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = Elem<SGMV_F16>::lo(word(v, i)), b = Elem<SGMV_F16>::hi(word(v, i));
    const float ha = __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    const float hb = __uint_as_float(__float_as_uint(b) & 0xffff0000u);
    h[i] = Elem<SGMV_BF16>::pack(ha, hb);
    // an infinity or a NaN is its own upper part (a NaN's payload sits in the upper bits)
    const bool fa = fabsf(a) < __builtin_inff(), fb = fabsf(b) < __builtin_inff();
    l[i] = Elem<SGMV_BF16>::pack(fa ? a - ha : 0.f, fb ? b - hb : 0.f);
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <int DT, bool MX, int CT>
struct Skinny {
  static constexpr int KU = MX ? 128 : 64;   // contracted elements of a unit
  static constexpr int XL = MX ? 4 : 2;      // x loads (MFMAs per column tile) of a unit
  static constexpr int WL = MX ? 1 : 2;      // weight loads of a column tile and unit

  template <int MT>
  static __device__ void run(const SkinnyArgs& A, const RowTile& t, int c0,
                             float (*sums)[16][16 * CT + 4]) {
    constexpr int UN = MT == 4 ? 1 : 2;      // units in flight
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
    const int K = A.h_in;
    // the element of a unit at which this lane's first piece starts
    const int k_lane = MX ? 32 * kq : 8 * kq;
    constexpr int k_step = MX ? 8 : 32;      // between its x pieces
    gptr<const uint16_t> xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      xp[m] = global_ptr(A.x) + A.share.div(A.T.row(t.row0 + min(16 * m + l16, t.rows - 1))) * A.ld_x + k_lane;
    gptr<const char> wp[CT];
    gptr<const uint8_t> sp[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int64_t col = min(c0 + 16 * c + l16, A.h_out - 1);
      const char* base = A.w + t.g * A.w_group;
      wp[c] = global_ptr(base) + (MX ? col * (K / 2) + 16 * kq : 2 * col * K + 16 * kq);
      if (MX) sp[c] = global_ptr(A.scales) + t.g * (A.w_group / 16) + col * (K / 32) + kq;
    }
    f32x4_t acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    uint4 xv[UN][MT][XL], wv[UN][CT][WL];
    uint32_t sv[UN][CT];
    // pieces past the row's end are zeros in both operands; their address is the row's start
    auto load = [&](int u, int unit, bool masked) {
      const int k0 = unit * KU;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int i = 0; i < WL; ++i) {
          const bool in = !masked || k0 + k_lane + i * 32 < K;
          const int64_t off = MX ? k0 / 2 : 2 * (k0 + 32 * i);
          const uint4 v = ld16((gptr<const uint16_t>)(wp[c] + (in ? off : -16 * kq)));
          wv[u][c][i] = in ? v : zero4();
        }
        if (MX) {
          const bool in = !masked || k0 + k_lane < K;
          const uint32_t b = sp[c][in ? k0 / 32 : -kq];
          sv[u][c] = in ? b : 127u;
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          const bool in = !masked || k0 + k_lane + i * k_step < K;
          const uint4 v = ld16(xp[m] + (in ? k0 + i * k_step : -k_lane));
          xv[u][m][i] = in ? v : zero4();
        }
    };
    auto multiply = [&](int u) {
      if constexpr (!MX) {
#pragma unroll
        for (int i = 0; i < XL; ++i)
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][c] = Elem<DT>::mfma(wv[u][c][i], xv[u][m][i], acc[m][c]);
      } else {
        bool fits = true;
        if constexpr (DT == SGMV_F16) {
          bool ok = true;
#pragma unroll
          for (int c = 0; c < CT; ++c) ok &= f16_holds(sv[u][c]);
          fits = __all(ok);
        }
        if (fits) {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const float s = mx_scale(sv[u][c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 e = mx_eight<DT>(word(wv[u][c][0], i), s);
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[m][c] = Elem<DT>::mfma(e, xv[u][m][i], acc[m][c]);
            }
          }
        } else {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 hi, lo;
              f16_split(xv[u][m][i], &hi, &lo);
#pragma unroll
              for (int c = 0; c < CT; ++c) {
                const uint4 e = mx_eight<SGMV_BF16>(word(wv[u][c][0], i), mx_scale(sv[u][c]));
                acc[m][c] = Elem<SGMV_BF16>::mfma(e, hi, acc[m][c]);
                acc[m][c] = Elem<SGMV_BF16>::mfma(e, lo, acc[m][c]);
              }
            }
        }
      }
    };
    const int whole = K / KU, units = (K + KU - 1) / KU;
    int u = w;
    for (; u + (UN - 1) * kSkinnyWaves < whole; u += UN * kSkinnyWaves) {
#pragma unroll
      for (int i = 0; i < UN; ++i) load(i, u + i * kSkinnyWaves, false);
#pragma unroll
      for (int i = 0; i < UN; ++i) multiply(i);
    }
    for (; u < units; u += kSkinnyWaves) {
      load(0, u, true);
      multiply(0);
    }

    // sums of the wavefronts, 16 rows at a time
    constexpr int COLS = 16 * CT;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m) __syncthreads();
#pragma unroll
      for (int c = 0; c < CT; ++c)
        *reinterpret_cast<f32x4_t*>(&sums[w][l16][16 * c + 4 * kq]) = acc[m][c];
      __syncthreads();
      for (int i = tid; i < 16 * COLS; i += 64 * kSkinnyWaves) {
        const int r = i / COLS, c = i % COLS;
        if (16 * m + r < t.rows && c0 + c < A.h_out) {
          float s = 0.f;
#pragma unroll
          for (int v = 0; v < kSkinnyWaves; ++v) s += sums[v][r][c];
          A.y[A.T.row(t.row0 + 16 * m + r) * A.ld_y + c0 + c] =
              static_cast<uint16_t>(Elem<DT>::pack(s, 0.f));
        }
      }
    }
  }
};

template <int DT, bool MX, int CT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(SkinnyArgs A) {
  __shared__ __attribute__((aligned(16))) float sums[kSkinnyWaves][16][16 * CT + 4];
  const int ct = (A.h_out + 16 * CT - 1) / (16 * CT);
  const TileList list(A.T, kSkinnyRows);
  const int m = blockIdx.x / ct, c0 = (blockIdx.x - m * ct) * 16 * CT;
  if (m >= list.count) return;
  const RowTile t = list.find(m);
  if (t.g == A.T.G) {  // rows of no group
    for (int i = threadIdx.x; i < t.rows * 16 * CT; i += blockDim.x) {
      const int c = c0 + i % (16 * CT);
      if (c < A.h_out) A.y[A.T.row(t.row0 + i / (16 * CT)) * A.ld_y + c] = 0;
    }
    return;
  }
  using S = Skinny<DT, MX, CT>;
  if (t.rows <= 16) S::template run<1>(A, t, c0, sums);
  else if (t.rows <= 32) S::template run<2>(A, t, c0, sums);
  else S::template run<4>(A, t, c0, sums);
}

// column tiles of a workgroup: few enough for two workgroups to a CU where the product has
// them, otherwise more, which share the reads of x
template <int DT, bool MX>
hipError_t launch_skinny(hipStream_t s, const SkinnyArgs& A, int64_t row_tiles) {
  constexpr int WIDE = MX ? 4 : 2;
  const int wide = (A.h_out + 16 * WIDE - 1) / (16 * WIDE);
  // row tiles that hold rows: at most the groups and the rows
  if (row_tiles * wide >= 512) {
    skinny_kernel<DT, MX, WIDE><<<static_cast<uint32_t>(row_tiles * wide), 64 * kSkinnyWaves, 0, s>>>(A);
  } else {
    const int64_t grid = row_tiles * ((A.h_out + 15) / 16);
    skinny_kernel<DT, MX, 1><<<static_cast<uint32_t>(grid), 64 * kSkinnyWaves, 0, s>>>(A);
  }
  return hipGetLastError();
}

}  // namespace sgmv_dev
