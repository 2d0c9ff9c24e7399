// Products of a few rows per group: the form for decode batches, bound by streaming the weight.
//
// One workgroup makes 16 * CT output columns for at most 32 rows of one group.  Its
// wavefronts take turns along the contracted dimension, a unit of 128 bytes of every weight row
// at a time, so the workgroup walks each row in order.  Each wavefront streams its units
// through a ring of its own in LDS, three units ahead, by direct loads whose lanes follow the
// rows' bytes (8 lanes to a row's line); loads straight into the MFMA operand's lanes, one row to
// a lane, took 98 us where the ring took 93 (4-bit, 8 experts of 5120 x 13824, 32 rows).  The
// rows of x, few and in the L2, go straight to registers one unit ahead.  Nothing is shared
// between wavefronts until they add their sums in LDS at the end, always in the same order.
//
// 4-bit weights: a unit is eight blocks of a row, each the operand of one MFMA: a lane takes 8
// elements of every block, as in the 16-bit form, so that 4 lanes read 64 bytes of x side by side
// (two whole blocks to a lane, and 16 bytes of x out of every 128 for each load: 10 % slower), and
// the scales of four units are fetched at once and dealt out between lanes.
// bfloat16 holds every element times its scale exactly for scales up to 2^125, so the scale goes
// in with the conversion.  float16 does for scales 2^-23 .. 2^13 (and for blocks of zeros); a
// workgroup that meets another one starts again with x taken apart into two bfloat16 (8 + 3 of its
// 11 bits), as two exact bfloat16 products.  With x in 4 bits too, both sides are bfloat16.  An
// element past bfloat16's range becomes an infinity, and so do the sums it is part of (or NaN): a
// workgroup with such sums looks for scales above 2^125, and computes its outputs again, another
// way, if it has one (mx_mend).
#pragma once

#include <type_traits>

#include "sgmv_rows.h"

namespace sgmv_dev {

struct SkinnyArgs {
  RowTab T;
  Share share;
  const uint16_t* x;         // 16-bit rows, or codes
  const uint8_t* x_scales;
  const char* w;             // 16-bit weights or codes
  const uint8_t* scales;
  uint16_t* y;
  int64_t ld_x, ld_y;        // elements
  int64_t w_group;           // bytes between groups of w
  int32_t h_in, h_out;
};

using sgmv_host::kSkinnyRows;

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;

// 2^(b - 127); NaN for 255
__device__ inline float mx_scale(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7fc00000u : (b ? b << 23 : 1u << 22));
}

// byte `at` of a word of scales, for mx_eight: of its scale the conversion reads the exponent's
// bits alone, as the format means them (0 is 2^-127, 255 NaN), so what stands beside them may stay
__device__ inline float mx_scale_at(uint32_t scales, int at) {
  return __uint_as_float(at == 3 ? scales >> 1 : scales << (23 - 8 * at));
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

// float16 holds these codes (or'd together) times the scale exactly
__device__ inline bool f16_holds(uint32_t b, uint32_t codes) {
  return b - 104u <= 36u || (codes & 0x77777777u) == 0;
}

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

__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) void tile_lds_void;
typedef __attribute__((address_space(1))) void tile_global_void;

// 16 bytes per lane from src into LDS at dst + 16 * lane (dst the same for the wavefront)
__device__ inline void to_lds(const char* src, u32x4_t* dst) {
  __builtin_amdgcn_global_load_lds((tile_global_void*)src, (tile_lds_void*)dst, 16, 0, 0);
}

template <int I, int N, class F>
__device__ __forceinline__ void tile_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    tile_for<I + 1, N>(f);
  }
}

// A product with 4-bit weights, for mx_any_scale
struct MxProduct {
  const RowTab& T;
  const Share& share;
  const uint16_t* x;         // 16-bit rows, or codes
  const uint8_t* x_scales;
  int64_t ld_x;              // elements (16-bit rows)
  const char* w;
  const uint8_t* scales;
  int64_t w_group;           // bytes between groups of w
  uint16_t* y;
  int64_t ld_y;
  int32_t h_in, h_out;
};

// Whether columns c0 .. c0 + cols - 1 of the tile's group (or the tile's rows of x) have a block
// whose scale, 2^126 or 2^127, may take an element past bfloat16's range.  By the whole workgroup.
template <bool XM>
__device__ __forceinline__ bool mx_past_range(const MxProduct& P, const RowTile& t, int c0, int cols) {
  const int blocks = P.h_in / 32;
  bool found = false;
  const uint8_t* const ws = P.scales + t.g * (P.w_group / 16) + static_cast<int64_t>(c0) * blocks;
  const int64_t mine = static_cast<int64_t>(min(cols, P.h_out - c0)) * blocks;
  for (int64_t i = threadIdx.x; i < mine; i += blockDim.x) found |= ws[i] - 253u <= 1u;
  if constexpr (XM) {
    for (int r = 0; r < t.rows; ++r) {
      const uint8_t* const xs = P.x_scales + P.share.div(P.T.row(t.row0 + r)) * static_cast<int64_t>(blocks);
      for (int b = threadIdx.x; b < blocks; b += blockDim.x) found |= xs[b] - 253u <= 1u;
    }
  }
  return __syncthreads_or(found);
}

// The outputs of a row tile's columns c0 .. c0 + cols - 1 for scales of any size, by the whole
// workgroup: an output to a thread, every block summed as if its scale were 2^-8 (no sum of 32
// products then passes float32) and scaled after.  Slow (every operand read again and again), for
// values past 2^127, which no weight of a model has.
template <int DT, bool XM>
__device__ __forceinline__ void mx_any_scale(const MxProduct& P, const RowTile& t, int c0, int cols) {
  const int blocks = P.h_in / 32;
  for (int i = threadIdx.x; i < t.rows * cols; i += blockDim.x) {
    const int c = c0 + i % cols;
    if (c >= P.h_out) continue;
    const int row = P.T.row(t.row0 + i / cols), of = P.share.div(row);
    const char* const w = P.w + t.g * P.w_group + static_cast<int64_t>(c) * (P.h_in / 2);
    const uint8_t* const ws = P.scales + t.g * (P.w_group / 16) + static_cast<int64_t>(c) * blocks;
    const uint16_t* const x = P.x + of * (XM ? static_cast<int64_t>(P.h_in) / 4 : P.ld_x);
    float acc = 0.f;
    for (int b = 0; b < blocks; ++b) {
      int power = ws[b] - 127 + 8;
      bool nan = ws[b] == 255;
      if constexpr (XM) {
        const uint32_t xb = P.x_scales[of * static_cast<int64_t>(blocks) + b];
        power += static_cast<int>(xb) - 127;
        nan |= xb == 255;
      }
      float sum = 0.f;
      for (int k = 0; k < 4; ++k) {
        const uint32_t codes = reinterpret_cast<const uint32_t*>(w)[4 * b + k];
        const uint4 v = mx_eight<SGMV_BF16>(codes, 0x1p-8f);
        const uint4 u = XM ? mx_eight<SGMV_BF16>(reinterpret_cast<const uint32_t*>(x)[4 * b + k], 1.f)
                           : ld16(x + 32 * b + 8 * k);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          using X = Elem<XM ? SGMV_BF16 : DT>;
          sum = fmaf(Elem<SGMV_BF16>::lo(word(v, h)), X::lo(word(u, h)), sum);
          sum = fmaf(Elem<SGMV_BF16>::hi(word(v, h)), X::hi(word(u, h)), sum);
        }
      }
      acc += nan ? __builtin_nanf("") : ldexpf(sum, power);
    }
    P.y[row * P.ld_y + c] = static_cast<uint16_t>(Elem<DT>::pack(acc, 0.f));
  }
}

// After a workgroup wrote its outputs, `finite` telling whether each thread's sums were: where some
// were not, because an element passed bfloat16's range, they are computed again.  The test at the
// end costs less than a hundredth of a call; looking at every scale in the loop cost bfloat16
// decode batches 1.5 to 3.5 hundredths.
template <int DT, bool XM>
__device__ __forceinline__ void mx_mend(const MxProduct& P, const RowTile& t, int c0, int cols, bool finite) {
  if (!__syncthreads_and(finite) && mx_past_range<XM>(P, t, c0, cols)) mx_any_scale<DT, XM>(P, t, c0, cols);
}

// XM: x in 4 bits (its rows dense), DT the type of y alone
template <int DT, bool MX, bool XM, int CT, int WAVES>
struct Skinny {
  static_assert(MX || !XM, "");
  static constexpr int CTYPE = XM ? SGMV_BF16 : DT;  // of the products
  static constexpr int KU = MX ? 256 : 64;   // contracted elements of a unit
  static constexpr int XL = MX ? 8 : 2;      // 8-element pieces of a lane and unit
  static constexpr int D = 4;                // units of the ring
  struct Ring {
    u32x4_t v[WAVES * CT * 128];             // [wavefront][column tile][row of 16][8 pieces]
  };

  // This wavefront's part of the products, in acc.  False where float16 did not hold a weight
  // (never with SPLIT, the exact way for scales up to 2^125).
  template <int MT, bool SPLIT>
  static __device__ __forceinline__ bool multiply_rows(const SkinnyArgs& A, const RowTile& t, int c0,
                                                       f32x4_t (*acc)[CT], Ring& r0, Ring& r1, Ring& r2,
                                                       Ring& r3) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
    const int K = A.h_in, row_bytes = MX ? K / 2 : 2 * K;
    // x: the element of a unit at which this lane's first piece starts, and from one to the next
    const int k_lane = 8 * kq;
    gptr<const uint16_t> xp[MT];
    gptr<const uint8_t> xs[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = A.share.div(A.T.row(t.row0 + min(16 * m + l16, t.rows - 1)));
      xp[m] = global_ptr(A.x) + (XM ? row * (static_cast<int64_t>(K) / 4) : row * A.ld_x) + k_lane / (XM ? 4 : 1);
      if constexpr (XM) {
        const int of = A.share.div(A.T.row(t.row0 + min(16 * m + (lane / 2) % 16, t.rows - 1)));
        xs[m] = global_ptr(A.x_scales) + of * (static_cast<int64_t>(K) / 32);
      }
    }
    // weights: lane l fetches a piece of row l / 8 of 8, the one that belongs in its slot (piece c
    // of row q of 16 sits in slot c ^ ((q >> 1) & 7): no bank conflicts for the reads below)
    const char* wp[CT][2];
    int wk[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) wk[h] = 16 * ((lane & 7) ^ (((8 * h + lane / 8) >> 1) & 7));
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const char* base = A.w + t.g * A.w_group;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wp[c][h] = base + static_cast<int64_t>(min(c0 + 16 * c + 8 * h + lane / 8, A.h_out - 1)) * row_bytes + wk[h];
    }
    // scales: lane l fetches those of column l / 2 (of row (l / 2) % 16 of x) for a whole round,
    // those of its units 0 and 1 in even lanes and 2 and 3 in odd ones
    gptr<const uint8_t> sp = global_ptr(A.scales);
    if (MX) sp += t.g * (A.w_group / 16) + static_cast<int64_t>(min(c0 + lane / 2 % (16 * CT), A.h_out - 1)) * (K / 32);
    const char* const zeros = reinterpret_cast<const char*>(kZeros);
    // this wavefront's units: w, w + WAVES, ...; n of them, the row's last one partial or whole
    const int units = (K + KU - 1) / KU, n = (units - w + WAVES - 1) / WAVES;
    bool held = true;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // the i-th unit of this wavefront; past the row's end (and past the last unit) zeros
    auto fetch = [&](Ring& to, int i) __attribute__((always_inline)) {
      const int at = (w + i * WAVES) * 128;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          to_lds(at + wk[h] < row_bytes ? wp[c][h] + at : zeros, &to.v[((w * CT + c) * 2 + h) * 64]);
    };
    using Piece = std::conditional_t<XM, uint32_t, uint4>;
    struct Rows {
      Piece x[MT][XL];
    };
    struct Scales {
      uint32_t w[2][2], x[MT][2][2];  // [unit][first or last four blocks]
    };
    // a unit's eight scales from block b0; past the row's end 1
    auto eight_scales = [&](uint32_t (&to)[2], gptr<const uint8_t> from, int b0, bool masked)
        __attribute__((always_inline)) {
      if (!masked || K % KU == 0) {
        __builtin_memcpy(to, (const uint8_t*)(from + (masked ? min(b0, K / 32 - 8) : b0)), 8);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          to[h] = 0;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int at = b0 + 4 * h + v;
            const uint32_t one = from[min(at, K / 32 - 1)];
            to[h] |= (at < K / 32 ? one : 127u) << (8 * v);
          }
        }
      }
    };
    // the scales of the round that starts with this wavefront's i-th unit
    auto scales_of = [&](Scales& S, int i, bool masked) __attribute__((always_inline)) {
      if constexpr (MX) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int b0 = (w + (i + 2 * (lane & 1) + u) * WAVES) * 8;
          eight_scales(S.w[u], sp, b0, masked);
          if constexpr (XM)
#pragma unroll
            for (int m = 0; m < MT; ++m) eight_scales(S.x[m][u], xs[m], b0, masked);
        }
      }
    };
    // the rows of x at the i-th unit
    auto rows_of = [&](Rows& R, int i, bool masked) __attribute__((always_inline)) {
      const int k0 = (w + i * WAVES) * KU;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int p = 0; p < XL; ++p) {
          const bool in = !masked || k0 + k_lane + 32 * p < K;
          const int at = in ? k0 + 32 * p : -k_lane;
          if constexpr (XM) {
            const uint32_t v = *reinterpret_cast<gptr<const uint32_t>>(xp[m] + at / 4);
            R.x[m][p] = in ? v : 0u;
          } else {
            const uint4 v = ld16(xp[m] + at);
            R.x[m][p] = in ? v : zero4();
          }
        }
      }
    };
    // 32-bit words of a ring: this lane's in the p-th piece (4-bit) or its two pieces (16-bit)
    const int at = (w * CT * 16 + l16) * 8, sw = (l16 >> 1) & 7;
    int slot[MX ? 8 : 2];
#pragma unroll
    for (int p = 0; p < (MX ? 8 : 2); ++p) {
      slot[p] = MX ? (at + (p ^ sw)) * 4 + kq : (at + ((4 * p + kq) ^ sw)) * 4;
      asm("" : "+v"(slot[p]));  // one lane offset: see the tiled product
    }
    // the eight scales of entry e (a column, or a row of x) at the round's unit j
    auto entry = [&](uint32_t (&to)[2], const uint32_t (&of)[2][2], int e, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) to[h] = __builtin_amdgcn_ds_bpermute(4 * (2 * e + (j >> 1)), of[j & 1][h]);
    };
    auto multiply = [&](const Ring& from, const Rows& R, const Scales& S, int unit) __attribute__((always_inline)) {
      const uint32_t* const words = reinterpret_cast<const uint32_t*>(from.v);
      if constexpr (!MX) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const u32x4_t wv = *reinterpret_cast<const u32x4_t*>(&words[slot[v] + c * 512]);
            const uint4 p = make_uint4(wv.x, wv.y, wv.z, wv.w);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][c] = Elem<DT>::mfma(p, R.x[m][v], acc[m][c]);
          }
      } else {
        uint32_t ws[CT][2], rs[MT][2], codes[CT][XL];
#pragma unroll
        for (int p = 0; p < XL; ++p)
#pragma unroll
          for (int c = 0; c < CT; ++c) codes[c][p] = words[slot[p] + c * 512];
        __builtin_amdgcn_sched_barrier(0);  // all of them first: one at a time, each was waited for
#pragma unroll
        for (int c = 0; c < CT; ++c) entry(ws[c], S.w, 16 * c + l16, unit);
        if constexpr (XM)
#pragma unroll
          for (int m = 0; m < MT; ++m) entry(rs[m], S.x[m], l16, unit);
#pragma unroll
        for (int p = 0; p < XL; ++p) {
          uint4 xv[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if constexpr (XM) xv[m] = mx_eight<SGMV_BF16>(R.x[m][p], mx_scale_at(rs[m][p / 4], p % 4));
            else xv[m] = R.x[m][p];
          }
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const uint32_t code = codes[c][p];
            const float s = mx_scale_at(ws[c][p / 4], p % 4);
            if constexpr (CTYPE == SGMV_F16 && !SPLIT) held &= f16_holds(ws[c][p / 4] >> (8 * (p % 4)) & 255u, code);
            if constexpr (SPLIT) {
              const uint4 e = mx_eight<SGMV_BF16>(code, s);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                uint4 hi, lo;
                f16_split(xv[m], &hi, &lo);
                acc[m][c] = Elem<SGMV_BF16>::mfma(e, hi, acc[m][c]);
                acc[m][c] = Elem<SGMV_BF16>::mfma(e, lo, acc[m][c]);
              }
              __builtin_amdgcn_sched_barrier(0);  // few registers, not speed
            } else {
              const uint4 e = mx_eight<CTYPE>(code, s);
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[m][c] = Elem<CTYPE>::mfma(e, xv[m], acc[m][c]);
            }
          }
        }
      }
    };
    auto ring = [&](auto k) __attribute__((always_inline)) -> Ring& {
      constexpr int j = decltype(k)::value % D;
      if constexpr (j == 0) return r0;
      else if constexpr (j == 1) return r1;
      else if constexpr (j == 2) return r2;
      else return r3;
    };
    // Rounds of D units, one to a ring buffer.  Loads of one wavefront arrive in order, so a
    // unit's weights are there once at most the loads behind them are in flight: those of three
    // units and of the rows of the next.
    static_assert(D == 4, "scales of a round");
    constexpr int W_LOADS = 2 * CT, X_LOADS = MT * XL;
    tile_for<0, D - 1>([&](auto k) __attribute__((always_inline)) { fetch(ring(k), decltype(k)::value); });
    Scales sn, sl;  // of this round and of the next
    scales_of(sn, 0, true);
    if constexpr (MT == 1 && !SPLIT) {
      Rows a, b;
      const int whole = n - (K % KU != 0 && (units - 1) % WAVES == w);
      if (n > 0) rows_of(a, 0, true);
      auto step = [&](auto k, int i, bool masked) __attribute__((always_inline)) {
        constexpr int j = decltype(k)::value;
        Rows &now = j % 2 ? b : a, &next = j % 2 ? a : b;
        if constexpr (j == 0) scales_of(sl, i + D, masked);
        if constexpr (j == D) sn = sl;
        rows_of(next, i + j + 1, masked);
        wait_reads();
        fetch(ring(std::integral_constant<int, j + D - 1>{}), i + j + D - 1);
        wait_loads<(D - 1) * W_LOADS + X_LOADS>();
        multiply(ring(k), now, sn, j % D);
      };
      constexpr int LAST = MX ? 2 * D : D + 1;  // rounds of whole units leave at most so many
      int i = 0;
      for (; i + LAST <= whole; i += D) {
        tile_for<0, D>([&](auto k) __attribute__((always_inline)) { step(k, i, false); });
        sn = sl;
      }
      tile_for<0, LAST>([&](auto k) __attribute__((always_inline)) {
        if (i + decltype(k)::value < n) step(k, i, true);
      });
    } else {  // two units' rows do not fit the registers
      Rows a;
      for (int i = 0; i < n; i += D) {
        scales_of(sl, i + D, true);
        tile_for<0, D>([&](auto k) __attribute__((always_inline)) {
          constexpr int j = decltype(k)::value;
          if (i + j < n) {
            rows_of(a, i + j, true);
            wait_reads();
            fetch(ring(std::integral_constant<int, j + D - 1>{}), i + j + D - 1);
            wait_loads<(D - 1) * W_LOADS>();
            multiply(ring(k), a, sn, j);
          }
        });
        sn = sl;
      }
    }
    wait_loads<0>();  // the last loads into LDS land before it is used again
    return held;
  }

  // at most N global loads of this wavefront are in flight
  template <int N>
  static __device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt range");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if constexpr (MX) __builtin_amdgcn_sched_barrier(0);  // a unit's use of its scales stays behind its wait
  }

  // Every LDS read of this wavefront has returned.  The buffer that a step fills is the one the
  // step before read, and a load into LDS is not held back by reads in flight.  (64 experts of
  // 4096 x 1024, 32 x 2 rows, with it: 66 to 70 us a call.)
  static __device__ __forceinline__ void wait_reads() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt 0
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }

  // false: some sum is an infinity or NaN
  template <int MT>
  static __device__ __forceinline__ bool run(const SkinnyArgs& A, const RowTile& t, int c0, Ring& r0, Ring& r1,
                                             Ring& r2, Ring& r3, float (*sums)[16][16 * CT + 4]) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
    constexpr int COLS = 16 * CT;
    f32x4_t acc[MT][CT];
    const bool held = multiply_rows<MT, false>(A, t, c0, acc, r0, r1, r2, r3);
    if constexpr (MX && CTYPE == SGMV_F16) {
      if (!__syncthreads_and(held)) multiply_rows<MT, true>(A, t, c0, acc, r0, r1, r2, r3);
    }
    float zero = 0.f;
    // sums of the wavefronts, 16 rows at a time
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m) __syncthreads();
#pragma unroll
      for (int c = 0; c < CT; ++c)
        *reinterpret_cast<f32x4_t*>(&sums[w][l16][16 * c + 4 * kq]) = acc[m][c];
      __syncthreads();
      for (int i = tid; i < 16 * COLS; i += 64 * WAVES) {
        const int r = i / COLS, c = i % COLS;
        if (16 * m + r < t.rows && c0 + c < A.h_out) {
          float s = 0.f;
#pragma unroll
          for (int v = 0; v < WAVES; ++v) s += sums[v][r][c];
          zero = fmaf(s, 0.f, zero);
          A.y[A.T.row(t.row0 + 16 * m + r) * A.ld_y + c0 + c] =
              static_cast<uint16_t>(Elem<DT>::pack(s, 0.f));
        }
      }
    }
    return zero == 0.f;
  }
};

template <int DT, bool MX, bool XM, int CT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, MX ? 2 : 4) void skinny_kernel(SkinnyArgs A) {
  using S = Skinny<DT, MX, XM, CT, WAVES>;
  __shared__ typename S::Ring r0, r1, r2, r3;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16][16 * CT + 4];
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
  const bool finite = t.rows <= 16 ? S::template run<1>(A, t, c0, r0, r1, r2, r3, sums)
                                   : S::template run<2>(A, t, c0, r0, r1, r2, r3, sums);
  if constexpr (MX)
    mx_mend<DT, XM>({A.T, A.share, A.x, A.x_scales, A.ld_x, A.w, A.scales, A.w_group, A.y, A.ld_y, A.h_in, A.h_out},
                    t, c0, 16 * CT, finite);
}

template <int DT, bool MX, bool XM, int CT, int WAVES>
hipError_t launch_skinny(hipStream_t s, const SkinnyArgs& A, const sgmv_host::Launch& L) {
  skinny_kernel<DT, MX, XM, CT, WAVES><<<static_cast<uint32_t>(L.workgroups), 64 * WAVES, 0, s>>>(A);
  return hipGetLastError();
}

template <bool MX, bool XM>
hipError_t launch_skinny(int32_t dtype, hipStream_t s, const SkinnyArgs& A) {
  const sgmv_host::Launch L = sgmv_host::skinny_launch(A.T.n, A.T.G, A.T.starts, A.h_out, MX);
  const bool f16 = dtype == SGMV_F16;
  if constexpr (!MX)
    return f16 ? launch_skinny<SGMV_F16, false, false, 1, 4>(s, A, L)
               : launch_skinny<SGMV_BF16, false, false, 1, 4>(s, A, L);
  else if (L.cols == 32)
    return f16 ? launch_skinny<SGMV_F16, true, XM, 2, 2>(s, A, L) : launch_skinny<SGMV_BF16, true, XM, 2, 2>(s, A, L);
  else
    return f16 ? launch_skinny<SGMV_F16, true, XM, 1, 8>(s, A, L) : launch_skinny<SGMV_BF16, true, XM, 1, 8>(s, A, L);
}

}  // namespace sgmv_dev
