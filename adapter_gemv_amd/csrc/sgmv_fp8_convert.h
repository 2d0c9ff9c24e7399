// 16-bit values taken to 8-bit floating point with one power of two for a block.
#pragma once

#include "sgmv_skinny.h"

namespace sgmv_dev {

typedef __attribute__((ext_vector_type(2))) short s16x2_t;

// the larger magnitude of each 16-bit half; magnitudes order like their patterns, infinity and NaN
// above all
__device__ inline uint32_t max_halves(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}
// of each half of 8 elements, and of both halves
__device__ inline uint32_t top_halves(const uint4& v) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return max_halves(max_halves(v.x & kMag, v.y & kMag), max_halves(v.z & kMag, v.w & kMag));
}
__device__ inline uint32_t top_of(uint32_t halves) { return max(halves & 0xffffu, halves >> 16); }
__device__ inline uint32_t top_of(const uint4& v) { return top_of(top_halves(v)); }

// The scale of a block whose largest magnitude has the 16 bits `top`: the least power of two,
// not below 2^-126, whose 448-fold is not below it; NaN for an infinity or a NaN.
template <int DT>
__device__ inline float block_scale(uint32_t top) {
  const float m = Elem<DT>::lo(top);
  const uint32_t b = __float_as_uint(m);
  if ((b >> 23) == 255) return __builtin_nanf("");
  // m = f * 2^p with 1 <= f < 2: 2^(p - 8) if f <= 1.75, 2^(p - 7) above
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// 8 elements divided by a power of two, as 8 codes (NaN: codes of no meaning)
template <int DT>
__device__ inline u32x2_t encode8(const uint4& v, float s) {
  s16x2_t c[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = word(v, 2 * i), b = word(v, 2 * i + 1);
    if constexpr (DT == SGMV_BF16) {
      c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c[i], __builtin_bit_cast(bf16x2_t, a), s, false);
      c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c[i], __builtin_bit_cast(bf16x2_t, b), s, true);
    } else {
      c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c[i], __builtin_bit_cast(f16x2_t, a), s, false);
      c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c[i], __builtin_bit_cast(f16x2_t, b), s, true);
    }
  }
  return {__builtin_bit_cast(uint32_t, c[0]), __builtin_bit_cast(uint32_t, c[1])};
}

// the same with codes 0 for a block whose scale is NaN
template <int DT>
__device__ inline u32x2_t encode8_finite(const uint4& v, float s) {
  const u32x2_t c = encode8<DT>(v, s);
  return s == s ? c : u32x2_t{0u, 0u};
}

}  // namespace sgmv_dev
