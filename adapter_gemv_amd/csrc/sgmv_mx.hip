// Microscaled 4-bit floating point: 16-bit values to the format and back, and products with
// weights (and rows) held in it.
#include <type_traits>

#include "sgmv_skinny.h"
#include "sgmv_tile.h"

using namespace sgmv_dev;
using namespace sgmv_host;

namespace {

constexpr int kMxBlock = 32;

// Both kernels move every byte once and are bound by that: four lanes to a block of 32, 8
// elements (16 bytes of values, 4 of codes) each, so a wavefront's accesses are whole lines, and
// kMxPer pieces a thread, all loads first.  Rows without gaps are one long row (no division).
constexpr int kMxPer = 4;

struct MxSpan {
  int64_t pieces, per_row, ld;  // pieces of 8 elements; elements between rows
  // the first element of piece i of a strided matrix
  __device__ int64_t at(int64_t i) const {
    if (per_row == 0) return 8 * i;
    const int64_t row = i / per_row;
    return row * ld + 8 * (i - row * per_row);
  }
};

// The scale byte of a block whose largest magnitude has the bits `top` (the magnitudes' patterns
// order like the magnitudes, with infinity and NaN above them all): the exponent of
// 2^(floor(log2) - 2) with bias 127, at least 0.
template <int DT>
__device__ inline uint32_t mx_scale_byte(uint32_t top) {
  if constexpr (DT == SGMV_BF16) {
    const int e = static_cast<int>(top >> 7);  // subnormals: below 2^-126, so 0 as well
    return static_cast<uint32_t>(max(e - 2, 0));
  } else {
    const uint32_t e = top >> 10;
    if (e) return e + 110;
    return top ? 101 + 31 - __builtin_clz(top) : 0;
  }
}

template <int DT>
__device__ inline uint32_t mx_encode8(const uint4& v, float scale) {
  uint32_t c = 0;
  if constexpr (DT == SGMV_BF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.x), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.y), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.z), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.w), scale, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.x), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.y), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.z), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, v.w), scale, 3);
  }
  return c;
}

// the larger of each 16-bit half
__device__ inline uint32_t max_halves(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}

template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales,
                                                          const uint16_t* __restrict__ x, MxSpan S) {
  constexpr uint32_t kMag = 0x7fff7fffu, kInf = DT == SGMV_BF16 ? 0x7f80u : 0x7c00u;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kMxPer) + threadIdx.x;
  uint4 v[kMxPer];
#pragma unroll
  for (int u = 0; u < kMxPer; ++u) v[u] = ld16(x + S.at(min(i0 + 256 * u, S.pieces - 1)));
#pragma unroll
  for (int u = 0; u < kMxPer; ++u) {
    const int64_t i = i0 + 256 * u;
    uint32_t top = max_halves(max_halves(v[u].x & kMag, v[u].y & kMag), max_halves(v[u].z & kMag, v[u].w & kMag));
    top = max(top & 0xffffu, top >> 16);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2)));
    const bool finite = top < kInf;
    const uint32_t b = finite ? mx_scale_byte<DT>(top) : 255u;
    const uint32_t c = mx_encode8<DT>(v[u], mx_scale(finite ? b : 127u));
    if (i < S.pieces) {  // the pieces are a multiple of 4: a block's lanes go together
      codes[i] = finite ? c : 0u;
      if ((i & 3) == 0) scales[i / 4] = static_cast<uint8_t>(b);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(uint16_t* __restrict__ y,
                                                            const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, MxSpan S) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kMxPer) + threadIdx.x;
  uint32_t w[kMxPer], b[kMxPer];
#pragma unroll
  for (int u = 0; u < kMxPer; ++u) {
    const int64_t i = min(i0 + 256 * u, S.pieces - 1);
    w[u] = codes[i];
    b[u] = scales[i / 4];
  }
#pragma unroll
  for (int u = 0; u < kMxPer; ++u) {
    const int64_t i = i0 + 256 * u;
    // exact in bfloat16; rounded to nearest even where float16 does not hold the value
    const uint4 v = mx_eight<DT>(w[u], mx_scale(b[u]));
    const uint32_t out[4] = {v.x, v.y, v.z, v.w};
    if (i < S.pieces) store_words<4>(y + S.at(i), out);
  }
}

inline MxSpan mx_span(int64_t rows, int32_t h, int64_t ld) {
  return {rows * (h / 8), rows == 1 || ld == h ? 0 : h / 8, ld};
}
inline uint32_t mx_grid(const MxSpan& S) {
  return static_cast<uint32_t>((S.pieces + 256 * kMxPer - 1) / (256 * kMxPer));
}

constexpr int64_t kMxMost = (int64_t(1) << 24) - 1;  // workgroups of 256 threads in a grid

inline int check_mx_rows(int64_t rows, int32_t h, int64_t ld) {
  if (rows < 0 || rows > kMxMost * (256 * kMxPer * 8) / h) return SGMV_ERR_SHAPE;
  if (h % kMxBlock != 0 || ld % 8 != 0) return SGMV_ERR_ALIGNMENT;
  return h < kMxBlock || h > kMaxDim || ld < h ? SGMV_ERR_SHAPE : SGMV_OK;
}

inline size_t rows_bytes16(int64_t rows, int64_t ld, int32_t h) {
  return rows <= 0 ? 0 : 2 * (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(h));
}

}  // namespace

extern "C" int sgmv_mx_quantize(hipStream_t stream, int32_t dtype, void* codes, void* scales,
                                const void* x, int64_t ld_x, int64_t rows, int32_t h) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (h < 1) return SGMV_ERR_SHAPE;
  if (int st = check_mx_rows(rows, h, ld_x)) return st;
  if (rows == 0) return SGMV_OK;
  if (!codes || !scales || !x) return SGMV_ERR_NULL;
  if (!aligned16(codes) || !aligned8(scales) || !aligned16(x)) return SGMV_ERR_ALIGNMENT;
  const size_t elems = static_cast<size_t>(rows) * h, x_bytes = rows_bytes16(rows, ld_x, h);
  if (ranges_overlap(codes, elems / 2, x, x_bytes) || ranges_overlap(scales, elems / 32, x, x_bytes) ||
      ranges_overlap(codes, elems / 2, scales, elems / 32))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const MxSpan S = mx_span(rows, h, ld_x);
  auto* c = static_cast<uint32_t*>(codes);
  auto* s = static_cast<uint8_t*>(scales);
  auto* p = static_cast<const uint16_t*>(x);
  if (dtype == SGMV_F16) mx_quantize_kernel<SGMV_F16><<<mx_grid(S), 256, 0, stream>>>(c, s, p, S);
  else mx_quantize_kernel<SGMV_BF16><<<mx_grid(S), 256, 0, stream>>>(c, s, p, S);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_mx_dequantize(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y,
                                  const void* codes, const void* scales, int64_t rows, int32_t h) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (h < 1) return SGMV_ERR_SHAPE;
  if (int st = check_mx_rows(rows, h, ld_y)) return st;
  if (rows == 0) return SGMV_OK;
  if (!codes || !scales || !y) return SGMV_ERR_NULL;
  if (!aligned16(codes) || !aligned8(scales) || !aligned16(y)) return SGMV_ERR_ALIGNMENT;
  const size_t elems = static_cast<size_t>(rows) * h, y_bytes = rows_bytes16(rows, ld_y, h);
  if (ranges_overlap(codes, elems / 2, y, y_bytes) || ranges_overlap(scales, elems / 32, y, y_bytes))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const MxSpan S = mx_span(rows, h, ld_y);
  auto* c = static_cast<const uint32_t*>(codes);
  auto* s = static_cast<const uint8_t*>(scales);
  auto* p = static_cast<uint16_t*>(y);
  if (dtype == SGMV_F16) mx_dequantize_kernel<SGMV_F16><<<mx_grid(S), 256, 0, stream>>>(p, c, s, S);
  else mx_dequantize_kernel<SGMV_BF16><<<mx_grid(S), 256, 0, stream>>>(p, c, s, S);
  return hip_status(hipGetLastError());
}

namespace {

// the checks that both products share; 0 when fine (n may be 0)
inline int check_mx_product(int32_t dtype, const void* y, int64_t ld_y, int32_t share,
                            const void* W_codes, const void* W_scales, const int32_t* starts,
                            const int32_t* perm, int32_t n, int32_t G, int32_t h_in,
                            int32_t h_out) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  int st;
  if ((st = check_groups(n, G, share, starts, perm)) || (st = check_dim(h_out, ld_y))) return st;
  if (h_in < 1) return SGMV_ERR_SHAPE;
  if ((st = check_mx_rows(0, h_in, h_in))) return st;
  if (n == 0) return SGMV_OK;
  if (!y || !W_codes || !W_scales) return SGMV_ERR_NULL;
  if (!aligned16(y) || !aligned16(W_codes) || !aligned8(W_scales)) return SGMV_ERR_ALIGNMENT;
  const size_t y_bytes = matrix_bytes(n, ld_y, h_out), elems = static_cast<size_t>(G) * h_in * h_out;
  if (over_tables(y, y_bytes, starts, perm, n, G) || ranges_overlap(y, y_bytes, W_codes, elems / 2) ||
      ranges_overlap(y, y_bytes, W_scales, elems / 32))
    return SGMV_ERR_ALIAS;
  return SGMV_OK;
}

}  // namespace

extern "C" int sgmv_mx_matmul(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y,
                              const void* x, int64_t ld_x, int32_t share, const void* W_codes,
                              const void* W_scales, const int32_t* starts, const int32_t* perm,
                              int32_t n, int32_t n_groups, int32_t h_in, int32_t h_out) {
  int st = check_mx_product(dtype, y, ld_y, share, W_codes, W_scales, starts, perm, n, n_groups, h_in,
                            h_out);
  if (st || (st = check_dim(h_in, ld_x))) return st;
  if (n == 0) return SGMV_OK;
  if (!x) return SGMV_ERR_NULL;
  if (!aligned16(x)) return SGMV_ERR_ALIGNMENT;
  if (ranges_overlap(y, matrix_bytes(n, ld_y, h_out), x, matrix_bytes(shared_rows(n, share), ld_x, h_in)))
    return SGMV_ERR_ALIAS;
  const Launch L = rows_launch(kMxW, n, n_groups, starts, h_in, h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if ((st = check_device())) return st;
  if (L.rows == kSkinnyRows) {
    SkinnyArgs S{};
    S.T = {starts, perm, n, n_groups};
    S.share = share_of(share);
    S.x = static_cast<const uint16_t*>(x);
    S.w = static_cast<const char*>(W_codes);
    S.scales = static_cast<const uint8_t*>(W_scales);
    S.y = static_cast<uint16_t*>(y);
    S.ld_x = ld_x, S.ld_y = ld_y, S.w_group = static_cast<int64_t>(h_in) * h_out / 2;
    S.h_in = h_in, S.h_out = h_out;
    return hip_status(launch_skinny<true, false>(dtype, stream, S));
  }
  TileArgs A{};
  A.T = {starts, perm, n, n_groups};
  A.share = share_of(share);
  A.r = static_cast<const char*>(x);
  A.c = static_cast<const char*>(W_codes);
  A.c_scale = static_cast<const uint8_t*>(W_scales);
  A.out = static_cast<uint16_t*>(y);
  A.ld_r = 2 * ld_x, A.ld_c = h_in / 2, A.ld_out = ld_y;
  A.c_group = static_cast<int64_t>(h_in) * h_out / 2;
  A.cols = h_out, A.depth = 2 * h_in;
  return hip_status(launch_tiles<kMxW>(dtype, stream, A, L));
}

extern "C" int sgmv_mx_matmul_quantized(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y,
                                        const void* x_codes, const void* x_scales, int32_t share,
                                        const void* W_codes, const void* W_scales,
                                        const int32_t* starts, const int32_t* perm, int32_t n,
                                        int32_t n_groups, int32_t h_in, int32_t h_out) {
  int st = check_mx_product(dtype, y, ld_y, share, W_codes, W_scales, starts, perm, n, n_groups, h_in,
                            h_out);
  if (st || n == 0) return st;
  if (!x_codes || !x_scales) return SGMV_ERR_NULL;
  if (!aligned16(x_codes) || !aligned8(x_scales)) return SGMV_ERR_ALIGNMENT;
  const size_t y_bytes = matrix_bytes(n, ld_y, h_out);
  const size_t elems = static_cast<size_t>(shared_rows(n, share)) * h_in;
  if (ranges_overlap(y, y_bytes, x_codes, elems / 2) || ranges_overlap(y, y_bytes, x_scales, elems / 32))
    return SGMV_ERR_ALIAS;
  const Launch L = rows_launch(kMxBoth, n, n_groups, starts, h_in, h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if ((st = check_device())) return st;
  if (L.rows == kSkinnyRows) {
    SkinnyArgs S{};
    S.T = {starts, perm, n, n_groups};
    S.share = share_of(share);
    S.x = static_cast<const uint16_t*>(x_codes);
    S.x_scales = static_cast<const uint8_t*>(x_scales);
    S.w = static_cast<const char*>(W_codes);
    S.scales = static_cast<const uint8_t*>(W_scales);
    S.y = static_cast<uint16_t*>(y);
    S.ld_y = ld_y, S.w_group = static_cast<int64_t>(h_in) * h_out / 2;
    S.h_in = h_in, S.h_out = h_out;
    return hip_status(launch_skinny<true, true>(dtype, stream, S));
  }
  TileArgs A{};
  A.T = {starts, perm, n, n_groups};
  A.share = share_of(share);
  A.r = static_cast<const char*>(x_codes);
  A.c = static_cast<const char*>(W_codes);
  A.r_scale = static_cast<const uint8_t*>(x_scales);
  A.c_scale = static_cast<const uint8_t*>(W_scales);
  A.out = static_cast<uint16_t*>(y);
  A.ld_r = h_in / 2, A.ld_c = h_in / 2, A.ld_out = ld_y;
  A.c_group = static_cast<int64_t>(h_in) * h_out / 2;
  A.cols = h_out, A.depth = h_in / 2;
  return hip_status(h_in % 256 == 0 ? launch_tiles<kMxBoth, true>(dtype, stream, A, L)
                                    : launch_tiles<kMxBoth, false>(dtype, stream, A, L));
}
