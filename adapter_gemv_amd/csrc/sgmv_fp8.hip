// 8-bit floating point with a scale for each block of 128: 16-bit values to the format and back,
// and products with both sides in it.
#include "sgmv_fp8_rules.h"
#include "sgmv_fp8_skinny.h"

using namespace sgmv_dev;
using namespace sgmv_host;

namespace {

constexpr int kBlock = 128;

// code * scale, rounded once to the 16-bit type: the product has at most 28 bits, which float64
// holds; what float32 cuts off is kept as its last bit (no later rounding is then misled)
template <int DT>
__device__ inline float decode1(float code, float scale) {
  const double exact = static_cast<double>(code) * static_cast<double>(scale);
  float f = static_cast<float>(exact);
  if (fabsf(f) < __builtin_inff() && static_cast<double>(f) != exact) {
    uint32_t b = __float_as_uint(f);
    if (fabs(static_cast<double>(f)) > fabs(exact)) --b;  // towards zero
    f = __uint_as_float(b | 1u);
  }
  return f;
}
template <int DT>
__device__ inline uint4 decode8(u32x2_t codes, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t c = i ? codes.y : codes.x;
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
    o[2 * i] = Elem<DT>::pack(decode1<DT>(a[0], scale), decode1<DT>(a[1], scale));
    o[2 * i + 1] = Elem<DT>::pack(decode1<DT>(b[0], scale), decode1<DT>(b[1], scale));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// the largest over the 16 lanes that hold a block
__device__ inline uint32_t block_top(uint32_t top) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  return top;
}

// Rows: 16 lanes to a block, 8 elements each; a wavefront takes four blocks of a row.  The largest
// magnitude is that of the bit patterns, one integer maximum for two elements.  Memory bounds it: 16384 x
// 4096, 201 MB in 35 us (5.8 TB/s, half of it from the Infinity Cache); 1531 x 5120 in 7.4 us.
struct Fp8Rows {
  int64_t rows, ld;
  int32_t h, pitch;  // of the codes: h, or h and zeros up to a multiple of 16
  int32_t units;     // of 512 elements of a row
};
template <int DT>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                           const uint16_t* __restrict__ x, Fp8Rows R) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
  const int64_t row = i / R.units;
  if (row >= R.rows) return;
  const int lane = threadIdx.x & 63, at = static_cast<int>(i - row * R.units) * 512 + 8 * lane;
  const bool in = at < R.h;
  const uint4 v = in ? ld16(x + row * R.ld + at) : zero4();
  const float s = block_scale<DT>(block_top(top_of(v)));
  if (at >= R.pitch) return;
  *reinterpret_cast<u32x2_t*>(codes + row * R.pitch + at) = encode8_finite<DT>(v, s);
  if (!in) return;
  if (at % kBlock == 0) scales[row * blocks_of(R.h) + at / kBlock] = s;
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(uint16_t* __restrict__ y, const uint8_t* __restrict__ codes,
                                                             const float* __restrict__ scales, Fp8Rows R) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
  const int64_t row = i / R.units;
  const int at = static_cast<int>(i - row * R.units) * 512 + 8 * (threadIdx.x & 63);
  if (row >= R.rows || at >= R.h) return;
  const uint4 v = decode8<DT>(*reinterpret_cast<const u32x2_t*>(codes + row * R.h + at),
                              scales[row * blocks_of(R.h) + at / kBlock]);
  const uint32_t o[4] = {v.x, v.y, v.z, v.w};
  store_words<4>(y + row * R.ld + at, o);
}

// Weights: a workgroup to a block of 128 x 128; a thread holds 8 elements of every 16th row, so that the
// block is read once.  Memory bounds it: 16 of 4096 x 4096, 805 MB in 141 us (5.7 TB/s); 4 of 8192 x 14336,
// 1.41 GB in 278 us, and back in 242 (5.8 TB/s).
struct Fp8Weights {
  int64_t stride;  // elements between groups of the 16-bit weight
  int32_t h_in, h_out;
};
template <int DT>
__global__ __launch_bounds__(256) void fp8_quantize_weight_kernel(uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                                  const uint16_t* __restrict__ W, Fp8Weights P) {
  __shared__ uint32_t tops[4];
  const int bi = blocks_of(P.h_in), bo = blocks_of(P.h_out);
  const int ib = blockIdx.x % bi, ob = blockIdx.x / bi % bo, g = blockIdx.x / bi / bo;
  const int c = ib * kBlock + 8 * (threadIdx.x % 16), r0 = ob * kBlock + threadIdx.x / 16;
  const uint16_t* const from = W + g * P.stride;
  uint4 v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    v[i] = c < P.h_in && r < P.h_out ? ld16(from + static_cast<int64_t>(r) * P.h_in + c) : zero4();
    top = max(top, top_of(v[i]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
  __syncthreads();
  const float s = block_scale<DT>(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
  uint8_t* const to = codes + static_cast<int64_t>(g) * P.h_in * P.h_out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (c < P.h_in && r < P.h_out)
      *reinterpret_cast<u32x2_t*>(to + static_cast<int64_t>(r) * P.h_in + c) = encode8_finite<DT>(v[i], s);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_dequantize_weight_kernel(uint16_t* __restrict__ W, const uint8_t* __restrict__ codes,
                                                                    const float* __restrict__ scales, Fp8Weights P) {
  const int bi = blocks_of(P.h_in), bo = blocks_of(P.h_out);
  const int ib = blockIdx.x % bi, ob = blockIdx.x / bi % bo, g = blockIdx.x / bi / bo;
  const int c = ib * kBlock + 8 * (threadIdx.x % 16), r0 = ob * kBlock + threadIdx.x / 16;
  const float s = scales[blockIdx.x];
  const uint8_t* const from = codes + static_cast<int64_t>(g) * P.h_in * P.h_out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (c >= P.h_in || r >= P.h_out) continue;
    const int64_t at = static_cast<int64_t>(r) * P.h_in + c;
    const uint4 v = decode8<DT>(*reinterpret_cast<const u32x2_t*>(from + at), s);
    const uint32_t o[4] = {v.x, v.y, v.z, v.w};
    store_words<4>(W + g * P.stride + at, o);
  }
}

// ------------------------------------------------------------------------------------
// products
// ------------------------------------------------------------------------------------
template <int DT, bool DX, bool NEAR>
hipError_t launch_fp8(hipStream_t s, const Fp8Args& A, const BlockLaunch& L) {
  const uint32_t grid = static_cast<uint32_t>(L.workgroups);
  if (L.rows == 256) fp8_tile_kernel<DT, DX, 256, 256, 2, 4, 2, NEAR><<<grid, 512, 0, s>>>(A);
  else if (L.rows == 64 && L.buffers == 8) fp8_tile_kernel<DT, DX, 64, 64, 2, 2, 8, NEAR><<<grid, 256, 0, s>>>(A);
  else if (L.rows == 64) fp8_tile_kernel<DT, DX, 64, 64, 2, 2, 4, NEAR><<<grid, 256, 0, s>>>(A);
  else if (L.buffers == 4) fp8_tile_kernel<DT, DX, 128, 128, 2, 2, 4, NEAR><<<grid, 256, 0, s>>>(A);
  else fp8_tile_kernel<DT, DX, 128, 128, 2, 2, 2, NEAR><<<grid, 256, 0, s>>>(A);
  return hipGetLastError();
}
template <bool DX>
hipError_t launch_fp8(int32_t dtype, hipStream_t s, const Fp8Args& A, const BlockLaunch& L) {
  const int32_t depth = DX ? A.h_out : A.h_in;
  const bool near = depth % 128 == 0 && static_cast<int64_t>(shared_rows(A.T.n, A.share_rows)) * A.ld_r <= UINT32_MAX &&
                    static_cast<int64_t>(A.h_in) * A.h_out <= UINT32_MAX;
  if (near) return dtype == SGMV_F16 ? launch_fp8<SGMV_F16, DX, true>(s, A, L) : launch_fp8<SGMV_BF16, DX, true>(s, A, L);
  return dtype == SGMV_F16 ? launch_fp8<SGMV_F16, DX, false>(s, A, L) : launch_fp8<SGMV_BF16, DX, false>(s, A, L);
}

template <int DT, bool X16>
hipError_t launch_fp8_skinny(hipStream_t s, const Fp8Args& A, const BlockLaunch& L) {
  const uint32_t grid = static_cast<uint32_t>(L.workgroups);
  if (L.cols == 16) fp8_skinny_kernel<DT, X16, 1, 8><<<grid, 512, 0, s>>>(A);
  else fp8_skinny_kernel<DT, X16, 2, 4><<<grid, 256, 0, s>>>(A);
  return hipGetLastError();
}
hipError_t launch_fp8_skinny(int32_t dtype, hipStream_t s, const Fp8Args& A, const BlockLaunch& L) {
  if (A.x) return dtype == SGMV_F16 ? launch_fp8_skinny<SGMV_F16, true>(s, A, L) : launch_fp8_skinny<SGMV_BF16, true>(s, A, L);
  return dtype == SGMV_F16 ? launch_fp8_skinny<SGMV_F16, false>(s, A, L) : launch_fp8_skinny<SGMV_BF16, false>(s, A, L);
}

// ------------------------------------------------------------------------------------
// host checks
// ------------------------------------------------------------------------------------
constexpr int64_t kMostGroups = (int64_t(1) << 24) - 1;  // workgroups of 256 threads in a grid

inline int check_fp8_dim(int32_t h, int unit = 16) {
  if (h < unit || h > kMaxDim) return SGMV_ERR_SHAPE;
  return h % unit != 0 ? SGMV_ERR_ALIGNMENT : SGMV_OK;
}
// of a weight: its rows are whole pieces
inline int check_fp8_dims(int32_t h_in, int32_t h_out) {
  if (int st = check_fp8_dim(h_in)) return st;
  return check_fp8_dim(h_out, 8);
}

// 16-bit rows that a launch of the quantiser takes
inline int check_rows16(int64_t rows, int32_t h, int64_t ld) {
  if (ld < h) return SGMV_ERR_SHAPE;
  if (ld % 8 != 0) return SGMV_ERR_ALIGNMENT;
  return rows < 0 || rows > kMostGroups * 4 / ((h + 511) / 512) ? SGMV_ERR_SHAPE : SGMV_OK;
}

inline int check_fp8_rows(int32_t dtype, int64_t rows, int32_t h, int64_t ld) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (int st = check_fp8_dim(h)) return st;
  return check_rows16(rows, h, ld);
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline size_t rows_bytes16(int64_t rows, int64_t ld, int32_t h) {
  return rows <= 0 ? 0 : 2 * (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(h));
}
inline size_t row_scales(int64_t rows, int32_t h) { return 4 * static_cast<size_t>(rows) * blocks_of(h); }
inline size_t weight_scales(int32_t G, int32_t h_in, int32_t h_out) {
  return 4 * static_cast<size_t>(G) * blocks_of(h_in) * blocks_of(h_out);
}

inline Fp8Rows fp8_rows(int64_t rows, int32_t h, int64_t ld, int32_t pitch) { return {rows, ld, h, pitch, (h + 511) / 512}; }
inline int32_t pitch_of(int32_t h) { return (h + 15) / 16 * 16; }
inline uint32_t fp8_grid(const Fp8Rows& R) { return static_cast<uint32_t>((R.rows * R.units + 3) / 4); }

hipError_t launch_quantize(int32_t dtype, hipStream_t s, void* codes, float* scales, const void* x, const Fp8Rows& R) {
  const auto kernel = dtype == SGMV_F16 ? fp8_quantize_kernel<SGMV_F16> : fp8_quantize_kernel<SGMV_BF16>;
  kernel<<<fp8_grid(R), 256, 0, s>>>(static_cast<uint8_t*>(codes), scales, static_cast<const uint16_t*>(x), R);
  return hipGetLastError();
}

// weights to the format (or back); 0 when fine
inline int check_fp8_weight(int32_t dtype, const void* W, int64_t stride, const void* codes, const void* scales,
                            int32_t G, int32_t h_in, int32_t h_out) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (int st = check_fp8_dims(h_in, h_out)) return st;
  const int64_t elems = static_cast<int64_t>(h_in) * h_out;
  if (G < 1 || stride < elems || static_cast<int64_t>(blocks_of(h_in)) * blocks_of(h_out) > kMostGroups / G)
    return SGMV_ERR_SHAPE;
  if (G > kMaxGroups) return SGMV_ERR_UNSUPPORTED;
  if (stride % 8 != 0) return SGMV_ERR_ALIGNMENT;
  if (!W || !codes || !scales) return SGMV_ERR_NULL;
  if (!aligned16(W) || !aligned16(codes) || !aligned4(scales)) return SGMV_ERR_ALIGNMENT;
  const size_t w = pool_bytes16(G, stride, elems), c = static_cast<size_t>(G) * elems, s = weight_scales(G, h_in, h_out);
  if (ranges_overlap(W, w, codes, c) || ranges_overlap(W, w, scales, s) || ranges_overlap(codes, c, scales, s))
    return SGMV_ERR_ALIAS;
  return SGMV_OK;
}

}  // namespace

extern "C" int sgmv_block_quantize(hipStream_t stream, int32_t dtype, void* codes, float* scales, const void* x,
                                 int64_t ld_x, int64_t rows, int32_t h) {
  if (int st = check_fp8_rows(dtype, rows, h, ld_x)) return st;
  if (rows == 0) return SGMV_OK;
  if (!codes || !scales || !x) return SGMV_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales) || !aligned16(x)) return SGMV_ERR_ALIGNMENT;
  const size_t c = static_cast<size_t>(rows) * h, s = row_scales(rows, h), xb = rows_bytes16(rows, ld_x, h);
  if (ranges_overlap(codes, c, x, xb) || ranges_overlap(scales, s, x, xb) || ranges_overlap(codes, c, scales, s))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  return hip_status(launch_quantize(dtype, stream, codes, scales, x, fp8_rows(rows, h, ld_x, h)));
}

extern "C" int sgmv_block_dequantize(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y, const void* codes,
                                   const float* scales, int64_t rows, int32_t h) {
  if (int st = check_fp8_rows(dtype, rows, h, ld_y)) return st;
  if (rows == 0) return SGMV_OK;
  if (!codes || !scales || !y) return SGMV_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales) || !aligned16(y)) return SGMV_ERR_ALIGNMENT;
  const size_t yb = rows_bytes16(rows, ld_y, h);
  if (ranges_overlap(codes, static_cast<size_t>(rows) * h, y, yb) || ranges_overlap(scales, row_scales(rows, h), y, yb))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const Fp8Rows R = fp8_rows(rows, h, ld_y, h);
  const auto kernel = dtype == SGMV_F16 ? fp8_dequantize_kernel<SGMV_F16> : fp8_dequantize_kernel<SGMV_BF16>;
  kernel<<<fp8_grid(R), 256, 0, stream>>>(static_cast<uint16_t*>(y), static_cast<const uint8_t*>(codes), scales, R);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_block_quantize_weight(hipStream_t stream, int32_t dtype, void* codes, float* scales, const void* W,
                                        int64_t W_stride, int32_t n_groups, int32_t h_in, int32_t h_out) {
  if (int st = check_fp8_weight(dtype, W, W_stride, codes, scales, n_groups, h_in, h_out)) return st;
  if (int st = check_device()) return st;
  const auto kernel = dtype == SGMV_F16 ? fp8_quantize_weight_kernel<SGMV_F16> : fp8_quantize_weight_kernel<SGMV_BF16>;
  kernel<<<n_groups * blocks_of(h_in) * blocks_of(h_out), 256, 0, stream>>>(
      static_cast<uint8_t*>(codes), scales, static_cast<const uint16_t*>(W), Fp8Weights{W_stride, h_in, h_out});
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_block_dequantize_weight(hipStream_t stream, int32_t dtype, void* W, int64_t W_stride, const void* codes,
                                          const float* scales, int32_t n_groups, int32_t h_in, int32_t h_out) {
  if (int st = check_fp8_weight(dtype, W, W_stride, codes, scales, n_groups, h_in, h_out)) return st;
  if (int st = check_device()) return st;
  const auto kernel = dtype == SGMV_F16 ? fp8_dequantize_weight_kernel<SGMV_F16> : fp8_dequantize_weight_kernel<SGMV_BF16>;
  kernel<<<n_groups * blocks_of(h_in) * blocks_of(h_out), 256, 0, stream>>>(
      static_cast<uint16_t*>(W), static_cast<const uint8_t*>(codes), scales, Fp8Weights{W_stride, h_in, h_out});
  return hip_status(hipGetLastError());
}

namespace {

struct Product {
  bool dx;
  int32_t dtype;
  void* out;
  int64_t ld_out;
  const void* r;       // 16-bit rows, or codes
  int64_t ld_r;        // 16-bit rows
  const float* r_scales;
  int32_t share;
  const void* w;
  const float* w_scales;
  const int32_t *starts, *perm;
  int32_t n, G, h_in, h_out;
  void* workspace;     // 16-bit rows
  size_t workspace_bytes;
  int32_t cols() const { return dx ? h_in : h_out; }
  int32_t depth() const { return dx ? h_out : h_in; }
  int32_t rows() const { return shared_rows(n, share); }
};

inline size_t codes_room(int64_t rows, int32_t h) { return align_up(static_cast<size_t>(rows) * pitch_of(h), 256); }
inline size_t rows_room(int64_t rows, int32_t h) { return rows <= 0 ? 0 : codes_room(rows, h) + row_scales(rows, h); }

int product(hipStream_t stream, const Product& P, bool quantized) {
  if (P.dtype != SGMV_F16 && P.dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  int st;
  if ((st = check_groups(P.n, P.G, P.share, P.starts, P.perm)) || (st = check_fp8_dims(P.h_in, P.h_out)) ||
      (st = check_dim(P.cols(), P.ld_out)) || (quantized && (st = check_fp8_dim(P.depth()))) ||
      (!quantized && (st = check_rows16(P.rows(), P.depth(), P.ld_r))))
    return st;
  const BlockLaunch L = fp8_launch(P.dx, P.n, P.G, P.starts, P.h_in, P.h_out);
  if (!L.fits()) return SGMV_ERR_SHAPE;
  if (P.n == 0) return SGMV_OK;
  if (!P.out || !P.r || (quantized && !P.r_scales) || !P.w || !P.w_scales) return SGMV_ERR_NULL;
  if (!aligned16(P.out) || !aligned16(P.r) || !aligned4(P.r_scales) || !aligned16(P.w) || !aligned4(P.w_scales))
    return SGMV_ERR_ALIGNMENT;
  const bool few = L.rows == kSkinnyRows;
  const size_t room = quantized || few ? 0 : rows_room(P.rows(), P.depth());
  if (room > 0 && (!P.workspace || P.workspace_bytes < room || !aligned16(P.workspace))) return SGMV_ERR_WORKSPACE;
  const size_t out_bytes = matrix_bytes(P.n, P.ld_out, P.cols()), elems = static_cast<size_t>(P.G) * P.h_in * P.h_out;
  const struct {
    const void* p;
    size_t bytes;
  } in[] = {{P.r, quantized ? static_cast<size_t>(P.rows()) * P.depth() : rows_bytes16(P.rows(), P.ld_r, P.depth())},
            {P.r_scales, quantized ? row_scales(P.rows(), P.depth()) : 0},
            {P.w, elems},
            {P.w_scales, weight_scales(P.G, P.h_in, P.h_out)}};
  if (over_tables(P.out, out_bytes, P.starts, P.perm, P.n, P.G)) return SGMV_ERR_ALIAS;
  if (room > 0 && (over_tables(P.workspace, room, P.starts, P.perm, P.n, P.G) ||
                   ranges_overlap(P.workspace, room, P.out, out_bytes)))
    return SGMV_ERR_ALIAS;
  for (const auto& i : in)
    if (i.bytes > 0 && (ranges_overlap(P.out, out_bytes, i.p, i.bytes) ||
                        (room > 0 && ranges_overlap(P.workspace, room, i.p, i.bytes))))
      return SGMV_ERR_ALIAS;
  if ((st = check_device())) return st;
  Fp8Args A{};
  A.T = {P.starts, P.perm, P.n, P.G};
  A.share = share_of(P.share);
  A.share_rows = P.share;
  A.ld_r = pitch_of(P.depth());
  if (quantized) {
    A.r = static_cast<const uint8_t*>(P.r);
    A.r_scale = P.r_scales;
  } else if (few) {
    A.x = static_cast<const uint16_t*>(P.r);
    A.ld_x = P.ld_r;
  } else {
    uint8_t* const codes = static_cast<uint8_t*>(P.workspace);
    float* const scales = reinterpret_cast<float*>(codes + codes_room(P.rows(), P.depth()));
    if (hipError_t e = launch_quantize(P.dtype, stream, codes, scales, P.r, fp8_rows(P.rows(), P.depth(), P.ld_r, pitch_of(P.depth()))))
      return hip_status(e);
    A.r = codes, A.r_scale = scales;
  }
  A.w = static_cast<const uint8_t*>(P.w);
  A.w_scale = P.w_scales;
  A.out = static_cast<uint16_t*>(P.out);
  A.ld_out = P.ld_out, A.h_in = P.h_in, A.h_out = P.h_out;
  if (few) return hip_status(launch_fp8_skinny(P.dtype, stream, A, L));
  return hip_status(P.dx ? launch_fp8<true>(P.dtype, stream, A, L) : launch_fp8<false>(P.dtype, stream, A, L));
}

}  // namespace

extern "C" size_t sgmv_block_workspace_bytes(int32_t n, int32_t share, int32_t n_groups, int32_t grouped, int32_t h_in,
                                           int32_t h_out) {
  if (n < 1 || share < 1 || n_groups < 1 || h_in < 1 || h_out < 1) return 0;
  if (fp8_launch(false, n, n_groups, grouped != 0, h_in, h_out).rows == kSkinnyRows) return 0;
  return rows_room(shared_rows(n, share), h_in);
}

extern "C" size_t sgmv_block_dx_workspace_bytes(int32_t n, int32_t h_out) {
  return n < 1 || h_out < 1 ? 0 : rows_room(n, h_out);
}

extern "C" int sgmv_block_matmul(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y, const void* x, int64_t ld_x,
                               int32_t share, const void* W_codes, const float* W_scales, const int32_t* starts,
                               const int32_t* perm, int32_t n, int32_t n_groups, int32_t h_in, int32_t h_out,
                               void* workspace, size_t workspace_bytes) {
  return product(stream, {false, dtype, y, ld_y, x, ld_x, nullptr, share, W_codes, W_scales, starts, perm, n, n_groups,
                          h_in, h_out, workspace, workspace_bytes}, false);
}

extern "C" int sgmv_block_matmul_quantized(hipStream_t stream, int32_t dtype, void* y, int64_t ld_y, const void* x_codes,
                                         const float* x_scales, int32_t share, const void* W_codes,
                                         const float* W_scales, const int32_t* starts, const int32_t* perm, int32_t n,
                                         int32_t n_groups, int32_t h_in, int32_t h_out) {
  return product(stream, {false, dtype, y, ld_y, x_codes, 0, x_scales, share, W_codes, W_scales, starts, perm, n,
                          n_groups, h_in, h_out, nullptr, 0}, true);
}

extern "C" int sgmv_block_matmul_dx(hipStream_t stream, int32_t dtype, void* dx, int64_t ld_dx, const void* dy,
                                  int64_t ld_dy, const void* W_codes, const float* W_scales, const int32_t* starts,
                                  const int32_t* perm, int32_t n, int32_t n_groups, int32_t h_in, int32_t h_out,
                                  void* workspace, size_t workspace_bytes) {
  return product(stream, {true, dtype, dx, ld_dx, dy, ld_dy, nullptr, 1, W_codes, W_scales, starts, perm, n, n_groups,
                          h_in, h_out, workspace, workspace_bytes}, false);
}

extern "C" int sgmv_block_matmul_dx_quantized(hipStream_t stream, int32_t dtype, void* dx, int64_t ld_dx,
                                            const void* dy_codes, const float* dy_scales, const void* W_codes,
                                            const float* W_scales, const int32_t* starts, const int32_t* perm, int32_t n,
                                            int32_t n_groups, int32_t h_in, int32_t h_out) {
  return product(stream, {true, dtype, dx, ld_dx, dy_codes, 0, dy_scales, 1, W_codes, W_scales, starts, perm, n,
                          n_groups, h_in, h_out, nullptr, 0}, true);
}
