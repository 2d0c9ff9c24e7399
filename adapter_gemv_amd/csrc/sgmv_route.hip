// Routing to experts and its gradient, and the weighted sum of each token's expert rows and its
// gradients.
#include "sgmv_device.h"
#include "sgmv_rules.h"

using namespace sgmv_dev;
using namespace sgmv_host;

namespace {

constexpr int kMaxRoutes = SGMV_MAX_ROUTES;
constexpr int kMaxExpertGroups = SGMV_MAX_EXPERT_GROUPS;

// ------------------------------------------------------------------------------------
// routing
// ------------------------------------------------------------------------------------
struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t n, E, k, groups, keep, best;
  float scale;
};

template <int DT>
__device__ inline float logit(const void* p, int64_t i) {
  if constexpr (DT == SGMV_F32) return static_cast<const float*>(p)[i];
  else return Elem<DT>::lo(static_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ inline void store_logit(void* p, int64_t i, float v) {
  if constexpr (DT == SGMV_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(Elem<DT>::pack(v, 0.f));
}

__device__ inline double wave_sum(double v) {
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ inline float wave_sum(float v) {
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ inline float wave_max(float v) {
  for (int d = 32; d; d /= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// an unsigned number that orders like the value, NaN above all; 0 stands for "not there"
__device__ inline uint64_t order(double v) {
  if (v != v) return ~uint64_t(0);
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 counts as 0
  return b >> 63 ? ~b : b | uint64_t(1) << 63;
}

// s_j over the sum of the chosen s, times a common factor that keeps the largest near 1: `top` is
// the largest chosen logit
template <bool SIGMOID, typename T>
__device__ inline T share_of_choice(T l, T top) {
  if constexpr (!SIGMOID) return exp(l - top);
  else return l >= 0 ? 1 / (1 + exp(-l)) : exp(l - (top < 0 ? top : T(0))) / (1 + exp(l));
}

// One wavefront to a token.  c in 64 bits: of the values that choose, a row's neighbours are
// often closer than float32's rounding.
template <int DT, bool SIGMOID>
__global__ __launch_bounds__(64) void route_kernel(RouteArgs A, bool normalize) {
  __shared__ uint64_t key[kMaxGroups];  // order of c; 0: not to be chosen
  __shared__ double val[kMaxGroups];
  __shared__ uint64_t group_key[kMaxExpertGroups];
  const int lane = threadIdx.x, t = blockIdx.x;
  const int64_t at = t * A.ld;
  float top = -__builtin_inff();
  bool bad = false;
  for (int e = lane; e < A.E; e += 64) {
    const float l = logit<DT>(A.logits, at + e);
    bad |= !(l < __builtin_inff());
    top = fmaxf(top, l);
  }
  bad = __any(bad);
  top = wave_max(top);
  double sum = 0;
  if (!SIGMOID) {
    for (int e = lane; e < A.E; e += 64) sum += exp(static_cast<double>(logit<DT>(A.logits, at + e)) - top);
    sum = wave_sum(sum);
  }
  auto score = [&](float l) -> double {
    if (SIGMOID) return 1 / (1 + exp(-static_cast<double>(l)));
    return bad ? __builtin_nan("") : exp(static_cast<double>(l) - top) / sum;
  };
  // scores grow with logits, so these choose as well where nothing is added to a score
  const bool by_logit = !A.bias && (A.keep == A.groups || A.best == 1);
  for (int e = lane; e < A.E; e += 64) {
    const float l = logit<DT>(A.logits, at + e);
    const double c = by_logit ? (!SIGMOID && bad ? __builtin_nan("") : static_cast<double>(l))
                              : score(l) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0);
    const bool out = l == -__builtin_inff() || c == -__builtin_inf();
    key[e] = out ? 0 : order(c);
    val[e] = c;
  }
  __syncthreads();
  if (A.keep < A.groups) {
    const int per = A.E / A.groups;
    if (lane < A.groups) {
      int b0 = -1, b1 = -1;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        if (key[e] == 0) continue;
        if (b0 < 0 || key[e] > key[b0]) b1 = b0, b0 = e;
        else if (b1 < 0 || key[e] > key[b1]) b1 = e;
      }
      group_key[lane] = b0 < 0 ? 0 : order(val[b0] + (A.best > 1 && b1 >= 0 ? val[b1] : 0.0));
    }
    __syncthreads();
    if (lane < A.groups) {
      int before = 0;
      for (int g = 0; g < A.groups; ++g)
        before += group_key[g] > group_key[lane] || (group_key[g] == group_key[lane] && g < lane);
      if (before >= A.keep)
        for (int e = lane * per; e < (lane + 1) * per; ++e) key[e] = 0;
    }
    __syncthreads();
  }
  int mine = -1;  // lane j: the j-th chosen expert
  for (int j = 0; j < A.k; ++j) {
    uint64_t k0 = 0;
    int e0 = 1 << 30;
    for (int e = lane; e < A.E; e += 64)
      if (key[e] > k0) k0 = key[e], e0 = e;
    for (int d = 32; d; d /= 2) {
      const uint64_t k1 = __shfl_xor(k0, d);
      const int e1 = __shfl_xor(e0, d);
      if (k1 > k0 || (k1 == k0 && e1 < e0)) k0 = k1, e0 = e1;
    }
    if (k0 == 0) break;
    if (lane == j) mine = e0;
    if (lane == 0) key[e0] = 0;
    __syncthreads();
  }
  const float l = mine < 0 ? -__builtin_inff() : logit<DT>(A.logits, at + mine);
  double w;
  if (normalize) {
    const float first = __any(mine >= 0 && l != l) ? __builtin_nanf("") : wave_max(l);
    const double u = mine < 0 ? 0 : share_of_choice<SIGMOID, double>(l, first);
    w = u / wave_sum(u);
    if (!SIGMOID && bad) w = __builtin_nan("");
  } else {
    w = score(l);
  }
  if (lane < A.k) {
    A.ids[static_cast<int64_t>(t) * A.k + lane] = mine;
    A.weights[static_cast<int64_t>(t) * A.k + lane] = mine < 0 ? 0.f : static_cast<float>(w * A.scale);
  }
}

struct RouteBackArgs {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t ld_d;
  int32_t n, E, k;
  float scale;
};

template <int DT, bool SIGMOID>
__global__ __launch_bounds__(64) void route_backward_kernel(RouteBackArgs A, bool normalize) {
  __shared__ float d[kMaxGroups];
  const int lane = threadIdx.x, t = blockIdx.x;
  const int64_t at = t * A.ld, to = t * A.ld_d;
  const int id = lane < A.k ? A.ids[static_cast<int64_t>(t) * A.k + lane] : -1;
  const float l = static_cast<uint32_t>(id) < static_cast<uint32_t>(A.E) ? logit<DT>(A.logits, at + id)
                                                                         : -__builtin_inff();
  const bool in = l != -__builtin_inff();  // takes part
  const float g = in ? A.scale * A.dweights[static_cast<int64_t>(t) * A.k + lane] : 0.f;
  float top = -__builtin_inff(), sum = 0.f, mine = 0.f, inner = 0.f;
  if (!SIGMOID && !normalize) {
    bool bad = false;
    for (int e = lane; e < A.E; e += 64) {
      const float v = logit<DT>(A.logits, at + e);
      bad |= !(v < __builtin_inff());
      top = fmaxf(top, v);
    }
    top = wave_max(top);
    for (int e = lane; e < A.E; e += 64) {
      const float v = logit<DT>(A.logits, at + e);
      if (v != -__builtin_inff()) sum += expf(v - top);
    }
    sum = wave_sum(sum);
    if (__any(bad)) sum = __builtin_nanf("");
    inner = wave_sum(in ? g * (expf(l - top) / sum) : 0.f);
    mine = g;
  } else if (normalize) {
    top = __any(in && l != l) ? __builtin_nanf("") : wave_max(l);
    float u = in ? share_of_choice<SIGMOID, float>(l, top) : 0.f;
    u /= wave_sum(u);
    inner = wave_sum(in ? g * u : 0.f);
    mine = in ? u * (g - inner) * (SIGMOID ? 1.f / (1.f + expf(l)) : 1.f) : 0.f;
  } else {
    mine = in ? g * (1.f / (1.f + expf(-l))) * (1.f / (1.f + expf(l))) : 0.f;
  }
  for (int e = lane; e < A.E; e += 64) d[e] = 0.f;
  __syncthreads();
  // one at a time, in order: the same expert may stand twice
  for (int j = 0; j < A.k; ++j) {
    if (lane == j && in) d[id] += mine;
    __syncthreads();
  }
  for (int e = lane; e < A.E; e += 64) {
    float v = d[e];
    if (!SIGMOID && !normalize) {
      const float x = logit<DT>(A.logits, at + e);
      v = x == -__builtin_inff() ? 0.f : expf(x - top) / sum * (v - inner);
    }
    store_logit<DT>(A.dlogits, to + e, v);
  }
}

// ------------------------------------------------------------------------------------
// the rows of a token's experts
// ------------------------------------------------------------------------------------
struct CombineArgs {
  uint16_t* out;       // dy
  int64_t ld_out;
  const uint16_t* y;
  int64_t ld_y;
  const float* weights;
  const uint16_t* dout;
  int64_t ld_dout;
  float* dweights;
  int32_t n, k, h;
};

// a thread to 8 columns of a token
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs A, bool add) {
  const int parts = (A.h + 2047) / 2048;
  const int t = blockIdx.x / parts, c = ((blockIdx.x - t * parts) * 256 + threadIdx.x) * 8;
  if (c >= A.h) return;
  float acc[8] = {};
  uint16_t* const out = A.out + t * A.ld_out + c;
  for (int j = 0; j < A.k; ++j) {
    const int64_t row = static_cast<int64_t>(t) * A.k + j;
    const uint4 v = ld16(A.y + row * A.ld_y + c);
    const float w = A.weights ? A.weights[row] : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, elem<DT>(v, i), acc[i]);
  }
  if (add) {
    const uint4 v = ld16(out);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += elem<DT>(v, i);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Elem<DT>::pack(acc[2 * i], acc[2 * i + 1]);
  store_words<4>(out, o);
}

// a workgroup to one row of y
template <int DT>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineArgs A) {
  __shared__ float sums[4];
  const int row = blockIdx.x, t = row / A.k, lane = threadIdx.x & 63;
  const float w = A.weights ? A.weights[row] : 1.f;
  float dot = 0.f;
  for (int c = threadIdx.x * 8; c < A.h; c += 2048) {
    const uint4 d = ld16(A.dout + t * A.ld_dout + c);
    if (A.dweights) dot = dot8<DT>(d, ld16(A.y + row * A.ld_y + c), dot);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = Elem<DT>::pack(w * elem<DT>(d, 2 * i), w * elem<DT>(d, 2 * i + 1));
    store_words<4>(A.out + row * A.ld_out + c, o);
  }
  dot = wave_sum(dot);
  if (lane == 0) sums[threadIdx.x / 64] = dot;
  __syncthreads();
  if (A.dweights && threadIdx.x == 0) A.dweights[row] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// ------------------------------------------------------------------------------------
// host checks
// ------------------------------------------------------------------------------------
inline int elem_bytes(int32_t dtype) { return dtype == SGMV_F32 ? 4 : 2; }

inline bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

inline size_t strided_bytes(int32_t n, int64_t ld, int32_t h, int one) {
  return n <= 0 ? 0 : one * (static_cast<size_t>(n - 1) * static_cast<size_t>(ld) + static_cast<size_t>(h));
}

// what both directions check; 0 when fine
inline int check_route(int32_t dtype, int32_t n, int32_t E, int32_t k, int32_t scores) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16 && dtype != SGMV_F32) return SGMV_ERR_UNSUPPORTED;
  if (scores != SGMV_SOFTMAX && scores != SGMV_SIGMOID) return SGMV_ERR_UNSUPPORTED;
  if (n < 0 || E < 1 || k < 1 || k > E) return SGMV_ERR_SHAPE;
  if (E > kMaxGroups || k > kMaxRoutes) return SGMV_ERR_UNSUPPORTED;
  return n > (1 << 25) ? SGMV_ERR_SHAPE : SGMV_OK;  // n * k fits 31 bits, and 64 threads a row a grid
}

inline int check_combine(int32_t dtype, int32_t n, int32_t k, int32_t h) {
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (n < 0 || k < 1 || static_cast<int64_t>(n) * k > kMaxGroupRows) return SGMV_ERR_SHAPE;
  // the threads of a grid
  if (h > 0 && static_cast<int64_t>(n) * std::max<int64_t>(k, (h + 2047) / 2048) > (1 << 24) - 1) return SGMV_ERR_SHAPE;
  return SGMV_OK;
}

}  // namespace

extern "C" int sgmv_route(hipStream_t stream, int32_t dtype, int32_t* ids, float* weights,
                          const void* logits, int64_t ld_logits, const float* bias, int32_t n,
                          int32_t n_experts, int32_t k, int32_t expert_groups, int32_t keep_groups,
                          int32_t group_best, int32_t scores, int32_t normalize, float scale) {
  if (int st = check_route(dtype, n, n_experts, k, scores)) return st;
  if (expert_groups < 1 || n_experts % expert_groups != 0 || keep_groups < 1 || keep_groups > expert_groups ||
      group_best < 1 || ld_logits < n_experts)
    return SGMV_ERR_SHAPE;
  if (expert_groups > kMaxExpertGroups || group_best > 2) return SGMV_ERR_UNSUPPORTED;
  if (n == 0) return SGMV_OK;
  if (!ids || !weights || !logits) return SGMV_ERR_NULL;
  if (!aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(bias, 4) || !aligned_to(logits, elem_bytes(dtype)))
    return SGMV_ERR_ALIGNMENT;
  const size_t out = 4 * static_cast<size_t>(n) * k, in = strided_bytes(n, ld_logits, n_experts, elem_bytes(dtype));
  if (ranges_overlap(ids, out, weights, out)) return SGMV_ERR_ALIAS;
  for (const void* p : {static_cast<const void*>(ids), static_cast<const void*>(weights)})
    if (ranges_overlap(p, out, logits, in) || (bias && ranges_overlap(p, out, bias, 4 * static_cast<size_t>(n_experts))))
      return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const RouteArgs A{logits, ld_logits, bias, ids, weights, n, n_experts, k, expert_groups, keep_groups, group_best, scale};
  const auto go = [&](auto kernel) { kernel<<<n, 64, 0, stream>>>(A, normalize != 0); };
  const bool sigmoid = scores == SGMV_SIGMOID;
  if (dtype == SGMV_F32) go(sigmoid ? route_kernel<SGMV_F32, true> : route_kernel<SGMV_F32, false>);
  else if (dtype == SGMV_F16) go(sigmoid ? route_kernel<SGMV_F16, true> : route_kernel<SGMV_F16, false>);
  else go(sigmoid ? route_kernel<SGMV_BF16, true> : route_kernel<SGMV_BF16, false>);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_route_backward(hipStream_t stream, int32_t dtype, void* dlogits, int64_t ld_dlogits,
                                   const float* dweights, const void* logits, int64_t ld_logits,
                                   const int32_t* ids, int32_t n, int32_t n_experts, int32_t k,
                                   int32_t scores, int32_t normalize, float scale) {
  if (int st = check_route(dtype, n, n_experts, k, scores)) return st;
  if (ld_dlogits < n_experts || ld_logits < n_experts) return SGMV_ERR_SHAPE;
  if (n == 0) return SGMV_OK;
  if (!dlogits || !dweights || !logits || !ids) return SGMV_ERR_NULL;
  const int one = elem_bytes(dtype);
  if (!aligned_to(ids, 4) || !aligned_to(dweights, 4) || !aligned_to(logits, one) || !aligned_to(dlogits, one))
    return SGMV_ERR_ALIGNMENT;
  const size_t out = strided_bytes(n, ld_dlogits, n_experts, one), chosen = 4 * static_cast<size_t>(n) * k;
  if (ranges_overlap(dlogits, out, logits, strided_bytes(n, ld_logits, n_experts, one)) ||
      ranges_overlap(dlogits, out, ids, chosen) || ranges_overlap(dlogits, out, dweights, chosen))
    return SGMV_ERR_ALIAS;
  if (int st = check_device()) return st;
  const RouteBackArgs A{logits, ld_logits, ids, dweights, dlogits, ld_dlogits, n, n_experts, k, scale};
  const auto go = [&](auto kernel) { kernel<<<n, 64, 0, stream>>>(A, normalize != 0); };
  const bool sigmoid = scores == SGMV_SIGMOID;
  if (dtype == SGMV_F32) go(sigmoid ? route_backward_kernel<SGMV_F32, true> : route_backward_kernel<SGMV_F32, false>);
  else if (dtype == SGMV_F16) go(sigmoid ? route_backward_kernel<SGMV_F16, true> : route_backward_kernel<SGMV_F16, false>);
  else go(sigmoid ? route_backward_kernel<SGMV_BF16, true> : route_backward_kernel<SGMV_BF16, false>);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_combine_rows(hipStream_t stream, int32_t dtype, void* out, int64_t ld_out,
                                 const void* y, int64_t ld_y, const float* weights, int32_t n,
                                 int32_t k, int32_t h, int32_t add) {
  int st;
  if ((st = check_combine(dtype, n, k, h)) || (st = check_dim(h, ld_out)) || (st = check_dim(h, ld_y))) return st;
  if (n == 0) return SGMV_OK;
  if (!out || !y) return SGMV_ERR_NULL;
  if (!aligned16(out) || !aligned16(y) || !aligned_to(weights, 4)) return SGMV_ERR_ALIGNMENT;
  const size_t out_bytes = matrix_bytes(n, ld_out, h);
  if (ranges_overlap(out, out_bytes, y, matrix_bytes(n * k, ld_y, h)) ||
      (weights && ranges_overlap(out, out_bytes, weights, 4 * static_cast<size_t>(n) * k)))
    return SGMV_ERR_ALIAS;
  if ((st = check_device())) return st;
  const CombineArgs A{static_cast<uint16_t*>(out), ld_out, static_cast<const uint16_t*>(y), ld_y, weights,
                      nullptr, 0, nullptr, n, k, h};
  const uint32_t grid = static_cast<uint32_t>(n) * ((h + 2047) / 2048);
  if (dtype == SGMV_F16) combine_kernel<SGMV_F16><<<grid, 256, 0, stream>>>(A, add != 0);
  else combine_kernel<SGMV_BF16><<<grid, 256, 0, stream>>>(A, add != 0);
  return hip_status(hipGetLastError());
}

extern "C" int sgmv_combine_rows_backward(hipStream_t stream, int32_t dtype, void* dy, int64_t ld_dy,
                                          float* dweights, const void* dout, int64_t ld_dout, const void* y,
                                          int64_t ld_y, const float* weights, int32_t n, int32_t k,
                                          int32_t h) {
  int st;
  if ((st = check_combine(dtype, n, k, h)) || (st = check_dim(h, ld_dy)) || (st = check_dim(h, ld_dout))) return st;
  if (weights && (st = check_dim(h, ld_y))) return st;
  if (n == 0) return SGMV_OK;
  if (!dy || !dout || (weights && (!dweights || !y))) return SGMV_ERR_NULL;
  if (!aligned16(dy) || !aligned16(dout) || (weights && !aligned16(y)) || !aligned_to(weights, 4) ||
      !aligned_to(dweights, 4))
    return SGMV_ERR_ALIGNMENT;
  const size_t dy_bytes = matrix_bytes(n * k, ld_dy, h), dout_bytes = matrix_bytes(n, ld_dout, h);
  const size_t chosen = 4 * static_cast<size_t>(n) * k;
  if (ranges_overlap(dy, dy_bytes, dout, dout_bytes)) return SGMV_ERR_ALIAS;
  if (weights) {
    const size_t y_bytes = matrix_bytes(n * k, ld_y, h);
    if (ranges_overlap(dy, dy_bytes, y, y_bytes) || ranges_overlap(dy, dy_bytes, weights, chosen) ||
        ranges_overlap(dy, dy_bytes, dweights, chosen) || ranges_overlap(dweights, chosen, dout, dout_bytes) ||
        ranges_overlap(dweights, chosen, y, y_bytes) || ranges_overlap(dweights, chosen, weights, chosen))
      return SGMV_ERR_ALIAS;
  }
  if ((st = check_device())) return st;
  const CombineArgs A{static_cast<uint16_t*>(dy), ld_dy, static_cast<const uint16_t*>(y), ld_y, weights,
                      static_cast<const uint16_t*>(dout), ld_dout, weights ? dweights : nullptr, n, k, h};
  if (dtype == SGMV_F16) combine_backward_kernel<SGMV_F16><<<n * k, 256, 0, stream>>>(A);
  else combine_backward_kernel<SGMV_BF16><<<n * k, 256, 0, stream>>>(A);
  return hip_status(hipGetLastError());
}
