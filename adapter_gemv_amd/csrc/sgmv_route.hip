// Routing to experts and its gradient, and the weighted sum of each token's expert rows and its
// gradients.
#include <type_traits>

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
__device__ inline float logit(int dtype, const void* p, int64_t i) {
  return dtype == SGMV_F32 ? logit<SGMV_F32>(p, i) : dtype == SGMV_F16 ? logit<SGMV_F16>(p, i) : logit<SGMV_BF16>(p, i);
}
template <int DT>
__device__ inline void store_logit(void* p, int64_t i, float v) {
  if constexpr (DT == SGMV_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(Elem<DT>::pack(v, 0.f));
}

// Reductions over the L lanes of a token (16: a row of the wavefront, by rotations within it; 64: then
// across rows), in every lane; all of them have to take part.
__device__ inline int from_lane(int v, int lane) { return __shfl(v, lane); }
template <int CTRL>
__device__ inline uint32_t rotated(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 15, 15, false));
}
template <int L, typename T, typename F>
__device__ inline T over_token(T v, F op) {
  static_assert((L == 16 || L == 64) && (sizeof(T) == 4 || sizeof(T) == 8), "");
  if constexpr (sizeof(T) == 4) {
    constexpr int kRotate = 0x120;  // row_ror
    const auto bits = [](T x) { return __builtin_bit_cast(uint32_t, x); };
    const auto back = [](uint32_t x) { return __builtin_bit_cast(T, x); };
    v = op(v, back(rotated<kRotate + 8>(bits(v))));
    v = op(v, back(rotated<kRotate + 4>(bits(v))));
    v = op(v, back(rotated<kRotate + 2>(bits(v))));
    v = op(v, back(rotated<kRotate + 1>(bits(v))));
    if constexpr (L == 64) {
      const auto h = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
      v = op(back(h[0]), back(h[1]));
      const auto q = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
      v = op(back(q[0]), back(q[1]));
    }
  } else {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v = op(v, __shfl_xor(v, d));
  }
  return v;
}
template <int L, typename T>
__device__ inline T token_sum(T v) {
  return over_token<L>(v, [](T a, T b) { return a + b; });
}
template <int L>
__device__ inline float token_max(float v) {
  return over_token<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ inline uint32_t token_most(uint32_t v) {
  return over_token<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ inline bool token_any(bool v) {
  const uint64_t set = __ballot(v);
  return L == 64 ? set != 0 : (set >> (threadIdx.x & 48) & 0xffffu) != 0;
}

constexpr float kInf = __builtin_inff();

// an unsigned number that orders like the value, NaN above all; 0 stands for "not there"
__device__ inline uint64_t order(double v) {
  if (v != v) return ~uint64_t(0);
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 counts as 0
  return b >> 63 ? ~b : b | uint64_t(1) << 63;
}
// the same for a value that is no NaN; 0 for minus infinity
__device__ inline uint32_t order(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v == -kInf ? 0u : b >> 31 ? ~b : b | 0x80000000u;
}

// s_j over the sum of the chosen s, times a common factor that keeps the largest near 1: `top` is
// the largest chosen logit (a sigmoid by itself: 0)
template <bool SIGMOID, typename T>
__device__ inline T share_of_choice(T l, T top) {
  if constexpr (!SIGMOID) return exp(l - top);
  else return l >= 0 ? 1 / (1 + exp(-l)) : exp(l - (top < 0 ? top : T(0))) / (1 + exp(l));
}

// the value that chooses an expert by its sigmoid
__device__ inline double exact_sigmoid(const RouteArgs& A, float l, int e) {
  return 1 / (1 + exp(-static_cast<double>(l))) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0);
}

// One token by the whole wavefront, with the values that choose in 64 bits: for tokens whose choice
// float32 leaves open, and for NaN.
template <int N>
struct ExactSpace {
  uint64_t key[N];  // order of c; 0: not to be chosen
  double val[N];
  uint64_t group_key[kMaxExpertGroups];
};
template <bool SIGMOID, int N>
__device__ __forceinline__ void route_exactly(const RouteArgs& A, int dtype, int t, bool normalize, ExactSpace<N>& S) {
  const int lane = threadIdx.x;
  const int64_t at = t * A.ld;
  float top = -kInf;
  bool bad = false;
  for (int e = lane; e < A.E; e += 64) {
    const float l = logit(dtype, A.logits, at + e);
    bad |= !(l < kInf);
    top = fmaxf(top, l);
  }
  bad = __any(bad);
  top = token_max<64>(top);
  double sum = 0;
  if (!SIGMOID) {
    for (int e = lane; e < A.E; e += 64) sum += exp(static_cast<double>(logit(dtype, A.logits, at + e)) - top);
    sum = token_sum<64>(sum);
  }
  auto score = [&](float l) -> double {
    if (SIGMOID) return 1 / (1 + exp(-static_cast<double>(l)));
    return bad ? __builtin_nan("") : exp(static_cast<double>(l) - top) / sum;
  };
  const bool by_logit = !A.bias && (A.keep == A.groups || A.best == 1);
  for (int e = lane; e < A.E; e += 64) {
    const float l = logit(dtype, A.logits, at + e);
    const double c = by_logit ? (!SIGMOID && bad ? __builtin_nan("") : static_cast<double>(l))
                     : SIGMOID ? exact_sigmoid(A, l, e)
                               : score(l) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0);
    S.key[e] = l == -kInf || c == -__builtin_inf() ? 0 : order(c);
    S.val[e] = c;
  }
  __syncthreads();
  if (A.keep < A.groups) {
    const int per = A.E / A.groups;
    if (lane < A.groups) {
      // the two best, as keys and where they are (no two places of one key: the first)
      uint64_t k0 = 0, k1 = 0;
      int b0 = 0, b1 = 0;
#pragma unroll 4
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const uint64_t k = S.key[e];
        const bool first = k > k0, second = k > k1;
        k1 = first ? k0 : second ? k : k1;
        b1 = first ? b0 : second ? e : b1;
        k0 = first ? k : k0;
        b0 = first ? e : b0;
      }
      S.group_key[lane] = k0 == 0 ? 0 : order(S.val[b0] + (A.best > 1 && k1 != 0 ? S.val[b1] : 0.0));
    }
    __syncthreads();
    if (lane < A.groups) {
      int before = 0;
      for (int g = 0; g < A.groups; ++g)
        before += S.group_key[g] > S.group_key[lane] || (S.group_key[g] == S.group_key[lane] && g < lane);
      if (before >= A.keep)
        for (int e = lane * per; e < (lane + 1) * per; ++e) S.key[e] = 0;
    }
    __syncthreads();
  }
  int mine = -1;  // lane j: the j-th chosen expert
  for (int j = 0; j < A.k; ++j) {
    uint64_t k0 = 0;
    int e0 = 1 << 30;
    for (int e = lane; e < A.E; e += 64)
      if (S.key[e] > k0) k0 = S.key[e], e0 = e;
    // the largest key, by halves, and the lowest place that has it
    const uint32_t high = token_most<64>(static_cast<uint32_t>(k0 >> 32));
    const uint32_t low = token_most<64>(static_cast<uint32_t>(k0 >> 32) == high ? static_cast<uint32_t>(k0) : 0u);
    const uint64_t k = static_cast<uint64_t>(high) << 32 | low;
    e0 = static_cast<int>(~token_most<64>(k0 == k ? ~static_cast<uint32_t>(e0) : 0u));
    if (k == 0) break;
    if (lane == j) mine = e0;
    if (lane == 0) S.key[e0] = 0;
    __syncthreads();
  }
  __syncthreads();
  const float l = mine < 0 ? -kInf : logit(dtype, A.logits, at + mine);
  double w;
  if (normalize) {
    const float first = __any(mine >= 0 && l != l) ? __builtin_nanf("") : token_max<64>(l);
    const double u = mine < 0 ? 0 : share_of_choice<SIGMOID, double>(l, first);
    w = u / token_sum<64>(u);
    if (!SIGMOID && bad) w = __builtin_nan("");
  } else {
    w = score(l);
  }
  if (lane < A.k) {
    A.ids[static_cast<int64_t>(t) * A.k + lane] = mine;
    A.weights[static_cast<int64_t>(t) * A.k + lane] = mine < 0 ? 0.f : static_cast<float>(w * A.scale);
  }
}

// L lanes to a token, each with V experts next to each other, so that the lowest of equal experts is
// in the lowest lane: k rounds of a maximum over a lane's experts and over the lanes (rotations within
// 16 lanes), in which the winner leaves.  For 256 experts a round costs 84 instructions for the four
// tokens of a wavefront, against 30 for one token with 64 lanes and 4 experts each.
//
// What chooses: where nothing is added to a score, the logits, which order like it.  Otherwise c in
// float32, with the least distance at which two of its values are sure to be in order.  Where closer ones
// stand among a token's first k + 1, or close sums of groups, sigmoids are taken again in 64 bits for
// these alone (the chosen ones and the next, each in its lane; the two best of each group); a token for
// which that is not enough, one with NaN, and a softmax, whose sum takes all experts, are done again
// by route_exactly.  Of 16384 tokens of float32 logits, 256 experts in 8 groups, 0.1 to 0.3 % have such
// values, and their wavefront is the last to end: all redone by route_exactly 25 us, so 18.3; 128 experts, 13.4
// and 10.4.  16-bit logits are often equal: without a bias, but with groups of two best, where the scores
// choose, 30 % of bfloat16 tokens have equal ones among their first nine: softmax 70 us (float32 25.6), sigmoid
// 32 (18).
//
// Distances: a sigmoid's float32 value is off by at most 2^-22 (its exponential by (|l| + 1) 2^-23 of
// itself, which the slope s (1 - s) takes to at most 0.48 * 2^-23; sum and reciprocal 2.5 * 2^-24), a
// softmax's by 2^-20 of the row's largest, most of it from the sum, and c by 2^-24 of itself.  Twice that
// between two values; all of it doubled.  A group's sum is off by what its two values are (by 2^-24 of each
// one's own size, which the sum need not have: biases of opposite sign cancel) and by 2^-24 of itself:
// between two sums that of both groups, doubled, is twice a value's distance and 2^-22 of the sizes.
template <int L, int V, bool SIGMOID, bool GROUPS>
__global__ __launch_bounds__(64) void route_kernel(RouteArgs A, int dtype, bool normalize, bool vectors,
                                                   bool bias_vectors) {
  constexpr int N = L * V;
  __shared__ union {
    ExactSpace<N> exact;
    struct {
      float c[64 / L][N + kMaxExpertGroups];  // a place more after each group: no bank conflicts
      float score[64 / L][kMaxExpertGroups];
    } g;
  } S;
  const int lane = threadIdx.x, l0 = lane % L, slot = lane / L;
  const int t0 = blockIdx.x * (64 / L), t = min(t0 + slot, A.n - 1);
  const int64_t at = t * A.ld + l0 * V;
  const int mine_n = min(V, A.E - l0 * V);  // may be negative
  float l[V];
  auto fetch = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    constexpr int W = DT == SGMV_F32 ? 4 : 8;  // elements of 16 bytes
    if (V % W == 0 && vectors && mine_n == V) {
#pragma unroll
      for (int v = 0; v + W <= V; v += W) {
        if constexpr (DT == SGMV_F32) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(A.logits) + at + v);
#pragma unroll
          for (int i = 0; i < 4; ++i) l[v + i] = x[i];
        } else {
          const uint4 x = ld16(static_cast<const uint16_t*>(A.logits) + at + v);
#pragma unroll
          for (int i = 0; i < 8; ++i) l[v + i] = elem<DT>(x, i);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = v < mine_n ? logit<DT>(A.logits, at + v) : -kInf;
    }
  };
  if (dtype == SGMV_F32) fetch(std::integral_constant<int, SGMV_F32>{});
  else if (dtype == SGMV_F16) fetch(std::integral_constant<int, SGMV_F16>{});
  else fetch(std::integral_constant<int, SGMV_BF16>{});

  const bool by_logit = !A.bias && (!GROUPS || A.best == 1);
  bool open = false;  // to be done in 64 bits
  float top = -kInf, sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    open |= SIGMOID ? l[v] != l[v] : !(l[v] < kInf);
    top = fmaxf(top, l[v]);
  }
  float c[V], near = 0.f;
  if (!SIGMOID && (!by_logit || !normalize)) {
    top = token_max<L>(top);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = l[v] == -kInf ? 0.f : __expf(l[v] - top);
      sum += c[v];
    }
    sum = token_sum<L>(sum);
  }
  if (by_logit) {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l[v];
  } else {
    const float one = 1.f / sum;  // the largest score
    near = SIGMOID ? 0x1p-20f : 0x1p-18f * one;
    float b[V];
    if (V % 4 == 0 && bias_vectors && mine_n == V) {
#pragma unroll
      for (int v = 0; v + 4 <= V; v += 4) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(A.bias + l0 * V + v);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[v + i] = x[i];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = A.bias && v < mine_n ? A.bias[l0 * V + v] : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float s = SIGMOID ? __builtin_amdgcn_rcpf(1.f + __expf(-l[v])) : c[v] * one;
      c[v] = l[v] == -kInf ? -kInf : s + b[v];
      open |= c[v] != c[v];
    }
  }
  const auto apart = [&](float a) { return by_logit ? 0.f : near + 0x1p-21f * fabsf(a); };

  if constexpr (GROUPS) {
    const int per = A.E / A.groups;
    float* const row = S.g.c[slot];
    const int g0 = l0 * V / per, in0 = l0 * V - g0 * per;  // this lane's first group, and place in it
#pragma unroll
    for (int v = 0, g = g0, in = in0; v < V; ++v) {
      if (v < mine_n) row[l0 * V + v + g] = c[v];
      if (++in == per) in = 0, ++g;
    }
    __syncthreads();
    for (int g = l0; g < A.groups; g += L) {
      float b0 = -kInf, b1 = -kInf;
#pragma unroll 8
      for (int e = 0; e < per; ++e) {
        const float x = row[g * (per + 1) + e];
        b1 = fmaxf(b1, fminf(b0, x));
        b0 = fmaxf(b0, x);
      }
      // of two best, half their sum: below infinity where both are, and minus infinity only without an expert
      const bool two = A.best > 1 && b1 > -kInf;
      const float half = A.best > 1 ? 0.5f : 1.f;
      b0 *= half;
      b1 = two ? b1 * half : 0.f;
      S.g.score[slot][g] = b0 + b1;
      // in the place after the group: how far from its exact sum this score may be, doubled; minus infinity,
      // which no distance is below, for logits and for infinities
      const float size = fabsf(b0) + fabsf(b1);
      row[g * (per + 1) + per] = by_logit || size == kInf ? -kInf : half * near + 0x1p-22f * size;
    }
    __syncthreads();
    uint64_t kept = 0;
    bool close = false;  // a group on the other side of the cut may be the better one
    for (int first = 0; first < A.groups; first += L) {
      const int g = first + l0;
      bool stay = false;
      if (g < A.groups) {
        const float mine = S.g.score[slot][g], off = row[g * (per + 1) + per];
        int before = 0, after = 0;  // surely better ones, and those that may be
        for (int h = 0; h < A.groups; ++h) {
          const float other = S.g.score[slot][h];
          before += other > mine || (other == mine && h < g);
          after += fabsf(other - mine) <= off + row[h * (per + 1) + per];
        }
        if (off > 0) --after;  // itself
        stay = before < A.keep;
        close |= after && before + after >= A.keep && before - after < A.keep;
      }
      const uint64_t set = __ballot(stay);
      kept |= (L == 64 ? set : set >> (lane & 48) & 0xffffu) << first;
    }
    if (!SIGMOID || A.groups > L) {
      open |= close;
    } else if (__any(close)) {  // the scores in 64 bits, if it is plain which experts make them up
      double score = -__builtin_inf();
      if (l0 < A.groups) {
        float b[3] = {-kInf, -kInf, -kInf};
        int e0 = 0, e1 = 0;
#pragma unroll 8
        for (int i = 0; i < per; ++i) {
          const float x = row[l0 * (per + 1) + i];
          const int e = l0 * per + i;
          const bool first = x > b[0], second = x > b[1];
          b[2] = fmaxf(b[2], fminf(b[1], x));
          e1 = first ? e0 : second ? e : e1;
          b[1] = first ? b[0] : second ? x : b[1];
          e0 = first ? e : e0;
          b[0] = first ? x : b[0];
        }
        const bool two = A.best > 1 && b[1] > -kInf;
        const float least = two ? b[1] : b[0], other = A.best > 1 ? b[2] : b[1];
        open |= other > -kInf && !(least - other > apart(least));
        if (b[0] > -kInf) {
          score = exact_sigmoid(A, logit(dtype, A.logits, t * A.ld + e0), e0);
          if (two) score += exact_sigmoid(A, logit(dtype, A.logits, t * A.ld + e1), e1);
        }
      }
      int before = 0;
      for (int h = 0; h < A.groups; ++h) {
        const double other = __shfl(score, lane - l0 + h);
        before += other > score || (other == score && h < l0);
      }
      const uint64_t set = __ballot(l0 < A.groups && before < A.keep);
      kept = L == 64 ? set : set >> (lane & 48) & 0xffffu;
    }
#pragma unroll
    for (int v = 0, g = g0, in = in0; v < V; ++v) {
      if (!(kept >> (g & 63) & 1)) c[v] = -kInf;
      if (++in == per) in = 0, ++g;
    }
    __syncthreads();
  }

  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = order(c[v]);
  int mine = -1;  // lane j of a token: its j-th expert
  uint32_t last = 0;
  const auto most = [&] {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    return best;
  };
  const auto take = [&](int j, uint32_t best, uint32_t m) {  // the first of the lanes that have the largest
    const uint64_t set = __ballot(best == m);
    const int first = __builtin_ctzll(L == 64 ? set : set >> (lane & 48) & 0xffffu);
    int v0 = 0;
#pragma unroll
    for (int v = V - 1; v > 0; --v) v0 = key[v] == m ? v : v0;
    v0 = key[0] == m ? 0 : v0;
    const int e = from_lane(l0 * V + v0, (lane - l0) + first);
    if (l0 == j) mine = m ? e : -1;
    const int leaves = l0 == first ? v0 : V;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = v == leaves ? 0u : key[v];
  };
  // whether the values that two keys stand for may be in another order
  const auto near_keys = [&](uint32_t more, uint32_t less) {
    const auto value = [](uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); };
    return less && !(value(more) - value(less) > apart(value(more)));
  };
  bool close = false;
  for (int j = 0; j < A.k; ++j) {
    const uint32_t best = most(), m = token_most<L>(best);
    if (!by_logit && j > 0) close |= near_keys(last, m);
    last = m;
    take(j, best, m);
  }
  if (!by_logit) {
    const uint32_t best = most(), next = token_most<L>(best);  // of those that are left
    const bool edge = near_keys(last, next);
    if (!SIGMOID) {
      open |= close || edge;
    } else if (__any(close || edge)) {
      // the chosen ones and the next in 64 bits, unless there are more that may belong to them
      take(A.k, best, next);
      const bool more = near_keys(last, token_most<L>(most()));  // by all lanes
      open |= edge && (A.k == L || more);
      const double c = mine < 0 ? 0 : exact_sigmoid(A, logit(dtype, A.logits, t * A.ld + mine), mine);
      int rank = 0;
      for (int h = 0; h < min(A.k + 1, L); ++h) {
        const double other = __shfl(c, lane - l0 + h);
        const int id = __shfl(mine, lane - l0 + h);
        rank += id >= 0 && (other > c || (other == c && id < mine));
      }
      if (mine < 0) rank = l0;
      mine = __builtin_amdgcn_ds_permute(4 * (lane - l0 + rank), mine);
      if (l0 >= A.k) mine = -1;
    }
  }

  const int64_t to = static_cast<int64_t>(t) * A.k + l0;
  const int64_t own = t * A.ld + mine;
  const float x = mine < 0 ? -kInf : logit(dtype, A.logits, own);
  float w;
  if (normalize) {
    const float first = token_max<L>(x);  // by all lanes
    const float u = mine < 0 ? 0.f : share_of_choice<SIGMOID, float>(x, first);
    w = u / token_sum<L>(u);
  } else {
    w = SIGMOID ? share_of_choice<SIGMOID, float>(x, 0.f) : expf(x - top) / sum;
  }
  open = token_any<L>(open);
  if (l0 < A.k && t0 + slot < A.n && !open) {
    A.ids[to] = mine;
    A.weights[to] = mine < 0 ? 0.f : w * A.scale;
  }
  const uint64_t again = __ballot(open && l0 == 0 && t0 + slot < A.n);
  for (int s = 0; s < 64 / L; ++s) {
    if (!(again >> (s * L) & 1)) continue;
    __syncthreads();
    route_exactly<SIGMOID>(A, dtype, t0 + s, normalize, S.exact);
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

// L lanes to a token; lane j has its j-th choice.  The row is put together in LDS and written in whole
// pieces; only a softmax that is not normalised reads all of it.  Bound by that write and the launch:
// 16384 tokens, 256 experts, float32: 6.9 us, 16.8 MB written.  Softmax not normalised reads the row three times,
// by single elements, and takes each exponential twice: 128 experts 9.2 to 10.0 us for 16.8 MB.
template <int DT, bool SIGMOID, int L, int N>
__global__ __launch_bounds__(64) void route_backward_kernel(RouteBackArgs A, bool normalize, bool vectors) {
  __shared__ __attribute__((aligned(16))) float rows[64 / L][N];
  const int lane = threadIdx.x, l0 = lane % L, slot = lane / L;
  const int t = min(static_cast<int>(blockIdx.x) * (64 / L) + slot, A.n - 1);
  const int64_t at = t * A.ld, to = t * A.ld_d;
  float* const row = rows[slot];
  const int id = l0 < A.k ? A.ids[static_cast<int64_t>(t) * A.k + l0] : -1;
  const float l = static_cast<uint32_t>(id) < static_cast<uint32_t>(A.E) ? logit<DT>(A.logits, at + id) : -kInf;
  const bool in = l != -kInf;  // takes part
  const float g = in ? A.scale * A.dweights[static_cast<int64_t>(t) * A.k + l0] : 0.f;
  const bool whole = !SIGMOID && !normalize;
  float top = -kInf, sum = 0.f, mine = 0.f, inner = 0.f;
  if (whole) {
    bool bad = false;
    for (int e = l0; e < A.E; e += L) {
      const float v = logit<DT>(A.logits, at + e);
      bad |= !(v < kInf);
      top = fmaxf(top, v);
    }
    top = token_max<L>(top);
    for (int e = l0; e < A.E; e += L) {
      const float v = logit<DT>(A.logits, at + e);
      if (v != -kInf) sum += expf(v - top);
    }
    sum = token_sum<L>(sum);
    if (token_any<L>(bad)) sum = __builtin_nanf("");
    inner = token_sum<L>(in ? g * (expf(l - top) / sum) : 0.f);
    mine = g;
  } else if (normalize) {
    const bool bad = token_any<L>(in && l != l);
    top = token_max<L>(l);
    if (bad) top = __builtin_nanf("");
    float u = in ? share_of_choice<SIGMOID, float>(l, top) : 0.f;
    u /= token_sum<L>(u);
    inner = token_sum<L>(in ? g * u : 0.f);
    mine = in ? u * (g - inner) * (SIGMOID ? 1.f / (1.f + expf(l)) : 1.f) : 0.f;
  } else {
    mine = in ? g * share_of_choice<SIGMOID, float>(l, 0.f) * (1.f / (1.f + expf(l))) : 0.f;
  }
  for (int e = 4 * l0; e < N; e += 4 * L) *reinterpret_cast<f32x4_t*>(&row[e]) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  // one at a time, in order: the same expert may stand twice
  for (int j = 0; j < A.k; ++j) {
    if (l0 == j && in) row[id] += mine;
    __syncthreads();
  }
  if (static_cast<int>(blockIdx.x) * (64 / L) + slot >= A.n) return;
  const auto value = [&](int e) {
    const float v = row[e];
    if (!whole) return v;
    const float x = logit<DT>(A.logits, at + e);
    return x == -kInf ? 0.f : expf(x - top) / sum * (v - inner);
  };
  constexpr int W = DT == SGMV_F32 ? 4 : 8;  // elements of 16 bytes
  const int tail = vectors ? A.E / W * W : 0;
  for (int e = W * l0; e < tail; e += W * L) {
    if constexpr (DT == SGMV_F32) {
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(A.dlogits) + to + e) =
          f32x4_t{value(e), value(e + 1), value(e + 2), value(e + 3)};
    } else {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = Elem<DT>::pack(value(e + 2 * i), value(e + 2 * i + 1));
      store_words<4>(static_cast<uint16_t*>(A.dlogits) + to + e, o);
    }
  }
  for (int e = tail + l0; e < A.E; e += L) store_logit<DT>(A.dlogits, to + e, value(e));
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

// A thread to 8 columns of a token; y is read once, in whole cache lines, and nothing is shared, so memory
// bounds it: 8191 tokens x 4 rows of 5120, 419 MB in 85 us (4.9 TB/s, as a copy).
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

// A workgroup to one row of y: a dot product and a scaled copy in one pass over y and dout, which the k
// workgroups of a token read from the cache: 8191 tokens x 4 rows of 5120, 755 MB in 140 us (5.4 TB/s).
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
  dot = token_sum<64>(dot);
  if (lane == 0) sums[threadIdx.x / 64] = dot;
  __syncthreads();
  if (A.dweights && threadIdx.x == 0) A.dweights[row] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// ------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------
// 16 lanes to a token, up to 256 experts of which up to 16 are chosen; 64 otherwise, whose places are 4, 8
// or 16 to a lane (16384 tokens, kernel and its launch in a graph, 16 lanes and 64: sigmoid, bias, 256
// experts in 8 groups 18.7 and 28.2 us, without groups 14.2 and 18.5; softmax 256 experts 10.5 and 14.6, 64
// experts 10.3 and 17.8, 8 experts 4.7 and 8.3; 512 experts with 8 places to a lane and with 16: 30 and 62).
template <int L, int V, bool SIGMOID>
void launch_route(hipStream_t s, const RouteArgs& A, int dtype, bool normalize, bool vectors) {
  const int grid = static_cast<int>(tiles_of(A.n, 64 / L));
  const bool bias_vectors = A.bias && aligned16(A.bias);
  if (A.keep < A.groups) route_kernel<L, V, SIGMOID, true><<<grid, 64, 0, s>>>(A, dtype, normalize, vectors, bias_vectors);
  else route_kernel<L, V, SIGMOID, false><<<grid, 64, 0, s>>>(A, dtype, normalize, vectors, bias_vectors);
}
template <bool SIGMOID>
void launch_route(hipStream_t s, const RouteArgs& A, int dtype, bool normalize, bool vectors) {
  const auto go = [&](auto lanes, auto each) {
    launch_route<decltype(lanes)::value, decltype(each)::value, SIGMOID>(s, A, dtype, normalize, vectors);
  };
  using std::integral_constant;
  const integral_constant<int, 16> some{};
  const integral_constant<int, 64> all{};
  if (A.k > 16 || A.E > 256) {
    if (A.E <= 256) go(all, integral_constant<int, 4>{});
    else if (A.E <= 512) go(all, integral_constant<int, 8>{});
    else go(all, integral_constant<int, 16>{});
  } else if (A.E <= 32) go(some, integral_constant<int, 2>{});
  else if (A.E <= 64) go(some, integral_constant<int, 4>{});
  else if (A.E <= 128) go(some, integral_constant<int, 8>{});
  else go(some, integral_constant<int, 16>{});
}

template <int DT>
void launch_back(hipStream_t s, const RouteBackArgs& A, int32_t scores, bool normalize, bool vectors) {
  const auto go = [&](auto kernel, int lanes) {
    kernel<<<static_cast<int>(tiles_of(A.n, 64 / lanes)), 64, 0, s>>>(A, normalize, vectors);
  };
  const bool sigmoid = scores == SGMV_SIGMOID;
  if (A.k > 16 || A.E > 256)
    go(sigmoid ? route_backward_kernel<DT, true, 64, kMaxGroups> : route_backward_kernel<DT, false, 64, kMaxGroups>, 64);
  else
    go(sigmoid ? route_backward_kernel<DT, true, 16, 256> : route_backward_kernel<DT, false, 16, 256>, 16);
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
  return n > (1 << 25) ? SGMV_ERR_SHAPE : SGMV_OK;  // 64 threads a row fit a grid; n * k may be 2^31: 64 bits
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
  const bool vectors = aligned16(logits) && ld_logits * elem_bytes(dtype) % 16 == 0;
  if (scores == SGMV_SIGMOID) launch_route<true>(stream, A, dtype, normalize != 0, vectors);
  else launch_route<false>(stream, A, dtype, normalize != 0, vectors);
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
  const bool vectors = aligned16(dlogits) && ld_dlogits * one % 16 == 0;
  if (dtype == SGMV_F32) launch_back<SGMV_F32>(stream, A, scores, normalize != 0, vectors);
  else if (dtype == SGMV_F16) launch_back<SGMV_F16>(stream, A, scores, normalize != 0, vectors);
  else launch_back<SGMV_BF16>(stream, A, scores, normalize != 0, vectors);
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
