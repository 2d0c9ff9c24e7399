// The tiled product of 8-bit operands with a scale for each block of 128, by group: rows of x times
// W^T, or rows of dy times W (DX).
//
// A workgroup makes BR rows x BC columns of the output; a stage is one block of the contracted
// dimension, 128 bytes of each row and column, brought by direct global-to-LDS loads into one of
// BUFS buffers while another is multiplied.  An MFMA 16x16x128 takes a whole block; its sums start from
// zero and are added to the tile's, times the block's two scales: 128 multiply-adds for 32 matrix
// instructions of a wavefront, which run beside them.
//
// This instruction, its own power-of-two scales left out, has twice the rate of bfloat16's.  It adds eight
// products at a time and cuts what lies 2^13 below the power of two of the largest (measured): at most
// 7 * 2^-13 of the sum of the magnitudes, where the rounding to 8 bits was off by up to 2^-4 of each
// element already.  Block sums are added in float32.
//
// Bound: 8192^3 reaches 2480 TFLOP/s on a card that has been at work (2050 to 2110 in the first 10 ms), its
// gradient 2440 (2100 to 2370), 4096^3 2240 and 2180.  MFMAs busy 67 % of what the CUs are (SQ_BUSY_CU_CYCLES, 4
// SIMDs each) and 62 % of the kernel's cycles (GRBM_GUI_ACTIVE); the barrier and LDS reads of a stage are the rest.
// Ragged groups add the empty half of a group's last tile, and workgroups that wait for the last ones:
// 1531 x 2 rows over 8 experts of 5120 x 13824, CUs busy 75 %, 328 to 343 us.
//
// x, dy and W lie along their rows where these are contracted: piece c (16 bytes) of tile row q sits
// in slot c ^ ((q >> 1) & 7), and a fragment is two 16-byte reads.  W of DX lies across: a stage is
// 128 contracted rows of BC bytes, a fragment four transposing reads (ds_read_b64_tr_b8, each of
// eight rows of one piece per 16 lanes).  Piece c of row k sits in slot c ^ swizzle(k), so that the 16
// rows of half a wavefront's read lie over all banks.  A lane has the same contracted positions in both
// forms: 16 * kq .. + 15 and 64 + 16 * kq .. + 15.
//
// Contracted positions past the end are zeros in both operands, tile rows and columns past the end
// repeat the last one and are not stored.
#pragma once

#include "sgmv_tile.h"

namespace sgmv_dev {

typedef __attribute__((ext_vector_type(2))) int i32x2_t;

struct Fp8Args {
  RowTab T;
  Share share;
  const uint16_t* x;      // rows in 16 bits, ld_x elements apart, or
  const uint8_t* r;       // rows of x or dy in 8 bits, ld_r apart, zeros up to a multiple of 16
  const float* r_scale;   // [rows, blocks]
  const uint8_t* w;       // [h_out, h_in]
  const float* w_scale;   // [blocks of h_out, blocks of h_in]
  uint16_t* out;
  int64_t ld_x, ld_r, ld_out;
  int32_t h_in, h_out;
  int32_t share_rows;     // rows that share one of r
};

__host__ __device__ inline int blocks_of(int h) { return (h + 127) / 128; }

template <int BR, int BC, int WR, int WC, int BUFS>
struct Fp8Tile {
  static constexpr int NW = WR * WC, TH = 64 * NW;
  static constexpr int NR = BR / WR / 16, NC = BC / WC / 16;  // fragments of a wavefront
  static constexpr int RI = BR / 8 / NW, CI = BC / 8 / NW;    // loads per stage
  static_assert(RI * 8 * NW == BR && CI * 8 * NW == BC && NC % 2 == 0 && NC <= 4 && NR * NC >= 4, "");
  static_assert(BR < TH && BR % 64 == 0, "a wavefront to 64 rows' scales, and one to the weight's");
  struct RBuf {
    u32x4_t v[BR * 8];
  };
  struct CBuf {
    u32x4_t v[BC * 8];
  };
  static constexpr int CB = (BC + 127) / 128;  // blocks of columns
  struct Scales {
    alignas(16) float r[BR];  // [wavefront rows][row of 16][fragment]
    float w[64];              // of the blocks of columns, in turn
  };
};

// at most N global loads of this wavefront are in flight, and every LDS access of it is done; then the
// workgroup's barrier
template <int N>
__device__ inline void wait_tile() {
  static_assert(N < 64, "vmcnt range");
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// the I-th buffer of its type in a kernel
template <class B, int I>
__device__ __forceinline__ B& stage_buffer() {
  __shared__ B b;
  return b;
}

// DX, tiles of B columns: where a piece of contracted row k is moved
template <int B>
__device__ inline int swizzle(int k) {
  static_assert(B == 256 || B == 128 || B == 64, "");
  return B == 256 ? (k & 7) | (k >> 1 & 8) : B == 128 ? (k >> 1 & 3) | (k >> 2 & 4) : (k >> 2 & 1) | (k >> 3 & 2);
}

// NEAR: the contracted dimension is a multiple of 128, and an offset into the rows, or into a group of
// W, fits 32 bits: loads are a uniform base and an offset of the lane's, and need no test (8192^3, with
// a number of stages that is known in rounds: 1822 TFLOP/s to 2020, the gradient 1599 to 2290).  Otherwise
// the lane's tests and 64-bit offsets do not fit beside the sums of 256 x 256: 31 registers are spilled (29 of
// DX; NEAR: none, 3 of DX), some read back in every round of stages.  8192 rows, 2880 x 2880, 102 us (1330
// TFLOP/s), where 2944 x 2944 takes 79 (1800).  Spills count among the loads in flight, but with two buffers
// every wait is for all of these.
template <int DT, bool DX, int BR, int BC, int WR, int WC, int BUFS, bool NEAR>
__global__ __launch_bounds__(64 * WR * WC, BUFS * BR >= 512 && BR < 256 ? 1 : 2) void fp8_tile_kernel(Fp8Args A) {
  using C = Fp8Tile<BR, BC, WR, WC, BUFS>;
  constexpr int NR = C::NR, NC = C::NC, RI = C::RI, CI = C::CI, CB = C::CB;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, kq = lane >> 4;
  const int wr = w / WC, wc = w % WC;
  const int cols = DX ? A.h_in : A.h_out, depth = DX ? A.h_out : A.h_in, bi = blocks_of(A.h_in);

  // which tile: workgroup b runs on XCD b % 8; each XCD takes a contiguous eighth of the tiles
  const int ct = (cols + BC - 1) / BC, xcd = blockIdx.x % kTileXcds, at = blockIdx.x / kTileXcds;
  const TileList list(A.T, BR);
  const int all = list.count * ct, per = all / kTileXcds, more = all % kTileXcds;
  if (at >= per + (xcd < more)) return;
  int m, c0;
  band_order(xcd * per + min(xcd, more) + at, list.count, ct, &m, &c0);
  const RowTile t = list.find(m);
  c0 *= BC;
  const int nst = t.g == A.T.G ? 0 : blocks_of(depth);  // rows of no group: zeros

  f32x4_t acc[NR][NC];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* const rbase = reinterpret_cast<const char*>(A.r);
  const char* const wbase = reinterpret_cast<const char*>(A.w) + static_cast<int64_t>(t.g) * A.h_in * A.h_out;
  // where this lane's pieces of the first stage are, and how far into the contracted dimension
  using Offset = std::conditional_t<NEAR, uint32_t, int64_t>;
  Offset rp[RI], cp[CI];
  int rk[RI], ck[CI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int q = (w * RI + i) * 8 + lane / 8;
    rk[i] = 16 * ((lane & 7) ^ ((q >> 1) & 7));
    const int j = nst ? A.share.div(A.T.row(t.row0 + min(q, t.rows - 1))) : 0;
    rp[i] = static_cast<Offset>(j) * static_cast<Offset>(A.ld_r) + rk[i];
  }
#pragma unroll
  for (int i = 0; i < CI; ++i) {
    if constexpr (!DX) {
      const int q = (w * CI + i) * 8 + lane / 8;
      ck[i] = 16 * ((lane & 7) ^ ((q >> 1) & 7));
      cp[i] = static_cast<Offset>(min(c0 + q, cols - 1)) * A.h_in + ck[i];
    } else {
      constexpr int L = BC / 16;  // lanes to a contracted row
      ck[i] = (w * CI + i) * (64 / L) + lane / L;
      cp[i] = static_cast<Offset>(ck[i]) * A.h_in + min(c0 + 16 * (lane % L ^ swizzle<BC>(ck[i])), cols - 16);
    }
  }
  // behind the last stage the last one again (NEAR), or zeros
  auto issue_r = [&](typename C::RBuf& to, int s, auto which) __attribute__((always_inline)) {
    constexpr int i = decltype(which)::value;
    const char* r = rbase + static_cast<int64_t>(NEAR ? min(s, nst - 1) : s) * 128 + rp[i];
    to_lds(NEAR || rk[i] < depth - s * 128 ? r : zeros, &to.v[(w * RI + i) * 64]);
  };
  auto issue_c = [&](typename C::CBuf& to, int s, auto which) __attribute__((always_inline)) {
    constexpr int i = decltype(which)::value;
    const char* c = wbase + static_cast<int64_t>(NEAR ? min(s, nst - 1) : s) * (DX ? 128 * static_cast<int64_t>(A.h_in) : 128) + cp[i];
    if constexpr (DX && !NEAR) asm("" : "+v"(c));  // keeps its computation out of a branch
    to_lds(NEAR || ck[i] < depth - s * 128 ? c : zeros, &to.v[(w * CI + i) * 64]);
  };
  constexpr int LOADS = RI + CI;
  auto issue_one = [&](typename C::RBuf& rt, typename C::CBuf& ct, int s, auto which) __attribute__((always_inline)) {
    constexpr int k = decltype(which)::value;
    if constexpr (k < RI) issue_r(rt, s, which);
    else issue_c(ct, s, std::integral_constant<int, k - RI>{});
  };

  // Scales come the same way, 4 bytes to a lane: the first wavefronts fetch the rows', in the order in
  // which a lane takes them, and the others the weight's.
  const int kb = blocks_of(depth);
  const float* sp = A.r_scale;
  int64_t step = 1;
  if (nst) {
    if (tid < BR) {
      const int q = (tid / (16 * NR) * NR + tid % NR) * 16 + tid / NR % 16;
      sp += static_cast<int64_t>(A.share.div(A.T.row(t.row0 + min(q, t.rows - 1)))) * kb;
    } else {
      const int cb = min(c0 + 128 * (lane % CB), cols - 1) / 128;
      sp = A.w_scale + static_cast<int64_t>(t.g) * bi * blocks_of(A.h_out) + (DX ? cb : cb * bi);
      if (DX) step = bi;
    }
  }
  auto issue_s = [&](typename C::Scales& to, int s) __attribute__((always_inline)) {
    float* const at = w * 64 < BR ? to.r + w * 64 : to.w;
    __builtin_amdgcn_global_load_lds((tile_global_void*)(sp + min(s, nst - 1) * step), (tile_lds_void*)at, 4, 0, 0);
  };

  // Fragment reads: a lane's offsets, made here, plus constants (so that the compiler tells LDS
  // buffers apart)
  int ro[2], co[4];
#pragma unroll
  for (int u = 0; u < 2; ++u) ro[u] = (wr * NR * 16 + l16) * 8 + ((u * 4 + kq) ^ ((l16 >> 1) & 7));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 16 * kq + l16 / 2;  // DX: the row whose half piece this lane points at
    co[u] = DX ? (k * (BC / 16) + ((wc * NC + u) ^ swizzle<BC>(k))) * 2 + (l16 & 1)  // 8-byte pieces
               : (wc * NC * 16 + l16) * 8 + (((u & 1) * 4 + kq) ^ ((l16 >> 1) & 7));
  }
  asm("" : "+v"(ro[0]), "+v"(ro[1]), "+v"(co[0]), "+v"(co[1]), "+v"(co[2]), "+v"(co[3]));
  auto join = [](u32x4_t a, u32x4_t b) __attribute__((always_inline)) {
    return i32x8_t{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
  };
  auto rfrag = [&](const typename C::RBuf& from, int i) __attribute__((always_inline)) {
    return join(from.v[ro[0] + i * 128], from.v[ro[1] + i * 128]);
  };
  auto cfrag = [&](const typename C::CBuf& from, int j) __attribute__((always_inline)) {
    if constexpr (!DX) {
      return join(from.v[co[0] + j * 128], from.v[co[1] + j * 128]);
    } else {
      typedef __attribute__((address_space(3))) i32x2_t lds2;
      const i32x2_t* const p = reinterpret_cast<const i32x2_t*>(from.v) + co[j];
      i32x8_t v;
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // rows + 8 * (q & 1) + 64 * (q >> 1)
        const i32x2_t x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2*)(p + (8 * (q & 1) + 64 * (q >> 1)) * (BC / 8)));
        v[2 * q] = x.x, v[2 * q + 1] = x.y;
      }
      return v;
    }
  };

  // One stage: NC MFMAs for each row fragment.  The multiply-adds of an MFMA's sums stand three MFMAs
  // behind it (those of the last three in the next stage), when they are there without a wait; the next
  // row fragment is read, and loads of the stage that is BUFS - 1 ahead are issued, meanwhile.  All of a
  // stage's fragments are read before its last one is multiplied: there the workgroup meets, the next
  // stage's first fragments are read during the last MFMAs, and the buffer is free for the loads of the
  // next stage (8192^3: a barrier between stages, 2030 TFLOP/s and 2290 for the gradient).
  constexpr int LAST = NR * NC, MEET = LAST - NC, CARRY = (LAST - 3) / NC;
  i32x8_t cv[NC], rv[2];
  f32x4_t sum[4];
  float sc[NR], ws, carried[NR];
  auto add = [&](auto which, auto& scale) __attribute__((always_inline)) {  // the n-th MFMA's sums
    constexpr int n = decltype(which)::value, i = n / NC, j = n % NC;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(sum[n & 3][q], scale[i], acc[i][j][q]);
    asm volatile("" : "+v"(acc[i][j]));  // here and not later, where sums would have to be kept
  };
  auto read_scales = [&](const typename C::Scales& sb) __attribute__((always_inline)) {
    constexpr int W = NR < 4 ? NR : 4;
    typedef __attribute__((ext_vector_type(W))) float part_t;
    const part_t* const from = reinterpret_cast<const part_t*>(&sb.r[(wr * 16 + l16) * NR]);
#pragma unroll
    for (int i = 0; i < NR / W; ++i) {
      const part_t v = from[i];
#pragma unroll
      for (int q = 0; q < W; ++q) sc[W * i + q] = v[q];
    }
    ws = sb.w[wc * 16 * NC / 128];
  };
  auto stage = [&](const typename C::RBuf& rb, const typename C::RBuf& r1, const typename C::CBuf& c1,
                   const typename C::Scales& s1, typename C::RBuf& rn, typename C::CBuf& cn, typename C::Scales& sn,
                   int s) __attribute__((always_inline)) {
    tile_for<0, LAST>([&](auto which) __attribute__((always_inline)) {
      constexpr int n = decltype(which)::value, i = n / NC, j = n % NC;
      if constexpr (n == MEET) wait_tile<(BUFS - 2) * (LOADS + 1)>();
      sum[n & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(cv[j], rv[i & 1], f32x4_t{0.f, 0.f, 0.f, 0.f},
                                                                    0, 0, 0, 0, 0, 0);
      // behind an MFMA, whose wait for its fragments would take these reads in
      if constexpr (j == 0 && i + 1 < NR) rv[(i + 1) & 1] = rfrag(rb, i + 1);
      tile_for<0, LOADS>([&](auto l) __attribute__((always_inline)) {
        if constexpr (decltype(l)::value * MEET * 3 / (5 * LOADS) == n) issue_one(rn, cn, s + BUFS - 1, l);
      });
      if constexpr (n == 1) issue_s(sn, s + BUFS - 1);
      if constexpr (n == MEET) rv[0] = rfrag(r1, 0);
      if constexpr (n >= MEET) cv[j] = cfrag(c1, j);
      if constexpr (n >= 3) {
        constexpr int m = n - 3;
        if constexpr (m % NC == 0) sc[m / NC] *= ws;
        add(std::integral_constant<int, m>{}, sc);
      } else {
        add(std::integral_constant<int, LAST - 3 + n>{}, carried);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int i = CARRY; i < NR; ++i) carried[i] = i * NC <= LAST - 4 ? sc[i] : sc[i] * ws;
    read_scales(s1);
  };
  // Buffers by number; each is an object of its own, by which the compiler tells them apart
  auto rbuf = [&](auto k) __attribute__((always_inline)) -> typename C::RBuf& {
    return stage_buffer<typename C::RBuf, decltype(k)::value % BUFS>();
  };
  auto cbuf = [&](auto k) __attribute__((always_inline)) -> typename C::CBuf& {
    return stage_buffer<typename C::CBuf, decltype(k)::value % BUFS>();
  };
  auto sbuf = [&](auto k) __attribute__((always_inline)) -> typename C::Scales& {
    return stage_buffer<typename C::Scales, decltype(k)::value % BUFS>();
  };
  if (nst > 0) {
    tile_for<0, BUFS - 1>([&](auto k) __attribute__((always_inline)) {
      tile_for<0, LOADS>([&](auto l) __attribute__((always_inline)) { issue_one(rbuf(k), cbuf(k), decltype(k)::value, l); });
      issue_s(sbuf(k), decltype(k)::value);
    });
    wait_tile<(BUFS - 2) * (LOADS + 1)>();
    // stages in rounds.  No branch inside the loop, which keeps the accumulators where they are.
    constexpr int ROUND = BUFS > 4 ? BUFS : 4;
    auto rounds = [&](auto&& nth) __attribute__((always_inline)) {
      int s = 0;
      for (; s + ROUND <= nst; s += ROUND) tile_for<0, ROUND>([&](auto k) __attribute__((always_inline)) { nth(k, s); });
      tile_for<0, ROUND - 1>([&](auto k) __attribute__((always_inline)) {
        if (s + decltype(k)::value < nst) nth(k, s);
      });
    };
    // stage s + k, k of a round.  The buffer that it fills is the one that the stage before read.
    if (wr * NR * 16 >= t.rows) {  // none of the tile's rows: this wavefront only fetches
      rounds([&](auto which, int s) __attribute__((always_inline)) {
        constexpr int k = decltype(which)::value;
        using Fill = std::integral_constant<int, k + BUFS - 1>;
        tile_for<0, LOADS>([&](auto l) __attribute__((always_inline)) { issue_one(rbuf(Fill{}), cbuf(Fill{}), s + k + BUFS - 1, l); });
        issue_s(sbuf(Fill{}), s + k + BUFS - 1);
        wait_tile<(BUFS - 2) * (LOADS + 1)>();
      });
    } else {
      using First = std::integral_constant<int, 0>;
      rv[0] = rfrag(rbuf(First{}), 0);
#pragma unroll
      for (int j = 0; j < NC; ++j) cv[j] = cfrag(cbuf(First{}), j);
      read_scales(sbuf(First{}));
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = CARRY; i < NR; ++i) carried[i] = 0.f;
      rounds([&](auto which, int s) __attribute__((always_inline)) {
        constexpr int k = decltype(which)::value;
        using Next = std::integral_constant<int, k + 1>;
        using Fill = std::integral_constant<int, k + BUFS - 1>;
        stage(rbuf(which), rbuf(Next{}), cbuf(Next{}), sbuf(Next{}), rbuf(Fill{}), cbuf(Fill{}), sbuf(Fill{}), s + k);
      });
      tile_for<LAST - 3, LAST>([&](auto n) __attribute__((always_inline)) { add(n, carried); });
    }
    wait_tile<0>();  // the last loads into LDS land before it is given back
  }

  // lane (l16, kq): row l16 of a fragment, columns 8 * (kq >> 1) .. + 7 of column tile
  // j + (kq & 1) after the exchange
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int q = (wr * NR + i) * 16 + l16;
    uint16_t* const to = A.out + A.T.row(t.row0 + min(q, t.rows - 1)) * A.ld_out;
#pragma unroll
    for (int j = 0; j < NC; j += 2) {
      using E = Elem<DT>;
      const f32x4_t a = acc[i][j], b = acc[i][j + 1];
      const auto lo = __builtin_amdgcn_permlane16_swap(E::pack(a[0], a[1]), E::pack(b[0], b[1]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(E::pack(a[2], a[3]), E::pack(b[2], b[3]), false, false);
      const int c = c0 + (wc * NC + j + (kq & 1)) * 16 + 8 * (kq >> 1);
      const uint32_t o[4] = {lo[0], hi[0], lo[1], hi[1]};
      if (q < t.rows && c < cols) store_words<4>(to + c, o);
    }
  }
}

}  // namespace sgmv_dev
