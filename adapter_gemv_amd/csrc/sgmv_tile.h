// The tiled matrix product behind the grouped calls.
//
// One workgroup makes a BR x BC tile of the output with MFMA 16x16 tiles: BR output rows (rows
// of a group, or rows of dW) by BC output columns.  Both operands come in stages of 128 bytes
// along the contracted dimension (64 16-bit elements, or 256 4-bit ones) by direct
// global-to-LDS loads into one of two or three stage buffers while another is multiplied, so a
// stage costs one barrier and its loads have at least most of the previous stage to arrive.
//
// An operand lies either along its rows (kAlong: each tile row's stage is 128 contiguous
// bytes, a fragment is one 16-byte LDS read per lane) or across them (kAcross: the contracted
// dimension is the row index; a stage is 64 rows of the tile's width, a fragment is two
// transposing LDS reads, ds_read_b64_tr_b16, each of a 4 x 16 block per 16 lanes).
//
// The direct loads put lane l's 16 bytes at l * 16, so the placement that keeps fragment
// reads free of bank conflicts is made on the global side: lane l fetches the piece that
// belongs in its slot.
//   kAlong:  piece c of tile row q sits in slot c ^ ((q >> 1) & 7) of the row's 8; the 16 rows
//            of a fragment then cover all 64 banks once.
//   kAcross: one load instruction fills a slab of 1 KB with the contracted rows that no one
//            transposing read takes together (those that differ in their place in the half
//            stage's eight, h, or in the half, u), and slabs are 32 bytes further apart than
//            they are long; the 16 rows of a read then lie in 16 slabs, over all banks, at
//            constant offsets from one address per lane.
//
// Weights in 4 bits against 16-bit rows (kMxW): a stage of a weight row is 32 bytes of codes
// (kCodes); a lane reads 16 codes, one half for each half of the stage, and converts them with
// their scale to the 16-bit operand, exactly in bfloat16 for scales up to 2^125.  float16 holds an
// element times its scale for scales 2^-23 .. 2^13 (and blocks of zeros); a tile that meets another
// one starts again in bfloat16, the rows taken apart into two bfloat16 parts (8 + 3 of their 11
// bits).  A tile with infinite sums looks for scales above 2^125, and is computed again by
// mx_any_scale if it has one, as in the streaming form.
// Both sides in 4 bits (kMxBoth): the fragments are the 16x16x128 scaled MFMA's operands, whose
// blocks of 32 are the format's own; the scale bytes go through LDS in the order in which its
// byte selectors take them.
//
// Output rows are the second MFMA operand and output columns the first, so a lane holds four
// neighbouring columns of one row; v_permlane16_swap pairs two column tiles into eight, and
// every store is 16 bytes.
//
// Contracted positions past the end are zeros in both operands (lanes there fetch a block of
// zeros), so what lies behind them in memory, NaN included, takes no part.  Tile rows and
// columns past the end repeat the last one and are not stored.
#pragma once

#include <type_traits>

#include "sgmv_skinny.h"

namespace sgmv_dev {

enum Form { kAlong, kAcross, kCodes };

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
// at most N (< 16) global loads of this wavefront are in flight, and every LDS access of it is
// done; then the workgroup's barrier
template <int N>
__device__ inline void wait_stage() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(N | (7 << 4));  // vmcnt N, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

struct TileArgs {
  RowTab T;
  Share share;
  const char *r, *c;                  // row and column operands
  const uint8_t *r_scale, *c_scale;   // kMxBoth, kMxW: dense, blocks / row as depth says
  uint16_t* out;
  int64_t ld_r, ld_c, ld_out;         // bytes between rows of r and c; elements of out
  int64_t c_group, out_group;         // bytes between groups of c; elements of out
  int32_t rows, cols, depth;          // dW: output rows; output columns; contracted bytes of a
                                      // row (kAlong) or contracted rows (kAcross)
};

// kAcross, tiles of B columns: pieces of 16 bytes between slabs, contracted rows of a slab
constexpr int kSlab = 66;
constexpr int slab_rows(int B) { return 512 / B; }
// the contracted row (of the stage's 64) that is row `in` of slab q
template <int B>
__device__ inline int slab_row(int q, int in) {
  static_assert(B == 256 || B == 128, "");
  return B == 256 ? (q >> 4) * 32 + ((q >> 2) & 3) * 8 + in * 4 + (q & 3)
                  : (in >> 1) * 32 + (q >> 2) * 8 + (in & 1) * 4 + (q & 3);
}

template <Mode M, int BR, int BC, int WR, int WC>
struct Tile {
  static constexpr Form RF = M == kDw ? kAcross : kAlong;
  static constexpr Form CF = M == kDx || M == kDw ? kAcross : M == kMxW ? kCodes : kAlong;
  static constexpr bool DW = M == kDw;
  static constexpr int NW = WR * WC, TH = 64 * NW;
  static constexpr int NR = BR / WR / 16, NC = BC / WC / 16;  // fragments of a wavefront
  static constexpr int CP = M == kMxW ? 2 : 8;                // 16-byte pieces of a column's stage
  static constexpr int RI = BR * 8 / 64 / NW, CI = BC * CP / 64 / NW;  // loads per stage
  static_assert(RI * 64 * NW == BR * 8 && CI * 64 * NW == BC * CP && NC % 2 == 0, "");
  static_assert(NR % 4 == 0 && NR >= NC, "runs of row fragments");
  static_assert(!DW || BR == BC, "dW shares its row indices between the operands");
  static_assert(M != kMxBoth || (BR == BC && BR + BC == TH), "one thread to a row's or column's scales");
  static constexpr int SB = M == kMxW ? 2 * BC / TH : 1;      // kMxW: a thread's scale bytes of a stage
  static_assert(M != kMxW || SB * TH == 2 * BC, "the same number of scale bytes for each thread");

  // scale bytes as a lane takes them.  kMxBoth: [lane group][wavefront tile][row of 16]
  // [fragment][half] of the rows, then of the columns; kMxW: [half][wavefront tile][row of 16]
  // [fragment] of the columns
  static constexpr int SC = M == kMxBoth ? 8 * BR : 0;  // where the columns' start
  struct MxScales {
    alignas(16) uint8_t b[M == kMxBoth ? 8 * (BR + BC) : M == kMxW ? 2 * BC : 16];
  };
  // LDS buffers.  kForward's 256 x 256 tile has room for a third one of the column operand: the
  // weight comes from HBM, the rows from the L2, so it is fetched two stages ahead.
  struct RBuf {
    u32x4_t v[RF == kAcross ? BR / 8 * kSlab : BR * 8];
  };
  struct CBuf {
    u32x4_t v[CF == kAcross ? BC / 8 * kSlab : BC * CP];
  };
  static constexpr int DC = M == kForward && BR == 256 ? 3 : 2;
};

using sgmv_host::kTileXcds;

// place `i` of R x C tiles taken in bands of 8 rows, columns outer within a band: the tiles
// that run together then share few row and column operands
__device__ inline void band_order(int i, int R, int C, int* r, int* c) {
  constexpr int H = 8;
  const int band = i / (H * C), in = i - band * H * C, h = min(H, R - band * H);
  *c = in / h;
  *r = band * H + in - *c * h;
}

// DT: type of the 16-bit operands and of the output.  WHOLE: kMxBoth, a row has a multiple of 8
// blocks, so a stage's 8 scale bytes are one aligned load; kDw, the rows come through perm.
template <int DT, Mode M, int BR, int BC, int WR, int WC, bool WHOLE = true>
__global__ __launch_bounds__(64 * WR * WC, 2) void tile_kernel(TileArgs A) {
  using C = Tile<M, BR, BC, WR, WC>;
  constexpr int NR = C::NR, NC = C::NC, RI = C::RI, CI = C::CI;
  constexpr Form RF = C::RF, CF = C::CF;
  constexpr bool DW = C::DW;
  __shared__ typename C::RBuf rb0, rb1;
  __shared__ typename C::CBuf cb0, cb1;
  __shared__ typename C::MxScales sb0, sb1;
  constexpr int DC = C::DC;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
  const int wr = w / WC, wc = w % WC;

  // which tile: workgroup b runs on XCD b % 8; each XCD takes a contiguous eighth of the tiles
  // (dW: of every group's tiles, whose costs differ from group to group)
  const int ct = (A.cols + BC - 1) / BC, xcd = blockIdx.x % kTileXcds, at = blockIdx.x / kTileXcds;
  RowTile t;
  int r0 = 0, c0, depth;
  if constexpr (DW) {
    const int rt = (A.rows + BR - 1) / BR, per = (rt * ct + kTileXcds - 1) / kTileXcds;
    const int in = xcd * per + at % per;
    t.g = at / per;
    if (in >= rt * ct) return;
    t.row0 = A.T.starts ? A.T.starts[t.g] : 0;
    t.rows = A.T.starts ? A.T.starts[t.g + 1] - t.row0 : A.T.n;
    band_order(in, rt, ct, &r0, &c0);
    r0 *= BR;
    depth = t.rows;
  } else {
    const TileList list(A.T, BR);
    const int all = list.count * ct, per = all / kTileXcds, more = all % kTileXcds;
    if (at >= per + (xcd < more)) return;
    int m;
    band_order(xcd * per + min(xcd, more) + at, list.count, ct, &m, &c0);
    t = list.find(m);
    depth = A.depth;
    if (t.g == A.T.G) depth = 0;  // rows of no group: zeros
  }
  c0 *= BC;

  f32x4_t acc[NR][NC];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  bool held = true;  // kMxW, float16: every weight so far, exactly

  const char* const zeros = reinterpret_cast<const char*>(kZeros);
  const char* const cbase = A.c + (DW ? 0 : static_cast<int64_t>(t.g) * A.c_group);
  // kAlong: where this lane's pieces of the stage start, and how far into the row
  const char *rp[RI], *cp[CI];
  int rk[RI], ck[CI];  // kAlong: byte of the row; kAcross: contracted row of the stage
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    if constexpr (RF == kAlong) {
      const int q = (w * RI + i) * 8 + lane / 8;
      rk[i] = 16 * ((lane & 7) ^ ((q >> 1) & 7));
      const int j = depth ? A.share.div(A.T.row(t.row0 + min(q, t.rows - 1))) : 0;
      rp[i] = A.r + j * A.ld_r + rk[i];
    } else {
      constexpr int L = BR / 8;  // lanes to a contracted row
      rk[i] = slab_row<BR>(w * RI + i, lane / L);
      rp[i] = A.r + 2 * min(r0 + 8 * (lane % L), A.rows - 8);
    }
  }
#pragma unroll
  for (int i = 0; i < CI; ++i) {
    if constexpr (CF == kAlong) {
      const int q = (w * CI + i) * 8 + lane / 8;
      ck[i] = 16 * ((lane & 7) ^ ((q >> 1) & 7));
      cp[i] = cbase + min(c0 + q, A.cols - 1) * A.ld_c + ck[i];
    } else if constexpr (CF == kCodes) {
      const int q = (w * CI + i) * 32 + lane / 2;
      ck[i] = 16 * (lane & 1);
      cp[i] = cbase + min(c0 + q, A.cols - 1) * A.ld_c + ck[i];
    } else {
      constexpr int L = BC / 8;
      ck[i] = slab_row<BC>(w * CI + i, lane / L);
      cp[i] = cbase + 2 * min(c0 + 8 * (lane % L), A.cols - 8) + (DW ? 0 : ck[i] * A.ld_c);
    }
  }
  constexpr int STEP = CF == kAcross ? 64 : 128;  // of `depth`
  const int nst = (depth + STEP - 1) / STEP;

  // dW: the rows of the next stage to be fetched (past the end the last one, whose address the
  // zeros then replace; the empty asm keeps the address from being computed under a branch)
  int jr[RI];
  auto rows_of = [&](int s) {
    if constexpr (DW) {
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const int k = t.row0 + min(s * 64 + rk[i], depth - 1);
        jr[i] = WHOLE ? A.T.perm[k] : k;
      }
    }
  };
  constexpr int RS = RF == kAcross ? kSlab : 64, CS = CF == kAcross ? kSlab : 64;
  // the k-th load of stage s (kDw: the k-th of each operand), of LOADS
  constexpr int LOADS = DW ? RI : RI + CI;
  auto issue_r = [&](typename C::RBuf& to, int s, auto which) __attribute__((always_inline)) {
    constexpr int i = decltype(which)::value;
    const int left = (depth - s * STEP) * (CF == kAcross ? 2 : 1);  // r lies along its rows: bytes
    to_lds(rk[i] < left ? rp[i] + static_cast<int64_t>(s) * 128 : zeros, &to.v[(w * RI + i) * RS]);
  };
  auto issue_c = [&](typename C::CBuf& to, int s, auto which) __attribute__((always_inline)) {
    constexpr int i = decltype(which)::value;
    const int64_t cs = CF == kAlong ? s * int64_t{128} : CF == kCodes ? s * int64_t{32} : s * 64 * A.ld_c;
    const int left = (depth - s * STEP) / (CF == kCodes ? 4 : 1);
    const char* c = cp[i] + cs;
    if constexpr (CF == kAcross) asm("" : "+v"(c));  // keeps its computation out of a branch
    to_lds(ck[i] < left ? c : zeros, &to.v[(w * CI + i) * CS]);
  };
  auto issue_dw = [&](typename C::RBuf& rt, typename C::CBuf& ct, int s, auto which) __attribute__((always_inline)) {
    constexpr int k = decltype(which)::value;
    const bool in = s * 64 + rk[k] < depth;
    const char *r = rp[k] + jr[k] * A.ld_r, *c = cp[k] + A.share.div_any(jr[k]) * A.ld_c;
    asm("" : "+v"(r), "+v"(c));
    to_lds(in ? r : zeros, &rt.v[(w * RI + k) * RS]);
    to_lds(in ? c : zeros, &ct.v[(w * CI + k) * CS]);
    if constexpr (k == LOADS - 1) rows_of(s + 1);
  };
  // one of the loads behind stage s: of the rows of the next one, or of the columns of the last
  // one that fits
  auto issue_one = [&](typename C::RBuf& rt, typename C::CBuf& ct, int s, auto which) __attribute__((always_inline)) {
    constexpr int k = decltype(which)::value;
    if constexpr (DW) issue_dw(rt, ct, s + 1, which);
    else if constexpr (k < RI) issue_r(rt, s + 1, which);
    else issue_c(ct, s + DC - 1, std::integral_constant<int, k - RI>{});
  };
  // scales: this thread's row or column of the tile, 8 bytes a stage (kMxBoth), or one block of
  // a column, 1 byte (kMxW); fetched a stage ahead and put into LDS behind the products
  const uint8_t* sp = nullptr;
  int blocks = 0;       // of a row
  int sto = 0;          // where in MxScales
  uint32_t sv[2] = {0, 0};
  if constexpr (M == kMxBoth) {
    blocks = depth / 16;
    const bool is_r = tid < BR;
    const int q = is_r ? tid : tid - BR, N = is_r ? NR : NC;
    sto = (is_r ? 0 : C::SC) + ((q / (16 * N)) * 16 + q % 16) * N * 2 + q / 16 % N * 2;
    static_assert(WR * NR == WC * NC, "one distance between lane groups");
    if (depth)
      sp = is_r ? A.r_scale + static_cast<int64_t>(A.share.div(A.T.row(t.row0 + min(q, t.rows - 1)))) * blocks
                : A.c_scale + (static_cast<int64_t>(t.g) * A.cols + min(c0 + q, A.cols - 1)) * blocks;
  } else if constexpr (M == kMxW) {
    blocks = depth / 64;
    const int q = tid % BC;  // and block tid / BC of the stage's two, or both
    sto = ((tid / BC * WC + q / (16 * NC)) * 16 + q % 16) * NC + q / 16 % NC;
    if (depth)
      sp = A.c_scale + (static_cast<int64_t>(t.g) * A.cols + min(c0 + q, A.cols - 1)) * blocks;
  }
  auto fetch_scales = [&](int s) {
    if constexpr (M == kMxBoth && WHOLE) {
      const u32x2_t v = *(gptr<const u32x2_t>)global_ptr(sp + 8 * min(s, blocks / 8 - 1));
      sv[0] = v.x, sv[1] = v.y;
    } else if constexpr (M == kMxBoth) {
      sv[0] = sv[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = global_ptr(sp)[min(8 * s + i, blocks - 1)];
        sv[i / 4] |= (8 * s + i < blocks ? b : 127u) << (8 * (i & 3));
      }
    } else if constexpr (M == kMxW) {
#pragma unroll
      for (int h = 0; h < C::SB; ++h) {
        const int k = 2 * s + tid / BC + h;
        const uint32_t b = global_ptr(sp)[min(k, blocks - 1)];
        sv[h] = k < blocks ? b : 127u;
      }
    }
  };
  auto store_scales = [&](typename C::MxScales& to) {  // no branch: see the loop below
    if constexpr (M == kMxBoth) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint16_t*>(to.b + sto + k * (WR * NR * 32)) =
            static_cast<uint16_t>(__builtin_amdgcn_perm(sv[1], sv[0], k | (4 + k) << 8));
    } else if constexpr (M == kMxW) {
#pragma unroll
      for (int h = 0; h < C::SB; ++h) to.b[sto + h * BC] = static_cast<uint8_t>(sv[h]);
    }
  };
  // Fragment reads.  Each address is one lane offset, made here, plus a constant: the compiler
  // tells LDS buffers apart (and so does not wait for loads into another one) only where the
  // address is a few steps from the buffer's name.
  auto lane_at = [&](auto form, int tile, int u) __attribute__((always_inline)) {
    constexpr Form F = decltype(form)::value;
    if constexpr (F == kAlong)  // 16-byte pieces
      return (tile * 16 + l16) * 8 + ((M == kMxW ? kq * 2 + u : u * 4 + kq) ^ ((l16 >> 1) & 7));
    else if constexpr (F == kCodes)  // 8-byte pieces
      return (tile * 16 + l16) * 4 + kq;
    else  // 8-byte pieces
      return (4 * kq + (l16 >> 2)) * kSlab * 2 + (l16 & 3) + 4 * tile;
  };
  using FormR = std::integral_constant<Form, RF>;
  using FormC = std::integral_constant<Form, CF>;
  int ro[2] = {lane_at(FormR{}, wr * NR, 0), lane_at(FormR{}, wr * NR, 1)};
  int co[2] = {lane_at(FormC{}, wc * NC, 0), lane_at(FormC{}, wc * NC, 1)};
  asm("" : "+v"(ro[0]), "+v"(ro[1]), "+v"(co[0]), "+v"(co[1]));
  auto fragment = [&](auto form, auto width, const u32x4_t* base, const int* at, int i,
                      int u) __attribute__((always_inline)) -> uint4 {
    if constexpr (decltype(form)::value == kAlong) {
      const u32x4_t v = base[at[u] + i * 128];
      return make_uint4(v.x, v.y, v.z, v.w);
    } else {
      constexpr int B = decltype(width)::value;
      typedef __attribute__((address_space(3))) s16x4_t lds4;
      const u32x2_t* p = reinterpret_cast<const u32x2_t*>(base) + at[0] + 4 * i +
                         u * (B == 256 ? 16 * kSlab * 2 : B / 2);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + B / 4));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return make_uint4(a.x, a.y, b.x, b.y);
    }
  };
  auto rfrag = [&](const typename C::RBuf& from, int i, int u) __attribute__((always_inline)) {
    return fragment(FormR{}, std::integral_constant<int, BR>{}, from.v, ro, i, u);
  };
  auto cfrag = [&](const typename C::CBuf& from, int j, int u) __attribute__((always_inline)) {
    return fragment(FormC{}, std::integral_constant<int, BC>{}, from.v, co, j, u);
  };
  // One stage: row fragments in runs of NQ, each 2 * NQ steps (both halves of the stage) of NC
  // MFMAs on one row fragment.  The next step's row fragment is read during a step, the second
  // half's column fragments during the first run's steps of the first half, and each of the
  // first steps issues one of the loads behind the stage: all at once, at the stage's start,
  // they hold up every wavefront for as long as the CU takes to accept 64 KB (8192^3, bfloat16:
  // forward 1370, dx 1350, dW 1270 TFLOP/s that way; 1470, 1400, 1300 spread out).  With two
  // workgroups to a CU the other one has work meanwhile, and what counts is that the loads
  // arrive in a stage of half the length (8 groups of 1024 rows, 4096 x 4096, 128 x 128 tiles:
  // 913 TFLOP/s at once, 871 spread out).  The fences keep the compiler from hoisting more reads
  // than there are registers for.
  constexpr int NQ = NR / 4;
  constexpr bool SPREAD = BC == 256;
  constexpr int PER = NC > NQ ? NC / NQ : 1, FROM = NQ - NC / PER;  // column fragments of a step
  auto stage = [&](const typename C::RBuf& rb, const typename C::CBuf& cb, const typename C::MxScales& sb,
                   typename C::RBuf& rn, typename C::CBuf& cn, typename C::MxScales& sn, int s,
                   auto split) __attribute__((always_inline)) {
    constexpr bool SPLIT = decltype(split)::value;
    constexpr int WT = SPLIT ? SGMV_BF16 : DT;  // kMxW: type of the converted weights
    uint4 cv[2][NC], rv[2];
    uint32_t rs[NR / 2], cs[NC / 2];
    if constexpr (M == kMxW) {
      u32x2_t codes[NC];
      static_assert(NC == 4, "a lane's scales are one word");
      const uint32_t scales = reinterpret_cast<const uint32_t*>(sb.b)[((kq >> 1) * WC + wc) * 16 + l16];
#pragma unroll
      for (int j = 0; j < NC; ++j)
        codes[j] = reinterpret_cast<const u32x2_t*>(cb.v)[co[0] + 64 * j];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float f = mx_scale_at(scales, j);
        if constexpr (DT == SGMV_F16 && !SPLIT) held &= f16_holds(scales >> (8 * j) & 255u, codes[j].x | codes[j].y);
        cv[0][j] = mx_eight<WT>(codes[j].x, f);
        cv[1][j] = mx_eight<WT>(codes[j].y, f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) cv[0][j] = cfrag(cb, j, 0);
    }
    if constexpr (M == kMxBoth) {
      const uint32_t* r = reinterpret_cast<const uint32_t*>(sb.b + ((kq * WR + wr) * 16 + l16) * NR * 2);
      const uint32_t* c = reinterpret_cast<const uint32_t*>(sb.b + C::SC + ((kq * WC + wc) * 16 + l16) * NC * 2);
#pragma unroll
      for (int i = 0; i < NR / 2; ++i) rs[i] = r[i];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) cs[j] = c[j];
    }
    rv[0] = rfrag(rb, 0, 0);
    fetch_scales(s + 1);
    if constexpr (!SPREAD) tile_for<0, LOADS>([&](auto k) __attribute__((always_inline)) { issue_one(rn, cn, s, k); });
    __builtin_amdgcn_sched_barrier(0);
    tile_for<0, 2 * NR>([&](auto step) __attribute__((always_inline)) {
      constexpr int n = decltype(step)::value, u = n / NQ % 2, i = n / (2 * NQ) * NQ + n % NQ;
      constexpr int n1 = n + 1, u1 = n1 / NQ % 2, i1 = n1 / (2 * NQ) * NQ + n1 % NQ;
      if constexpr (n1 < 2 * NR) rv[n1 & 1] = rfrag(rb, i1, u1);
      if constexpr (SPREAD && n < LOADS) issue_one(rn, cn, s, step);
      if constexpr (M != kMxW && n < NQ && n >= FROM) {
#pragma unroll
        for (int j = 0; j < PER; ++j) cv[1][(n - FROM) * PER + j] = cfrag(cb, (n - FROM) * PER + j, 1);
      }
      uint4 hi, lo;
      if constexpr (SPLIT) f16_split(rv[n & 1], &hi, &lo);
      tile_for<0, NC>([&](auto col) __attribute__((always_inline)) {
        constexpr int j = decltype(col)::value;
        if constexpr (M == kMxBoth) {
          const uint4 a = cv[u][j], b = rv[n & 1];
          const i32x8_t av = {int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};
          const i32x8_t bv = {int(b.x), int(b.y), int(b.z), int(b.w), 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              av, bv, acc[i][j], 4, 4, (j % 2) * 2 + u, cs[j / 2], (i % 2) * 2 + u, rs[i / 2]);
        } else if constexpr (SPLIT) {
          acc[i][j] = Elem<SGMV_BF16>::mfma(cv[u][j], hi, acc[i][j]);
          acc[i][j] = Elem<SGMV_BF16>::mfma(cv[u][j], lo, acc[i][j]);
        } else {
          acc[i][j] = Elem<DT>::mfma(cv[u][j], rv[n & 1], acc[i][j]);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    store_scales(sn);
  };

  // No branch inside the loop, which keeps the accumulators where they are: stages go in pairs
  // (an odd count's last one is zeros), or in sixes where the columns have three buffers, with
  // the remainder behind the loop; what is fetched behind the end is zeros.
  auto all_stages = [&](auto split) __attribute__((always_inline)) {
    rows_of(0);
    fetch_scales(0);
    if constexpr (DW) {
      tile_for<0, RI>([&](auto k) __attribute__((always_inline)) { issue_dw(rb0, cb0, 0, k); });
    } else {
      tile_for<0, RI>([&](auto k) __attribute__((always_inline)) { issue_r(rb0, 0, k); });
      tile_for<0, CI>([&](auto k) __attribute__((always_inline)) { issue_c(cb0, 0, k); });
    }
    store_scales(sb0);
    if constexpr (DC == 2) {
      for (int s = 0; s < nst; s += 2) {
        wait_stage<0>();
        stage(rb0, cb0, sb0, rb1, cb1, sb1, s, split);
        wait_stage<0>();
        stage(rb1, cb1, sb1, rb0, cb0, sb0, s + 1, split);
      }
    } else {
      __shared__ typename C::CBuf cb2;
      tile_for<0, CI>([&](auto k) __attribute__((always_inline)) { issue_c(cb1, 1, k); });
      auto nth = [&](auto which, int s) __attribute__((always_inline)) {
        constexpr int k = decltype(which)::value;
        typename C::RBuf &r = k % 2 ? rb1 : rb0, &rn = k % 2 ? rb0 : rb1;
        typename C::CBuf &c = k % 3 == 0 ? cb0 : k % 3 == 1 ? cb1 : cb2;
        typename C::CBuf &cn = k % 3 == 0 ? cb2 : k % 3 == 1 ? cb0 : cb1;
        wait_stage<CI>();
        stage(r, c, sb0, rn, cn, sb0, s + k, split);
      };
      int s = 0;
      for (; s + 6 <= nst; s += 6) tile_for<0, 6>([&](auto k) __attribute__((always_inline)) { nth(k, s); });
      tile_for<0, 5>([&](auto k) __attribute__((always_inline)) {
        if (s + decltype(k)::value < nst) nth(k, s);
      });
    }
    wait_stage<0>();  // the last loads into LDS land before it is used again or given back
  };
  if (nst > 0) {
    all_stages(std::false_type{});
    if constexpr (M == kMxW && DT == SGMV_F16) {
      if (!__syncthreads_and(held)) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int j = 0; j < NC; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        all_stages(std::true_type{});
      }
    }
  }

  // lane (l16, kq): row l16 of a fragment, columns 8 * (kq >> 1) .. + 7 of column tile
  // j + (kq & 1) after the exchange
  int row[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int q = (wr * NR + i) * 16 + l16;
    row[i] = DW ? r0 + q : t.row0 + min(q, t.rows - 1);
  }
  if (!DW && A.T.perm) {
#pragma unroll
    for (int i = 0; i < NR; ++i) row[i] = A.T.perm[row[i]];
  }
  float zero = 0.f;  // kMxW: NaN once a sum is not finite
  uint16_t* const out = A.out + (DW ? static_cast<int64_t>(t.g) * A.out_group : 0);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int q = (wr * NR + i) * 16 + l16;
    const bool in = DW ? row[i] < A.rows : q < t.rows;
    uint16_t* to = out + row[i] * A.ld_out;
#pragma unroll
    for (int j = 0; j < NC; j += 2) {
      using E = Elem<DT>;
      const f32x4_t a = acc[i][j], b = acc[i][j + 1];
      const auto lo = __builtin_amdgcn_permlane16_swap(E::pack(a[0], a[1]), E::pack(b[0], b[1]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(E::pack(a[2], a[3]), E::pack(b[2], b[3]), false, false);
      const int c = c0 + (wc * NC + j + (kq & 1)) * 16 + 8 * (kq >> 1);
      const uint32_t o[4] = {lo[0], hi[0], lo[1], hi[1]};
      if (in && c < A.cols) store_words<4>(to + c, o);
      if constexpr (M == kMxW)
#pragma unroll
        for (int v = 0; v < 4; ++v) zero = fmaf(a[v], 0.f, fmaf(b[v], 0.f, zero));
    }
  }
  if constexpr (M == kMxW) {
    if (nst > 0)
      mx_mend<DT, false>({A.T, A.share, reinterpret_cast<const uint16_t*>(A.r), nullptr, A.ld_r / 2, A.c, A.c_scale,
                          A.c_group, A.out, A.ld_out, A.depth / 2, A.cols}, t, c0, BC, zero == 0.f);
  }
}

template <int DT, Mode M, int BR, int BC, int WR, int WC, bool WHOLE = true>
hipError_t launch_tile(hipStream_t s, const TileArgs& A, const sgmv_host::Launch& L) {
  tile_kernel<DT, M, BR, BC, WR, WC, WHOLE><<<static_cast<uint32_t>(L.workgroups), 64 * WR * WC, 0, s>>>(A);
  return hipGetLastError();
}

template <Mode M, bool WHOLE = true>
hipError_t launch_tiles(int32_t dtype, hipStream_t s, const TileArgs& A, const sgmv_host::Launch& L) {
  const bool f16 = dtype == SGMV_F16;
  if constexpr (M == kMxW)
    if (L.rows == 128 && L.cols == 256)
      return f16 ? launch_tile<SGMV_F16, M, 128, 256, 1, 4, WHOLE>(s, A, L)
                 : launch_tile<SGMV_BF16, M, 128, 256, 1, 4, WHOLE>(s, A, L);
  if (L.rows == 256)
    return f16 ? launch_tile<SGMV_F16, M, 256, 256, 2, 4, WHOLE>(s, A, L)
               : launch_tile<SGMV_BF16, M, 256, 256, 2, 4, WHOLE>(s, A, L);
  return f16 ? launch_tile<SGMV_F16, M, 128, 128, 2, 2, WHOLE>(s, A, L)
             : launch_tile<SGMV_BF16, M, 128, 128, 2, 2, WHOLE>(s, A, L);
}

}  // namespace sgmv_dev
