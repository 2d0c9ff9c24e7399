// The tiled matrix product behind the grouped calls.
//
// One workgroup makes a BR x BC tile of the output with MFMA 16x16 tiles: BR output rows (rows
// of a group, or rows of dW) by BC output columns.  Both operands come in stages of 128 bytes
// along the contracted dimension (64 16-bit elements, or 256 4-bit ones) by direct
// global-to-LDS loads into one of two stage buffers while the other is multiplied, so a stage
// costs one barrier and its loads have the whole previous stage to arrive.
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
//   kAcross: 32-byte column block p of contracted row k sits in block p ^ spread(k); the 16
//            rows that one transposing read touches then cover the banks evenly.
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

#include "sgmv_rows.h"

namespace sgmv_dev {

enum Form { kAlong, kAcross };
constexpr int kMx4 = 2;  // element type of the tile product beside SGMV_F16 and SGMV_BF16

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) void tile_lds_void;
typedef __attribute__((address_space(1))) void tile_global_void;

__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// 16 bytes per lane from src into LDS at dst + 16 * lane (dst the same for the wavefront)
__device__ inline void to_lds(const char* src, uint4* dst) {
  __builtin_amdgcn_global_load_lds((tile_global_void*)src, (tile_lds_void*)dst, 16, 0, 0);
}

// every global load of this wavefront has landed, and every LDS access of it is done
__device__ inline void wait_stage() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt 0, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

struct TileArgs {
  RowTab T;
  Share share;
  const char *r, *c;                  // row and column operands
  const uint8_t *r_scale, *c_scale;   // kMx4
  uint16_t* out;
  int64_t ld_r, ld_c, ld_out;         // bytes between rows of r and c; elements of out
  int64_t c_group, out_group;         // bytes between groups of c; elements of out
  int32_t rows, cols, depth;          // dW: output rows; output columns; contracted bytes of a
                                      // row (kAlong) or contracted rows (kAcross)
};

template <int DT, Form RF, Form CF, bool DW, int BR, int BC, int WR, int WC>
struct Tile {
  static constexpr int NW = WR * WC, TH = 64 * NW;
  static constexpr int NR = BR / WR / 16, NC = BC / WC / 16;  // fragments of a wavefront
  static constexpr int RI = BR / 8 / NW, CI = BC / 8 / NW;    // loads of a wavefront per stage
  static_assert(RI * 8 * NW == BR && CI * 8 * NW == BC && NC % 2 == 0, "");
  static_assert(NR >= NC, "column fragments are fetched one to a row step");
  static_assert(!DW || BR == BC, "dW shares its row indices between the operands");

  struct Stage {
    uint4 r[BR * 8];
    uint4 c[BC * 8];
  };
  struct Scales {  // [lane group][wavefront tile][row of 16][fragment][half stage]
    uint8_t r[4][WR][16][NR][2];
    uint8_t c[4][WC][16][NC][2];
  };

  static __device__ int spread(int B, int k) {
    const int j = k & 3, q = (k >> 3) & 3;
    return B >= 256 ? j | (q << 2) : B == 128 ? j | ((q & 1) << 2) : (j >> 1) | ((q & 1) << 1);
  }
};

constexpr int kTileXcds = 8;

// place `i` of R x C tiles taken in bands of 8 rows, columns outer within a band: the tiles
// that run together then share few row and column operands
__device__ inline void band_order(int i, int R, int C, int* r, int* c) {
  constexpr int H = 8;
  const int band = i / (H * C), in = i - band * H * C, h = min(H, R - band * H);
  *c = in / h;
  *r = band * H + in - *c * h;
}

template <int DT, Form RF, Form CF, bool DW, int BR, int BC, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void tile_kernel(TileArgs A) {
  using C = Tile<DT, RF, CF, DW, BR, BC, WR, WC>;
  constexpr int NR = C::NR, NC = C::NC, RI = C::RI, CI = C::CI;
  constexpr int OUT = DT;
  __shared__ typename C::Stage b0, b1;
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
    const TileList list(A.T, BR, true);
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
      rk[i] = (w * RI + i) * (64 / L) + lane / L;
      const int p = lane % L, col = 16 * ((p >> 1) ^ C::spread(BR, rk[i])) + 8 * (p & 1);
      rp[i] = A.r + 2 * min(r0 + col, A.rows - 8);
    }
  }
#pragma unroll
  for (int i = 0; i < CI; ++i) {
    if constexpr (CF == kAlong) {
      const int q = (w * CI + i) * 8 + lane / 8;
      ck[i] = 16 * ((lane & 7) ^ ((q >> 1) & 7));
      cp[i] = cbase + min(c0 + q, A.cols - 1) * A.ld_c + ck[i];
    } else {
      constexpr int L = BC / 8;
      ck[i] = (w * CI + i) * (64 / L) + lane / L;
      const int p = lane % L, col = 16 * ((p >> 1) ^ C::spread(BC, ck[i])) + 8 * (p & 1);
      cp[i] = cbase + 2 * min(c0 + col, A.cols - 8) + (DW ? 0 : ck[i] * A.ld_c);
    }
  }
  constexpr int STEP = CF == kAlong ? 128 : 64;  // of `depth`
  const int nst = (depth + STEP - 1) / STEP;

  // dW: rows of the stage after the next one to be fetched
  int jr[RI];
  auto rows_of = [&](int s) {
    if constexpr (DW) {
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const int k = s * 64 + rk[i];
        jr[i] = k < depth ? A.T.row(t.row0 + k) : -1;
      }
    }
  };
  auto issue = [&](typename C::Stage& st, int s) {
    if constexpr (DW) {
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const bool in = jr[i] >= 0;
        to_lds(in ? rp[i] + jr[i] * A.ld_r : zeros, &st.r[(w * RI + i) * 64]);
        to_lds(in ? cp[i] + A.share.div(jr[i]) * A.ld_c : zeros, &st.c[(w * CI + i) * 64]);
      }
      rows_of(s + 1);
    } else {
      const int64_t rs = static_cast<int64_t>(s) * 128;
      const int64_t cs = CF == kAlong ? rs : s * 64 * A.ld_c;
      const int left = depth - s * STEP;
      const int rleft = CF == kAlong ? left : 2 * left;  // r lies along its rows: bytes
#pragma unroll
      for (int i = 0; i < RI; ++i)
        to_lds(rk[i] < rleft ? rp[i] + rs : zeros, &st.r[(w * RI + i) * 64]);
#pragma unroll
      for (int i = 0; i < CI; ++i)
        to_lds(ck[i] < left ? cp[i] + cs : zeros, &st.c[(w * CI + i) * 64]);
    }
  };
  auto fragment = [&](auto form, auto width, const uint4* base, int tile16, int u) -> uint4 {
    if constexpr (decltype(form)::value == kAlong) {
      return base[(tile16 * 16 + l16) * 8 + ((u * 4 + kq) ^ ((l16 >> 1) & 7))];
    } else {
      constexpr int B = decltype(width)::value;
      const int k = u * 32 + kq * 8 + (l16 >> 2);
      const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + k * B +
                          16 * (tile16 ^ C::spread(B, k)) + 4 * (l16 & 3);
      typedef __attribute__((address_space(3))) s16x4_t lds4;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * B));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return make_uint4(a.x, a.y, b.x, b.y);
    }
  };
  auto rfrag = [&](const typename C::Stage& st, int i, int u) {
    return fragment(std::integral_constant<Form, RF>{}, std::integral_constant<int, BR>{}, st.r,
                    wr * NR + i, u);
  };
  auto cfrag = [&](const typename C::Stage& st, int j, int u) {
    return fragment(std::integral_constant<Form, CF>{}, std::integral_constant<int, BC>{}, st.c,
                    wc * NC + j, u);
  };
  // One stage: 2 * NR steps of NC MFMAs, one row fragment each.  The next step's row fragment
  // is read during a step, and the second half's column fragments during the first half's last
  // steps; the fences keep the compiler from hoisting more reads than there are registers for.
  auto stage = [&](const typename C::Stage& st, typename C::Stage& next, int s) {
    uint4 cv[2][NC], rv[2];
#pragma unroll
    for (int j = 0; j < NC; ++j) cv[0][j] = cfrag(st, j, 0);
    rv[0] = rfrag(st, 0, 0);
    issue(next, s + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 2 * NR; ++n) {
      const int u = n / NR, i = n % NR;
      if (n + 1 < 2 * NR) rv[(n + 1) & 1] = rfrag(st, (n + 1) % NR, (n + 1) / NR);
      if (u == 0 && i >= NR - NC) cv[1][i - (NR - NC)] = cfrag(st, i - (NR - NC), 1);
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[i][j] = Elem<DT>::mfma(cv[u][j], rv[n & 1], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // stages in pairs, one to a buffer (an odd count's last stage, and the one fetched behind the
  // end, are zeros): no branch inside the loop, which keeps the accumulators where they are
  if (nst > 0) {
    rows_of(0);
    issue(b0, 0);
    for (int s = 0; s < nst; s += 2) {
      wait_stage();
      stage(b0, b1, s);
      wait_stage();
      stage(b1, b0, s + 1);
    }
    wait_stage();  // the last loads into LDS land before the workgroup can end
  }

  // lane (l16, kq): row l16 of a fragment, columns 8 * (kq >> 1) .. + 7 of column tile
  // j + (kq & 1) after the exchange
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int q = (wr * NR + i) * 16 + l16;
    bool in;
    int64_t row;
    if constexpr (DW) {
      in = r0 + q < A.rows;
      row = r0 + q;
    } else {
      in = q < t.rows;
      row = in ? A.T.row(t.row0 + q) : 0;
    }
    uint16_t* to = A.out + (DW ? static_cast<int64_t>(t.g) * A.out_group : 0) + row * A.ld_out;
#pragma unroll
    for (int j = 0; j < NC; j += 2) {
      using E = Elem<OUT>;
      const f32x4_t a = acc[i][j], b = acc[i][j + 1];
      const auto lo = __builtin_amdgcn_permlane16_swap(E::pack(a[0], a[1]), E::pack(b[0], b[1]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(E::pack(a[2], a[3]), E::pack(b[2], b[3]), false, false);
      const int c = c0 + (wc * NC + j + (kq & 1)) * 16 + 8 * (kq >> 1);
      const uint32_t o[4] = {lo[0], hi[0], lo[1], hi[1]};
      if (in && c < A.cols) store_words<4>(to + c, o);
    }
  }
}

}  // namespace sgmv_dev
