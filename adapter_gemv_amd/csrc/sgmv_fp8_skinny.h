// Products of a few rows per group with 8-bit weights: the form for decode batches, bound by
// streaming the weight.
//
// As for 16-bit weights, one workgroup makes 16 output columns for at most 32 rows of one group, its
// wavefronts take turns along the contracted dimension, and each streams its units through a ring of
// its own in LDS, three units ahead; their sums are added at the end, in the same order always.  A
// unit is one block of 128: 128 bytes of each of 16 weight rows, one MFMA 16x16x128 for 16 rows of x,
// whose sums are added to the wavefront's times the block's two scales.
//
// x comes in 8 bits, or in 16 (X16) and is taken to 8 here, by every workgroup for itself: a lane has
// 32 of a block's elements (16 * kq .. + 15 and 64 + 16 * kq .. + 15 of row l16), so that the largest is
// two exchanges away.
//
// Bound by the stream of the weight, or by the launch and one pass over the depth: 4096 x 4096, one
// row, 6.3 us (2.7 TB/s); 5120 x 13824, one row, 21.4 us with weights from memory (3.3 TB/s); 64 rows over 46
// of 64 experts of 4096 x 1024, 34 to 38 us (5.0 to 5.7 TB/s); 16 rows over 7 of 8 of 5120 x 13824, 4.6 TB/s.
#pragma once

#include "sgmv_fp8_convert.h"
#include "sgmv_fp8_tile.h"

namespace sgmv_dev {

template <int DT, bool X16, int CT, int WAVES>
struct Fp8Skinny {
  static constexpr int D = 4;                // units of the ring
  struct Ring {
    u32x4_t v[WAVES * CT * 128];             // [wavefront][column tile][row of 16][8 pieces]
  };

  // a block of a lane's row of x
  struct Block {
    uint4 v[X16 ? 4 : 2];
    float scale;                             // !X16
  };

  template <int MT>
  static __device__ __forceinline__ void multiply_rows(const Fp8Args& A, const RowTile& t, int c0, f32x4_t (&acc)[MT][CT],
                                                       Ring& r0, Ring& r1, Ring& r2, Ring& r3) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
    const int K = A.h_in, kb = blocks_of(K);
    gptr<const uint8_t> xp[MT];
    gptr<const uint16_t> xh[MT];
    gptr<const float> xs[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = A.share.div(A.T.row(t.row0 + min(16 * m + l16, t.rows - 1)));
      if constexpr (X16) {
        xh[m] = global_ptr(A.x) + row * A.ld_x + 16 * kq;
      } else {
        xp[m] = global_ptr(A.r) + row * A.ld_r + 16 * kq;
        xs[m] = global_ptr(A.r_scale) + row * kb;
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // weights: lane l fetches a piece of row l / 8 of 8, the one that belongs in its slot (piece c
    // of row q of 16 sits in slot c ^ ((q >> 1) & 7): no bank conflicts for the reads below)
    const char* wp[CT][2];
    int wk[2];
    const char* const base = reinterpret_cast<const char*>(A.w) + static_cast<int64_t>(t.g) * A.h_in * A.h_out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      wk[h] = 16 * ((lane & 7) ^ (((8 * h + lane / 8) >> 1) & 7));
#pragma unroll
      for (int c = 0; c < CT; ++c)
        wp[c][h] = base + static_cast<int64_t>(min(c0 + 16 * c + 8 * h + lane / 8, A.h_out - 1)) * K + wk[h];
    }
    // columns of a workgroup are 16 * CT of a multiple of that: of one block
    gptr<const float> ws = global_ptr(A.w_scale) + (static_cast<int64_t>(t.g) * blocks_of(A.h_out) + c0 / 128) * kb;
    const char* const zeros = reinterpret_cast<const char*>(kZeros);
    const int n = (kb - w + WAVES - 1) / WAVES;  // this wavefront's units: w, w + WAVES, ...

    // the i-th unit of this wavefront; past the row's end (and past the last unit) zeros
    auto fetch = [&](Ring& to, int i) __attribute__((always_inline)) {
      const int at = (w + i * WAVES) * 128;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) to_lds(at + wk[h] < K ? wp[c][h] + at : zeros, &to.v[((w * CT + c) * 2 + h) * 64]);
    };
    // x at the i-th unit (past the last unit: at the row's first block), and the weight's scale
    struct Rows {
      Block x[MT];
      float ws;
    };
    auto rows_of = [&](Rows& R, int i) __attribute__((always_inline)) {
      const int b = i < n ? w + i * WAVES : 0, k0 = b * 128;
      R.ws = ws[b];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bool in = k0 + 64 * u + 16 * kq < K;
          const int at = in ? k0 + 64 * u : -16 * kq;
          if constexpr (X16) {
            R.x[m].v[2 * u] = ld16(xh[m] + at);
            R.x[m].v[2 * u + 1] = ld16(xh[m] + at + 8);
          } else {
            const u32x4_t a = *reinterpret_cast<gptr<const u32x4_t>>(xp[m] + at);
            R.x[m].v[u] = make_uint4(a.x, a.y, a.z, a.w);
          }
        }
        if constexpr (!X16) R.x[m].scale = xs[m][b];
      }
    };
    int slot[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      slot[u] = (w * CT * 16 + l16) * 8 + ((4 * u + kq) ^ ((l16 >> 1) & 7));
      asm("" : "+v"(slot[u]));  // one lane offset: see the tiled product
    }
    auto multiply = [&](const Ring& from, Rows& R, int i) __attribute__((always_inline)) {
      if (const int left = K - (w + i * WAVES) * 128; left < 128) {  // the row ends in this block
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int q = 0; q < (X16 ? 4 : 2); ++q)
            if (64 * (X16 ? q / 2 : q) + 16 * kq >= left) R.x[m].v[q] = zero4();
      }
      i32x8_t wv[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const u32x4_t a = from.v[slot[0] + c * 128], b = from.v[slot[1] + c * 128];
        wv[c] = i32x8_t{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Block& x = R.x[m];
        i32x8_t xv;
        float s;
        if constexpr (X16) {
          uint32_t top = max_halves(max_halves(top_halves(x.v[0]), top_halves(x.v[1])),
                                    max_halves(top_halves(x.v[2]), top_halves(x.v[3])));
          // of the lanes 16 and 32 apart, the four that hold the block
          const auto h = __builtin_amdgcn_permlane16_swap(top, top, false, false);
          top = max_halves(h[0], h[1]);
          const auto q = __builtin_amdgcn_permlane32_swap(top, top, false, false);
          s = block_scale<DT>(top_of(max_halves(q[0], q[1])));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2_t c = encode8<DT>(x.v[q], s);
            xv[2 * q] = int(c.x), xv[2 * q + 1] = int(c.y);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) xv[q] = int(word(x.v[q / 4], q % 4));
          s = x.scale;
        }
        s *= R.ws;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const f32x4_t sum = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv[c], xv, f32x4_t{0.f, 0.f, 0.f, 0.f},
                                                                               0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][c][q] = fmaf(sum[q], s, acc[m][c][q]);
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
    // Loads of one wavefront arrive in order: once the rows of this unit are there, so is its weight.
    // That leaves two units' weights and the next one's rows in flight.  Two units' rows of two row
    // tiles in 16 bits do not fit the registers: they are loaded in their own step.
    constexpr int X_LOADS = 1 + MT * (X16 ? 4 : 3);
    constexpr bool AHEAD = !X16 || MT == 1;
    tile_for<0, D - 1>([&](auto k) __attribute__((always_inline)) { fetch(ring(k), decltype(k)::value); });
    Rows a, b;
    if constexpr (AHEAD) rows_of(a, 0);
    for (int i = 0; i < n; i += D)
      tile_for<0, D>([&](auto k) __attribute__((always_inline)) {
        constexpr int j = decltype(k)::value;
        Rows &now = j % 2 ? b : a, &next = j % 2 ? a : b;
        if (i + j < n) {
          if constexpr (AHEAD) rows_of(next, i + j + 1);
          else rows_of(a, i + j);
          wait_reads();
          fetch(ring(std::integral_constant<int, j + D - 1>{}), i + j + D - 1);
          wait_loads<AHEAD ? 4 * CT + X_LOADS : 6 * CT>();
          multiply(ring(k), AHEAD ? now : a, i + j);
        }
      });
    wait_loads<0>();  // the last loads into LDS land before it is used again
  }

  // at most N global loads of this wavefront are in flight
  template <int N>
  static __device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt range");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }

  // every LDS read of this wavefront has returned: the buffer that a step fills is the one the step
  // before read, and a load into LDS is not held back by reads in flight
  static __device__ __forceinline__ void wait_reads() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt 0
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }

  template <int MT>
  static __device__ __forceinline__ void run(const Fp8Args& A, const RowTile& t, int c0, Ring& r0, Ring& r1, Ring& r2,
                                             Ring& r3, float (*sums)[16][16 * CT + 4]) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, kq = lane >> 4;
    constexpr int COLS = 16 * CT;
    f32x4_t acc[MT][CT];
    multiply_rows<MT>(A, t, c0, acc, r0, r1, r2, r3);
    // sums of the wavefronts, 16 rows at a time
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m) __syncthreads();
#pragma unroll
      for (int c = 0; c < CT; ++c) *reinterpret_cast<f32x4_t*>(&sums[w][l16][16 * c + 4 * kq]) = acc[m][c];
      __syncthreads();
      for (int i = tid; i < 16 * COLS; i += 64 * WAVES) {
        const int r = i / COLS, c = i % COLS;
        if (16 * m + r < t.rows && c0 + c < A.h_out) {
          float s = 0.f;
#pragma unroll
          for (int v = 0; v < WAVES; ++v) s += sums[v][r][c];
          A.out[A.T.row(t.row0 + 16 * m + r) * A.ld_out + c0 + c] = static_cast<uint16_t>(Elem<DT>::pack(s, 0.f));
        }
      }
    }
  }
};

template <int DT, bool X16, int CT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, CT == 1 ? 4 : 2) void fp8_skinny_kernel(Fp8Args A) {
  using S = Fp8Skinny<DT, X16, CT, WAVES>;
  constexpr int COLS = 16 * CT;
  static_assert(128 % COLS == 0, "columns of one block");
  __shared__ typename S::Ring r0, r1, r2, r3;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16][COLS + 4];
  const int ct = (A.h_out + COLS - 1) / COLS;
  const TileList list(A.T, sgmv_host::kSkinnyRows);
  const int m = blockIdx.x / ct, c0 = (blockIdx.x - m * ct) * COLS;
  if (m >= list.count) return;
  const RowTile t = list.find(m);
  if (t.g == A.T.G) {  // rows of no group
    for (int i = threadIdx.x; i < t.rows * COLS; i += blockDim.x)
      if (c0 + i % COLS < A.h_out) A.out[A.T.row(t.row0 + i / COLS) * A.ld_out + c0 + i % COLS] = 0;
    return;
  }
  if (t.rows <= 16) S::template run<1>(A, t, c0, r0, r1, r2, r3, sums);
  else S::template run<2>(A, t, c0, r0, r1, r2, r3, sums);
}

}  // namespace sgmv_dev
