// fp8_rows.hip -- products with E4M3 weights (an FP32 scale per 128 x 128 block) for
// few rows, plain and gated, one matrix or grouped by expert.
//
//   y[s][n] = sum over blocks j of k:  s_x(s, j) s_w(n / 128, j)  sum over k in j of xe we
//
// with x in BF16 (xe = x, s_x = 1) or converted on the way to E4M3 with a scale per 1 x
// 128 (ACT8).  Elements go through the matrix unit as BF16, which holds them exactly (see
// fp8_tile.hip for why not as bytes); the sum over a block is scaled once and added
// to the running FP32 sum.
//
// A stream over the weights, built as the MXFP4 kernel of experts_rows.hip: a wave
// owns 16 R rows (64 as a rule, 16 or 32 of narrow matrices, 20 to 44 where even shares
// fill the chip better) and walks every NWth window of 128 k, one block of scales, which it
// sends to a ring of its own in LDS, 16 R rows of 128 bytes, piece p of row r at 16
// (p ^ (r / 2 % 8)); the waves' sums meet in LDS and are added in a fixed order.
// ACT8: a lane's 32 values of x become elements by the maximum over the four lanes
// that hold a block, which the wait for the weights hides.
#include <algorithm>

#include "experts_rows.h"
#include "fp8.h"

namespace uw {
namespace {

template <int R, int Q, bool GATED, bool ACT8, bool XL, int NW, typename RR>
__global__ __launch_bounds__(64 * NW) void k_experts_fp8(ExpertsView vw, ExpertsView vu, RR rr,
                                                         const uint16_t* __restrict__ x, void* __restrict__ y,
                                                         int ntiles, int chunks, int most) {
  constexpr int RT = GATED ? R / 2 : R;
  constexpr bool kBelow = !GATED && !ACT8 && R > 1;   // tiles of `most` rows, which may end in the next row of blocks
  const int span = kBelow ? most : 16 * RT;
  constexpr int kW = 16 * R * 128;   // a wave's weights of a window
  constexpr int kX = XL ? 16 * 256 : 4;
  __shared__ __attribute__((aligned(128))) char w0[NW * kW], w1[NW * kW];
  __shared__ __attribute__((aligned(128))) char x0[NW * kX], x1[NW * kX];
  __shared__ typename Finder<RR>::Lds found;
  Finder<RR> finder;
  if (!finder.template begin<NW>(rr, found)) return;
  for (int turn = 0;; ++turn) {
    unsigned tile;
    Share sh;
    if (!finder.find(rr, found, turn, (unsigned)ntiles, (unsigned)chunks, vw.count, 16 * Q, tile, sh)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int64_t N = vw.n;
    const int K = (int)vw.k, nwin = (int)fp8_blocks(K);
    const int64_t n0 = (int64_t)tile * span;
    const int64_t rows = N - n0 < span ? N - n0 : span;
    auto weights = [&](const ExpertsView& v) __attribute__((always_inline)) {
      return rsrc_of(v.w + (int64_t)sh.expert * v.w_stride + n0 * K, (uint64_t)(rows * K));
    };
    // The row of blocks that holds n0 and, kBelow, the next; the upper half of the wave
    // loads that one's.
    const int row_blocks = (int)(fp8_blocks(N) - (n0 >> 7));
    auto scales = [&](const ExpertsView& v) __attribute__((always_inline)) {
      return rsrc_of(v.scale + (int64_t)sh.expert * v.scale_stride + (n0 >> 7) * nwin * 4,
                     (uint64_t)nwin * (kBelow && row_blocks > 1 ? 8 : 4));
    };
    const __amdgpu_buffer_rsrc_t ww = weights(vw), ws = scales(vw);
    const __amdgpu_buffer_rsrc_t uw = GATED ? weights(vu) : ww, us = GATED ? scales(vu) : ws;
    const int upper = 128 - (int)(n0 & 127);   // rows of the tile in the first of them

    // x rows of this lane's slots
    const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, (uint64_t)rr.x_rows * 2 * (uint64_t)K);
    constexpr int XR = XL ? 4 : Q;
    uint32_t xrow[XR];
    int32_t row[XR];
    auto slot = [&](int q) __attribute__((always_inline)) { return XL ? 4 * q + g : 16 * q + i16; };
    finder.rows(rr, found, sh, row, slot);

    f32x4_t acc[R][Q];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int q = 0; q < Q; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Load i takes rows 8 i .. 8 i + 7, eight lanes a row; of the 16 R rows
    // the gated form has W's first, then U's.
    const int pr = lane >> 3;
    auto load_w = [&](int j, char* wbuf) __attribute__((always_inline)) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what was read from the buffer has been
      const int k0 = 128 * j;
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) {
        const bool u = GATED && i >= R;
        const int r = 8 * (u ? i - R : i) + pr, piece = (lane & 7) ^ ((8 * i + pr) >> 1 & 7);
        const uint32_t off = k0 + 16 * piece < K ? (uint32_t)(r * K + (k0 + 16 * piece)) : kOutside;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(u ? uw : ww, (lds_char*)(wbuf + wave * kW + 1024 * i), 16, (int)off, 0,
                                                 0, 0);
      }
    };
    struct Win {
      uint4 xv[Q][4];
      float s[2];   // the blocks' scales (gated: W's and U's), 0 past the last window
    };
    auto load_x = [&](int j, char* xbuf, Win& w) __attribute__((always_inline)) {
      const int k0 = 128 * j;
      if constexpr (XL) {   // rows 4 i .. 4 i + 3, sixteen lanes a row; piece p of row r at 16 (p ^ r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + 8 * (i16 ^ (4 * i + g));
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_char*)(xbuf + wave * kX + 1024 * i), 16,
                                                   (int)(k < K ? xrow[i] + 2u * (uint32_t)k : kOutside), 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = k0 + 32 * g + 8 * i;
            w.xv[q][i] = bload16(rx, k < K ? xrow[q] + 2u * (uint32_t)k : kOutside);
          }
      }
      const int at = j < nwin ? 4 * (kBelow ? j + (lane >> 5) * nwin : j) : (int)kOutside;
      w.s[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ws, at, 0, 0));
      if constexpr (GATED) w.s[1] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(us, at, 0, 0));
    };
    auto compute = [&](const char* wbuf, const char* xbuf, Win& w) __attribute__((always_inline)) {
      if constexpr (XL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w.xv[0][i] = *reinterpret_cast<const uint4*>(xbuf + wave * kX + i16 * 256 + (((4 * g + i) ^ i16) << 4));
      }
      uint4 d[R][2];
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const int r = 16 * t + i16;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          d[t][u] = *reinterpret_cast<const uint4*>(wbuf + wave * kW + r * 128 + (((2 * g + u) ^ (r >> 1 & 7)) << 4));
      }
      f32x4_t part[R][Q];
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int q = 0; q < Q; ++q) part[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      float sx[Q];
      uint4 xv[Q][4];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        sx[q] = 1.0f;
        if constexpr (ACT8) {   // the block's maximum is over the four lane groups
          uint32_t m = max_halves(max_halves(bf16_top8(w.xv[q][0]), bf16_top8(w.xv[q][1])),
                                  max_halves(bf16_top8(w.xv[q][2]), bf16_top8(w.xv[q][3])));
          m = max_halves(m, (uint32_t)__shfl_xor((int)m, 16));
          m = max_halves(m, (uint32_t)__shfl_xor((int)m, 32));
          const Fp8Scale f = fp8_scale(top_bits(m));
          sx[q] = f.scale;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 e = fp8_pack8(w.xv[q][i], f.inv);
            xv[q][i] = fp8_unpack8(e.x, e.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[q][i] = w.xv[q][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const uint4& h = d[t][i >> 1];
          const bf16x8_t a = __builtin_bit_cast(bf16x8_t, i & 1 ? fp8_unpack8(h.z, h.w) : fp8_unpack8(h.x, h.y));
#pragma unroll
          for (int q = 0; q < Q; ++q)
            part[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, xv[q][i]), part[t][q],
                                                                 0, 0, 0);
        }
      float sw[R];
      if constexpr (kBelow) {
        auto half = [&](int l) __attribute__((always_inline)) {
          return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w.s[0]), l));
        };
        const float first = half(0), below = half(32);
#pragma unroll
        for (int t = 0; t < R; ++t) sw[t] = 16 * t + 4 * g < upper ? first : below;
      } else {
#pragma unroll
        for (int t = 0; t < R; ++t) sw[t] = w.s[t >= RT ? 1 : 0];
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const float s = ACT8 ? sx[q] * sw[t] : sw[t];
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[t][q][c] = __builtin_fmaf(part[t][q][c], s, acc[t][q][c]);
        }
    };

    // windows past the last (whole rounds of the waves) lie past K: zeros, scaled by 0
    Win wa, wb;
    load_w(wave, w0);   // on its way while the row indices arrive
#pragma unroll
    for (int q = 0; q < XR; ++q) {
      const bool in = (slot(q) < sh.count) & (row[q] >= 0) & (row[q] < rr.x_rows);
      xrow[q] = in ? (uint32_t)((int64_t)row[q] * K) * 2u : kOutside;
    }
    load_x(wave, x0, wa);
    for (int j = wave; j < nwin; j += 2 * NW) {
      load_w(j + NW, w1);
      load_x(j + NW, x1, wb);
      compute(w0, x0, wa);
      load_w(j + 2 * NW, w0);
      load_x(j + 2 * NW, x0, wa);
      compute(w1, x1, wb);
    }

    __builtin_amdgcn_s_waitcnt(0);   // nothing travels to LDS any more
    __syncthreads();
    f32x4_t* red = reinterpret_cast<f32x4_t*>(w0);
    static_assert(R * Q * 64 * 16 <= kW, "the sums fit one ring buffer");
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int q = 0; q < Q; ++q) red[((wave * R + t) * Q + q) * 64 + lane] = acc[t][q];
    __syncthreads();
    finish<R, Q, GATED, NW>(red, sh, n0, rows, N, y);
    if constexpr (!Finder<RR>::kWalks) return;
    __syncthreads();   // the sums have been read
  }
}

// One matrix and BF16 x: where whole tiles fill the rounds of blocks on the CUs to less than
// three quarters, each block gets as few rows as make no more rounds, in fours, half its tile
// at least.  (us, whole tiles / so, weights out of every cache: 5001x8224, 157 / 251 blocks, 1
// row 15.9 / 14.8, 13 rows 17.7 / 16.4; 9000x4096 13.6 / 12.9, 16.2 / 15.1; 18432x5120 26.1 / 21.8,
// 33.3 / 29.3.  With less to even out a block's own work counts: 7168x2048, 224 / 256 blocks,
// 1 row 6.0 / 6.2; so does x's conversion, which every block makes: 5001x8224, 13 rows, weights
// in the last-level cache 15.5 / 16.1.)
template <int R, int Q, bool GATED, bool ACT8, bool XL, int NW>
hipError_t launch_one(const ExpertsCall& c, hipStream_t s) {
  const int64_t chunks = max_chunks(c.r.slots, c.w.count, 16 * Q, c.r.offsets != nullptr);
  int64_t rows = GATED ? 8 * R : 16 * R, ntiles = (c.w.n + rows - 1) / rows;
  if (!c.r.offsets && !ACT8 && R > 1) {
    const int64_t cus = device_cus(), most = (ntiles * chunks + cus - 1) / cus * cus / chunks;
    const int64_t even = ((c.w.n + most - 1) / most + 3) / 4 * 4;
    if (4 * even < 3 * rows) rows = even > rows / 2 ? even : rows / 2;
    ntiles = (c.w.n + rows - 1) / rows;
  }
  const int64_t grid = (chunks * ntiles + 7) / 8 * 8;
  if (!grid_fits(grid, 64 * NW)) return hipErrorNotSupported;
  if (c.check) return hipSuccess;
  hipLaunchKernelGGL((k_experts_fp8<R, Q, GATED, ACT8, XL, NW, RaggedRows>), dim3((unsigned)grid), dim3(64 * NW), 0, s,
                     c.w, c.u, c.r, c.x, c.y, (int)ntiles, (int)chunks, (int)rows);
  return hipGetLastError();
}
// One matrix: 64 rows of it a wave, or 32 and eight waves a block where that makes too
// few blocks, or 16 where those fit the chip at once (32 / 16 a wave, us, 13 rows of x:
// 1000x16384 12.6 / 9.8, 4096x4096 6.5 / 5.7, 5001x8224, 313 blocks of 16, 17.3 / 21.7); x
// through LDS, like the weights, once its loads are many, or two groups of sixteen rows
// where the blocks still make three quarters of the chip.  Measured (us; 64 rows, 64 with x in LDS, 32 with
// eight waves, the same with x in LDS, two groups; x in BF16):
//   14336x4096   1 row 14.4 / 15.6 / 14.2 / 15.8, 16 rows 15.3 / 16.0 / 17.5 / 17.5, 32 rows 21.5 / 22.2 / 26.8 / 26.7 / 19.2
//   5001x8224    1 row 21.7 / 24.1 / 15.0 / 15.6, 16 rows 28.2 / 25.4 / 18.9 / 17.9, 32 rows 26.6 / 24.1 / 29.5 / 27.3 / 39.8
//   4096x4096    1 row  7.9 /  8.6 /  5.8 /  6.1, 16 rows  9.2 /  8.9 /  8.2 /  6.7, 32 rows  9.3 /  8.7 /  8.4 /  7.0 / 13.0
//   28672x8192  16 rows 47.8 / 47.2 / 55.5 / 52.9, in 8 bits 51.3 / 45.9 / 67.1 / 57.3
// Two groups with 192 to 255 blocks, us, one group with x in LDS / two, weights out of every cache:
//   12288x4096  17 rows 20.8 / 15.1, 32 rows 21.4 / 18.5, in 8 bits 21.9 / 18.7, 22.0 / 19.2
//   14336x4096  17 rows 21.5 / 15.9, 32 rows 22.0 / 19.2, in 8 bits 22.4 / 19.2, 22.3 / 19.9
//   6144x4096   64 rows 18.4 / 15.5, in 8 bits 21.4 / 17.1;  16049x12224, 24 rows in 8 bits 57.9 / 50.0
// Sixteen rows, x past LDS / through it: 28672x2048 15.5 / 16.7, 28672x4096 29.1 / 29.0, 28672x8192 52.2 / 48.7.
template <bool ACT8>
hipError_t launch_matrix(const ExpertsCall& c, hipStream_t s) {
  const int64_t cus = device_cus(), rows = c.r.slots, tiles = (c.w.n + 63) / 64;
  if (rows > 16 && tiles * ((rows + 31) / 32) >= cus * 3 / 4) return launch_one<4, 2, false, ACT8, false, 4>(c, s);
  const int64_t blocks = tiles * ((rows + 15) / 16);
  if (blocks >= cus * 3 / 4)
    return rows > (ACT8 ? 8 : 15) ? launch_one<4, 1, false, ACT8, true, 4>(c, s)
                                  : launch_one<4, 1, false, ACT8, false, 4>(c, s);
  if ((c.w.n + 15) / 16 * ((rows + 15) / 16) <= cus) return launch_one<1, 1, false, ACT8, true, 8>(c, s);
  return rows > 8 ? launch_one<2, 1, false, ACT8, true, 8>(c, s) : launch_one<2, 1, false, ACT8, false, 8>(c, s);
}

// Grouped by expert: two groups of sixteen slots where experts have more as a rule.
template <bool GATED>
hipError_t launch_grouped(const ExpertsCall& c, hipStream_t s) {
  const int64_t avg = (c.r.slots + c.w.count - 1) / c.w.count, rows = GATED ? 32 : 64;
  const int64_t blocks = (c.w.n + rows - 1) / rows * max_chunks(c.r.slots, c.w.count, 32, true);
  if (avg <= 12 || blocks < device_cus()) return launch_one<4, 1, GATED, false, false, 4>(c, s);
  return launch_one<4, 2, GATED, false, false, 4>(c, s);
}

template <int R, int NW>
hipError_t launch_routed(const ExpertsCall& c, const RouteCall& r, hipStream_t s) {
  const int64_t ntiles = (c.w.n + 8 * R - 1) / (8 * R), grid = routed_grid(r, ntiles, 2);
  if (!grid_fits(grid, 64 * NW)) return hipErrorNotSupported;
  return with_routed(r, [&](auto rr) {
    hipLaunchKernelGGL((k_experts_fp8<R, 1, true, false, false, NW, decltype(rr)>), dim3((unsigned)grid), dim3(64 * NW),
                       0, s, c.w, c.u, rr, c.x, c.y, (int)ntiles, 0, 0);
    return hipGetLastError();
  });
}

}  // namespace

// 32 outputs a tile, or where that makes fewer tiles than blocks fit the chip 16 and eight
// waves, so that all of a wave's windows are on their way at once (layer of one token, 8 of 64
// experts, us with 32 / 16: 512x7168 32.6 / 28.4, 1408x2048 23.0 / 22.2; two of eight 2048x4096
// 22.8 / 19.2; beyond the rule, 16 tokens over 64 of 1408x2048, the product alone 63 / 67).
hipError_t launch_layer_gated_fp8(const ExpertsCall& c, const RouteCall& r, hipStream_t s) {
  const int64_t pairs = r.tokens * r.topk;
  if ((c.w.n + 31) / 32 * (pairs < r.experts ? pairs : r.experts) < 2 * device_cus()) return launch_routed<2, 8>(c, r, s);
  return launch_routed<4, 4>(c, r, s);
}

hipError_t launch_fp8_rows(const ExpertsCall& c, bool act8, hipStream_t s) {
  if (!c.r.offsets) return act8 ? launch_matrix<true>(c, s) : launch_matrix<false>(c, s);
  return c.gated ? launch_grouped<true>(c, s) : launch_grouped<false>(c, s);
}

namespace {

// Estimates in us, fitted to measured times (some 650 of one matrix, 1 to 1024 rows, 300 x 9600 to
// 28672 x 8192, the tiles' within 16 % rms; 350 of 8 to 64 experts, 4 to 256 rows each):
//   tiles  rounds of one block a CU, each its steps of 128 k and three more, at 1.15 (64 rows) or
//          1.55 (128 rows);
//   rows   3 and the weights once per group of rows.
double tile_us(int64_t blocks, int64_t steps, int rows, int64_t cus) {
  return (double)((blocks + cus - 1) / cus * (steps + 3)) * (rows == 64 ? 1.15 : 1.55);
}

}  // namespace

// Grouped by expert.  The chunks of rows that the plan will make are not known here: one an
// expert at least, and half a chunk an expert more than whole ones.  Weights pass the rows
// kernel at 5 TB/s, in groups of 16 rows or, with more than 12 an expert, 32, and the tiles
// at 4.7 TB/s at most.  (us, measured rows / 64 / 128: 32 experts 2048x2048 of 4 rows 31 /
// 29 / 31, of 32 rows 43 / 31 / 32, of 64 rows 65 / 50 / 37; 8 of 2048x4096, 64 rows 32 / 38 /
// 46, 256 rows - / 81 / 59.)
hipError_t launch_fp8_experts(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.w.count, slots = c.r.slots, avg = (slots + e - 1) / e, with_rows = slots < e ? slots : e;
  const int64_t ntiles = (c.w.n + (c.gated ? 127 : 255)) / (c.gated ? 128 : 256);
  auto chunks = [&](int64_t rows) {
    const int64_t n = slots / rows + with_rows / 2;
    return n > with_rows ? n : with_rows;
  };
  const bool spread = avg <= 96;
  // x past 2 GiB goes by pointers, in 128-row tiles
  if (c.r.x_rows * 2 * c.w.k > kOutside) return launch_fp8_tile(c, Fp8Tile{128, spread, 0, 1, nullptr, nullptr}, s);
  const double weights = (c.gated ? 2.0 : 1.0) * (double)c.w.n * (double)c.w.k * 1e-6;
  const int64_t steps = fp8_blocks(c.w.k);
  const int64_t cus = device_cus();
  const double t64 = tile_us(ntiles * chunks(64), steps, 64, cus), t128 = tile_us(ntiles * chunks(128), steps, 128, cus);
  const double least = (double)with_rows * weights / 4.7, best = t64 < t128 ? t64 : t128;
  if (3 + (double)chunks(avg > 12 ? 32 : 16) * weights / 5 < (best > least ? best : least))
    return launch_fp8_rows(c, false, s);
  return launch_fp8_tile(c, Fp8Tile{t64 < t128 ? 64 : 128, spread, 0, 1, nullptr, nullptr}, s);
}

// One matrix.  The tiles of the last, partly filled round go in slices of K where that is
// faster: it costs 6.5 and the slices' sums at 5.3 TB/s.  The weights pass the tiles at
// 2.5 TB/s at most; the rows kernel takes them once per 16 rows of x at 7 TB/s, or per 32 at
// 6.2 where that fills the chip.  (us without / with slices: 5001x8224, 200 rows 55 / 40;
// 4096x14336, 333 rows 173 / 56.)  Two groups on three quarters of the chip, which launch_matrix
// takes, are not counted at 6.2 here: that would send long rows of few tiles there (us as it is /
// so: 6328x8160, 64 rows 29.1 / 34.4; 3037x10176, 119 rows 26.4 / 33.4; 2018x5600, 200 rows
// 22.6 / 16.1).  Slices hold 512 rows of 256 sums a CU at most, which no
// plan of a million shapes tried wanted to pass (1 to 60000 x 32 to 32768, 17 to 20000 rows).
Fp8Plan plan_fp8(int64_t n, int64_t k, int64_t batch, bool act8) {
  auto pad = [](uint64_t b) { return (b + 255) / 256 * 256; };
  Fp8Plan p{};
  const bool big = batch * 2 * k > kOutside;
  const int64_t cus = device_cus(), steps = fp8_blocks(k);
  const double weights = (double)n * (double)k * 1e-6;
  double best = 0;
  constexpr int kSplits = 16;
  const int64_t slice_rows = 4 * 128 * cus;
  auto tiles_of = [&](int rows) { return (batch + rows - 1) / rows * ((n + 255) / 256); };
  for (int rows = big ? 128 : 64; rows <= 128; rows *= 2) {
    const int64_t tiles = tiles_of(rows), tail = tiles % cus;
    for (int splits = 1; splits <= kSplits && (splits == 1 || (tail && steps >= 2 * splits && tail * splits * rows <= slice_rows));
         ++splits) {
      double us = tile_us(splits > 1 ? tiles - tail : tiles, steps, rows, cus);
      if (splits > 1)
        us += tile_us(tail * splits, (steps + splits - 1) / splits, rows, cus) + 6.5 +
              (double)(tail * splits * rows) * 2048e-6 / 5.3;
      if (us < weights / 2.5) us = weights / 2.5;
      if (best == 0 || us < best) {
        best = us;
        p.tile = Fp8Tile{rows, batch <= 96, splits > 1 ? (int)tail : 0, splits, nullptr, nullptr};
      }
    }
  }
  if (batch <= 256 && !big) {   // (beyond, x's share of the traffic would count)
    const double sixteens = (double)((batch + 15) / 16) * weights / 7, twos = (double)((batch + 31) / 32) * weights / 6.2;
    const bool fills = (n + 63) / 64 * ((batch + 31) / 32) >= cus;
    p.few = 3 + (fills && twos < sixteens ? twos : sixteens) < best;
    if (p.few) return p;
  }
  if (act8) {
    p.x_bytes = pad(2 * (uint64_t)batch * (uint64_t)k);
    p.scale_bytes = pad(4 * (uint64_t)batch * (uint64_t)steps);
  }
  p.part_bytes = pad((uint64_t)p.tile.tail * (uint64_t)p.tile.splits * (uint64_t)p.tile.rows * 1024);
  const int64_t splits = steps / 2 < kSplits ? steps / 2 : kSplits;
  int64_t slices = 0;   // rows of the largest tail in most slices, as far as the tiles reach
  for (int rows = 64; rows <= 128 && splits > 1; rows *= 2) {
    const int64_t tiles = tiles_of(rows), tail = tiles < cus ? tiles : cus - 1;
    slices = std::max(slices, tail * splits * rows);
  }
  p.bytes = p.x_bytes + p.scale_bytes + 1024 * (uint64_t)std::min(slices, slice_rows);
  return p;
}

hipError_t launch_fp8_product(const ExpertsCall& c, const Fp8Plan& p, bool act8, void* ws, hipStream_t s) {
  if (p.few) return launch_fp8_rows(c, act8, s);
  char* const at = static_cast<char*>(ws);
  ExpertsCall call = c;
  Fp8Tile t = p.tile;
  t.part = reinterpret_cast<float*>(at + p.x_bytes + p.scale_bytes);
  if (act8) {
    uint16_t* const xe = reinterpret_cast<uint16_t*>(at);
    float* const xs = reinterpret_cast<float*>(at + p.x_bytes);
    const hipError_t e = launch_round_fp8(c.x, c.r.slots, c.w.k, xe, xs, s);
    if (e != hipSuccess) return e;
    call.x = xe;
    t.act = xs;
  }
  return launch_fp8_tile(call, t, s);
}

}  // namespace uw
