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
// owns 64 rows and walks every NWth window of 128 k, one block of scales, which it
// sends to a ring of its own in LDS, 64 rows of 128 bytes, piece p of row r at 16
// (p ^ (r / 2 % 8)); the waves' sums meet in LDS and are added in a fixed order.
// ACT8: a lane's 32 values of x become elements by the maximum over the four lanes
// that hold a block, which the wait for the weights hides.
#include "experts_rows.h"
#include "fp8.h"

namespace uw {
namespace {

template <int Q, bool GATED, bool ACT8, int NW, typename RR>
__global__ __launch_bounds__(64 * NW) void k_experts_fp8(ExpertsView vw, ExpertsView vu, RR rr,
                                                         const uint16_t* __restrict__ x, void* __restrict__ y,
                                                         int ntiles, int chunks) {
  constexpr int R = 4, RT = GATED ? 2 : 4, kRows = 16 * RT;
  constexpr int kW = 64 * 128;   // a wave's weights of a window
  __shared__ __attribute__((aligned(128))) char w0[NW * kW], w1[NW * kW];
  __shared__ typename Finder<RR>::Lds found;
  unsigned tile;
  Share sh;
  if (!Finder<RR>::find(rr, found, (unsigned)ntiles, (unsigned)chunks, vw.count, 16 * Q, tile, sh)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t N = vw.n;
  const int K = (int)vw.k, nwin = (int)fp8_blocks(K);
  const int64_t n0 = (int64_t)tile * kRows;
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  auto weights = [&](const ExpertsView& v) __attribute__((always_inline)) {
    return rsrc_of(v.w + (int64_t)sh.expert * v.w_stride + n0 * K, (uint64_t)(rows * K));
  };
  auto scales = [&](const ExpertsView& v) __attribute__((always_inline)) {   // the row of blocks that holds n0
    return rsrc_of(v.scale + (int64_t)sh.expert * v.scale_stride + (n0 >> 7) * nwin * 4, (uint64_t)nwin * 4);
  };
  const __amdgpu_buffer_rsrc_t ww = weights(vw), ws = scales(vw);
  const __amdgpu_buffer_rsrc_t uw = GATED ? weights(vu) : ww, us = GATED ? scales(vu) : ws;

  // x rows of this lane's slots
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, (uint64_t)rr.x_rows * 2 * (uint64_t)K);
  uint32_t xrow[Q];
  int32_t row[Q];
  auto slot = [&](int q) __attribute__((always_inline)) { return 16 * q + i16; };
  Finder<RR>::rows(rr, found, sh, row, slot);

  f32x4_t acc[R][Q];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // Load i of eight takes rows 8 i .. 8 i + 7, eight lanes a row; of the 64 rows
  // the gated form has W's first, then U's.
  const int pr = lane >> 3;
  auto load_w = [&](int j, char* wbuf) __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what was read from the buffer has been
    const int k0 = 128 * j;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool u = GATED && i >= 4;
      const int r = 8 * (u ? i - 4 : i) + pr, piece = (lane & 7) ^ ((8 * i + pr) >> 1 & 7);
      const uint32_t off = k0 + 16 * piece < K ? (uint32_t)(r * K + (k0 + 16 * piece)) : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(u ? uw : ww, (lds_char*)(wbuf + wave * kW + 1024 * i), 16, (int)off, 0,
                                               0, 0);
    }
  };
  struct Win {
    uint4 xv[Q][4];
    float s[2];   // the blocks' scales, 0 past the last window
  };
  auto load_x = [&](int j, Win& w) __attribute__((always_inline)) {
    const int k0 = 128 * j;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 32 * g + 8 * i;
        w.xv[q][i] = bload16(rx, k < K ? xrow[q] + 2u * (uint32_t)k : kOutside);
      }
    const int at = j < nwin ? 4 * j : (int)kOutside;
    w.s[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ws, at, 0, 0));
    w.s[1] = GATED ? __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(us, at, 0, 0)) : w.s[0];
  };
  auto compute = [&](const char* wbuf, const Win& w) __attribute__((always_inline)) {
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
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float sw = w.s[t >= RT ? 1 : 0], s = ACT8 ? sx[q] * sw : sw;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][q][c] = __builtin_fmaf(part[t][q][c], s, acc[t][q][c]);
      }
  };

  // windows past the last (whole rounds of the waves) lie past K: zeros, scaled by 0
  Win wa, wb;
  load_w(wave, w0);   // on its way while the row indices arrive
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const bool in = (slot(q) < sh.count) & (row[q] >= 0) & (row[q] < rr.x_rows);
    xrow[q] = in ? (uint32_t)((int64_t)row[q] * K) * 2u : kOutside;
  }
  load_x(wave, wa);
  for (int j = wave; j < nwin; j += 2 * NW) {
    load_w(j + NW, w1);
    load_x(j + NW, wb);
    compute(w0, wa);
    load_w(j + 2 * NW, w0);
    load_x(j + 2 * NW, wa);
    compute(w1, wb);
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
  finish<R, Q, GATED, NW>(red, sh, n0, N, y);
}

template <int Q, bool GATED, bool ACT8>
hipError_t launch_one(const ExpertsCall& c, hipStream_t s) {
  const int64_t rows = GATED ? 32 : 64, ntiles = (c.w.n + rows - 1) / rows;
  const int64_t chunks = max_chunks(c.r.slots, c.w.count, 16 * Q, c.r.offsets != nullptr);
  const int64_t grid = (chunks * ntiles + 7) / 8 * 8;
  if (!grid_fits(grid, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_experts_fp8<Q, GATED, ACT8, 4, RaggedRows>), dim3((unsigned)grid), dim3(256), 0, s, c.w, c.u,
                     c.r, c.x, c.y, (int)ntiles, (int)chunks);
  return hipGetLastError();
}

template <bool GATED, bool ACT8>
hipError_t launch_q(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1, avg = (c.r.slots + e - 1) / e;
  const int64_t rows = GATED ? 32 : 64;
  const int64_t blocks = (c.w.n + rows - 1) / rows * max_chunks(c.r.slots, c.w.count, 32, c.r.offsets != nullptr);
  if (avg <= (c.r.offsets ? 12 : 16) || blocks < device_cus()) return launch_one<1, GATED, ACT8>(c, s);
  return launch_one<2, GATED, ACT8>(c, s);
}

}  // namespace

hipError_t launch_layer_gated_fp8(const ExpertsCall& c, const RouteCall& r, hipStream_t s) {
  const int64_t ntiles = (c.w.n + 31) / 32, grid = routed_grid(r, ntiles);
  if (!grid_fits(grid, 256)) return hipErrorNotSupported;
  return with_routed(r, [&](auto rr) {
    hipLaunchKernelGGL((k_experts_fp8<1, true, false, 4, decltype(rr)>), dim3((unsigned)grid), dim3(256), 0, s, c.w,
                       c.u, rr, c.x, c.y, (int)ntiles, 0);
    return hipGetLastError();
  });
}

hipError_t launch_fp8_rows(const ExpertsCall& c, bool act8, hipStream_t s) {
  if (act8) return launch_q<false, true>(c, s);
  return c.gated ? launch_q<true, false>(c, s) : launch_q<false, false>(c, s);
}

// Which kernel, by the rows an expert has on average if every slot is used.
hipError_t launch_fp8(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1, avg = (c.r.slots + e - 1) / e;
  const bool big = c.r.x_rows * 2 * c.w.k > kOutside;   // x past 2 GiB: by pointers
  const bool spread = avg <= 96;
  if (avg <= 32 && !big) return launch_fp8_rows(c, false, s);
  return launch_fp8_tile(c, nullptr, avg <= 64 ? 64 : 128, spread, s);
}

hipError_t launch_fp8_act(const ExpertsCall& c, uint16_t* xe, float* xs, hipStream_t s) {
  if (c.r.slots <= kFp8RowsMax) return launch_fp8_rows(c, true, s);
  const hipError_t e = launch_round_fp8(c.x, c.r.slots, c.w.k, xe, xs, s);
  if (e != hipSuccess) return e;
  ExpertsCall t = c;
  t.x = xe;
  return launch_fp8_tile(t, xs, c.r.slots <= 64 ? 64 : 128, c.r.slots <= 96, s);
}

}  // namespace uw
