// experts_rows.hip -- products grouped by expert for few rows an expert:
// y[s] = x[row(s)] . W_e^T for the slots s of expert e, weights BF16, UWF1
// (palette indices) or MXFP4, and the gated form silu(x . G_e^T) * (x . U_e^T).
//
// With few rows an expert the product is a stream over the weights of the
// experts that have rows, so the kernel keeps many bytes of them in flight and
// reuses nothing but x:
//   * a block owns 16 R rows of one expert's weights and up to 16 Q of its
//     slots; its waves (four as a rule) walk interleaved windows of K, each loading its
//     weights two windows deep, BF16 and UWF1 straight into registers, MXFP4
//     through LDS, and feeding v_mfma_f32_16x16x32_bf16 with the weights as A
//     (16 output features) and x as B (16 slots);
//   * the order of k inside an MFMA is free as long as A and B agree.  BF16:
//     MFMA m of a 128-wide window takes k 32 m + 8 g .. +7 in lane group g, so
//     a load reads 64 contiguous bytes of each of 16 rows.  The byte and
//     nibble forms give lane group g a run of 32 (MXFP4: 64) consecutive k, so
//     that a lane's weights lie in one UWF1 group or whole MXFP4 blocks;
//   * the waves' sums meet in LDS and are added in a fixed order.
#include "experts.h"

namespace uw {
namespace {

__device__ __forceinline__ uint32_t word4(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Every load goes through a buffer resource (or, for a UWF1 expert's
// exponents, a selected pointer): what must count as nothing -- weights and
// x beyond K, rows beyond N, slots beyond the share, row indices outside x --
// has an offset past the resource's end and reads zero, so the loop holds no
// selects.  This is what a UWF1 expert's lane reads there:
__device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0, 0, 0, 0};

// BF16 and UWF1: k of MFMA m's eight weights in lane group g, from the start of
// a window of 128
template <int FORM>
__device__ __forceinline__ int k_off(int m, int g) {
  return FORM == kFormBf16 ? 32 * m + 8 * g : 32 * g + 8 * m;
}

// A block's rows [n0, n0 + rows) of one expert's matrix.
template <int FORM>
struct Mat {
  __amdgpu_buffer_rsrc_t w;   // BF16: from row n0
  ExpertEntry t;              // UWF1
  uint32_t el0, el_end;       // ... its elements [n0 K, (n0 + rows) K)
};

template <int FORM>
__device__ __forceinline__ Mat<FORM> matrix_of(const ExpertsView& v, int e, int64_t n0, int span) {
  Mat<FORM> m{};
  const int64_t rows = v.n - n0 < span ? v.n - n0 : span;
  if constexpr (form_is_pal(FORM)) {
    m.t = v.table[e];
    m.el0 = (uint32_t)(n0 * v.k);
    m.el_end = (uint32_t)((n0 + rows) * v.k);
    m.w = rsrc_of(m.t.sm + n0 * v.k, (uint64_t)(rows * v.k));
  } else {
    m.w = rsrc_of(v.w + (int64_t)e * v.w_stride + n0 * 2 * v.k, (uint64_t)(rows * 2 * v.k));
  }
  return m;
}

// A lane's weights of one window of one row, as loaded:
//   BF16: d[m] = the eight of MFMA m;  UWF1: d[0], d[1] = 32 sign+mantissa
//   bytes, d[2] = 32 index nibbles, or d[2], d[3] = 32 exponent bytes when f
//   (verbatim group)
struct Raw {
  uint4 d[4];
  uint32_t f;
};

// flag and rank words of the lane's group (UWF1), loaded a window ahead
struct Flags {
  uint32_t fw, rw;
};

// row: from n0
template <int FORM>
__device__ __forceinline__ void load_flags(const Mat<FORM>& m, int row, int K, int k, Flags& f) {
  if constexpr (form_is_pal(FORM)) {
    const uint32_t el = m.el0 + (uint32_t)row * (uint32_t)K + (uint32_t)k;
    const uint32_t w = (k < K && el < m.el_end ? el : m.el0) >> 11;
    f.fw = gload<uint32_t>(m.t.vflags + w);
    f.rw = gload<uint32_t>(m.t.vrank + w);
  }
}

// k0: the window's start (K or more: nothing)
template <int FORM>
__device__ __forceinline__ void load_raw(const Mat<FORM>& m, int row, int K, int k0, int g, const Flags& fl, Raw& r) {
  if constexpr (FORM == kFormBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + k_off<FORM>(i, g);
      r.d[i] = bload16(m.w, k < K ? (uint32_t)(row * K + k) * 2u : kOutside);
    }
  } else {
    const int k = k0 + k_off<FORM>(0, g);
    const uint32_t at = (uint32_t)row * (uint32_t)K + (uint32_t)k, el = m.el0 + at;
    const bool in = k < K && el < m.el_end;
    r.d[0] = bload16(m.w, in ? at : kOutside);
    r.d[1] = bload16(m.w, in ? at + 16u : kOutside);
    const uint32_t grp = el >> 6;
    const bool v = in && group_verbatim(fl.fw, grp);
    const uint32_t vo = group_rank(fl.fw, fl.rw, grp) * 64u + (el & 63u);
    // outside the matrix the exponents are zeros, as of a verbatim group
    const uint8_t* p = v ? m.t.vexp + vo : in ? m.t.pidx + el / 2 : reinterpret_cast<const uint8_t*>(g_zero16);
    r.d[2] = gload16(p);
    r.d[3] = make_uint4(0u, 0u, 0u, 0u);
    if (v) r.d[3] = gload16(p + 16);   // (rarely any lane: a fourth load for all would cost 10 %)
    r.f = v || !in ? 1u : 0u;
  }
}

// A operand of MFMA m
template <int FORM>
__device__ __forceinline__ bf16x8_t a_frag(const Mat<FORM>& mt, const Raw& r, int m) {
  uint4 o;
  if constexpr (FORM == kFormBf16) {
    o = r.d[m];
  } else {
    const int wi = 2 * (m & 1);
    uint32_t e0, e1;
    pal8<FORM == kFormPalRun>(word4(r.d[2], m), mt.t.pal, e0, e1);
    e0 = r.f ? word4(r.d[2 + (m >> 1)], wi) : e0;
    e1 = r.f ? word4(r.d[2 + (m >> 1)], wi + 1) : e1;
    rebuild4(word4(r.d[m >> 1], wi), e0, o.x, o.y);
    rebuild4(word4(r.d[m >> 1], wi + 1), e1, o.z, o.w);
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

// A block's tile of output rows and chunk of slots.  The chunks of one matrix
// read the same weights, so a tile's chunks follow each other on one XCD and
// share them in its L2 (MXFP4 5001x8224, 45 rows: 18.1 -> 15.2 us).  Experts'
// chunks share little, and all XCDs walking through an expert together do
// better (MXFP4 layer of 37 tokens over 32 experts: 109 us against 118).
struct Place {
  unsigned tile, chunk;
};
__device__ __forceinline__ Place place_of(const RaggedRows& rr, unsigned ntiles, unsigned chunks) {
  if (rr.offsets) return {blockIdx.x % ntiles, blockIdx.x / ntiles};
  const unsigned turn = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);   // (the grid is a multiple of 8)
  return {turn / chunks, turn % chunks};
}

// The waves' sums, added in wave order and stored.  red: per wave and tile
// the MFMA's D: lane l holds output features 4 (l / 16) .. +3 of slot l % 16.
template <int R, int Q, bool GATED, int NW>
__device__ __forceinline__ void finish(const f32x4_t* red, const Share& sh, int64_t n0, int64_t N, void* __restrict__ y) {
  constexpr int RT = GATED ? R / 2 : R;
  for (int i = threadIdx.x; i < RT * Q * 64; i += 64 * NW) {
    const int ln = i & 63, q = (i >> 6) % Q, t = (i >> 6) / Q;
    auto sum = [&](int tt) __attribute__((always_inline)) {
      f32x4_t s = red[(tt * Q + q) * 64 + ln];
#pragma unroll
      for (int v = 1; v < NW; ++v) s += red[((v * R + tt) * Q + q) * 64 + ln];
      return s;
    };
    f32x4_t s = sum(t);
    const int b = 16 * q + (ln & 15);
    const int64_t n = n0 + 16 * t + 4 * (ln >> 4);
    if (b >= sh.count || n >= N) continue;
    const int64_t at = (sh.first + b) * N + n;
    if constexpr (GATED) {
      const f32x4_t u = sum(t + RT);
#pragma unroll
      for (int c = 0; c < 4; ++c) s[c] = silu(s[c]) * u[c];
      uint16_t* o = static_cast<uint16_t*>(y) + at;
      const uint32_t lo = bf16_pair(s[0], s[1]), hi = bf16_pair(s[2], s[3]);
      if ((N & 3) == 0) {
        *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n + c < N) o[c] = (uint16_t)((c < 2 ? lo : hi) >> (16 * (c & 1)));
      }
    } else {
      float* o = static_cast<float*>(y) + at;
      if ((N & 3) == 0) {
        *reinterpret_cast<f32x4_t*>(o) = s;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n + c < N) o[c] = s[c];
      }
    }
  }
}

// R weight tiles of 16 rows (gated: the first half from W, the second the
// same rows of U), Q groups of 16 slots
template <int FORM, int R, int Q, bool GATED>
__global__ __launch_bounds__(256) void k_experts_rows(ExpertsView vw, ExpertsView vu, RaggedRows rr,
                                                      const uint16_t* __restrict__ x, void* __restrict__ y,
                                                      int ntiles, int chunks) {
  constexpr int W = 128;
  constexpr int RT = GATED ? R / 2 : R;   // distinct output tiles
  __shared__ f32x4_t red[4 * R * Q * 64];
  const Place at = place_of(rr, (unsigned)ntiles, (unsigned)chunks);
  if (at.tile >= (unsigned)ntiles || at.chunk >= (unsigned)chunks) return;
  const Share sh = find_share(rr, vw.count, at.chunk, 16 * Q);
  if (sh.count == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t N = vw.n;
  const int K = (int)vw.k;
  const int64_t n0 = (int64_t)at.tile * (16 * RT);
  const Mat<FORM> mw = matrix_of<FORM>(vw, sh.expert, n0, 16 * RT);
  Mat<FORM> mu = mw;
  if constexpr (GATED) mu = matrix_of<FORM>(vu, sh.expert, n0, 16 * RT);
  auto mat = [&](int t) __attribute__((always_inline)) -> const Mat<FORM>& { return GATED && t >= RT ? mu : mw; };
  auto row_of = [&](int t) __attribute__((always_inline)) { return 16 * (t % RT) + i16; };

  // x rows of this lane's slots
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, (uint64_t)rr.x_rows * 2 * (uint64_t)K);
  uint32_t xrow[Q];
  int32_t row[Q];   // (fewer than 2^31 slots)
#pragma unroll
  for (int q = 0; q < Q; ++q) row[q] = (int32_t)sh.first + (16 * q + i16 < sh.count ? 16 * q + i16 : 0);
  if (rr.rows) {
#pragma unroll
    for (int q = 0; q < Q; ++q) row[q] = rr.rows[row[q]];
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const bool in = (16 * q + i16 < sh.count) & (row[q] >= 0) & (row[q] < rr.x_rows);
    xrow[q] = in ? (uint32_t)((int64_t)row[q] * K) * 2u : kOutside;
  }

  const int nwin = (K + W - 1) / W;
  f32x4_t acc[R][Q];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  struct Win {
    Raw r[R];
    uint4 xv[Q][4];
  };
  auto flags = [&](int j, Flags (&f)[R]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < R; ++t) load_flags<FORM>(mat(t), row_of(t), K, W * j + k_off<FORM>(0, g), f[t]);
  };
  // windows past the last (whole rounds of four) lie past K and load zeros
  auto load = [&](int j, const Flags (&f)[R], Win& w) __attribute__((always_inline)) {
    const int k0 = W * j;
#pragma unroll
    for (int t = 0; t < R; ++t) load_raw<FORM>(mat(t), row_of(t), K, k0, g, f[t], w.r[t]);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + k_off<FORM>(i, g);
        w.xv[q][i] = bload16(rx, k < K ? xrow[q] + 2u * (uint32_t)k : kOutside);
      }
  };
  auto compute = [&](const Win& w) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const bf16x8_t a = a_frag<FORM>(mat(t), w.r[t], i);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, w.xv[q][i]), acc[t][q],
                                                              0, 0, 0);
      }
  };

  Win wa, wb;
  Flags fa[R], fb[R];
  flags(wave, fa);
  flags(wave + 4, fb);
  load(wave, fa, wa);
  flags(wave + 8, fa);
  for (int j = wave; j < nwin; j += 8) {
    load(j + 4, fb, wb);
    flags(j + 12, fb);
    compute(wa);
    load(j + 8, fa, wa);
    flags(j + 16, fa);
    compute(wb);
  }
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) red[((wave * R + t) * Q + q) * 64 + lane] = acc[t][q];
  __syncthreads();
  finish<R, Q, GATED, 4>(red, sh, n0, N, y);
}

// MXFP4.  Its weights are few bytes a lane, and a wave that loads operands
// straight into registers asks for 16 pieces of one K position in 16 rows at a
// time: the load unit takes them one by one and was what the kernel waited for
// (70 % busy).  So a wave sends its weights and scales to a ring of its own in
// LDS, rows in whole lines, and reads its operands there; nothing but the wave's
// own loads is waited for (layer of 37 tokens over 32 experts: 128 -> 109 us, 105 now;
// 4096x4096, 256 rows: 34 -> 25 us).
// A window is 256 k wide: 64 rows of 128 bytes, piece p of row r at 16 (p ^
// (r / 2 % 8)), so that the 16 lanes of a read hit all banks.
// XL: x goes the same way, 16 rows of 512 bytes, piece p of row r at 16 (p ^ r).
// That leaves room for one block of four waves a CU instead of two, which one matrix does not
// mind (14336x4096, without / with: 4 rows 8.5 / 9.1 us, 7 rows 8.9 / 9.1, 10 rows
// 9.8 / 9.1, 32 rows 17.9 / 15.1), but layers do (32 experts 2048x2048 of 8 rows: 22 / 31 us).
// With more blocks than CUs it runs two waves a block, two blocks a CU (us with
// four / two waves: 5120x5120, 64 rows, 320 blocks 18.5 / 14.4; 14336x4096, 32 rows, 448
// blocks 15.1 / 13.0; 14 rows, 224 blocks 9.5 / 11.5).  Without XL four waves it is (two /
// four / eight: one row of 14336x4096 9.7 / 8.0 / 9.3, layer of 37 tokens 111 / 104 / 146).
template <int Q, bool GATED, bool XL, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_mx4(ExpertsView vw, ExpertsView vu, RaggedRows rr,
                                                     const uint16_t* __restrict__ x, void* __restrict__ y,
                                                     int ntiles, int chunks) {
  constexpr int R = 4, RT = GATED ? 2 : 4, kRows = 16 * RT;
  constexpr int kW = 64 * 128, kS = 64 * 8;   // a wave's weights and scales of a window
  __shared__ __attribute__((aligned(128))) char w0[NW * kW], w1[NW * kW], s0[NW * kS], s1[NW * kS];
  constexpr int kX = XL ? 16 * 512 : 4;
  __shared__ __attribute__((aligned(128))) char x0[NW * kX], x1[NW * kX];
  const Place at = place_of(rr, (unsigned)ntiles, (unsigned)chunks);
  if (at.tile >= (unsigned)ntiles || at.chunk >= (unsigned)chunks) return;
  const Share sh = find_share(rr, vw.count, at.chunk, 16 * Q);
  if (sh.count == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t N = vw.n;
  const int K = (int)vw.k, st = (int)mx4_scale_stride(K);
  const int64_t n0 = (int64_t)at.tile * kRows;
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  auto weights = [&](const ExpertsView& v) __attribute__((always_inline)) {
    return rsrc_of(v.w + (int64_t)sh.expert * v.w_stride + n0 * (K / 2), (uint64_t)(rows * (K / 2)));
  };
  auto scales = [&](const ExpertsView& v) __attribute__((always_inline)) {
    return rsrc_of(v.scale + (int64_t)sh.expert * v.scale_stride + n0 * st, (uint64_t)(rows * st));
  };
  const __amdgpu_buffer_rsrc_t ww = weights(vw), ws = scales(vw);
  const __amdgpu_buffer_rsrc_t uw = GATED ? weights(vu) : ww, us = GATED ? scales(vu) : ws;

  // x rows of this lane's slots
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, (uint64_t)rr.x_rows * 2 * (uint64_t)K);
  constexpr int XR = XL ? 8 : Q;
  uint32_t xrow[XR];
  int32_t row[XR];
  auto slot = [&](int q) __attribute__((always_inline)) { return XL ? 2 * q + (lane >> 5) : 16 * q + i16; };
#pragma unroll
  for (int q = 0; q < XR; ++q) row[q] = (int32_t)sh.first + (slot(q) < sh.count ? slot(q) : 0);   // (fewer than 2^31 slots)
  if (rr.rows) {
#pragma unroll
    for (int q = 0; q < XR; ++q) row[q] = rr.rows[row[q]];
  }

  f32x4_t acc[R][Q];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint32_t top[R] = {};   // the largest scale byte of the lane's rows

  // Load i of eight takes rows 8 i .. 8 i + 7, eight lanes a row; of the 64 rows
  // the gated form has W's first, then U's.
  const int pr = lane >> 3;                                   // row of the eight
  auto load_w = [&](int j, char* wbuf, char* sbuf) __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what was read from the buffer has been
    const int k0 = 256 * j;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool u = GATED && i >= 4;
      const int r = 8 * (u ? i - 4 : i) + pr, piece = (lane & 7) ^ ((8 * i + pr) >> 1 & 7);
      const uint32_t off = k0 + 32 * piece < K ? (uint32_t)(r * (K / 2) + (k0 / 2 + 16 * piece)) : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(u ? uw : ww, (lds_char*)(wbuf + wave * kW + 1024 * i), 16, (int)off, 0,
                                               0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // scales, two lanes a row
      const int r = GATED ? lane >> 1 : 32 * i + (lane >> 1);
      const uint32_t off = k0 + 128 * (lane & 1) < K ? (uint32_t)(r * st + 8 * j + 4 * (lane & 1)) : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(GATED && i ? us : ws, (lds_char*)(sbuf + wave * kS + 256 * i), 4,
                                               (int)off, 0, 0, 0);
    }
  };
  auto load_x = [&](int j, char* xbuf, uint4 (&xv)[Q][8]) __attribute__((always_inline)) {
    const int k0 = 256 * j;
    if constexpr (XL) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 8 * ((lane & 31) ^ (2 * i + (lane >> 5)));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_char*)(xbuf + wave * kX + 1024 * i), 16,
                                                 (int)(k < K ? xrow[i] + 2u * (uint32_t)k : kOutside), 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = k0 + 64 * g + 8 * i;
          xv[q][i] = bload16(rx, k < K ? xrow[q] + 2u * (uint32_t)k : kOutside);
        }
    }
  };
  auto compute = [&](int j, const char* wbuf, const char* sbuf, const char* xbuf, const uint4 (&xv)[Q][8]) __attribute__((always_inline)) {
    const bool in0 = 256 * j + 64 * g < K, in1 = 256 * j + 64 * g + 32 < K;
    float scale[R][2];
    uint4 d[R][2];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int r = 16 * t + i16;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        d[t][u] = *reinterpret_cast<const uint4*>(wbuf + wave * kW + r * 128 + (((2 * g + u) ^ (r >> 1 & 7)) << 4));
      const uint32_t f = *reinterpret_cast<const uint16_t*>(sbuf + wave * kS + r * 8 + 2 * g);
      const uint32_t lo = in0 ? f & 255u : 0u, hi = in1 ? f >> 8 : 0u;
      scale[t][0] = e8m0_float(lo);
      scale[t][1] = e8m0_float(hi);
      top[t] = max(top[t], max(lo, hi));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 xl;
      if constexpr (XL) xl = *reinterpret_cast<const uint4*>(xbuf + wave * kX + i16 * 512 + (((8 * g + i) ^ i16) << 4));
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const bf16x8_t a = __builtin_bit_cast(bf16x8_t, mx4_unpack8(word4(d[t][i / 4], i % 4), scale[t][i / 4]));
#pragma unroll
        for (int q = 0; q < Q; ++q)
          acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, XL ? xl : xv[q][i]), acc[t][q],
                                                              0, 0, 0);
      }
    }
  };

  // windows past the last (whole rounds of the waves) lie past K and load zeros
  const int nwin = (K + 255) / 256;
  uint4 xa[Q][8], xb[Q][8];
  load_w(wave, w0, s0);   // on its way while the row indices arrive
#pragma unroll
  for (int q = 0; q < XR; ++q) {
    const bool in = (slot(q) < sh.count) & (row[q] >= 0) & (row[q] < rr.x_rows);
    xrow[q] = in ? (uint32_t)((int64_t)row[q] * K) * 2u : kOutside;
  }
  load_x(wave, x0, xa);
  for (int j = wave; j < nwin; j += 2 * NW) {
    load_w(j + NW, w1, s1);
    load_x(j + NW, x1, xb);
    compute(j, w0, s0, x0, xa);
    load_w(j + 2 * NW, w0, s0);
    load_x(j + 2 * NW, x0, xa);
    compute(j + NW, w1, s1, x1, xb);
  }
  // a NaN scale makes its row's outputs NaN: one more MFMA, NaN times zero
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const uint32_t n = top[t] == 255u ? 0x7FC07FC0u : 0u;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(n, n, n, n)),
                                                          __builtin_bit_cast(bf16x8_t, zero), acc[t][q], 0, 0, 0);
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

template <int FORM, int R, int Q, bool GATED>
hipError_t launch_one(const ExpertsCall& c, hipStream_t s) {
  const int64_t rows = 16 * (GATED ? R / 2 : R), ntiles = (c.w.n + rows - 1) / rows;
  const int64_t chunks = max_chunks(c.r.slots, c.w.count, 16 * Q, c.r.offsets != nullptr);
  const int64_t grid = (chunks * ntiles + 7) / 8 * 8;
  if (!grid_fits(grid, 256)) return hipErrorNotSupported;
  if constexpr (FORM == kFormMx4) {
    auto k = k_experts_mx4<Q, GATED, false, 4>;
    int waves = 4;
    if constexpr (Q == 1 && !GATED) {
      if (!c.r.offsets && c.r.slots > 7) {   // one matrix, slots mostly filled
        waves = grid > device_cus() ? 2 : 4;
        k = waves == 2 ? k_experts_mx4<1, false, true, 2> : k_experts_mx4<1, false, true, 4>;
      }
    }
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(64 * waves), 0, s, c.w, c.u, c.r, c.x, c.y, (int)ntiles, (int)chunks);
  } else {
    hipLaunchKernelGGL((k_experts_rows<FORM, R, Q, GATED>), dim3((unsigned)grid), dim3(256), 0, s, c.w, c.u, c.r, c.x,
                       c.y, (int)ntiles, (int)chunks);
  }
  return hipGetLastError();
}

// Tiles a wave: two and more waves for BF16 and UWF1 (one token, two of eight
// experts, us with 2 / 4: BF16 84 / 115, UWF1 70 / 75).
template <int FORM, int Q, bool GATED>
hipError_t launch_r(const ExpertsCall& c, hipStream_t s) {
  return launch_one<FORM, FORM == kFormMx4 ? 4 : 2, Q, GATED>(c, s);
}

// Two groups of 16 slots where experts have more than 16 rows as a rule and the
// blocks still fill the chip (us with one / two:
// MXFP4 14336x4096, 64 rows 27.5 / 25.3; 5001x8224, 200 rows 65 / 58; BF16 5120x5120, 64 rows 57 / 40).
template <int FORM, bool GATED>
hipError_t launch_form(const ExpertsCall& c, int64_t avg, hipStream_t s) {
  const int64_t rows = 16 * (FORM == kFormMx4 ? 4 : 2) / (GATED ? 2 : 1);
  const int64_t blocks =
      (c.w.n + rows - 1) / rows * max_chunks(c.r.slots, c.w.count, 32, c.r.offsets != nullptr);
  if (avg <= (c.r.offsets ? 12 : 16) || blocks < device_cus()) return launch_r<FORM, 1, GATED>(c, s);
  return launch_r<FORM, 2, GATED>(c, s);
}

template <int FORM>
hipError_t launch_gated(const ExpertsCall& c, int64_t avg, hipStream_t s) {
  return c.gated ? launch_form<FORM, true>(c, avg, s) : launch_form<FORM, false>(c, avg, s);
}

}  // namespace

hipError_t launch_experts_rows(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1, avg = (c.r.slots + e - 1) / e;
  switch (c.w.form) {
    case kFormBf16: return launch_gated<kFormBf16>(c, avg, s);
    case kFormPal: return launch_gated<kFormPal>(c, avg, s);
    case kFormPalRun: return launch_gated<kFormPalRun>(c, avg, s);
    default: return launch_gated<kFormMx4>(c, avg, s);
  }
}

// Which kernel: by the rows an expert has on average if every slot is used
// (the counts themselves are on the device) and the blocks that makes.  The LDS
// tiles read each weight once per tile of 64, 128 or 256 rows, but need a block
// on every CU: with fewer, smaller tiles, and below three quarters of the CUs
// the register-fed kernel, up to the rows where its reloading of weights costs
// more.  It also takes UWF1 and MXFP4 weights, which the tiles pass through
// registers, of experts with few rows.  Measured (us, register-fed / 64 / 128 / 256):
//   BF16 gated, one token, 2 of 8 experts 14336x4096: 85 / 82 / 82 / 83
//   BF16, 32 experts 2048x2048, 16 rows: 73 / 51 / 51 / 52
//   BF16, 16 experts 2048x2048, 64 rows: 69 / 38 / 41 / 46
//   BF16, 24 experts 1500x1024, 167 rows: 114 / 40 / 33 / 33
//   BF16 layer, 64 experts 1408x2048, 281 rows: 1902 / 628 / 489 / 469
//   BF16 gated, 64 experts 1408x2048, 512 rows: 1985 / 600 / 441 / 402
//   UWF1 gated, 16 experts 2048x2048, 1024 rows: 1438 / 579 / 464 / 356
//   UWF1, 32 experts 2048x4096, 3 rows: 75 / 106 / 108 / 114;  16 experts 2048x2048, 48 rows 62 / 53 / 54
//   MXFP4, 16 experts 2048x2048: 32 rows 25 / 29 / 31, 64 rows 38 / 33 / 35, 128 rows 61 / 46 / 37
//   MXFP4 14336x4096: 64 rows 25 / 52 / 59, 128 rows 45 / 55 / 60, 256 rows 74 / 58 / 61
//   MXFP4, few tiles: 5001x8224, 200 rows 58 / 109 / 125; 4096x4096, 256 rows 25 / 52 / 63
hipError_t launch_experts(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1;
  const int64_t avg = (c.r.slots + e - 1) / e;
  if (c.r.x_rows * 2 * c.w.k > kOutside) return launch_experts_tile(c, 256, false, s);   // x past 2 GiB: by pointers
  const int64_t cus = device_cus(), ntiles = (c.w.n + (c.gated ? 127 : 255)) / (c.gated ? 128 : 256);
  auto blocks = [&](int rows) { return ntiles * max_chunks(c.r.slots, c.w.count, rows, c.r.offsets != nullptr); };
  const bool spread = avg <= 96;   // few rows: the weights' way from memory is what counts
  int rows = spread ? 64 : avg <= 256 ? 128 : 256;
  while (rows > 64 && blocks(rows) < cus) rows /= 2;
  const int64_t few = c.w.form == kFormBf16 ? 0 : c.w.form == kFormMx4 ? 40 : 12;
  if (avg <= few || (avg <= 256 && blocks(rows) < cus * 3 / 4))
    return launch_experts_rows(c, s);
  return launch_experts_tile(c, rows, spread, s);
}

}  // namespace uw
