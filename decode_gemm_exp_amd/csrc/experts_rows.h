// experts_rows.h -- what the kernels for few rows an expert share: a lane's weights
// of one window as loaded and as an MFMA takes them (BF16, UWF1), a block's place in
// the grid, and the end of a block.
#pragma once

#include "route.h"

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
  const unsigned eighth = (ntiles * chunks + 7) / 8;   // (of the grid, a multiple of 8: one argument less to load)
  const unsigned turn = (blockIdx.x & 7) * eighth + (blockIdx.x >> 3);
  return {turn / chunks, turn % chunks};
}

// A block's tiles and experts, and the rows of x its slots multiply.  RaggedRows: one
// tile, by the plan in memory.  RoutedRows: by its own choice, block 0 writing the plan
// and the others walking through the tiles of every expert that has pairs, so that a block
// routes once however many tiles there are.
template <typename RR>
struct Finder;

template <>
struct Finder<RaggedRows> {
  static constexpr bool kWalks = false;
  struct Lds {};
  // false: the block has nothing (more) to do
  template <int NW>
  __device__ __forceinline__ bool begin(const RaggedRows&, Lds&) { return true; }
  __device__ __forceinline__ bool find(const RaggedRows& rr, Lds&, int, unsigned ntiles, unsigned chunks, int experts,
                                       int most, unsigned& tile, Share& sh) const {
    const Place at = place_of(rr, ntiles, chunks);
    if (at.tile >= ntiles || at.chunk >= chunks) return false;
    tile = at.tile;
    sh = find_share(rr, experts, at.chunk, most);
    return sh.count != 0;
  }
  // row[q]: of slot slot(q), those behind the share's last as its first
  template <int N, typename F>
  __device__ __forceinline__ void rows(const RaggedRows& rr, const Lds&, const Share& sh, int32_t (&row)[N], F&& slot) const {
#pragma unroll
    for (int q = 0; q < N; ++q) row[q] = (int32_t)sh.first + (slot(q) < sh.count ? slot(q) : 0);   // (fewer than 2^31 slots)
    if (rr.rows) {
#pragma unroll
      for (int q = 0; q < N; ++q) row[q] = rr.rows[row[q]];
    }
  }
};

template <int L, int NV>
struct Finder<RoutedRows<L, NV>> {
  static constexpr bool kWalks = true;
  using Lds = RoutedLds;
  int items;
  template <int NW>
  __device__ __forceinline__ bool begin(const RoutedRows<L, NV>& rr, Lds& lds) {
    if (blockIdx.x == 0) {
      write_few<L, NV, NW>(rr.c, lds);
      return false;
    }
    items = __builtin_amdgcn_readfirstlane(route_few<L, NV, NW>(rr.c, lds));
    return true;
  }
  // the block's turn-th tile
  __device__ __forceinline__ bool find(const RoutedRows<L, NV>&, Lds& lds, int turn, unsigned ntiles, unsigned, int, int,
                                       unsigned& tile, Share& sh) const {
    const unsigned at = blockIdx.x - 1 + (unsigned)turn * (gridDim.x - 1), item = at / ntiles;
    if (item >= (unsigned)items) return false;
    tile = at - item * ntiles;
    sh.expert = __builtin_amdgcn_readfirstlane(lds.expert[item]);
    sh.first = __builtin_amdgcn_readfirstlane(lds.first[item]);
    sh.count = __builtin_amdgcn_readfirstlane(lds.first[item + 1]) - (int)sh.first;
    return true;
  }
  template <int N, typename F>
  __device__ __forceinline__ void rows(const RoutedRows<L, NV>&, const Lds& lds, const Share& sh, int32_t (&row)[N], F&& slot) const {
    const uint32_t tokens = lds.tokens[sh.expert];
#pragma unroll
    for (int q = 0; q < N; ++q) row[q] = nth_bit(tokens, slot(q) < sh.count ? slot(q) : 0);
  }
};

// The waves' sums, added in wave order and stored.  red: per wave and tile
// the MFMA's D: lane l holds output features 4 (l / 16) .. +3 of slot l % 16.
// rows: the block's, up to N - n0 of them or a multiple of four.
template <int R, int Q, bool GATED, int NW>
__device__ __forceinline__ void finish(const f32x4_t* red, const Share& sh, int64_t n0, int64_t rows, int64_t N,
                                       void* __restrict__ y) {
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
    const int f = 16 * t + 4 * (ln >> 4);
    const int64_t n = n0 + f;
    if (b >= sh.count || f >= rows) continue;
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

}  // namespace
}  // namespace uw
