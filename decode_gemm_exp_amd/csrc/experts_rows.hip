// experts_rows.hip -- products grouped by expert for few rows an expert:
// y[s] = x[row(s)] . W_e^T for the slots s of expert e, weights BF16, UWF1
// (palette indices) or MXFP4, and the gated form silu(x . G_e^T) * (x . U_e^T).
//
// With few rows an expert the product is a stream over the weights of the
// experts that have rows, so the kernel keeps many bytes of them in flight and
// reuses nothing but x:
//   * a block owns 16 R rows of one expert's weights and up to 16 Q of its
//     slots; its four waves walk interleaved windows of K, each loading its
//     weights straight into registers, two windows deep, and feeding
//     v_mfma_f32_16x16x32_bf16 with the weights as A (16 output features) and
//     x as B (16 slots);
//   * the order of k inside an MFMA is free as long as A and B agree.  BF16:
//     MFMA m of a 128-wide window takes k 32 m + 8 g .. +7 in lane group g, so
//     a load reads 64 contiguous bytes of each of 16 rows.  The byte and
//     nibble forms give lane group g a run of 32 (MXFP4: 64) consecutive k, so
//     that a lane's weights lie in one UWF1 group or whole MXFP4 blocks;
//   * the four waves' sums meet in LDS and are added in a fixed order.
#include "experts.h"

namespace uw {
namespace {

__device__ __forceinline__ uint32_t word4(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// units of 32 weights a lane takes of a window, and the window's width
template <int FORM> constexpr int units() { return FORM == kFormMx4 ? 2 : 1; }
template <int FORM> constexpr int window() { return 128 * units<FORM>(); }

// k of MFMA (u, m)'s eight weights in lane group g, from the window's start
template <int FORM>
__device__ __forceinline__ int k_off(int u, int m, int g) {
  return FORM == kFormBf16 ? 32 * m + 8 * g : 32 * units<FORM>() * g + 32 * u + 8 * m;
}

// one expert's matrix
struct Mat {
  const uint8_t* w;
  const uint8_t* scale;
  ExpertEntry t;
};

template <int FORM>
__device__ __forceinline__ Mat matrix_of(const ExpertsView& v, int e) {
  Mat m{};
  if constexpr (form_is_pal(FORM)) {
    m.t = v.table[e];
  } else {
    m.w = v.w + (int64_t)e * v.w_stride;
    if constexpr (FORM == kFormMx4) m.scale = v.scale + (int64_t)e * v.scale_stride;
  }
  return m;
}

// A lane's weights of one window of one row, as loaded:
//   BF16: d[m] = the eight of MFMA m;  MXFP4: d[u] = 32 elements, f = the two
//   scale bytes;  UWF1: d[0], d[1] = 32 sign+mantissa bytes, d[2] = 32 index
//   nibbles, or d[2], d[3] = 32 exponent bytes when f (verbatim group)
struct Raw {
  uint4 d[4];
  uint32_t f;
};

// flag and rank words of the lane's group (UWF1), loaded a window ahead
struct Flags {
  uint32_t fw, rw;
};

template <int FORM>
__device__ __forceinline__ void load_flags(const Mat& m, int64_t row, int64_t K, int64_t k, bool ok, Flags& f) {
  if constexpr (form_is_pal(FORM)) {
    const uint64_t w = ok ? (uint64_t)(row * K + k) >> 11 : 0;
    f.fw = gload<uint32_t>(m.t.vflags + w);
    f.rw = gload<uint32_t>(m.t.vrank + w);
  }
}

// row: inside the matrix; k0: the window's start; weights at k >= K are not
// loaded (the row's first are, and are zeroed when unpacked)
template <int FORM>
__device__ __forceinline__ void load_raw(const Mat& m, int64_t row, int64_t K, int64_t k0, int g, const Flags& fl, Raw& r) {
  if constexpr (FORM == kFormBf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(m.w) + row * K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + k_off<FORM>(0, i, g);
      r.d[i] = *reinterpret_cast<const uint4*>(p + (k < K ? k : 0));
    }
  } else if constexpr (FORM == kFormMx4) {
    const uint8_t* p = m.w + row * (K / 2);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = k0 + k_off<FORM>(u, 0, g);
      r.d[u] = *reinterpret_cast<const uint4*>(p + (k < K ? k : 0) / 2);
    }
    const int64_t k = k0 + k_off<FORM>(0, 0, g);   // a multiple of 64: the pair of scales is aligned
    r.f = *reinterpret_cast<const uint16_t*>(m.scale + row * mx4_scale_stride(K) + (k < K ? k : 0) / 32);
  } else {
    const int64_t k = k0 + k_off<FORM>(0, 0, g);
    const uint64_t el = (uint64_t)(row * K + (k < K ? k : 0));
    r.d[0] = gload16(m.t.sm + el);
    r.d[1] = gload16(m.t.sm + el + 16);
    const uint64_t grp = el >> 6;
    const bool v = k < K && group_verbatim(fl.fw, grp);
    const uint8_t* p = v ? m.t.vexp + (uint64_t)group_rank(fl.fw, fl.rw, grp) * 64 + (el & 63) : m.t.pidx + el / 2;
    r.d[2] = gload16(p);
    if (v) r.d[3] = gload16(p + 16);
    r.f = v ? 1u : 0u;
  }
}

// A operand of MFMA (u, m)
template <int FORM>
__device__ __forceinline__ bf16x8_t a_frag(const Mat& mt, const Raw& r, int u, int m, bool ok) {
  uint4 o;
  if constexpr (FORM == kFormBf16) {
    o = r.d[m];
  } else if constexpr (FORM == kFormMx4) {
    o = mx4_unpack8(word4(r.d[u], m), e8m0_float((r.f >> (8 * u)) & 255u));
    // (scale 255 is NaN, whatever the element)
    if (((r.f >> (8 * u)) & 255u) == 255u) o = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
  } else {
    const int wi = 2 * (m & 1);
    uint32_t e0, e1;
    pal8<FORM == kFormPalRun>(word4(r.d[2], m), mt.t.pal, e0, e1);
    e0 = r.f ? word4(r.d[2 + (m >> 1)], wi) : e0;
    e1 = r.f ? word4(r.d[2 + (m >> 1)], wi + 1) : e1;
    rebuild4(word4(r.d[m >> 1], wi), e0, o.x, o.y);
    rebuild4(word4(r.d[m >> 1], wi + 1), e1, o.z, o.w);
  }
  o.x = ok ? o.x : 0u;
  o.y = ok ? o.y : 0u;
  o.z = ok ? o.z : 0u;
  o.w = ok ? o.w : 0u;
  return __builtin_bit_cast(bf16x8_t, o);
}

// R weight tiles of 16 rows (gated: the first half from W, the second the
// same rows of U), Q groups of 16 slots
template <int FORM, int R, int Q, bool GATED>
__global__ __launch_bounds__(256) void k_experts_rows(ExpertsView vw, ExpertsView vu, RaggedRows rr,
                                                      const uint16_t* __restrict__ x, void* __restrict__ y,
                                                      int ntiles) {
  constexpr int U = units<FORM>(), W = window<FORM>();
  constexpr int RT = GATED ? R / 2 : R;   // distinct output tiles
  __shared__ f32x4_t red[4 * R * Q * 64];
  const Share sh = find_share(rr, vw.count, blockIdx.x / (unsigned)ntiles, 16 * Q);
  if (sh.count == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t N = vw.n, K = vw.k;
  const int64_t n0 = (int64_t)(blockIdx.x % (unsigned)ntiles) * (16 * RT);
  const Mat mw = matrix_of<FORM>(vw, sh.expert);
  Mat mu = mw;
  if constexpr (GATED) mu = matrix_of<FORM>(vu, sh.expert);
  auto mat = [&](int t) __attribute__((always_inline)) -> const Mat& { return GATED && t >= RT ? mu : mw; };

  // x rows of this lane's slots; slots past the share and rows outside x read
  // row 0 and are zeroed
  const uint16_t* xrow[Q];
  bool xok[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int b = 16 * q + i16;
    int64_t row = sh.first + (b < sh.count ? b : 0);
    if (rr.rows) row = rr.rows[row];
    xok[q] = b < sh.count && row >= 0 && row < rr.x_rows;
    xrow[q] = x + (xok[q] ? row : 0) * K;
  }
  // weight rows of this lane, clamped into the matrix (those past it are not stored)
  int64_t wrow[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int64_t n = n0 + 16 * (t % RT) + i16;
    wrow[t] = n < N ? n : N - 1;
  }

  const int nwin = (int)((K + W - 1) / W);
  f32x4_t acc[R][Q];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  struct Win {
    Raw r[R];
    uint4 xv[Q][4 * U];
  };
  auto flags = [&](int j, Flags (&f)[R]) __attribute__((always_inline)) {
    const int64_t k = (int64_t)W * j + k_off<FORM>(0, 0, g);
#pragma unroll
    for (int t = 0; t < R; ++t) load_flags<FORM>(mat(t), wrow[t], K, k, j < nwin && k < K, f[t]);
  };
  auto load = [&](int j, const Flags (&f)[R], Win& w) __attribute__((always_inline)) {
    const int64_t k0 = j < nwin ? (int64_t)W * j : 0;
#pragma unroll
    for (int t = 0; t < R; ++t) load_raw<FORM>(mat(t), wrow[t], K, k0, g, f[t], w.r[t]);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4 * U; ++i) {
        const int64_t k = k0 + k_off<FORM>(i / 4, i % 4, g);
        w.xv[q][i] = *reinterpret_cast<const uint4*>(xrow[q] + (k < K ? k : 0));
      }
  };
  auto compute = [&](int j, const Win& w) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)W * j;
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) {
      const bool ok = j < nwin && k0 + k_off<FORM>(i / 4, i % 4, g) < K;
      bf16x8_t b[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        uint4 v = w.xv[q][i];
        const bool in = ok && xok[q];
        v.x = in ? v.x : 0u;
        v.y = in ? v.y : 0u;
        v.z = in ? v.z : 0u;
        v.w = in ? v.w : 0u;
        b[q] = __builtin_bit_cast(bf16x8_t, v);
      }
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const bf16x8_t a = a_frag<FORM>(mat(t), w.r[t], i / 4, i % 4, ok);
#pragma unroll
        for (int q = 0; q < Q; ++q) acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[q], acc[t][q], 0, 0, 0);
      }
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
    compute(j, wa);
    load(j + 8, fa, wa);
    flags(j + 16, fa);
    compute(j + 4, wb);
  }

  // the waves' sums, added in wave order.  D of the MFMA: lane l holds output
  // features 4 (l / 16) .. +3 of slot l % 16
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int q = 0; q < Q; ++q) red[((wave * R + t) * Q + q) * 64 + lane] = acc[t][q];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * Q * 64; i += 256) {
    const int ln = i & 63, q = (i >> 6) % Q, t = (i >> 6) / Q;
    auto sum = [&](int tt) __attribute__((always_inline)) {
      f32x4_t s = red[(tt * Q + q) * 64 + ln];
#pragma unroll
      for (int v = 1; v < 4; ++v) s += red[((v * R + tt) * Q + q) * 64 + ln];
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

template <int FORM, int Q>
hipError_t launch_q(const ExpertsCall& c, hipStream_t s) {
  const int64_t chunks = max_chunks(c.r.slots, c.w.count, 16 * Q, c.r.offsets != nullptr);
  const int64_t ntiles = (c.w.n + (c.gated ? 15 : 31)) / (c.gated ? 16 : 32);
  if (chunks * ntiles > INT32_MAX) return hipErrorNotSupported;
  const dim3 grid((unsigned)(chunks * ntiles));
  if (c.gated)
    hipLaunchKernelGGL((k_experts_rows<FORM, 2, Q, true>), grid, dim3(256), 0, s, c.w, c.u, c.r, c.x, c.y, (int)ntiles);
  else
    hipLaunchKernelGGL((k_experts_rows<FORM, 2, Q, false>), grid, dim3(256), 0, s, c.w, c.w, c.r, c.x, c.y, (int)ntiles);
  return hipGetLastError();
}

template <int FORM>
hipError_t launch_form(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1;
  const int64_t avg = (c.r.slots + e - 1) / e;
  if (avg <= 16) return launch_q<FORM, 1>(c, s);
  if (avg <= 32) return launch_q<FORM, 2>(c, s);
  return launch_q<FORM, 4>(c, s);
}

}  // namespace

hipError_t launch_experts_rows(const ExpertsCall& c, hipStream_t s) {
  switch (c.w.form) {
    case kFormBf16: return launch_form<kFormBf16>(c, s);
    case kFormPal: return launch_form<kFormPal>(c, s);
    case kFormPalRun: return launch_form<kFormPalRun>(c, s);
    default: return launch_form<kFormMx4>(c, s);
  }
}

// Which kernel: by the rows an expert has on average if every slot is used
// (the counts themselves are on the device).  The register-fed kernel streams
// weights for few rows; the LDS tiles rebuild and read each weight once per
// tile of 64, 128 or 256 rows.  Measured (us, register-fed / 64 / 128 / 256):
//   BF16, 16 experts 2048x2048, 64 rows: 69 / 42 / 44 / 53
//   BF16 gated, 64 experts 1408x2048, 512 rows: 1985 / 581 / 529 / 450
//   BF16 layer, 64 experts 1408x2048, 281 rows: 1902 / 601 / 593 / 539
//   UWF1 gated, 16 experts 2048x2048, 1024 rows: 1438 / 772 / 495 / 409
//   UWF1, 32 experts 2048x4096, 3 rows: 78 / 106 / 110 / 135
hipError_t launch_experts(const ExpertsCall& c, hipStream_t s) {
  const int64_t e = c.r.offsets ? c.w.count : 1;
  const int64_t avg = (c.r.slots + e - 1) / e;
  if (avg <= 8) return launch_experts_rows(c, s);
  return launch_experts_tile(c, avg <= 96 ? 64 : avg <= 160 ? 128 : 256, s);
}

}  // namespace uw
