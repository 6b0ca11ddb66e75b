// layer.hip -- the second of the two kernels of a mixture-of-experts layer for a few
// tokens (the first: the routed gated product, experts_rows.hip and fp8_rows.hip):
//   out[t] = BF16( sum over e  w[t][e]  h[slot(t, e)] . D_e^T )
// over the experts e of token t, D_e [n][k] in any form.
//
// A stream over the rows of D of every expert that has tokens.  A block owns 16 / P
// output features and walks all those experts, so the weighted sum ends in one
// block and needs neither partial sums in memory nor a third launch.  Its waves cut
// the list of (expert, window of k) into contiguous runs; a window is a few MFMAs
// with the weights as A (16 features) and h as B (16 tokens), whose sum is
// weighted per token and added to the wave's.  A token without the expert keeps its
// sum: its column could hold an infinity's product with zero.  The waves' sums meet
// in LDS and are added in a fixed order.
//
// P > 1, few tokens and few features: the sixteen rows of an MFMA are 16 / P
// features at P places of k, the columns 16 / P tokens at the same P places.  Where
// the two places agree D holds a product, elsewhere nothing that is used.  Blocks
// are then P times as many, each with P times as much of k in a window.
#include "experts_rows.h"
#include "fp8.h"

namespace uw {
namespace {

constexpr int kNW = 8, kNT = 64 * kNW;

struct LayerDown {
  ExpertsView d;
  const int32_t *ids, *slots;   // [tokens][topk]
  const float* weights;
  const uint16_t* h;            // [pairs][k]
  uint16_t* out;                // [tokens][n]
  int tokens, topk;
};

// The pairs by expert: number of experts with pairs, which, and per expert and
// token its slot (-1: none) and weight.
struct PairsLds {
  int32_t by_slot[kLayerPairs], index[kLayerPairs];
  int32_t expert[kLayerPairs];
  int16_t slot[kLayerPairs][kLayerTokens];
  float weight[kLayerPairs][kLayerTokens];
};

__device__ __forceinline__ int sort_pairs(const LayerDown& c, PairsLds& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, pairs = c.tokens * c.topk;
  int id = -1, slot = -1;
  float w = 0.0f;
  if (tid < pairs) {
    id = c.ids[tid];
    slot = c.slots[tid];
    w = c.weights[tid];
  }
  if (tid < kLayerPairs) s.by_slot[tid] = -1;
  static_assert(sizeof(s.slot) == 16 * kNT, "one store a thread");
  reinterpret_cast<uint4*>(s.slot)[tid] = make_uint4(~0u, ~0u, ~0u, ~0u);
  __syncthreads();
  if (slot >= 0) s.by_slot[slot] = id;
  __syncthreads();
  int experts = 0;   // with pairs; every wave counts them all, the first four write
#pragma unroll
  for (int i = 0; i < kLayerPairs / 64; ++i) {
    const int at = 64 * i + lane, e = s.by_slot[at];
    const bool first = e >= 0 && (at == 0 || s.by_slot[at == 0 ? 0 : at - 1] != e);
    const uint64_t mask = __ballot(first);
    const int mine = experts + __popcll(mask & ((2ull << lane) - 1ull)) - 1;
    if (wave == i) {
      s.index[at] = mine;
      if (first) s.expert[mine] = e;
    }
    experts += __popcll(mask);
  }
  __syncthreads();
  if (slot >= 0) {
    const int i = s.index[slot], t = tid / c.topk;
    s.slot[i][t] = (int16_t)slot;
    s.weight[i][t] = w;
  }
  __syncthreads();
  return experts;
}

// k of a window, and the eight k of an MFMA in lane group g from the window's start
template <int FORM> constexpr int kWindow = FORM == kFormMx4 ? 256 : 128;
template <int FORM> constexpr int kMfmas = kWindow<FORM> / 32;
template <int FORM>
__device__ __forceinline__ int down_k(int m, int g) {
  if constexpr (FORM == kFormMx4) return 128 * (m >> 2) + 32 * g + 8 * (m & 3);
  else if constexpr (FORM == kFormFp8) return 64 * (m >> 1) + 16 * g + 8 * (m & 1);
  else return k_off<FORM>(m, g);
}

template <int FORM, int P>
__global__ __launch_bounds__(kNT) void k_layer_down(LayerDown c) {
  constexpr int kRows = 16 / P, kTokens = 16 / P, W = kWindow<FORM>, M = kMfmas<FORM>;
  __shared__ PairsLds pairs;
  __shared__ f32x4_t red[kNW * 64];
  const int experts = sort_pairs(c, pairs);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int place = i16 / kRows, row = i16 % kRows, token = i16 % kTokens;
  const int64_t n0 = (int64_t)blockIdx.x * kRows, N = c.d.n;
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  const int K = (int)c.d.k, nwin = (K + P * W - 1) / (P * W);
  const __amdgpu_buffer_rsrc_t rh = rsrc_of(c.h, (uint64_t)c.tokens * c.topk * 2 * (uint64_t)K);

  const int total = __builtin_amdgcn_readfirstlane(experts) * nwin;
  const int begin = (int)((int64_t)total * wave / kNW), end = (int)((int64_t)total * (wave + 1) / kNW);

  // The walk: expert `at` of the list, window `j`.  It runs ahead of the sums, past
  // the end as well, where everything reads zeros.
  struct Walk {
    int at, j, left;
  };
  auto next = [&](Walk& w) __attribute__((always_inline)) {
    --w.left;
    if (++w.j == nwin) {
      w.j = 0;
      ++w.at;
    }
  };
  struct Win {
    Raw r;
    PalView pal;
    uint32_t sc[2];    // MXFP4: two blocks' scale bytes; FP8: the block's scale
    uint4 xv[M];
    float weight;
    bool has;
  };
  Walk wl{begin / nwin, begin % nwin, end - begin}, wf = wl;
  Flags fa[3];

  // UWF1: the flag and rank words, a window ahead of its data
  auto flags = [&](Flags& f) __attribute__((always_inline)) {
    if constexpr (form_is_pal(FORM)) {
      const int e = __builtin_amdgcn_readfirstlane(pairs.expert[wf.left > 0 ? wf.at : 0]);
      const Mat<FORM> m = matrix_of<FORM>(c.d, e, n0, kRows);
      load_flags(m, row, K, wf.left > 0 ? P * W * wf.j + W * place + k_off<FORM>(0, g) : K, f);
      next(wf);
    }
  };
  auto load = [&](const Flags& f, Win& w) __attribute__((always_inline)) {
    const bool in = wl.left > 0;
    const int at = in ? wl.at : 0, e = __builtin_amdgcn_readfirstlane(pairs.expert[at]);
    const int slot = token < c.tokens ? pairs.slot[at][token] : -1;
    w.weight = pairs.weight[at][token];
    w.has = in && slot >= 0;
    const int k0 = in ? P * W * wl.j + W * place : K;
    if constexpr (FORM == kFormBf16 || form_is_pal(FORM)) {
      const Mat<FORM> m = matrix_of<FORM>(c.d, e, n0, kRows);
      load_raw(m, row, K, k0, g, f, w.r);
      if constexpr (form_is_pal(FORM)) w.pal = m.t.pal;
    } else if constexpr (FORM == kFormFp8) {
      const __amdgpu_buffer_rsrc_t rw = rsrc_of(c.d.w + (int64_t)e * c.d.w_stride + n0 * K, (uint64_t)(rows * K));
      const int nb = (int)fp8_blocks(K);
      const __amdgpu_buffer_rsrc_t rs =
          rsrc_of(c.d.scale + (int64_t)e * c.d.scale_stride + (n0 >> 7) * nb * 4, (uint64_t)nb * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = k0 + 64 * i + 16 * g;
        w.r.d[i] = bload16(rw, k < K ? (uint32_t)(row * K + k) : kOutside);
      }
      w.sc[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, k0 < K ? (k0 >> 7) * 4 : (int)kOutside, 0, 0);
    } else {
      const int st = (int)mx4_scale_stride(K);
      const __amdgpu_buffer_rsrc_t rw =
          rsrc_of(c.d.w + (int64_t)e * c.d.w_stride + n0 * (K / 2), (uint64_t)(rows * (K / 2)));
      const __amdgpu_buffer_rsrc_t rs =
          rsrc_of(c.d.scale + (int64_t)e * c.d.scale_stride + n0 * st, (uint64_t)(rows * st));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = k0 + 128 * i + 32 * g;
        w.r.d[i] = bload16(rw, k < K ? (uint32_t)(row * (K / 2) + k / 2) : kOutside);
        w.sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, k < K ? (int)(row * st + k / 32) : (int)kOutside, 0, 0);
      }
    }
    const uint32_t hrow = slot >= 0 ? (uint32_t)slot * 2u * (uint32_t)K : kOutside;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int k = k0 + down_k<FORM>(m, g);
      w.xv[m] = bload16(rh, k < K ? hrow + 2u * (uint32_t)k : kOutside);
    }
    next(wl);
  };

  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Win& w) __attribute__((always_inline)) {
    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < M; ++m) {
      bf16x8_t a;
      if constexpr (FORM == kFormFp8) {
        const uint4& d = w.r.d[m >> 1];
        a = __builtin_bit_cast(bf16x8_t, m & 1 ? fp8_unpack8(d.z, d.w) : fp8_unpack8(d.x, d.y));
      } else if constexpr (FORM == kFormMx4) {
        a = __builtin_bit_cast(bf16x8_t, mx4_unpack8(word4(w.r.d[m >> 2], m & 3), e8m0_float(w.sc[m >> 2] & 255u)));
      } else {
        Mat<FORM> mt{};
        mt.t.pal = w.pal;
        a = a_frag(mt, w.r, m);
      }
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, w.xv[m]), part, 0, 0, 0);
    }
    float scale = w.weight;
    if constexpr (FORM == kFormFp8) {
      scale = __builtin_bit_cast(float, w.sc[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) part[i] *= scale;
      scale = w.weight;
    }
    if constexpr (FORM == kFormMx4) {   // a NaN scale makes its row NaN: one more MFMA, NaN times zero
      const bool nan = (w.sc[0] & 255u) == 255u || (w.sc[1] & 255u) == 255u;
      if (__ballot(nan)) {
        const uint32_t n = nan ? 0x7FC07FC0u : 0u;
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(n, n, n, n)),
                                                       __builtin_bit_cast(bf16x8_t, make_uint4(0u, 0u, 0u, 0u)), part, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = w.has ? __builtin_fmaf(part[i], scale, acc[i]) : acc[i];
  };

  if (end > begin) {
    Win wa, wb, wc;
    flags(fa[0]);
    flags(fa[1]);
    load(fa[0], wa);
    flags(fa[2]);
    load(fa[1], wb);
    flags(fa[0]);
    for (int i = begin; i < end; i += 3) {
      load(fa[2], wc);
      flags(fa[1]);
      compute(wa);
      load(fa[0], wa);
      flags(fa[2]);
      compute(wb);
      load(fa[1], wb);
      flags(fa[0]);
      compute(wc);
    }
  }
  red[wave * 64 + lane] = acc;
  __syncthreads();
  // D: lane l holds rows 4 (l / 16) .. +3 of column l % 16
  const float* r = reinterpret_cast<const float*>(red);
  for (int i = threadIdx.x; i < kRows * c.tokens; i += kNT) {
    const int t = i / kRows, f = i % kRows;
    if (f >= rows) continue;
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int dr = p * kRows + f, at = ((dr >> 2) * 16 + p * kTokens + t) * 4 + (dr & 3);
#pragma unroll
      for (int v = 0; v < kNW; ++v) s += r[v * 256 + at];
    }
    c.out[(int64_t)t * N + n0 + f] = (uint16_t)bf16_pair(s, s);
  }
}

template <int FORM, int P>
hipError_t launch_p(const LayerDown& c, hipStream_t s) {
  const int64_t grid = (c.d.n + 16 / P - 1) / (16 / P);   // (n is at most 2^20)
  hipLaunchKernelGGL((k_layer_down<FORM, P>), dim3((unsigned)grid), dim3(kNT), 0, s, c);
  return hipGetLastError();
}

template <int FORM>
hipError_t launch_form(const LayerDown& c, hipStream_t s) {
  const int64_t cus = device_cus();
  if (c.d.n / 16 >= cus || c.tokens > 8) return launch_p<FORM, 1>(c, s);
  if (c.d.n / 8 >= cus || c.tokens > 4) return launch_p<FORM, 2>(c, s);
  return launch_p<FORM, 4>(c, s);
}

}  // namespace

hipError_t launch_layer_down(const ExpertsView& d, const RouteCall& r, const uint16_t* h, uint16_t* out, hipStream_t s) {
  const LayerDown c{d, r.ids, r.slots, r.weights, h, out, (int)r.tokens, r.topk};
  switch (d.form) {
    case kFormBf16: return launch_form<kFormBf16>(c, s);
    case kFormPal: return launch_form<kFormPal>(c, s);
    case kFormPalRun: return launch_form<kFormPalRun>(c, s);
    case kFormFp8: return launch_form<kFormFp8>(c, s);
    default: return launch_form<kFormMx4>(c, s);
  }
}

}  // namespace uw
