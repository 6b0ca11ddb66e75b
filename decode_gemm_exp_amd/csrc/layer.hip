// layer.hip -- the second of the two kernels of a mixture-of-experts layer for a few
// tokens (the first: the routed gated product, experts_rows.hip and fp8_rows.hip):
//   out[t] = BF16( sum over e  w[t][e]  h[slot(t, e)] . D_e^T )
// over the experts e of token t, D_e [n][k] in any form.
//
// h is BF16, as uw_matmul_experts_gated gives it: the matrix unit takes it so, and FP32 sums follow
// (out is off by 0.0023 to 0.0024 of its norm, 0.0017 of which is its own rounding to BF16).
//
// A stream over the rows of D of every expert that has tokens.  A block owns 16 / P
// output features and walks all those experts, so the weighted sum ends in one
// block and needs neither partial sums in memory nor a third launch.  An item is an
// expert and up to C of its tokens; the waves cut the list of (item, window of k)
// into contiguous runs.  A window is a few MFMAs with the weights as A and h as B; at
// the end of an item (or of a run) a wave adds its tokens' sums, weighted, to sums of
// its own in LDS, and the waves' are added in a fixed order at last.
//
// Rows and columns of an MFMA are used to the full:
//   P > 1: its sixteen rows are 16 / P features at P places of k, its columns 16 / P
//     at the same P places.  Where the two places agree D holds a product, elsewhere
//     nothing that is used.  Blocks are P times as many: 2048 features are 128 tiles
//     of sixteen, half the CUs (16 tokens over 64 experts 1408x2048, P = 1 / 2: BF16 94 / 60 us, FP8
//     63 / 42; MXFP4 over 160 experts, C = 4, 45.5 / 30.2: 4 TB/s of weights).
//   C < 16 / P: few tokens have an expert in common, and the columns behind the C-th of a
//     place would hold nothing.  A load of h then fetches the pieces of 16 / (P C)
//     MFMAs at once, one in each run of C columns, and each MFMA but the first moves
//     its pieces to the first run.
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

// returns the number of items
template <int C>
__device__ __forceinline__ int sort_pairs(const LayerDown& c, PairsLds& s) {
  const int tid = threadIdx.x, pairs = c.tokens * c.topk;
  int id = -1, slot = -1;
  float w = 0.0f;
  if (tid < pairs) {
    id = c.ids[tid];
    slot = c.slots[tid];
    w = c.weights[tid];
  }
  if (tid < kLayerPairs) s.expert[tid] = -1;
  __syncthreads();
  if (slot >= 0) {
    s.expert[slot] = id;
    s.token[slot] = tid / c.topk;
    s.weight[slot] = w;
  }
  __syncthreads();
  return list_items<C>(s);
}

// k of a window, and the eight k of an MFMA in lane group g from the window's start
template <int FORM> constexpr int kWindow = FORM == kFormMx4 ? 256 : 128;
template <int FORM> constexpr int kMfmas = kWindow<FORM> / 32;
// windows a wave has on their way
template <int FORM> constexpr int kDepth = FORM == kFormMx4 ? 4 : 3;
template <int FORM>
__device__ __forceinline__ int down_k(int m, int g) {
  if constexpr (FORM == kFormMx4) return 128 * (m >> 2) + 32 * g + 8 * (m & 3);
  else if constexpr (FORM == kFormFp8) return 64 * (m >> 1) + 16 * g + 8 * (m & 1);
  else return k_off<FORM>(m, g);
}

// lane i takes lane i + N's (within sixteen)
template <int N>
__device__ __forceinline__ uint4 from_right(const uint4& v) {
  auto move = [](uint32_t x) __attribute__((always_inline)) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x100 + N, 0xF, 0xF, true);
  };
  return make_uint4(move(v.x), move(v.y), move(v.z), move(v.w));
}

template <int FORM, int P, int C>
__global__ __launch_bounds__(kNT) void k_layer_down(LayerDown c) {
  constexpr int kRows = 16 / P, X = kRows / C;   // X: MFMAs whose pieces of h one load fetches
  constexpr int W = kWindow<FORM>, M = kMfmas<FORM>;
  static_assert(M % X == 0, "loads of h are whole");
  __shared__ PairsLds pairs;
  __shared__ float sums[kNW][P][kLayerTokens][kRows];
  const int items = sort_pairs<C>(c, pairs);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int place = i16 / kRows, row = i16 % kRows, piece = row / C, token = row % C;
  const int64_t n0 = (int64_t)blockIdx.x * kRows, N = c.d.n;
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  const int K = (int)c.d.k, nwin = (K + P * W - 1) / (P * W);
  const __amdgpu_buffer_rsrc_t rh = rsrc_of(c.h, (uint64_t)c.tokens * c.topk * 2 * (uint64_t)K);
  for (int i = lane; i < P * kLayerTokens * kRows; i += 64) (&sums[wave][0][0][0])[i] = 0.0f;

  const int total = __builtin_amdgcn_readfirstlane(items) * nwin;
  const int begin = (int)((int64_t)total * wave / kNW), end = (int)((int64_t)total * (wave + 1) / kNW);

  // The walk: item `at`, window `j`.  It runs ahead of the sums, past the end as well,
  // where everything reads zeros.
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
    uint4 xv[M / X];
    float weight;      // of the item's token in this lane's column
    int to;            // that token, -1: none
    bool ends;         // the item's last window, or the run's
  };
  Walk wl{begin / nwin, begin % nwin, end - begin}, wf = wl;
  constexpr int D = kDepth<FORM>;
  Flags fl[D];

  // UWF1: the flag and rank words, a window ahead of its data; of the expert that is
  // being loaded its table entry, of the one whose flags are, which may be the next, a copy
  Mat<FORM> mat{}, fmat{};
  int flagged = -1;
  auto flags = [&](Flags& f) __attribute__((always_inline)) {
    if constexpr (form_is_pal(FORM)) {
      const bool in = wf.left > 0;
      if (in && wf.at != flagged) {
        flagged = wf.at;
        fmat = matrix_of<FORM>(c.d, __builtin_amdgcn_readfirstlane(pairs.item_expert[flagged]), n0, kRows);
      }
      load_flags(fmat, row, K, in ? P * W * wf.j + W * place + k_off<FORM>(0, g) : K, f);
      next(wf);
    }
  };
  // A lane's offsets in its matrix, scales and row of h for window 0; the window goes by
  // the loads' scalar offset.  The last window may pass K and has offsets of its own.
  constexpr int NW_ = FORM == kFormBf16 ? 4 : 2, NX = M / X;
  uint32_t wo[2][NW_], so[2][2], xo[2][NX];
  const int last = P * W * (nwin - 1);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int end_k = t ? K - last : W * P;   // from the window's start
    auto at = [&](int k, uint32_t off) __attribute__((always_inline)) { return k < end_k ? off : kOutside; };
    const int kp = W * place, st = (int)mx4_scale_stride(K);
#pragma unroll
    for (int i = 0; i < NW_; ++i) {
      const int k = kp + (FORM == kFormBf16 ? 32 * i + 8 * g : FORM == kFormFp8 ? 64 * i + 16 * g : 128 * i + 32 * g);
      wo[t][i] = at(k, FORM == kFormBf16 ? (uint32_t)(row * K + k) * 2u
                                         : FORM == kFormFp8 ? (uint32_t)(row * K + k) : (uint32_t)(row * (K / 2) + k / 2));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      so[t][i] = FORM == kFormFp8 ? at(kp, 4u * place) : at(kp + 128 * i + 32 * g, (uint32_t)(row * st + (kp + 128 * i + 32 * g) / 32));
#pragma unroll
    for (int l = 0; l < NX; ++l) {
      int k = kp + down_k<FORM>(X * l, g);
#pragma unroll
      for (int x = 1; x < X; ++x) k = piece == x ? kp + down_k<FORM>(X * l + x, g) : k;
      xo[t][l] = at(k, 2u * (uint32_t)k);
    }
  }
  // the item that is being loaded
  __amdgpu_buffer_rsrc_t rw = rh, rs = rh;
  uint32_t hrow = kOutside;
  float weight = 0.0f;
  int to = -1, loaded = -1;      // the token of this lane's column, -1: none
  // what LDS says of the next one, read an item ahead
  int next_e = 0, next_slot = 0, next_end = 0;
  auto look = [&](int item) __attribute__((always_inline)) {
    next_e = pairs.item_expert[item];
    next_slot = pairs.item_first[item] + token;
    next_end = pairs.item_first[item + 1];
  };
  auto load = [&](const Flags& f, Win& w) __attribute__((always_inline)) {
    const bool in = wl.left > 0;
    if (in && wl.at != loaded) {
      loaded = wl.at;
      const int e = __builtin_amdgcn_readfirstlane(next_e);
      const bool has = next_slot < next_end;   // (slots up to the next item's first are the item's)
      hrow = has ? (uint32_t)next_slot * 2u * (uint32_t)K : kOutside;
      weight = pairs.weight[has ? next_slot : 0];
      to = has ? pairs.token[next_slot] : -1;
      look(loaded + 1);
      const uint8_t* base = c.d.w + (int64_t)e * c.d.w_stride;
      if constexpr (FORM == kFormBf16) {
        rw = rsrc_of(base + n0 * 2 * K, (uint64_t)(rows * 2 * K));
      } else if constexpr (FORM == kFormFp8) {
        const int nb = (int)fp8_blocks(K);
        rw = rsrc_of(base + n0 * K, (uint64_t)(rows * K));
        rs = rsrc_of(c.d.scale + (int64_t)e * c.d.scale_stride + (n0 >> 7) * nb * 4, (uint64_t)nb * 4);
      } else if constexpr (FORM == kFormMx4) {
        const int st = (int)mx4_scale_stride(K);
        rw = rsrc_of(base + n0 * (K / 2), (uint64_t)(rows * (K / 2)));
        rs = rsrc_of(c.d.scale + (int64_t)e * c.d.scale_stride + n0 * st, (uint64_t)(rows * st));
      } else {
        mat = matrix_of<FORM>(c.d, e, n0, kRows);
      }
    }
    w.weight = weight;
    w.to = to;
    w.ends = in && (wl.j == nwin - 1 || wl.left == 1);
    const bool tail = wl.j == nwin - 1;
    const int k0 = P * W * wl.j;
    auto pick = [&](uint32_t most, uint32_t end) __attribute__((always_inline)) {
      return in ? tail ? end : most : kOutside;
    };
    if constexpr (form_is_pal(FORM)) {
      load_raw(mat, row, K, in ? k0 + W * place : K, g, f, w.r);
      w.pal = mat.t.pal;
    } else {
#pragma unroll
      for (int i = 0; i < NW_; ++i) {
        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)pick(wo[0][i], wo[1][i]), FORM == kFormBf16 ? 2 * k0 : FORM == kFormFp8 ? k0 : k0 / 2, 0);
        w.r.d[i] = make_uint4(v.x, v.y, v.z, v.w);
      }
      if constexpr (FORM == kFormFp8)
        w.sc[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)pick(so[0][0], so[1][0]), k0 / 32, 0);
      if constexpr (FORM == kFormMx4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w.sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)pick(so[0][i], so[1][i]), k0 / 32, 0);
      }
    }
#pragma unroll
    for (int l = 0; l < NX; ++l) {
      const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(rh, (int)(hrow + pick(xo[0][l], xo[1][l])), 2 * k0, 0);
      w.xv[l] = make_uint4(v.x, v.y, v.z, v.w);
    }
    next(wl);
  };

  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Win& w) __attribute__((always_inline)) {
    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FORM != kFormFp8) part = acc;
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
      uint4 b = w.xv[m / X];
      if constexpr (X > 1) {
        if (m % X == 1) b = from_right<C>(b);
        if constexpr (X > 2) {
          if (m % X == 2) b = from_right<2 * C>(b);
          if (m % X == 3) b = from_right<3 * C>(b);
        }
      }
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, b), part, 0, 0, 0);
    }
    if constexpr (FORM == kFormMx4) {   // a NaN scale makes its row NaN: one more MFMA, NaN times zero
      const bool nan = (w.sc[0] & 255u) == 255u || (w.sc[1] & 255u) == 255u;
      if (__ballot(nan)) {
        const uint32_t n = nan ? 0x7FC07FC0u : 0u;
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(n, n, n, n)),
                                                       __builtin_bit_cast(bf16x8_t, make_uint4(0u, 0u, 0u, 0u)), part, 0, 0, 0);
      }
    }
    if constexpr (FORM == kFormFp8) {
      const float scale = __builtin_bit_cast(float, w.sc[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], scale, acc[i]);
    } else {
      acc = part;
    }
    if (w.ends) {
      // D: lane l holds rows 4 (l / 16) .. +3 of column l % 16
      if (piece == 0 && 4 * g / kRows == place && w.to >= 0) {
        f32x4_t* to = reinterpret_cast<f32x4_t*>(&sums[wave][place][w.to][4 * g % kRows]);
        f32x4_t s = *to;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __builtin_fmaf(acc[i], w.weight, s[i]);
        *to = s;
      }
      acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };

  if (end > begin) {
    look(wl.at);
    // D sets of registers in turn: a set's load is D - 1 windows ahead of its sums, its
    // flags a window ahead of its load
    Win w[D];
    flags(fl[0]);
#pragma unroll
    for (int d = 0; d < D - 1; ++d) {
      flags(fl[d + 1]);
      load(fl[d], w[d]);
    }
    for (int i = begin; i < end; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        flags(fl[d]);
        load(fl[(d + D - 1) % D], w[(d + D - 1) % D]);
        // (loads before the wait for the oldest; UWF1, whose exponents come under a branch, does better
        // without: 39.7 -> 35.6 us)
        if constexpr (!form_is_pal(FORM)) __builtin_amdgcn_sched_barrier(0);
        compute(w[d]);
        if constexpr (!form_is_pal(FORM)) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * c.tokens; i += kNT) {
    const int t = i / kRows, f = i % kRows;
    if (f >= rows) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kNW; ++v)
#pragma unroll
      for (int p = 0; p < P; ++p) s += sums[v][p][t][f];
    c.out[(int64_t)t * N + n0 + f] = (uint16_t)bf16_pair(s, s);
  }
}

template <int FORM, int P, int C>
hipError_t launch_one(const LayerDown& c, hipStream_t s) {
  const int64_t grid = (c.d.n + 16 / P - 1) / (16 / P);   // (n is at most 2^20)
  hipLaunchKernelGGL((k_layer_down<FORM, P, C>), dim3((unsigned)grid), dim3(kNT), 0, s, c);
  return hipGetLastError();
}

// Places until every CU has a block; columns for the tokens that an expert has, about twice
// their average so that hardly any expert is two items.  (us with all 16 / P columns / so:
// 16 tokens, 6 of 160 MXFP4 experts 1408x2048 38.5 / 30.2, 8 tokens, 8 of 64 BF16 ones 53 / 43.5,
// one token, FP8 8.2 / 7.7, two tokens, 2 of 8 FP8 experts 14336x4096 52.7 / 33.7.)
template <int FORM>
hipError_t launch_form(const LayerDown& c, hipStream_t s) {
  const int64_t cus = device_cus();
  const int pairs = c.tokens * c.topk, most = c.tokens < (2 * pairs + c.d.count - 1) / c.d.count + 1
                                                  ? c.tokens
                                                  : (2 * pairs + c.d.count - 1) / c.d.count + 1;
  if (c.d.n / 16 >= cus || most > 8)
    return most > 4 ? launch_one<FORM, 1, 16>(c, s) : launch_one<FORM, 1, 4>(c, s);
  if (c.d.n / 8 >= cus || most > 4)
    return most > 4 ? launch_one<FORM, 2, 8>(c, s) : most > 2 ? launch_one<FORM, 2, 4>(c, s) : launch_one<FORM, 2, 2>(c, s);
  return launch_one<FORM, 4, 4>(c, s);
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
