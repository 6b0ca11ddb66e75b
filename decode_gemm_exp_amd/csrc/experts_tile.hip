// experts_tile.hip -- products grouped by expert for many rows an expert:
// LDS-tiled v_mfma_f32_32x32x16_bf16, weights BF16, UWF1 (palette indices) or
// MXFP4, plain (fp32 out) and gated (silu(x G^T) * (x U^T), BF16 out).
//
// A block computes BM slots of one expert times 256 weight rows (gated: 128
// gate rows and the same 128 up rows, 32 by 32 interleaved so that a wave
// holds both factors of its outputs).  Eight waves, two along the slots and
// four along the columns, each BM/2 x 64.  K advances 64 at a time through two
// LDS buffers:
//   * step s runs its MFMAs from one buffer, fragments one 16-wide slice ahead
//     of use, while every thread moves step s+1 from registers into the other
//     buffer (weights rebuilt to BF16 on the way, once per block) and asks for
//     the data of step s+2;
//   * the one barrier of a step stands before its last slice's MFMAs, so the
//     next step's first fragments travel while those run;
//   * LDS rows are 128 bytes without padding; 16-byte piece c of row r sits at
//     c ^ (r & 7), so eight rows of one fragment column meet eight different
//     piece columns and neither reads nor writes collide.
// Gathered rows of x cost nothing extra: a thread keeps the pointers of its
// rows.  Waves whose slots all lie behind the expert's last row skip their
// MFMAs.
#include "experts.h"

namespace uw {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4_t;

constexpr int kBK = 64, kBN = 256, kNT = 512;
constexpr uint32_t kOutside = 0x7FFF0000u;   // past the end of every buffer resource here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t byte) {
  const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)byte, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint32_t piece_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }

// A thread's share of the weight tile: what it loads for a step and how it
// becomes BF16 in LDS.  Rows: LDS row c of the tile is weight row row_of(c).
// K tails and rows past N read zero.
template <int FORM>
struct Weights;

// BF16: four pieces of eight weights, LDS rows tid / 8 + 64 i
template <>
struct Weights<kFormBf16> {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[4], col;
  uint4 d[4];
  template <typename RowOf>
  __device__ __forceinline__ void init(const ExpertsView& w, const ExpertsView& u, int e, int64_t n0, RowOf&& row_of) {
    const int tid = threadIdx.x;
    col = 8u * (tid & 7);
    int first_up = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bool up;
      const int n = row_of(tid / 8 + 64 * i, up);
      off[i] = (uint32_t)n * (uint32_t)(2 * w.k) + 2u * col;
      first_up = up;   // the same for a wave's rows and for each i
    }
    const ExpertsView& m = __builtin_amdgcn_readfirstlane(first_up) ? u : w;
    const int64_t rows = m.n - n0 < kBN ? m.n - n0 : kBN;
    r = rsrc_of(m.w + (int64_t)e * m.w_stride + n0 * 2 * m.k, (uint64_t)rows * 2 * m.k);
  }
  __device__ __forceinline__ void load(int64_t k0, int64_t K) {
    const uint32_t ko = k0 + col < K ? (uint32_t)(2 * k0) : kOutside;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = bload16(r, off[i] + ko);
  }
  __device__ __forceinline__ void store(char* lds, int part) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 2 * part; i < 2 * part + 2; ++i)
      *reinterpret_cast<uint4*>(lds + piece_at(tid / 8 + 64 * i, tid & 7)) = d[i];
  }
};

// MXFP4: one block of 32 weights, LDS row tid / 2
template <>
struct Weights<kFormMx4> {
  __amdgpu_buffer_rsrc_t r, rs;
  uint32_t off, soff, col;
  uint4 d;
  uint32_t sc;
  template <typename RowOf>
  __device__ __forceinline__ void init(const ExpertsView& w, const ExpertsView& u, int e, int64_t n0, RowOf&& row_of) {
    const int tid = threadIdx.x;
    col = 32u * (tid & 1);
    bool up;
    const int n = row_of(tid / 2, up);
    off = (uint32_t)n * (uint32_t)(w.k / 2) + col / 2;
    soff = (uint32_t)n * (uint32_t)mx4_scale_stride(w.k) + col / 32;
    const ExpertsView& m = __builtin_amdgcn_readfirstlane((int)up) ? u : w;   // 32 rows a wave: all gate or all up
    const int64_t rows = m.n - n0 < kBN ? m.n - n0 : kBN;
    r = rsrc_of(m.w + (int64_t)e * m.w_stride + n0 * (m.k / 2), (uint64_t)rows * (m.k / 2));
    rs = rsrc_of(m.scale + (int64_t)e * m.scale_stride + n0 * mx4_scale_stride(m.k), (uint64_t)rows * mx4_scale_stride(m.k));
  }
  __device__ __forceinline__ void load(int64_t k0, int64_t K) {
    const bool in = k0 + col < K;
    d = bload16(r, off + (in ? (uint32_t)(k0 / 2) : kOutside));
    sc = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(soff + (in ? (uint32_t)(k0 / 32) : kOutside)), 0, 0);
  }
  __device__ __forceinline__ void store(char* lds, int part) const {
    const int tid = threadIdx.x;
    const float s = e8m0_float(sc & 255u);
    const bool nan = (sc & 255u) == 255u;
    const uint32_t q[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 2 * part; i < 2 * part + 2; ++i) {
      uint4 v = mx4_unpack8(q[i], s);
      if (nan) v = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      *reinterpret_cast<uint4*>(lds + piece_at(tid / 2, (int)(col / 8) + i)) = v;
    }
  }
};

// UWF1: two pieces of 16 weights, LDS rows tid / 4 + 128 i; a row's 64 k of a
// step are one group, whose flag and rank words are loaded a step ahead of
// its data
template <bool RUN>
struct WeightsPal {
  const ExpertEntry* t;
  int64_t el[2];     // element of the piece at k = 0
  uint4 s[2];
  uint2 a[2], b[2];
  uint32_t fw[2], rw[2], verb;
  template <typename RowOf>
  __device__ __forceinline__ void init(const ExpertsView& w, const ExpertsView& u, int e, int64_t n0, RowOf&& row_of) {
    const int tid = threadIdx.x;
    int first_up = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bool up;
      int64_t n = n0 + row_of(tid / 4 + 128 * i, up);
      n = n < w.n ? n : w.n - 1;   // rows past N are not stored
      el[i] = n * w.k + 16 * (tid & 3);
      first_up = up;               // 16 rows a wave, 128 apart: all gate or all up
    }
    t = (__builtin_amdgcn_readfirstlane(first_up) ? u : w).table + e;
    verb = 0;
    flags(0, w.k);
  }
  __device__ __forceinline__ void flags(int64_t k0, int64_t K) {
    const int64_t k = k0 < K ? k0 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fw[i] = t->vflags[(uint64_t)(el[i] + k) >> 11];
      rw[i] = t->vrank[(uint64_t)(el[i] + k) >> 11];
    }
  }
  __device__ __forceinline__ void load(int64_t k0, int64_t K) {   // K % 64 == 0: a step is whole or absent
    const int64_t k = k0 < K ? k0 : 0;
    verb = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t x = (uint64_t)(el[i] + k), g = x >> 6;
      s[i] = *reinterpret_cast<const uint4*>(t->sm + x);
      const bool v = group_verbatim(fw[i], g);
      const uint8_t* p = v ? t->vexp + (uint64_t)group_rank(fw[i], rw[i], g) * 64 + (x & 63) : t->pidx + x / 2;
      a[i] = *reinterpret_cast<const uint2*>(p);
      b[i] = *reinterpret_cast<const uint2*>(p + (v ? 8 : 0));
      verb |= (v ? 1u : 0u) << i;
    }
    flags(k0 + kBK, K);
  }
  __device__ __forceinline__ void store(char* lds, int part) const {
    const int tid = threadIdx.x, i = part;
    uint4 e = pal16<RUN>(a[i].x, a[i].y, t->pal);
    if ((verb >> i) & 1u) e = make_uint4(a[i].x, a[i].y, b[i].x, b[i].y);
    uint32_t o[8];
    rebuild16(s[i], e, o);
    const int row = tid / 4 + 128 * i, c = 2 * (tid & 3);
    *reinterpret_cast<uint4*>(lds + piece_at(row, c)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(lds + piece_at(row, c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
};
template <> struct Weights<kFormPal> : WeightsPal<false> {};
template <> struct Weights<kFormPalRun> : WeightsPal<true> {};

template <int FORM, int BM, bool GATED>
__global__ __launch_bounds__(kNT) void k_experts_tile(ExpertsView vw, ExpertsView vu, RaggedRows rr,
                                                      const uint16_t* __restrict__ x, void* __restrict__ y,
                                                      int ntiles) {
  constexpr int TM = BM / 64;                 // 32-row tiles of a wave; two column tiles
  constexpr int XP = BM / 64;                 // pieces of x a thread moves per step
  constexpr int OUT = GATED ? 128 : 256;      // output columns of a block
  constexpr int kStage = (BM + kBN) * 128;
  extern __shared__ __attribute__((aligned(128))) char lds[];

  Share sh;
  const int nt = find_tile(rr, vw.count, blockIdx.x, ntiles, BM, sh);
  if (nt < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t N = vw.n, K = vw.k;
  const int64_t n0 = (int64_t)nt * OUT;

  // x: LDS rows tid / 8 + 64 i, piece tid % 8
  const uint16_t* xp[XP];
  uint32_t xok = 0;
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int b = tid / 8 + 64 * i;
    int64_t row = sh.first + (b < sh.count ? b : 0);
    if (rr.rows) row = rr.rows[row];
    const bool ok = row >= 0 && row < rr.x_rows;   // outside: a row of zeros
    xok |= (ok ? 1u : 0u) << i;
    xp[i] = x + (ok ? row : 0) * K;
  }
  const int xcol = 8 * (tid & 7);
  uint4 xd[XP];
  bool xin = false;
  auto load_x = [&](int64_t k0) __attribute__((always_inline)) {
    xin = k0 + xcol < K;
#pragma unroll
    for (int i = 0; i < XP; ++i) xd[i] = *reinterpret_cast<const uint4*>(xp[i] + (xin ? k0 + xcol : 0));
  };
  auto store_x = [&](char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const bool ok = xin && ((xok >> i) & 1u);
      uint4 v = xd[i];
      v.x = ok ? v.x : 0u;
      v.y = ok ? v.y : 0u;
      v.z = ok ? v.z : 0u;
      v.w = ok ? v.w : 0u;
      *reinterpret_cast<uint4*>(buf + piece_at(tid / 8 + 64 * i, tid & 7)) = v;
    }
  };

  Weights<FORM> w;
  w.init(vw, vu, sh.expert, n0, [](int c, bool& up) __attribute__((always_inline)) {
    up = GATED && (c & 32);
    return GATED ? (c >> 6) * 32 + (c & 31) : c;
  });

  f32x16_t acc[TM][2];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
  bf16x8_t fa[2][TM], fb[2][2];
  const int frow = lane & 31, fpiece = lane >> 5;
  auto read = [&](const char* buf, int slice, int p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      fa[p][i] = *reinterpret_cast<const bf16x8_t*>(buf + piece_at(wm * (BM / 2) + 32 * i + frow, 2 * slice + fpiece));
#pragma unroll
    for (int j = 0; j < 2; ++j)
      fb[p][j] = *reinterpret_cast<const bf16x8_t*>(buf + BM * 128 + piece_at(wn * 64 + 32 * j + frow, 2 * slice + fpiece));
  };
  auto mma = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[p][i], fb[p][j], acc[i][j], 0, 0, 0);
  };

  const int steps = (int)((K + kBK - 1) / kBK);
  load_x(0);
  w.load(0, K);
  store_x(lds);
  w.store(lds + BM * 128, 0);
  w.store(lds + BM * 128, 1);
  load_x(kBK);
  w.load(kBK, K);
  __syncthreads();
  if (wm * (BM / 2) < sh.count) {
    read(lds, 0, 0);
    for (int s = 0; s < steps; ++s) {
      char* cur = lds + (s & 1) * kStage;
      char* nxt = lds + ((s + 1) & 1) * kStage;
      read(cur, 1, 1);
      store_x(nxt);
      mma(0);
      read(cur, 2, 0);
      w.store(nxt + BM * 128, 0);
      mma(1);
      read(cur, 3, 1);
      w.store(nxt + BM * 128, 1);
      load_x((int64_t)kBK * (s + 2));
      w.load((int64_t)kBK * (s + 2), K);
      mma(0);
      __syncthreads();
      read(nxt, 0, 0);
      mma(1);
    }
  } else {
    for (int s = 0; s < steps; ++s) {   // moves data for the other waves
      char* nxt = lds + ((s + 1) & 1) * kStage;
      store_x(nxt);
      w.store(nxt + BM * 128, 0);
      w.store(nxt + BM * 128, 1);
      load_x((int64_t)kBK * (s + 2));
      w.load((int64_t)kBK * (s + 2), K);
      __syncthreads();
    }
    return;
  }

  // D of the MFMA: lane l, register r: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int b = wm * (BM / 2) + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (b >= sh.count) continue;
      if constexpr (GATED) {
        const int64_t n = n0 + wn * 32 + frow;
        const float h = silu(acc[i][0][r]) * acc[i][1][r];
        if (n < N) static_cast<uint16_t*>(y)[(sh.first + b) * N + n] = (uint16_t)bf16_pair(h, h);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = n0 + wn * 64 + 32 * j + frow;
          if (n < N) static_cast<float*>(y)[(sh.first + b) * N + n] = acc[i][j][r];
        }
      }
    }
}

template <int FORM, int BM, bool GATED>
hipError_t launch_one(const ExpertsCall& c, hipStream_t s) {
  constexpr int bytes = 2 * (BM + kBN) * 128;
  const auto k = k_experts_tile<FORM, BM, GATED>;
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(k), bytes);
  if (e != hipSuccess) return e;
  const int64_t out = GATED ? 128 : 256, ntiles = (c.w.n + out - 1) / out;
  // a multiple of 8 blocks: every XCD's eighth of the list, rounded up, has its blocks
  const int64_t tiles = max_chunks(c.r.slots, c.w.count, BM, c.r.offsets != nullptr) * ntiles;
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid > INT32_MAX) return hipErrorNotSupported;
  hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(kNT), bytes, s, c.w, c.u, c.r, c.x, c.y, (int)ntiles);
  return hipGetLastError();
}

template <int FORM, bool GATED>
hipError_t launch_rows(const ExpertsCall& c, int rows, hipStream_t s) {
  if (rows <= 64) return launch_one<FORM, 64, GATED>(c, s);
  if (rows <= 128) return launch_one<FORM, 128, GATED>(c, s);
  return launch_one<FORM, 256, GATED>(c, s);
}

template <int FORM>
hipError_t launch_form(const ExpertsCall& c, int rows, hipStream_t s) {
  return c.gated ? launch_rows<FORM, true>(c, rows, s) : launch_rows<FORM, false>(c, rows, s);
}

}  // namespace

hipError_t launch_experts_tile(const ExpertsCall& c, int rows, hipStream_t s) {
  switch (c.w.form) {
    case kFormBf16: return launch_form<kFormBf16>(c, rows, s);
    case kFormPal: return launch_form<kFormPal>(c, rows, s);
    case kFormPalRun: return launch_form<kFormPalRun>(c, rows, s);
    default: return launch_form<kFormMx4>(c, rows, s);
  }
}

}  // namespace uw
