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
//     of use.  x and BF16 weights go straight from memory to LDS (16 bytes a
//     lane, no registers); UWF1 and MXFP4 weights through registers, rebuilt
//     to BF16 once per block, loaded two steps ahead and stored one ahead;
//   * the one barrier of a step stands before its last slice's MFMAs, so the
//     next step's first fragments travel while those run, and the buffer the
//     step leaves is refilled for the step after the next right behind it;
//   * LDS rows are 128 bytes without padding; 16-byte piece c of row r sits at
//     c ^ (r / 2 % 8).  LDS has 64 banks, two rows' worth, and serves 16 lanes of
//     a 16-byte read at a time: 16 rows of one fragment column then meet all
//     of them once.  (With c ^ r % 8 rows eight apart shared banks: four lost
//     cycles for each of the reads, a quarter of the kernel's cycles.)
// Gathered rows of x cost nothing extra: a thread keeps the offsets of its rows
// in a buffer resource over x, and what must read as zero (a K tail, a row
// index outside x) lies past the resource's end.  Beyond 2 GiB of x the rows go
// by 64-bit pointers instead (BIG, 256-row tiles only): those loads are of the
// flat kind, whose counters the compiler must drain before any LDS read, about
// 10 % of the time.  Waves whose slots all lie behind the expert's last row skip their
// MFMAs.
#include <type_traits>

#include "experts.h"

namespace uw {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;

constexpr int kBK = 64, kBN = 256, kNT = 512;
constexpr uint32_t kOutside = 0x7FFF0000u;   // past the end of every buffer resource here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t byte) {
  const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)byte, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint32_t piece_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ ((row >> 1) & 7)) << 4)); }

// A thread's share of the weight tile: what it loads for a step and how it
// becomes BF16 in LDS.  Rows: LDS row c of the tile is weight row row_of(c).
// K tails and rows past N read zero.
template <int FORM>
struct Weights;

// what a K tail or a row index outside x reads where x goes by pointers
__device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) char lds_char;

// the piece of its LDS row that lands at this thread's place (see piece_at)
__device__ __forceinline__ int own_piece() { return (threadIdx.x ^ (threadIdx.x >> 4)) & 7; }

// BF16: four pieces of eight weights, LDS rows tid / 8 + 64 i, straight to LDS
template <>
struct Weights<kFormBf16> {
  static constexpr bool kDirect = true;
  __amdgpu_buffer_rsrc_t r;
  uint32_t off[4], col;
  template <typename RowOf>
  __device__ __forceinline__ void init(const ExpertsView& w, const ExpertsView& u, int e, int64_t n0, RowOf&& row_of) {
    const int tid = threadIdx.x;
    col = 8u * own_piece();
    bool up = false;   // the same for a wave's rows and for each i
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = (uint32_t)row_of(tid / 8 + 64 * i, up) * (uint32_t)(2 * w.k) + 2u * col;
    const ExpertsView& m = __builtin_amdgcn_readfirstlane((int)up) ? u : w;
    const int64_t rows = m.n - n0 < kBN ? m.n - n0 : kBN;
    r = rsrc_of(m.w + (int64_t)e * m.w_stride + n0 * 2 * m.k, (uint64_t)rows * 2 * m.k);
  }
  __device__ __forceinline__ void direct(int64_t k0, int64_t K, lds_char* to) const {
    const uint32_t ko = k0 + col < K ? (uint32_t)(2 * k0) : kOutside;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to + 8192 * i, 16, (int)(off[i] + ko), 0, 0, 0);
  }
};

// MXFP4: one block of 32 weights, LDS row tid / 2
template <>
struct Weights<kFormMx4> {
  __amdgpu_buffer_rsrc_t r, rs;
  static constexpr bool kDirect = false;
  uint32_t off, soff, col;
  uint4 d[2];
  uint32_t sc[2];
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
  __device__ __forceinline__ void load(int64_t k0, int64_t K, int set) {
    const bool in = k0 + col < K;
    d[set] = bload16(r, off + (in ? (uint32_t)(k0 / 2) : kOutside));
    sc[set] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(soff + (in ? (uint32_t)(k0 / 32) : kOutside)), 0, 0);
  }
  __device__ __forceinline__ void store(char* lds, int part, int set) const {
    const int tid = threadIdx.x;
    const uint32_t byte = sc[set] & 255u;
    const float s = e8m0_float(byte);
    const bool nan = byte == 255u;
    const uint32_t q[4] = {d[set].x, d[set].y, d[set].z, d[set].w};
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
  static constexpr bool kDirect = false;
  ExpertEntry t;
  uint32_t el[2];    // element of the piece at k = 0 (a matrix has fewer than 2^32)
  uint4 s[2][2];
  uint2 a[2][2], b[2][2];
  uint32_t fw[2], rw[2], verb[2];
  template <typename RowOf>
  __device__ __forceinline__ void init(const ExpertsView& w, const ExpertsView& u, int e, int64_t n0, RowOf&& row_of) {
    const int tid = threadIdx.x;
    bool up = false;                 // 16 rows a wave, 128 apart: all gate or all up
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int64_t n = n0 + row_of(tid / 4 + 128 * i, up);
      n = n < w.n ? n : w.n - 1;     // rows past N are not stored
      el[i] = (uint32_t)(n * w.k) + 16u * (tid & 3);
    }
    t = (__builtin_amdgcn_readfirstlane((int)up) ? u : w).table[e];
    flags(0, w.k);
  }
  __device__ __forceinline__ void flags(int64_t k0, int64_t K) {
    const uint32_t k = k0 < K ? (uint32_t)k0 : 0u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fw[i] = gload<uint32_t>(t.vflags + ((el[i] + k) >> 11));
      rw[i] = gload<uint32_t>(t.vrank + ((el[i] + k) >> 11));
    }
  }
  __device__ __forceinline__ void load(int64_t k0, int64_t K, int set) {   // K % 64 == 0: a step is whole or absent
    const uint32_t k = k0 < K ? (uint32_t)k0 : 0u;
    verb[set] = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = el[i] + k, g = x >> 6;
      s[set][i] = gload16(t.sm + x);
      const bool v = group_verbatim(fw[i], g);
      const uint8_t* p = v ? t.vexp + (uint64_t)group_rank(fw[i], rw[i], g) * 64 + (x & 63) : t.pidx + x / 2;
      a[set][i] = gload8(p);
      b[set][i] = gload8(p + (v ? 8 : 0));
      verb[set] |= (v ? 1u : 0u) << i;
    }
    flags(k0 + kBK, K);
  }
  __device__ __forceinline__ void store(char* lds, int part, int set) const {
    const int tid = threadIdx.x, i = part;
    uint4 e = pal16<RUN>(a[set][i].x, a[set][i].y, t.pal);
    if ((verb[set] >> i) & 1u) e = make_uint4(a[set][i].x, a[set][i].y, b[set][i].x, b[set][i].y);
    uint32_t o[8];
    rebuild16(s[set][i], e, o);
    const int row = tid / 4 + 128 * i, c = 2 * (tid & 3);
    *reinterpret_cast<uint4*>(lds + piece_at(row, c)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(lds + piece_at(row, c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
};
template <> struct Weights<kFormPal> : WeightsPal<false> {};
template <> struct Weights<kFormPalRun> : WeightsPal<true> {};

template <int FORM, int BM, bool GATED, bool BIG>
__global__ __launch_bounds__(kNT) void k_experts_tile(ExpertsView vw, ExpertsView vu, RaggedRows rr,
                                                      const uint16_t* __restrict__ x, void* __restrict__ y,
                                                      int ntiles) {
  constexpr int TM = BM / 64;                 // 32-row tiles of a wave; two column tiles
  constexpr int XP = BM / 64;                 // pieces of x a thread moves per step
  using W = Weights<FORM>;
  constexpr int OUT = GATED ? 128 : 256;      // output columns of a block
  // objects of their own rather than parts of one, so that the compiler sees that
  // what is read from or stored to one does not wait for what travels into
  // another
  __shared__ __attribute__((aligned(128))) char xa[BM * 128], xb[BM * 128];
  __shared__ __attribute__((aligned(128))) char wa[kBN * 128], wb[kBN * 128];

  Share sh;
  const int nt = find_tile(rr, vw.count, blockIdx.x, ntiles, BM, sh);
  if (nt < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t N = vw.n, K = vw.k;
  const int64_t n0 = (int64_t)nt * OUT;

  // x: LDS rows tid / 8 + 64 i
  const int xcol = 8 * own_piece();
  uint32_t xo[XP];          // byte offset of the row
  const uint16_t* xp[XP];   // BIG: its address, NULL for a row of zeros
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int b = tid / 8 + 64 * i;
    int64_t row = sh.first + (b < sh.count ? b : 0);
    if (rr.rows) row = rr.rows[row];
    const bool in = row >= 0 && row < rr.x_rows;
    xo[i] = in ? (uint32_t)(2 * (row * K + xcol)) : kOutside;
    xp[i] = in ? x + row * K + xcol : nullptr;
  }
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, BIG ? 0 : (uint64_t)rr.x_rows * 2 * K);
  auto direct_x = [&](int64_t k0, lds_char* to) __attribute__((always_inline)) {
    if constexpr (BIG) {
#pragma unroll
      for (int i = 0; i < XP; ++i) {
        const void* p = xp[i] && k0 + xcol < K ? (const void*)(xp[i] + k0) : (const void*)g_zero16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, to + 8192 * i, 16, 0, 0);
      }
    } else {
      const uint32_t ko = k0 + xcol < K ? (uint32_t)(2 * k0) : kOutside;
#pragma unroll
      for (int i = 0; i < XP; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, to + 8192 * i, 16, (int)(xo[i] + ko), 0, 0, 0);
    }
  };
  // the step from k0, as far as it goes straight to LDS
  W w;
  auto direct = [&](int64_t k0, char* xbuf, char* wbuf) __attribute__((always_inline)) {
    direct_x(k0, (lds_char*)(xbuf + wave * 1024));
    if constexpr (W::kDirect) w.direct(k0, K, (lds_char*)(wbuf + wave * 1024));
  };
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
  // Piece 2 slice + lane / 32 of row r lies at r * 128 + 16 ((lane / 32 ^ r / 2 % 8)
  // ^ 2 slice): one base for x and one for the weights, the slice flipping
  // two of its bits, a row tile 4096 bytes further.  (The empty asm makes a base
  // opaque, or the compiler keeps all sixteen addresses of two buffers in
  // registers, and spills.)
  const uint32_t base_a = piece_at(wm * (BM / 2) + frow, fpiece), base_b = piece_at(wn * 64 + frow, fpiece);
  auto read = [&](const char* xbuf, const char* wbuf, int slice, int p) __attribute__((always_inline)) {
    uint32_t a = base_a, b = base_b;
    asm volatile("" : "+v"(a), "+v"(b));
    a ^= 32u * slice;
    b ^= 32u * slice;
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[p][i] = *reinterpret_cast<const bf16x8_t*>(xbuf + a + 4096 * i);
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[p][j] = *reinterpret_cast<const bf16x8_t*>(wbuf + b + 4096 * j);
  };
  auto mma = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[p][i], fb[p][j], acc[i][j], 0, 0, 0);
  };

  const int steps = (int)((K + kBK - 1) / kBK);
  auto store = [&](char* wbuf, int part, int set) __attribute__((always_inline)) {
    if constexpr (!W::kDirect) w.store(wbuf, part, set);
  };
  auto load = [&](int64_t k0, int set) __attribute__((always_inline)) {
    if constexpr (!W::kDirect) w.load(k0, K, set);
  };
  direct(0, xa, wa);
  load(0, 0);
  load(kBK, 1);
  store(wa, 0, 0);
  store(wa, 1, 0);
  direct(kBK, xb, wb);
  load(2 * kBK, 0);
  asm volatile("" : : "s"(y));   // its scalar load ends here: pending, it would make the loop's first LDS wait a full one
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  const bool active = wm * (BM / 2) < sh.count;
  if (active) read(xa, wa, 0, 0);
  // two steps an iteration, so that buffers and register sets are constants;
  // step s of parity q finds its data in xcur and wcur, that of s + 1 in set
  // 1 - q and on its way to xnxt and wnxt
  auto step = [&](int s, char* xcur, char* wcur, char* xnxt, char* wnxt, auto Q, auto Active) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    constexpr bool kActive = decltype(Active)::value;
    if constexpr (kActive) {
      // (the scheduling barriers keep each slice's reads ahead of the MFMAs of
      // the slice before, which cover their latency)
      read(xcur, wcur, 1, 1);
      __builtin_amdgcn_sched_barrier(0);
      store(wnxt, 0, 1 - q);
      mma(0);
      __builtin_amdgcn_sched_barrier(0);
      read(xcur, wcur, 2, 0);
      __builtin_amdgcn_sched_barrier(0);
      store(wnxt, 1, 1 - q);
      mma(1);
      __builtin_amdgcn_sched_barrier(0);
      read(xcur, wcur, 3, 1);
      __builtin_amdgcn_sched_barrier(0);
      mma(0);
      __builtin_amdgcn_sched_barrier(0);
    } else {   // moves data for the other waves
      store(wnxt, 0, 1 - q);
      store(wnxt, 1, 1 - q);
    }
    // this thread's part of step s + 1 has landed, and this wave has read all
    // of step s: after the barrier both hold for the block
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    direct((int64_t)kBK * (s + 2), xcur, wcur);
    load((int64_t)kBK * (s + 3), 1 - q);
    if constexpr (kActive) {
      read(xnxt, wnxt, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      mma(1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto run = [&](auto Active) __attribute__((always_inline)) {
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      step(s, xa, wa, xb, wb, std::integral_constant<int, 0>{}, Active);
      step(s + 1, xb, wb, xa, wa, std::integral_constant<int, 1>{}, Active);
    }
    if (s < steps) step(s, xa, wa, xb, wb, std::integral_constant<int, 0>{}, Active);
  };
  // (a wave takes one of the two loops as a whole; both pass the same barriers)
  if (!active) {
    run(std::false_type{});
    return;
  }
  run(std::true_type{});

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

// x up to here goes through a buffer resource (an offset past it plus a K tail's
// kOutside stays below 2^32)
constexpr int64_t kBigBytes = kOutside;

template <int FORM, int BM, bool GATED, bool BIG = false>
hipError_t launch_one(const ExpertsCall& c, hipStream_t s) {
  const int64_t out = GATED ? 128 : 256, ntiles = (c.w.n + out - 1) / out;
  // a multiple of 8 blocks: every XCD's eighth of the list, rounded up, has its blocks
  const int64_t tiles = max_chunks(c.r.slots, c.w.count, BM, c.r.offsets != nullptr) * ntiles;
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid > INT32_MAX) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_experts_tile<FORM, BM, GATED, BIG>), dim3((unsigned)grid), dim3(kNT), 0, s, c.w, c.u, c.r, c.x, c.y, (int)ntiles);
  return hipGetLastError();
}

template <int FORM, bool GATED>
hipError_t launch_rows(const ExpertsCall& c, int rows, hipStream_t s) {
  if (c.r.x_rows * 2 * c.w.k > kBigBytes) return launch_one<FORM, 256, GATED, true>(c, s);
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
