// experts_tile.hip -- products grouped by expert for many rows an expert:
// LDS-tiled v_mfma_f32_32x32x16_bf16, weights BF16, UWF1 (palette indices) or
// MXFP4, plain (fp32 out) and gated (silu(x G^T) * (x U^T), BF16 out).
//
// A block computes BM slots of one expert times 256 weight rows (gated: 128
// gate rows and the same 128 up rows, 32 by 32 interleaved so that a wave
// holds both factors of its outputs).  Eight waves, two along the slots and
// four along the columns, each BM/2 x 64.  K advances 64 at a time:
//   * K goes through a ring of LDS buffers; step s runs its MFMAs from one,
//     fragments one 16-wide slice ahead of use.  x and BF16 weights go straight
//     from memory to LDS (16 bytes a lane, no registers); UWF1 and MXFP4 weights
//     through registers, rebuilt to BF16 once per block, loaded two steps ahead
//     and stored one ahead;
//   * the one barrier of a step stands before its last slice's MFMAs, so the
//     next step's first fragments travel while those run, and the buffer the
//     step leaves is refilled right behind it;
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
// 10 % of the time.
//
// A wave's row tiles alternate with the other's along the slots, and what lies
// behind the expert's last row is skipped by halves of a wave's rows, so a partly
// filled block costs both waves of a SIMD about what it holds.
//
// Where x and weights both go straight to LDS (BF16), as many steps as LDS holds
// are on their way at once: four buffers of 64-row tiles, three of 128-row ones,
// and for 256 rows three of weights, which come from HBM, and two of x, which
// mostly comes from L2, together all 160 KiB.  Gated, 64 experts 1408x2048 of 512
// rows each, us: 128-row tiles with two buffers 515, three 441; 256-row tiles
// with two 414, three of weights 402 (0.94 PFLOP/s; 8192^3 in one matrix 1.28,
// a library's BF16 product of that size 1.35 on the same card).  Without any
// loads in the loop (a timing copy) it took 347: the rest is LDS reads, barriers
// and the matrix unit at the clock it holds.
#include <type_traits>

#include "experts.h"

namespace uw {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;

constexpr int kBK = 64, kBN = 256, kNT = 512;

// A thread's share of the weight tile: what it loads for a step and how it
// becomes BF16 in LDS.  Rows: LDS row c of the tile is weight row row_of(c).
// K tails and rows past N read zero.
template <int FORM>
struct Weights;

// what a K tail or a row index outside x reads where x goes by pointers
__device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0, 0, 0, 0};

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
  __device__ __forceinline__ void direct(int k0, int K, lds_char* to, int i) const {   // piece i of four
    const uint32_t ko = k0 + (int)col < K ? 2u * (uint32_t)k0 : kOutside;
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
  __device__ __forceinline__ void first(int, int) {}
  // the step from k0 (the one after it begins at k1)
  __device__ __forceinline__ void load(int k0, int, int K, int set) {
    const bool in = k0 + (int)col < K;
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
  }
  __device__ __forceinline__ void flags(int k0, int K) {
    const uint32_t k = k0 < K ? (uint32_t)k0 : 0u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fw[i] = gload<uint32_t>(t.vflags + ((el[i] + k) >> 11));
      rw[i] = gload<uint32_t>(t.vrank + ((el[i] + k) >> 11));
    }
  }
  __device__ __forceinline__ void first(int k0, int K) { flags(k0, K); }
  __device__ __forceinline__ void load(int k0, int k1, int K, int set) {   // K % 64 == 0: a step is whole or absent
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
    flags(k1, K);
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
                                                      int ntiles, int spread) {
  constexpr int TM = BM / 64;                 // 32-row tiles of a wave; two column tiles
  constexpr int XP = BM / 64;                 // pieces of x a thread moves per step
  using W = Weights<FORM>;
  constexpr int OUT = GATED ? 128 : 256;      // output columns of a block
  // buffers of x and of weights
  constexpr int SX = !W::kDirect || BM == 256 ? 2 : BM == 128 ? 3 : 4;
  constexpr int SW = W::kDirect && BM == 256 && !BIG ? 3 : SX;
  // objects of their own rather than parts of one, so that the compiler sees that
  // what is read from or stored to one does not wait for what travels into
  // another
  constexpr int kX = BM * 128, kW = kBN * 128;
  __shared__ __attribute__((aligned(128))) char x0[kX], x1[kX], w0[kW], w1[kW];
  __shared__ __attribute__((aligned(16))) char x2[SX > 2 ? kX : 16], x3[SX > 3 ? kX : 16], w2[SW > 2 ? kW : 16],
      w3[SW > 3 ? kW : 16];   // (those of 16 bytes are never touched and take no space)
  char* const xbufs[4] = {x0, x1, x2, x3};
  char* const wbufs[4] = {w0, w1, w2, w3};

  // row tiles come in groups of G, a wave's groups alternating with the other's
  constexpr int G = TM == 4 ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int K = (int)vw.k;
  const int xcol = 8 * own_piece();
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(x, BIG ? 0 : (uint64_t)rr.x_rows * 2 * K);

  // The block's tile: its slots and columns, and where its x and weights lie.
  struct Tile {
    Share sh;
    int nt;
    uint32_t xo[XP];          // x, LDS rows tid / 8 + 64 i: byte offset of the row
    const uint16_t* xp[XP];   // BIG: its address, NULL for a row of zeros
    W w;
  } t;
  t.nt = find_tile(rr, vw.count, blockIdx.x & 7, blockIdx.x >> 3, ntiles, BM, t.sh);
  if (t.nt < 0) return;
  int32_t rows[XP];   // (fewer than 2^31 slots); all indices loaded before one is used
#pragma unroll
  for (int i = 0; i < XP; ++i) rows[i] = (int32_t)t.sh.first + (tid / 8 + 64 * i < t.sh.count ? tid / 8 + 64 * i : 0);
  if (rr.rows) {
#pragma unroll
    for (int i = 0; i < XP; ++i) rows[i] = rr.rows[rows[i]];
  }
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int64_t row = rows[i];
    const bool in = (row >= 0) & (row < rr.x_rows);
    t.xo[i] = in ? (uint32_t)(2 * (row * K + xcol)) : kOutside;
    t.xp[i] = in ? x + row * K + xcol : nullptr;
  }
  t.w.init(vw, vu, t.sh.expert, (int64_t)t.nt * OUT, [](int c, bool& up) __attribute__((always_inline)) {
    up = GATED && (c & 32);
    return GATED ? (c >> 6) * 32 + (c & 31) : c;
  });

  // what goes straight to LDS of the step from k0: x's piece i of XP, the weights' of WP
  constexpr int WP = W::kDirect ? 4 : 0;
  auto direct_x = [&](int k0, char* buf, int i) __attribute__((always_inline)) {
    lds_char* to = (lds_char*)(buf + wave * 1024 + 8192 * i);
    if constexpr (BIG) {
      const void* p = t.xp[i] && k0 + xcol < K ? (const void*)(t.xp[i] + k0) : (const void*)g_zero16;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, to, 16, 0, 0);
    } else {
      const uint32_t ko = k0 + xcol < K ? 2u * (uint32_t)k0 : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, to, 16, (int)(t.xo[i] + ko), 0, 0, 0);
    }
  };
  auto direct_w = [&](int k0, char* buf, int i) __attribute__((always_inline)) {
    if constexpr (W::kDirect) t.w.direct(k0, K, (lds_char*)(buf + wave * 1024), i);
  };

  f32x16_t acc[TM][2];
  bf16x8_t fa[2][TM], fb[2][2];
  const int frow = lane & 31, fpiece = lane >> 5;
  // first slot, within the tile, of the wave's row tile i
  auto slot_of = [&](int i) __attribute__((always_inline)) { return ((i / G) * 2 + wm) * (32 * G) + (i % G) * 32; };
  // Piece 2 slice + lane / 32 of row r lies at r * 128 + 16 ((lane / 32 ^ r / 2 % 8)
  // ^ 2 slice): one base for x and one for the weights, the slice flipping
  // two of its bits, a row tile a constant further.  (The empty asm makes a base
  // opaque, or the compiler keeps all sixteen addresses of two buffers in
  // registers, and spills.)
  const uint32_t base_a = piece_at(wm * (32 * G) + frow, fpiece), base_b = piece_at(wn * 64 + frow, fpiece);
  auto read = [&](const char* xbuf, const char* wbuf, int slice, int p, auto TA) __attribute__((always_inline)) {
    uint32_t a = base_a, b = base_b;
    asm volatile("" : "+v"(a), "+v"(b));
    a ^= 32u * slice;
    b ^= 32u * slice;
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
      fa[p][i] = *reinterpret_cast<const bf16x8_t*>(xbuf + a + (i / G) * (64 * G * 128) + (i % G) * 4096);
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[p][j] = *reinterpret_cast<const bf16x8_t*>(wbuf + b + 4096 * j);
  };
  auto mma_one = [&](int p, int t) __attribute__((always_inline)) {
    acc[t / 2][t % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[p][t / 2], fb[p][t % 2], acc[t / 2][t % 2], 0, 0, 0);
  };
  auto mma = [&](int p, auto TA) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2 * decltype(TA)::value; ++t) mma_one(p, t);
  };

  const int steps = (K + kBK - 1) / kBK;
  // spread: each block starts its walk along K elsewhere.  Rows are a power of two
  // apart as a rule, and blocks that all read the same columns at once meet on
  // the same memory channels: 32 BF16 experts 2048x2048 of 16 rows 67 -> 51 us
  // (5.3 TB/s).  With many rows an expert, blocks in step share more through L2
  // than that costs (8192^3: 856 -> 972 us), so the launcher decides.  Steps past
  // the last lie past K and fetch zeros.
  const int rot = spread ? (int)((blockIdx.x * 5u) % (unsigned)steps) : 0;
  auto step_k = [&](int s) __attribute__((always_inline)) {
    const int ss = s + rot;
    return kBK * (s >= steps ? steps : ss >= steps ? ss - steps : ss);
  };
  auto store = [&](char* wbuf, int part, int set) __attribute__((always_inline)) {
    if constexpr (!W::kDirect) t.w.store(wbuf, part, set);
  };
  auto load = [&](int s, int set) __attribute__((always_inline)) {
    if constexpr (!W::kDirect) t.w.load(step_k(s), step_k(s + 1), K, set);
  };
  // Step s: its data is in buffers J % SX and J % SW, that of s + 1 in register
  // set (J + 1) % 2 (what goes through registers) and on its way to the next
  // buffers.  TA: the wave's row tiles that hold slots (0: it moves data for the
  // others).
  auto step = [&](int s, auto J, auto TA) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    constexpr bool kActive = decltype(TA)::value > 0;
    char* const xcur = xbufs[j % SX];
    char* const wcur = wbufs[j % SW];
    char* const xnxt = xbufs[(j + 1) % SX];
    char* const wnxt = wbufs[(j + 1) % SW];
    if constexpr (kActive) {
      // (the scheduling barriers keep each slice's reads ahead of the MFMAs of
      // the slice before, which cover their latency)
      read(xcur, wcur, 1, 1, TA);
      __builtin_amdgcn_sched_barrier(0);
      store(wnxt, 0, (j + 1) % 2);
      mma(0, TA);
      __builtin_amdgcn_sched_barrier(0);
      read(xcur, wcur, 2, 0, TA);
      __builtin_amdgcn_sched_barrier(0);
      store(wnxt, 1, (j + 1) % 2);
      mma(1, TA);
      __builtin_amdgcn_sched_barrier(0);
      read(xcur, wcur, 3, 1, TA);
      __builtin_amdgcn_sched_barrier(0);
      mma(0, TA);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      store(wnxt, 0, (j + 1) % 2);
      store(wnxt, 1, (j + 1) % 2);
    }
    // This thread's part of step s + 1 has landed, and this wave has read all
    // of step s: after the barrier both hold for the block.  What may still
    // travel, all of it issued after s + 1's pieces: with SX = SW the S - 2
    // later steps, with one buffer more of weights the weights of s + 2.
    constexpr int kLater = !W::kDirect ? 0 : SX == SW ? (XP + WP) * (SX - 2) : WP;
    static_assert(kLater < 16 && (SX == SW || (SX == 2 && SW == 3)), "the counter's low field; what is issued when");
    __builtin_amdgcn_s_waitcnt(0x70 | kLater);   // vmcnt kLater, lgkmcnt 0
    bare_barrier();
    if constexpr (kActive) {
      read(xnxt, wnxt, 0, 0, TA);
      __builtin_amdgcn_sched_barrier(0);
    }
    // The pieces that refill this step's buffers, x first, one behind each MFMA:
    // all at once they fill the memory pipe, and what the wave issues next waits.
    constexpr int kMma = 2 * decltype(TA)::value, kPieces = XP + WP;
#pragma unroll
    for (int i = 0; i < (kMma > kPieces ? kMma : kPieces); ++i) {
      if (i < kMma) mma_one(1, i);
      if (i < XP) direct_x(step_k(s + SX), xcur, i);
      else if (i < kPieces) direct_w(step_k(s + SW), wcur, i - XP);
      __builtin_amdgcn_sched_barrier(0);
    }
    load(s + 3, (j + 1) % 2);
  };
  // D of the MFMA: lane l, register r: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
  // The tile's rows of y are one buffer resource, so rows behind the last slot
  // are dropped by its bound, as are columns past N, by an offset outside.
  auto write = [&](auto TA) __attribute__((always_inline)) {
    constexpr int kSize = GATED ? 2 : 4, kCols = GATED ? 1 : 2;
    const __amdgpu_buffer_rsrc_t ry =
        rsrc_of(static_cast<char*>(y) + t.sh.first * vw.n * kSize, (uint64_t)t.sh.count * (uint64_t)vw.n * kSize);
    int N = (int)vw.n;
    asm volatile("" : "+s"(N));   // or every row's offset is worked out before the loop and kept in registers
    uint32_t at[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int n = t.nt * OUT + (GATED ? wn * 32 : wn * 64 + 32 * j) + frow;
      at[j] = n < N ? (uint32_t)(4 * (lane >> 5) * N + n) * kSize : kOutside;
    }
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t row = (uint32_t)((slot_of(i) + 8 * (r >> 2) + (r & 3)) * N) * kSize;
        if constexpr (GATED) {
          const float h = silu(acc[i][0][r]) * acc[i][1][r];
          __builtin_amdgcn_raw_buffer_store_b16((short)bf16_pair(h, h), ry, (int)(at[0] + row), 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float v = acc[i][j][r];   // (a bit cast of the vector's element itself takes element 0)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned int, v), ry, (int)(at[j] + row), 0, 0);
          }
        }
      }
  };
  // a whole tile
  auto run = [&](auto TA) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
    if constexpr (decltype(TA)::value > 0) read(x0, w0, 0, 0, TA);
    // Whole rounds of the buffers, then what is left (breaks inside the loop
    // would cost a full wait at its head).  What the last steps fetch lies
    // past K: zeros.
    constexpr int kRound = SX == SW ? SX : SX * SW;
    auto steps_from = [&](int s, auto J, auto self) __attribute__((always_inline)) {
      step(s, J, TA);
      constexpr int j = decltype(J)::value + 1;
      if constexpr (j < kRound) self(s + 1, std::integral_constant<int, j>{}, self);
    };
    auto rest_from = [&](int s, auto J, auto self) __attribute__((always_inline)) {
      if (s >= steps) return;
      step(s, J, TA);
      constexpr int j = decltype(J)::value + 1;
      if constexpr (j + 1 < kRound) self(s + 1, std::integral_constant<int, j>{}, self);
    };
    int s = 0;
    for (; s + kRound <= steps; s += kRound) steps_from(s, std::integral_constant<int, 0>{}, steps_from);
    rest_from(s, std::integral_constant<int, 0>{}, rest_from);
    write(TA);   // (here, so that the loops' accumulators need not meet in the same registers)
  };

  // the buffers' first filling, in the order in which the steps go on
  auto fill = [&](int i) __attribute__((always_inline)) {
    if (SX != SW && i < SW)
#pragma unroll
      for (int p = 0; p < WP; ++p) direct_w(step_k(i), wbufs[i], p);
    if (i < SX)
#pragma unroll
      for (int p = 0; p < XP; ++p) direct_x(step_k(i), xbufs[i], p);
    if (SX == SW && i < SW)
#pragma unroll
      for (int p = 0; p < WP; ++p) direct_w(step_k(i), wbufs[i], p);
  };
  fill(0);
  if constexpr (!W::kDirect) t.w.first(step_k(0), K);
  load(0, 0);
  load(1, 1);
  store(w0, 0, 0);
  store(w0, 1, 0);
  fill(1);
  if constexpr (SW > 2) fill(2);
  if constexpr (SW > 3) fill(3);
  load(2, 0);
  asm volatile("" : : "s"(y));   // its scalar load ends here: pending, it would make the loop's first LDS wait a full one
  // step 0 has landed
  constexpr int kAhead = !W::kDirect ? 0 : WP * (SW - 1) + XP * (SX - 1);
  __builtin_amdgcn_s_waitcnt(0x70 | (kAhead < 16 ? kAhead : 15));
  bare_barrier();
  // (a wave takes one of the loops as a whole; all pass the same barriers)
  if (t.sh.count > (TM > 1 ? (2 + wm) * (32 * G) : wm * 32)) {
    run(std::integral_constant<int, TM>{});
  } else if (TM > 1 && t.sh.count > wm * (32 * G)) {
    run(std::integral_constant<int, TM == 1 ? 1 : TM / 2>{});
  } else {
    run(std::integral_constant<int, 0>{});
  }
  __builtin_amdgcn_s_waitcnt(0);   // nothing travels to LDS any more when the block gives it back
}

template <int FORM, int BM, bool GATED, bool BIG = false>
hipError_t launch_one(const ExpertsCall& c, bool spread, hipStream_t s) {
  const int64_t out = GATED ? 128 : 256, ntiles = (c.w.n + out - 1) / out;
  // a multiple of 8 blocks: every XCD's eighth of the list, rounded up, has its blocks
  const int64_t tiles = max_chunks(c.r.slots, c.w.count, BM, c.r.offsets != nullptr) * ntiles;
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (!grid_fits(grid, kNT)) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_experts_tile<FORM, BM, GATED, BIG>), dim3((unsigned)grid), dim3(kNT), 0, s, c.w, c.u, c.r, c.x,
                     c.y, (int)ntiles, (int)spread);
  return hipGetLastError();
}

template <int FORM, bool GATED>
hipError_t launch_rows(const ExpertsCall& c, int rows, bool spread, hipStream_t s) {
  if (c.r.x_rows * 2 * c.w.k > kOutside) return launch_one<FORM, 256, GATED, true>(c, spread, s);
  if (rows <= 64) return launch_one<FORM, 64, GATED>(c, spread, s);
  if (rows <= 128) return launch_one<FORM, 128, GATED>(c, spread, s);
  return launch_one<FORM, 256, GATED>(c, spread, s);
}

template <int FORM>
hipError_t launch_form(const ExpertsCall& c, int rows, bool spread, hipStream_t s) {
  return c.gated ? launch_rows<FORM, true>(c, rows, spread, s) : launch_rows<FORM, false>(c, rows, spread, s);
}

}  // namespace

hipError_t launch_experts_tile(const ExpertsCall& c, int rows, bool spread, hipStream_t s) {
  switch (c.w.form) {
    case kFormBf16: return launch_form<kFormBf16>(c, rows, spread, s);
    case kFormPal: return launch_form<kFormPal>(c, rows, spread, s);
    case kFormPalRun: return launch_form<kFormPalRun>(c, rows, spread, s);
    default: return launch_form<kFormMx4>(c, rows, spread, s);
  }
}

}  // namespace uw
