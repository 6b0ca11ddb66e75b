// mx4_gemm.hip -- y = x . W^T with both operands in MXFP4, on the matrix unit's
// block-scaled form v_mfma_scale_f32_32x32x64_f8f6f4.
//
// A lane's share of an operand is one whole block (32 elements, 16 bytes) and
// its scale byte, so elements go from HBM to the matrix unit without being
// unpacked, and the product of two blocks is scaled inside the instruction
// (exact: both scales are powers of two).
//
// The loop is that of experts_tile.hip (a block BM x 256, eight waves of BM/2
// x 64, LDS buffers filled directly, one barrier a step, row tiles of the two wave
// rows alternating): its 128-byte LDS rows hold 256 k here, four slices of 64.  A
// row's eight scale bytes of a step are stored beside it, those of even blocks
// before those of odd ones: lanes 0..31 take the even blocks and lanes 32..63 the
// odd ones, so a lane's four are one dword and the instruction picks the
// slice's byte.
//
// 28672x8192 at 1024 rows: see the launcher.
#include <type_traits>

#include "experts.h"

namespace uw {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

constexpr int kStep = 256, kBN = 256, kNT = 512;

template <int BM>
__global__ __launch_bounds__(kNT) void k_mx4_tile(const uint8_t* __restrict__ we, const uint8_t* __restrict__ ws,
                                                  int64_t N, int K, const uint8_t* __restrict__ xe,
                                                  const uint8_t* __restrict__ xs, int64_t B, float* __restrict__ y,
                                                  int ntiles) {
  constexpr int TM = BM / 64;
  constexpr int G = TM == 4 ? 2 : 1;          // row tiles come in groups of G, a wave's alternating with the other's
  constexpr int XP = BM / 64, P = XP + 4;     // pieces a thread moves per step: x, then weights
  constexpr int kRows = BM + kBN;
  constexpr int S = BM == 256 ? 2 : 3;        // buffers: as many as fit
  // objects of their own rather than parts of one, so that the compiler sees that
  // what is read from or stored to one does not wait for what travels into
  // another
  __shared__ __attribute__((aligned(128))) char r0[kRows * 128], r1[kRows * 128], r2[S > 2 ? kRows * 128 : 16];
  __shared__ __attribute__((aligned(128))) char c0[kNT * 8], c1[kNT * 8], c2[S > 2 ? kNT * 8 : 16];
  char* const rows[3] = {r0, r1, r2};
  char* const scales[3] = {c0, c1, c2};

  Share sh;
  const int nt = find_tile(RaggedRows{nullptr, nullptr, B, B}, 1, blockIdx.x & 7, blockIdx.x >> 3, ntiles, BM, sh);
  if (nt < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t n0 = (int64_t)nt * kBN, m0 = sh.first;
  const int64_t rows_w = N - n0 < kBN ? N - n0 : kBN;
  const int row_bytes = K / 2, stride = (int)mx4_scale_stride(K);
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(xe + m0 * row_bytes, (uint64_t)sh.count * row_bytes);
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(we + n0 * row_bytes, (uint64_t)rows_w * row_bytes);
  // thread t carries the scales of LDS row t (those beyond the rows carry zeros
  // to a place of their own, without a branch)
  const bool is_x = tid < BM;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_readfirstlane((int)is_x) ? rsrc_of(xs + m0 * stride, (uint64_t)sh.count * stride)
                                                : rsrc_of(ws + n0 * stride, (uint64_t)rows_w * stride);
  const uint32_t soff = tid < kRows ? (uint32_t)(is_x ? tid : tid - BM) * (uint32_t)stride : kOutside;
  // elements travel straight to LDS: thread t's pieces are those at t's place,
  // which the swizzle gives to piece t % 8 ^ (row / 2) % 8 of row t / 8 + 64 i
  const int piece = (tid ^ (tid >> 4)) & 7;
  const uint32_t off = (uint32_t)(tid / 8) * (uint32_t)row_bytes + 16u * piece;
  const uint32_t rows64 = 64u * (uint32_t)row_bytes;

  auto direct = [&](int k0, char* buf, int i) __attribute__((always_inline)) {   // piece i of P
    const uint32_t ko = k0 + 32 * piece < K ? (uint32_t)(k0 / 2) : kOutside;     // past K: zero
    __builtin_amdgcn_raw_ptr_buffer_load_lds(i < XP ? rx : rw, (lds_char*)(buf + wave * 1024) + 8192 * i, 16,
                                             (int)(off + ko + (uint32_t)(i < XP ? i : i - XP) * rows64), 0, 0, 0);
  };
  // a row's scales are loaded two steps ahead of their store, in two register sets
  uint32_t s0[2] = {}, s1[2] = {};
  auto load_scales = [&](int k0, int set) __attribute__((always_inline)) {
    const u32x2_t v =
        __builtin_amdgcn_raw_buffer_load_b64(rs, (int)(soff + (k0 < K ? (uint32_t)(k0 / 32) : kOutside)), 0, 0);
    s0[set] = v.x;
    s1[set] = v.y;
  };
  auto store_scales = [&](int k0, char* buf, int set) __attribute__((always_inline)) {
    // bytes of blocks past K are another row's scales, maybe NaN: zero them
    auto keep = [](int blocks) __attribute__((always_inline)) {
      return (uint32_t)((1ull << (8 * min(max(blocks, 0), 4))) - 1ull);
    };
    const int left = (K - k0) >> 5;
    const uint32_t a = s0[set] & keep(left), b = s1[set] & keep(left - 4);
    *reinterpret_cast<uint2*>(buf + tid * 8) =
        make_uint2(__builtin_amdgcn_perm(b, a, 0x06040200u), __builtin_amdgcn_perm(b, a, 0x07050301u));
  };

  f32x16_t acc[TM][2];
  uint4 fa[2][TM], fb[2][2];
  int sa[2][TM], sb[2][2];   // scales of a step, current and next
  const int frow = lane & 31, half = lane >> 5;
  auto slot_of = [&](int i) __attribute__((always_inline)) { return ((i / G) * 2 + wm) * (32 * G) + (i % G) * 32; };
  // one base a fragment column, the slice flipping two of its bits (the empty asm
  // keeps the compiler from holding every slice's address in a register)
  const uint32_t base_a = piece_at(wm * (32 * G) + frow, half), base_b = piece_at(BM + wn * 64 + frow, half);
  const uint32_t scale_a = half * 4 + (wm * (32 * G) + frow) * 8, scale_b = half * 4 + (BM + wn * 64 + frow) * 8;
  auto read = [&](const char* buf, int slice, int p, auto TA) __attribute__((always_inline)) {
    uint32_t a = base_a, b = base_b;
    asm volatile("" : "+v"(a), "+v"(b));
    a ^= 32u * slice;
    b ^= 32u * slice;
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
      fa[p][i] = *reinterpret_cast<const uint4*>(buf + a + (i / G) * (64 * G * 128) + (i % G) * 4096);
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[p][j] = *reinterpret_cast<const uint4*>(buf + b + 4096 * j);
  };
  auto read_scales = [&](const char* buf, int p, auto TA) __attribute__((always_inline)) {
    uint32_t a = scale_a, b = scale_b;
    asm volatile("" : "+v"(a), "+v"(b));
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
      sa[p][i] = *reinterpret_cast<const int*>(buf + a + (i / G) * (64 * G * 8) + (i % G) * 256);
#pragma unroll
    for (int j = 0; j < 2; ++j) sb[p][j] = *reinterpret_cast<const int*>(buf + b + 256 * j);
  };
  auto op = [](const uint4& v) __attribute__((always_inline)) {
    return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  };
  // MFMA t of slice SL of the step whose scales are in sa[q], sb[q]; fragments p
  auto mma_one = [&](auto SL, int p, int q, int t) __attribute__((always_inline)) {
    constexpr int sl = decltype(SL)::value;
    acc[t / 2][t % 2] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        op(fa[p][t / 2]), op(fb[p][t % 2]), acc[t / 2][t % 2], 4, 4, sl, sa[q][t / 2], sl, sb[q][t % 2]);
  };
  auto mma = [&](auto SL, int p, int q, auto TA) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2 * decltype(TA)::value; ++t) mma_one(SL, p, q, t);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;

  const int steps = (K + kStep - 1) / kStep;
  // Step s finds its data in buffers J % S, its scales in sa[J % 2] and sb[J % 2];
  // TA: the wave's row tiles that hold rows (0: it moves data for the others)
  auto step = [&](int s, auto J, auto TA) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value, q = j % 2;
    constexpr bool kActive = decltype(TA)::value > 0;
    char* const cur = rows[j % S];
    char* const nxt = rows[(j + 1) % S];
    char* const nxt_scales = scales[(j + 1) % S];
    store_scales(kStep * (s + 1), nxt_scales, 1 - q);
    load_scales(kStep * (s + 3), 1 - q);
    if constexpr (kActive) {
      // (the scheduling barriers keep each slice's reads ahead of the MFMAs of
      // the slice before, which cover their latency)
      read(cur, 1, 1, TA);
      __builtin_amdgcn_sched_barrier(0);
      mma(I0{}, 0, q, TA);
      __builtin_amdgcn_sched_barrier(0);
      read(cur, 2, 0, TA);
      __builtin_amdgcn_sched_barrier(0);
      mma(I1{}, 1, q, TA);
      __builtin_amdgcn_sched_barrier(0);
      read(cur, 3, 1, TA);
      __builtin_amdgcn_sched_barrier(0);
      mma(I2{}, 0, q, TA);
      __builtin_amdgcn_sched_barrier(0);
    }
    // This thread's part of step s + 1 has landed, and this wave has read all
    // of step s: after the barrier both hold for the block.  What may still
    // travel, all issued after s + 1's pieces: those of the S - 2 later steps
    // (the scale loads among them only make the wait stricter).
    __builtin_amdgcn_s_waitcnt(0x70 | (P * (S - 2)));   // vmcnt, lgkmcnt 0
    bare_barrier();
    if constexpr (kActive) {
      read(nxt, 0, 0, TA);
      read_scales(nxt_scales, 1 - q, TA);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the pieces that refill this step's buffer, one behind each MFMA
    constexpr int kMma = 2 * decltype(TA)::value;
#pragma unroll
    for (int i = 0; i < (kMma > P ? kMma : P); ++i) {
      if (i < kMma) mma_one(I3{}, 1, q, i);
      if (i < P) direct(kStep * (s + S), cur, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // D of the MFMA: lane l, register r: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
  // The tile's rows of y are one buffer resource: rows behind the last are dropped
  // by its bound, as are columns past N, by an offset outside.
  auto write = [&](auto TA) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t ry = rsrc_of(y + m0 * N, (uint64_t)sh.count * (uint64_t)N * 4);
    uint32_t at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = n0 + wn * 64 + 32 * j + frow;
      at[j] = n < N ? (uint32_t)(4 * half * (int)N + (int)n) * 4u : kOutside;
    }
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t row = (uint32_t)((slot_of(i) + 8 * (r >> 2) + (r & 3)) * (int)N) * 4u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float v = acc[i][j][r];   // (a bit cast of the vector's element itself takes element 0)
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned int, v), ry, (int)(at[j] + row), 0, 0);
        }
      }
  };
  auto run = [&](auto TA) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < decltype(TA)::value; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
    if constexpr (decltype(TA)::value > 0) {
      read(r0, 0, 0, TA);
      read_scales(c0, 0, TA);
    }
    // whole rounds of buffers and register sets, then what is left; what the
    // last steps fetch lies past K: zeros
    constexpr int kRound = S == 2 ? 2 : 6;
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
    for (; s + kRound <= steps; s += kRound) steps_from(s, I0{}, steps_from);
    rest_from(s, I0{}, rest_from);
    write(TA);
  };

  load_scales(0, 0);
#pragma unroll
  for (int b = 0; b < S; ++b)
#pragma unroll
    for (int i = 0; i < P; ++i) direct(kStep * b, rows[b], i);
  store_scales(0, c0, 0);
  load_scales(kStep, 1);
  load_scales(2 * kStep, 0);
  asm volatile("" : : "s"(y));   // its scalar load ends here: pending, it would make the loop's first LDS wait a full one
  __builtin_amdgcn_s_waitcnt(0x70 | (P * (S - 1) < 16 ? P * (S - 1) : 15));   // step 0 has landed
  bare_barrier();
  // (a wave takes one of the loops as a whole; all pass the same barriers)
  if (sh.count > (TM > 1 ? (2 + wm) * (32 * G) : wm * 32)) {
    run(std::integral_constant<int, TM>{});
  } else if (TM > 1 && sh.count > wm * (32 * G)) {
    run(std::integral_constant<int, TM == 1 ? 1 : TM / 2>{});
  } else {
    run(std::integral_constant<int, 0>{});
  }
  __builtin_amdgcn_s_waitcnt(0);   // nothing travels to LDS any more when the block gives it back
}

template <int BM>
hipError_t launch_bm(const uint8_t* we, const uint8_t* ws, int64_t n, int64_t k, const uint8_t* xe, const uint8_t* xs,
                     int64_t batch, float* y, hipStream_t s) {
  const int64_t ntiles = (n + kBN - 1) / kBN, tiles = (batch + BM - 1) / BM * ntiles, grid = (tiles + 7) / 8 * 8;
  if (!grid_fits(grid, kNT)) return hipErrorNotSupported;
  hipLaunchKernelGGL(k_mx4_tile<BM>, dim3((unsigned)grid), dim3(kNT), 0, s, we, ws, n, (int)k, xe, xs, batch, y,
                     (int)ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_tile(const uint8_t* we, const uint8_t* ws, int64_t n, int64_t k, const uint8_t* xe,
                           const uint8_t* xs, int64_t batch, float* y, hipStream_t s) {
  // The tallest tile that still gives three quarters of the CUs a block.  Measured (us,
  // 64 / 128 / 256 rows, quantisation of x included): 28672x8192 at 1024 rows 252 / 191 / 150
  // (3.2 PFLOP/s), 14336x4096 at 1000 rows (224 tall tiles) 77 / 56 / 47, 5001x2048 at 512
  // rows 16.4 / 18.1 / 22.3, 4096x4096 at 256 rows 22.1 / 24.1 / 32.7.
  const int64_t blocks = (int64_t)device_cus() * 3 / 4, ntiles = (n + kBN - 1) / kBN;
  if (batch > 128 && (batch + 255) / 256 * ntiles >= blocks) return launch_bm<256>(we, ws, n, k, xe, xs, batch, y, s);
  if (batch > 64 && (batch + 127) / 128 * ntiles >= blocks) return launch_bm<128>(we, ws, n, k, xe, xs, batch, y, s);
  return launch_bm<64>(we, ws, n, k, xe, xs, batch, y, s);
}

}  // namespace uw
