// mx4_gemm.hip -- y = x . W^T with both operands in MXFP4, on the matrix unit's
// block-scaled form v_mfma_scale_f32_32x32x64_f8f6f4.
//
// A lane's share of an operand is one whole block (32 elements, 16 bytes) and
// its scale byte, so elements go from HBM to the matrix unit without being
// unpacked, and the product of two blocks is scaled inside the instruction
// (exact: both scales are powers of two).
//
// The loop is that of experts_tile.hip (a block BM x 256, eight waves of BM/2
// x 64, two LDS buffers, one barrier a step): its 128-byte LDS rows hold 256 k
// here, four slices of 64.  A row's eight scale bytes of a step are stored
// beside it, those of even blocks before those of odd ones: lanes 0..31 take
// the even blocks and lanes 32..63 the odd ones, so a lane's four are one dword
// and the instruction picks the slice's byte.
#include <type_traits>

#include "experts.h"

namespace uw {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

constexpr int kStep = 256, kBN = 256, kNT = 512;
constexpr uint32_t kOutside = 0x7FFF0000u;   // past the end of every buffer resource here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint32_t piece_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ ((row >> 1) & 7)) << 4)); }

template <int BM>
__global__ __launch_bounds__(kNT) void k_mx4_tile(const uint8_t* __restrict__ we, const uint8_t* __restrict__ ws,
                                                  int64_t N, int K, const uint8_t* __restrict__ xe,
                                                  const uint8_t* __restrict__ xs, int64_t B, float* __restrict__ y,
                                                  int ntiles) {
  constexpr int TM = BM / 64;
  constexpr int XP = BM / 64, P = XP + 4;     // pieces a thread moves per step: x, then weights
  constexpr int kRows = BM + kBN;
  // objects of their own rather than parts of one, so that the compiler sees that
  // what is read from or stored to one does not wait for what travels into
  // another
  __shared__ __attribute__((aligned(128))) char lds_a[kRows * 128], lds_b[kRows * 128];
  __shared__ __attribute__((aligned(128))) char scales_a[kRows * 8], scales_b[kRows * 8];

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
  // thread t < kRows carries the scales of LDS row t
  const bool is_x = tid < BM;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_readfirstlane((int)is_x) ? rsrc_of(xs + m0 * stride, (uint64_t)sh.count * stride)
                                                : rsrc_of(ws + n0 * stride, (uint64_t)rows_w * stride);
  const uint32_t soff = (uint32_t)(is_x ? tid : tid - BM) * (uint32_t)stride;
  // elements travel straight to LDS: thread t's pieces are those at t's place,
  // which the swizzle gives to piece t % 8 ^ (row / 2) % 8 of row t / 8 + 64 i
  const int piece = (tid ^ (tid >> 4)) & 7;
  const uint32_t off = (uint32_t)(tid / 8) * (uint32_t)row_bytes + 16u * piece;
  const uint32_t rows64 = 64u * (uint32_t)row_bytes;

  auto load = [&](int k0, char* buf) __attribute__((always_inline)) {
    const uint32_t ko = k0 + 32 * piece < K ? (uint32_t)(k0 / 2) : kOutside;   // past K: zero
    __attribute__((address_space(3))) char* to =
        (__attribute__((address_space(3))) char*)(buf + wave * 1024);
#pragma unroll
    for (int i = 0; i < P; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i < XP ? rx : rw, to + 8192 * i, 16,
                                               (int)(off + ko + (uint32_t)(i < XP ? i : i - XP) * rows64), 0, 0, 0);
  };
  // a row's scales are loaded one step ahead of their store
  uint32_t s0 = 0, s1 = 0;
  auto load_scales = [&](int k0) __attribute__((always_inline)) {
    if (kRows == kNT || tid < kRows) {
      const u32x2_t v =
          __builtin_amdgcn_raw_buffer_load_b64(rs, (int)(soff + (k0 < K ? (uint32_t)(k0 / 32) : kOutside)), 0, 0);
      s0 = v.x;
      s1 = v.y;
    }
  };
  auto store_scales = [&](int k0, char* buf) __attribute__((always_inline)) {
    if (kRows == kNT || tid < kRows) {
      // bytes of blocks past K are another row's scales, maybe NaN: zero them
      auto keep = [](int blocks) __attribute__((always_inline)) {
        return (uint32_t)((1ull << (8 * min(max(blocks, 0), 4))) - 1ull);
      };
      const int left = (K - k0) >> 5;
      const uint32_t a = s0 & keep(left), b = s1 & keep(left - 4);
      *reinterpret_cast<uint2*>(buf + tid * 8) =
          make_uint2(__builtin_amdgcn_perm(b, a, 0x06040200u), __builtin_amdgcn_perm(b, a, 0x07050301u));
    }
  };

  f32x16_t acc[TM][2];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
  uint4 fa[2][TM], fb[2][2];
  int sa[2][TM], sb[2][2];   // scales of a step, current and next
  const int frow = lane & 31, half = lane >> 5;
  // one base a fragment column, the slice flipping two of its bits (the empty asm
  // keeps the compiler from holding every slice's address in a register)
  const uint32_t base_a = piece_at(wm * (BM / 2) + frow, half), base_b = piece_at(BM + wn * 64 + frow, half);
  const uint32_t scale_a = half * 4 + (wm * (BM / 2) + frow) * 8,
                 scale_b = half * 4 + (BM + wn * 64 + frow) * 8;
  auto read = [&](const char* buf, int slice, int p) __attribute__((always_inline)) {
    uint32_t a = base_a, b = base_b;
    asm volatile("" : "+v"(a), "+v"(b));
    a ^= 32u * slice;
    b ^= 32u * slice;
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[p][i] = *reinterpret_cast<const uint4*>(buf + a + 4096 * i);
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[p][j] = *reinterpret_cast<const uint4*>(buf + b + 4096 * j);
  };
  auto read_scales = [&](const char* buf, int p) __attribute__((always_inline)) {
    uint32_t a = scale_a, b = scale_b;
    asm volatile("" : "+v"(a), "+v"(b));
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[p][i] = *reinterpret_cast<const int*>(buf + a + 256 * i);
#pragma unroll
    for (int j = 0; j < 2; ++j) sb[p][j] = *reinterpret_cast<const int*>(buf + b + 256 * j);
  };
  auto op = [](const uint4& v) __attribute__((always_inline)) {
    return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  };
  // slice SL of the step whose scales are in sa[q], sb[q]; fragments p
#define UW_MX4_MMA(SL, p, q)                                                                                         \
  _Pragma("unroll") for (int i = 0; i < TM; ++i) _Pragma("unroll") for (int j = 0; j < 2; ++j)                       \
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(op(fa[p][i]), op(fb[p][j]), acc[i][j], 4, 4, SL,   \
                                                                  sa[q][i], SL, sb[q][j])

  const int steps = (K + kStep - 1) / kStep;
  load(0, lds_a);
  load_scales(0);
  load(kStep, lds_b);
  store_scales(0, scales_a);
  load_scales(kStep);
  asm volatile("" : : "s"(y));   // its scalar load ends here: pending, it would make the loop's first LDS wait a full one
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  const bool active = wm * (BM / 2) < sh.count;
  if (active) {
    read(lds_a, 0, 0);
    read_scales(scales_a, 0);
  }
  // two steps an iteration, so that buffers and scale registers are constants
  auto step = [&](int s, char* cur, char* nxt, char* nxt_scales, auto Q, auto Active) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    constexpr bool kActive = decltype(Active)::value;
    store_scales(kStep * (s + 1), nxt_scales);
    load_scales(kStep * (s + 2));
    if constexpr (kActive) {
      // (the scheduling barriers keep each slice's reads ahead of the MFMAs of
      // the slice before, which cover their latency)
      read(cur, 1, 1);
      __builtin_amdgcn_sched_barrier(0);
      UW_MX4_MMA(0, 0, q);
      __builtin_amdgcn_sched_barrier(0);
      read(cur, 2, 0);
      __builtin_amdgcn_sched_barrier(0);
      UW_MX4_MMA(1, 1, q);
      __builtin_amdgcn_sched_barrier(0);
      read(cur, 3, 1);
      __builtin_amdgcn_sched_barrier(0);
      UW_MX4_MMA(2, 0, q);
      __builtin_amdgcn_sched_barrier(0);
    }
    // step s + 1 has landed (this thread's part of it), and this wave has read
    // all of step s: after the barrier both hold for the block
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    load(kStep * (s + 2), cur);
    if constexpr (kActive) {
      read(nxt, 0, 0);
      read_scales(nxt_scales, 1 - q);
      __builtin_amdgcn_sched_barrier(0);
      UW_MX4_MMA(3, 1, q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto run = [&](auto Active) __attribute__((always_inline)) {
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      step(s, lds_a, lds_b, scales_b, std::integral_constant<int, 0>{}, Active);
      step(s + 1, lds_b, lds_a, scales_a, std::integral_constant<int, 1>{}, Active);
    }
    if (s < steps) step(s, lds_a, lds_b, scales_b, std::integral_constant<int, 0>{}, Active);
  };
  // (a wave takes one of the two loops as a whole; both pass the same barriers)
  if (!active) {
    run(std::false_type{});
    __builtin_amdgcn_s_waitcnt(0);   // nothing travels to LDS any more when the block gives it back
    return;
  }
  run(std::true_type{});
  __builtin_amdgcn_s_waitcnt(0);
#undef UW_MX4_MMA

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int b = wm * (BM / 2) + 32 * i + 8 * (r >> 2) + 4 * half + (r & 3);
      if (b >= sh.count) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wn * 64 + 32 * j + frow;
        if (n < N) y[(m0 + b) * N + n] = acc[i][j][r];
      }
    }
}

template <int BM>
hipError_t launch_bm(const uint8_t* we, const uint8_t* ws, int64_t n, int64_t k, const uint8_t* xe, const uint8_t* xs,
                     int64_t batch, float* y, hipStream_t s) {
  const int64_t ntiles = (n + kBN - 1) / kBN, tiles = (batch + BM - 1) / BM * ntiles, grid = (tiles + 7) / 8 * 8;
  if (grid > INT32_MAX) return hipErrorNotSupported;
  hipLaunchKernelGGL(k_mx4_tile<BM>, dim3((unsigned)grid), dim3(kNT), 0, s, we, ws, n, (int)k, xe, xs, batch, y,
                     (int)ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_tile(const uint8_t* we, const uint8_t* ws, int64_t n, int64_t k, const uint8_t* xe,
                           const uint8_t* xs, int64_t batch, float* y, hipStream_t s) {
  // the tallest tile that still gives every CU a block
  const int64_t cus = device_cus(), ntiles = (n + kBN - 1) / kBN;
  if (batch > 128 && (batch + 255) / 256 * ntiles >= cus) return launch_bm<256>(we, ws, n, k, xe, xs, batch, y, s);
  if (batch > 64 && (batch + 127) / 128 * ntiles >= cus) return launch_bm<128>(we, ws, n, k, xe, xs, batch, y, s);
  return launch_bm<64>(we, ws, n, k, xe, xs, batch, y, s);
}

}  // namespace uw
