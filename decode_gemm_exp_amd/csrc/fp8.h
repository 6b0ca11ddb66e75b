// fp8.h -- E4M3 with an FP32 scale per block of 128, shared by the conversion and
// the products: a block's scale, packing and unpacking.
//
// A block's largest magnitude m, at least 2^-110, gives scale = m / 448 and inv =
// 448 / m, both divided exactly and rounded once to FP32 (448 is the largest E4M3
// value, and the floor keeps both normal numbers).  Elements are v inv, rounded
// to FP32, then to E4M3 to nearest even: at most 448 (1 + 2^-23), which rounds to
// 448.  A block with an infinity or a NaN has scale NaN and elements 0.
#pragma once

#include "experts.h"

namespace uw {

constexpr int kFp8Block = 128;
__host__ __device__ constexpr int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Fp8Scale {
  float scale, inv;   // inv 0: elements are zeros
};

// top: the FP32 bits of the largest magnitude
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
  const bool finite = top < 0x7F800000u;
  const float m = fmaxf(__builtin_bit_cast(float, top), 0x1p-110f);
  const float s = __fdiv_rn(m, 448.0f), i = __fdiv_rn(448.0f, m);
  return {finite ? s : __builtin_nanf(""), finite ? i : 0.0f};
}

// four values times inv -> four E4M3 bytes
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, q, true);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// eight BF16 -> eight bytes.  A block that is not finite: inv is 0 and the
// product could be NaN, so its elements are set apart
__device__ __forceinline__ uint2 fp8_pack8(const uint4& v, float inv) {
  const uint2 q = make_uint2(fp8_pack4(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv, bf16_lo(v.y) * inv, bf16_hi(v.y) * inv),
                             fp8_pack4(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv, bf16_lo(v.w) * inv, bf16_hi(v.w) * inv));
  return inv != 0.0f ? q : make_uint2(0u, 0u);
}

// the largest magnitude among eight BF16, as FP32 bits' upper half in either
// half of the result
__device__ __forceinline__ uint32_t bf16_top8(const uint4& v) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  auto mag = [](uint32_t w) __attribute__((always_inline)) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
  const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(v.x), mag(v.y)),
                                            __builtin_elementwise_max(mag(v.z), mag(v.w)));
  return __builtin_bit_cast(uint32_t, m);
}
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// both halves of bf16_top8's result -> FP32 bits
__device__ __forceinline__ uint32_t top_bits(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }

// eight E4M3 bytes -> eight BF16, exact
__device__ __forceinline__ uint4 fp8_unpack8(uint32_t a, uint32_t b) {
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
  return o;
}

hipError_t launch_quantize_fp8(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, int block_rows,
                               uint8_t* elem, float* scale, hipStream_t s);
hipError_t launch_dequantize_fp8(const uint8_t* elem, const float* scale, int64_t rows, int64_t cols, int block_rows,
                                 uint16_t* out, int64_t ld, hipStream_t s);
// rows of x -> their elements per 1 x 128 as BF16 numbers, unscaled, and scales
hipError_t launch_round_fp8(const uint16_t* x, int64_t rows, int64_t cols, uint16_t* out, float* scale, hipStream_t s);

// Products with E4M3 weights.  How the tiles run one:
struct Fp8Tile {
  int rows;           // of a tile: 64 or 128
  bool spread;
  int tail, splits;   // one matrix, plain: the last `tail` tiles' K goes in slices, summed by a second kernel
  float* part;        // tail * splits tiles of rows * 256
  const float* act;   // x's scales when c.x holds E4M3 values as BF16
};
hipError_t launch_fp8_tile(const ExpertsCall& c, const Fp8Tile& t, hipStream_t s);
hipError_t launch_fp8_rows(const ExpertsCall& c, bool act8, hipStream_t s);
// experts' rows
hipError_t launch_fp8_experts(const ExpertsCall& c, hipStream_t s);

// One matrix: which kernel serves it, and the workspace that takes.
struct Fp8Plan {
  bool few;           // launch_fp8_rows
  Fp8Tile tile;       // (pointers not set)
  uint64_t x_bytes, scale_bytes, part_bytes;   // of the workspace, in this order
  // What a caller provides: never less for more rows, 0 with `few`.  Slices go up and down
  // with the rows, so their share is a bound that all plans of as many rows or fewer keep.
  uint64_t bytes;
  bool uses_workspace() const { return x_bytes + scale_bytes + part_bytes != 0; }
};
Fp8Plan plan_fp8(int64_t n, int64_t k, int64_t batch, bool act8);
hipError_t launch_fp8_product(const ExpertsCall& c, const Fp8Plan& p, bool act8, void* ws, hipStream_t s);

}  // namespace uw
