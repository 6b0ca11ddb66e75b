// mx4.hip -- MXFP4 conversion (OCP Microscaling Formats: E2M1 elements, one
// E8M0 scale per 32 along a row) from and to BF16 / FP32.
//
// A block's scale is 2^(floor(log2 max|v|) - 2), 2 being the exponent of the
// largest E2M1 value, kept within 2^-127 .. 2^127: read off the exponent field
// of the largest magnitude (a block of zeros, and one whose maximum is
// subnormal, take 2^-127).  Elements are v / scale rounded to nearest, ties to
// the even code, at most 6 in magnitude.  A block holding an infinity or a NaN
// has scale byte 255 (NaN) and elements 0.
//
// Bound: HBM, 2 (or 4) + 0.53 bytes an element.  Four lanes share a block,
// eight elements each, so every load and store of a wave is contiguous, and
// the block's maximum takes two lane permutes.  The scaled conversion
// instructions round as the definition does.  14336x4096: quantise 23 us, dequantise
// 22 us (149 MB each, 6.5 TB/s, part of it cached; by shifts and compares 47 us).
#include "experts.h"

namespace uw {
namespace {

constexpr int kUnroll = 4;   // pieces of eight elements a thread has in flight

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);   // lanes 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);            // lanes 2 3 0 1
  return v > o ? v : o;
}

// scale byte of a block whose largest magnitude has FP32 bits `top` (BF16
// bits in the upper half serve as well: the exponent field is the same)
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// Eight values as loaded: BF16 pairs, or floats.
template <bool F32>
struct Eight {
  uint32_t w[F32 ? 8 : 4];
};

template <bool F32>
__device__ __forceinline__ Eight<F32> load8(const void* src, int64_t at) {
  Eight<F32> e;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(src) + at * (F32 ? 4 : 2));
  const uint4 a = p[0];
  e.w[0] = a.x; e.w[1] = a.y; e.w[2] = a.z; e.w[3] = a.w;
  if constexpr (F32) {
    const uint4 b = p[1];
    e.w[4] = b.x; e.w[5] = b.y; e.w[6] = b.z; e.w[7] = b.w;
  }
  return e;
}

// the largest magnitude's bits, as of a float
template <bool F32>
__device__ __forceinline__ uint32_t top8(const Eight<F32>& e) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < (F32 ? 8 : 4); ++i) {
    if constexpr (F32) {
      m = max(m, e.w[i] & 0x7FFFFFFFu);
    } else {
      m = max(m, max((e.w[i] & 0x7FFFu) << 16, e.w[i] & 0x7FFF0000u));
    }
  }
  return m;
}

// Codes of eight values over the block's scale.  The scaled conversion divides by
// the power of two in its scale operand's exponent field, rounds to nearest even
// and saturates; seven comparisons an element instead took 1.6 times the whole
// kernel's time.
template <bool F32>
__device__ __forceinline__ uint32_t pack8(const Eight<F32>& e, uint32_t byte) {
  const float s = e8m0_float(byte);
  uint32_t q = 0;
  if constexpr (F32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, e.w[i]);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
  } else {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, e.w[0]), s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, e.w[1]), s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, e.w[2]), s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, e.w[3]), s, 3);
  }
  return byte == 255u ? 0u : q;
}

// pieces: rows * cols / 8, of which cols / 8 a row
template <bool F32>
__global__ __launch_bounds__(256) void k_quantize_mx4(const void* __restrict__ src, int64_t pieces, uint32_t per_row,
                                                      int64_t ld, uint8_t* __restrict__ elem,
                                                      uint8_t* __restrict__ scale, int64_t stride) {
  const int64_t base = (int64_t)blockIdx.x * (256 * kUnroll) + threadIdx.x;
  Eight<F32> e[kUnroll];
  int64_t row[kUnroll];
  uint32_t col[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t p = base + 256 * u < pieces ? base + 256 * u : pieces - 1;
    row[u] = p / per_row;
    col[u] = (uint32_t)(p - row[u] * per_row);
    e[u] = load8<F32>(src, row[u] * ld + 8 * (int64_t)col[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    // pieces is a multiple of four, so a block's four lanes are in or out together
    const uint32_t byte = scale_byte(quad_max(top8(e[u])));
    const int64_t p = base + 256 * u;
    if (p >= pieces) continue;
    reinterpret_cast<uint32_t*>(elem)[p] = pack8(e[u], byte);
    const uint32_t b = col[u] >> 2;
    if ((col[u] & 3) == 0) {
      scale[row[u] * stride + b] = (uint8_t)byte;
      // the row's last block also clears the bytes that pad its scales
      if (4 * (b + 1) == per_row)
        for (int64_t i = b + 1; i < stride; ++i) scale[row[u] * stride + i] = 0;
    }
  }
}

__device__ __forceinline__ uint4 unpack8(uint32_t q, uint32_t byte) {
  return byte == 255u ? make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u)
                      : mx4_unpack8(q, e8m0_float(byte));
}

__global__ __launch_bounds__(256) void k_dequantize_mx4(const uint8_t* __restrict__ elem,
                                                        const uint8_t* __restrict__ scale, int64_t pieces,
                                                        uint32_t per_row, int64_t stride, uint16_t* __restrict__ out,
                                                        int64_t ld) {
  const int64_t base = (int64_t)blockIdx.x * (256 * kUnroll) + threadIdx.x;
  uint32_t q[kUnroll], byte[kUnroll];
  int64_t at[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t p = base + 256 * u < pieces ? base + 256 * u : pieces - 1;
    const int64_t row = p / per_row;
    const uint32_t col = (uint32_t)(p - row * per_row);
    q[u] = reinterpret_cast<const uint32_t*>(elem)[p];
    byte[u] = scale[row * stride + (col >> 2)];
    at[u] = row * ld + 8 * (int64_t)col;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (base + 256 * u < pieces) *reinterpret_cast<uint4*>(out + at[u]) = unpack8(q[u], byte[u]);
}

__global__ __launch_bounds__(256) void k_round_mx4(const uint16_t* __restrict__ x, int64_t pieces,
                                                   uint16_t* __restrict__ out) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const Eight<false> e = load8<false>(x, 8 * (p < pieces ? p : pieces - 1));
  const uint32_t byte = scale_byte(quad_max(top8(e)));
  if (p < pieces) reinterpret_cast<uint4*>(out)[p] = unpack8(pack8(e, byte), byte);
}

int64_t blocks_for(int64_t pieces) { return (pieces + 256 * kUnroll - 1) / (256 * kUnroll); }

}  // namespace

hipError_t launch_quantize_mx4(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* elem,
                               uint8_t* scale, hipStream_t s) {
  const int64_t pieces = rows * (cols / 8);
  if (!grid_fits(blocks_for(pieces), 256)) return hipErrorNotSupported;
  const dim3 grid((unsigned)blocks_for(pieces));
  if (f32)
    hipLaunchKernelGGL(k_quantize_mx4<true>, grid, dim3(256), 0, s, src, pieces, (uint32_t)(cols / 8), ld, elem, scale,
                       mx4_scale_stride(cols));
  else
    hipLaunchKernelGGL(k_quantize_mx4<false>, grid, dim3(256), 0, s, src, pieces, (uint32_t)(cols / 8), ld, elem, scale,
                       mx4_scale_stride(cols));
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t* elem, const uint8_t* scale, int64_t rows, int64_t cols, uint16_t* out,
                                 int64_t ld, hipStream_t s) {
  const int64_t pieces = rows * (cols / 8);
  if (!grid_fits(blocks_for(pieces), 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL(k_dequantize_mx4, dim3((unsigned)blocks_for(pieces)), dim3(256), 0, s, elem, scale, pieces,
                     (uint32_t)(cols / 8), mx4_scale_stride(cols), out, ld);
  return hipGetLastError();
}

hipError_t launch_round_mx4(const uint16_t* x, int64_t rows, int64_t cols, uint16_t* out, hipStream_t s) {
  const int64_t pieces = rows * (cols / 8);
  hipLaunchKernelGGL(k_round_mx4, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, x, pieces, out);
  return hipGetLastError();
}

}  // namespace uw
