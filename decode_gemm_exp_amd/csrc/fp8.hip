// fp8.hip -- conversion between BF16 / FP32 and E4M3 with an FP32 scale per block
// of 1 x 128 (a row's) or 128 x 128 (a matrix's); see fp8.h for the arithmetic.
//
// Bound: HBM, 2 (or 4) + 1 bytes an element; 14336x4096 BF16 in 128 x 128 takes 30 to 32 us,
// back 30 (176 MB: 5.5 to 5.9 TB/s).  One pass: what a block's maximum is
// taken over stays in registers until it is converted.  A thread holds pieces of
// eight elements, sixteen lanes a row of a block, so that loads and stores run
// over whole rows of blocks.
#include "fp8.h"

namespace uw {
namespace {

// Eight values as loaded: BF16 pairs, or floats.
template <bool F32>
struct Eight {
  uint4 a, b;   // b: floats only
};

template <bool F32>
__device__ __forceinline__ Eight<F32> load8(const void* src, int64_t at) {
  // (read once: kept out of the caches, 14336x4096 34.5 -> 30.5 us)
  const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(src) + at * (F32 ? 4 : 2));
  auto piece = [](const u32x4_t& v) __attribute__((always_inline)) { return make_uint4(v.x, v.y, v.z, v.w); };
  Eight<F32> e;
  e.a = piece(__builtin_nontemporal_load(p));
  if constexpr (F32) e.b = piece(__builtin_nontemporal_load(p + 1));
  return e;
}

// the largest magnitude's FP32 bits
template <bool F32>
__device__ __forceinline__ uint32_t top8(const Eight<F32>& e) {
  if constexpr (F32) {
    auto mag = [](uint32_t w) __attribute__((always_inline)) { return w & 0x7FFFFFFFu; };
    return max(max(max(mag(e.a.x), mag(e.a.y)), max(mag(e.a.z), mag(e.a.w))),
               max(max(mag(e.b.x), mag(e.b.y)), max(mag(e.b.z), mag(e.b.w))));
  } else {
    return top_bits(bf16_top8(e.a));
  }
}

template <bool F32>
__device__ __forceinline__ uint2 pack(const Eight<F32>& e, float inv) {
  if constexpr (F32) {
    auto f = [&](uint32_t w) __attribute__((always_inline)) { return __builtin_bit_cast(float, w) * inv; };
    const uint2 q = make_uint2(fp8_pack4(f(e.a.x), f(e.a.y), f(e.a.z), f(e.a.w)),
                               fp8_pack4(f(e.b.x), f(e.b.y), f(e.b.z), f(e.b.w)));
    return inv != 0.0f ? q : make_uint2(0u, 0u);
  } else {
    return fp8_pack8(e.a, inv);
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return v > o ? v : o;
}
// over the sixteen lanes of a row: quads, then mirrored halves, then the row mirrored
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v))));
}

// A block of threads takes 16 U rows of one column of blocks.  BIG: U = 8, they are
// one block of 128 x 128; else each row's 128 elements are one.  AS16: elements are
// written as the BF16 numbers they are (exact), two bytes each.
template <bool F32, int U, bool BIG, bool AS16>
__global__ __launch_bounds__(256) void k_quantize_fp8(const void* __restrict__ src, int64_t rows, int64_t cols,
                                                      int64_t ld, void* __restrict__ elem,
                                                      float* __restrict__ scale, uint32_t nb) {
  static_assert(!BIG || U == 8, "a block of 128 rows");
  const uint32_t rb = blockIdx.x / nb, cb = blockIdx.x - rb * nb;
  const int lane16 = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t col = (int64_t)cb * 128 + 8 * lane16, row0 = (int64_t)rb * (16 * U) + r;
  const bool in_col = col < cols;
  Eight<F32> e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {   // what is not there reads the block's first piece, and does not count
    const int64_t row = row0 + 16 * u;
    const bool in = in_col && row < rows;
    e[u] = load8<F32>(src, in ? row * ld + col : (int64_t)rb * (16 * U) * ld + (int64_t)cb * 128);
  }
  uint32_t top[U];
#pragma unroll
  for (int u = 0; u < U; ++u) top[u] = in_col && row0 + 16 * u < rows ? top8(e[u]) : 0u;
  if constexpr (BIG) {
    __shared__ uint32_t part[16];
    uint32_t m = top[0];
#pragma unroll
    for (int u = 1; u < U; ++u) m = max(m, top[u]);
    m = row_max(m);
    if (lane16 == 0) part[r] = m;
    __syncthreads();
    m = row_max(part[lane16]);
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = m;
    if (threadIdx.x == 0) scale[(int64_t)rb * nb + cb] = fp8_scale(m).scale;
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = row_max(top[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + 16 * u;
    const Fp8Scale f = fp8_scale(top[u]);
    if (row >= rows) continue;
    if (!BIG && lane16 == 0) scale[row * nb + cb] = f.scale;
    if (!in_col) continue;
    const uint2 q = pack(e[u], f.inv);
    if constexpr (AS16) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(elem) + row * cols + col) = fp8_unpack8(q.x, q.y);
    else *reinterpret_cast<uint2*>(static_cast<uint8_t*>(elem) + row * cols + col) = q;
  }
}

// A block of threads takes 64 rows of 256 columns, a thread eight elements of every
// eighth row, so that a wave's stores are whole lines.
__global__ __launch_bounds__(256) void k_dequantize_fp8(const uint8_t* __restrict__ elem,
                                                        const float* __restrict__ scale, int64_t rows, int64_t cols,
                                                        int block_rows, uint16_t* __restrict__ out, int64_t ld,
                                                        uint32_t nt) {
  constexpr int U = 8;
  const uint32_t rt = blockIdx.x / nt, ct = blockIdx.x - rt * nt;
  const int64_t col = (int64_t)ct * 256 + 8 * (threadIdx.x & 31), row0 = (int64_t)rt * 64 + (threadIdx.x >> 5);
  if (col >= cols) return;
  const int64_t nb = fp8_blocks(cols);
  uint2 q[U];
  float f[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + 8 * u < rows ? row0 + 8 * u : rows - 1;
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(elem + row * cols + col);
    q[u] = make_uint2(v.x, v.y);
    f[u] = scale[(block_rows == 1 ? row : row >> 7) * nb + (col >> 7)];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + 8 * u;
    if (row >= rows) break;
    auto two = [&](uint32_t w, bool hi) __attribute__((always_inline)) {
      typedef __attribute__((ext_vector_type(2))) float f2;
      const f2 v = hi ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
      return bf16_pair(v.x * f[u], v.y * f[u]);
    };
    *reinterpret_cast<uint4*>(out + row * ld + col) =
        make_uint4(two(q[u].x, false), two(q[u].x, true), two(q[u].y, false), two(q[u].y, true));
  }
}

template <bool F32, int U, bool BIG, bool AS16 = false>
hipError_t launch_quantize(const void* src, int64_t rows, int64_t cols, int64_t ld, void* elem, float* scale,
                           hipStream_t s) {
  const int64_t nb = fp8_blocks(cols), grid = nb * ((rows + 16 * U - 1) / (16 * U));
  if (!grid_fits(grid, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_quantize_fp8<F32, U, BIG, AS16>), dim3((unsigned)grid), dim3(256), 0, s, src, rows, cols, ld, elem,
                     scale, (uint32_t)nb);
  return hipGetLastError();
}

template <bool F32, bool AS16>
hipError_t launch_rows(const void* src, int64_t rows, int64_t cols, int64_t ld, void* elem, float* scale, hipStream_t s) {
  // four rows a thread where that still makes a block for every CU
  if ((rows + 63) / 64 * fp8_blocks(cols) >= device_cus())
    return launch_quantize<F32, 4, false, AS16>(src, rows, cols, ld, elem, scale, s);
  return launch_quantize<F32, 1, false, AS16>(src, rows, cols, ld, elem, scale, s);
}

}  // namespace

hipError_t launch_quantize_fp8(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, int block_rows,
                               uint8_t* elem, float* scale, hipStream_t s) {
  if (block_rows != 1)
    return f32 ? launch_quantize<true, 8, true>(src, rows, cols, ld, elem, scale, s)
               : launch_quantize<false, 8, true>(src, rows, cols, ld, elem, scale, s);
  return f32 ? launch_rows<true, false>(src, rows, cols, ld, elem, scale, s)
             : launch_rows<false, false>(src, rows, cols, ld, elem, scale, s);
}

hipError_t launch_round_fp8(const uint16_t* x, int64_t rows, int64_t cols, uint16_t* out, float* scale, hipStream_t s) {
  return launch_rows<false, true>(x, rows, cols, cols, out, scale, s);
}

hipError_t launch_dequantize_fp8(const uint8_t* elem, const float* scale, int64_t rows, int64_t cols, int block_rows,
                                 uint16_t* out, int64_t ld, hipStream_t s) {
  const int64_t nt = (cols + 255) / 256, grid = nt * ((rows + 63) / 64);
  if (!grid_fits(grid, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL(k_dequantize_fp8, dim3((unsigned)grid), dim3(256), 0, s, elem, scale, rows, cols, block_rows, out,
                     ld, (uint32_t)nt);
  return hipGetLastError();
}

}  // namespace uw
