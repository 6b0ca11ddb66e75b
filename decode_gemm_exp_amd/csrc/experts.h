// experts.h -- shared declarations of the mixture-of-experts and MXFP4
// operators: the experts' weights as the kernels see them, the search of a
// block's share of ragged rows, MXFP4 unpacking, and the launchers.
#pragma once

#include "rebuild.h"

namespace uw {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 16;
// Tokens of a layer that goes in two kernels; a block of 256 threads or more holds all their pairs, and
// sixteen are the columns of an MFMA.  us, two kernels / router, both products and the weighted sum, 1, 8 and 16 tokens:
//   FP8, 8 of 64 experts 1408x2048    18.8 / 27.8    65 / 86      99 / 110
//   MXFP4, 6 of 160 1408x2048         16.4 / 23.2    51 / 61      84 / 96
//   BF16, 8 of 64 1408x2048           29.1 / 38.2   125 / 147    183 / 193
//   BF16, 2 of 16 512x1024            11.1 / 17.3    17 / 22      20 / 26
//   UWF1, 4 of 32 2048x4096           34.7 / 39.4   175 / 175    234 / 235
//   BF16, 2 of 8 14336x4096            124 / 130    496 / 493    507 / 500
//   FP8, 2 of 8 14336x4096              67 / 78     228 / 223    265 / 254
// Few large experts, which all have tokens by eight, lose up to 4 % to what they win elsewhere.
constexpr int kLayerTokens = UW_LAYER_TOKENS, kLayerPairs = kLayerTokens * kMaxTopk;

// Weight forms of the expert products, a template argument of the kernels.
// kFormPal serves UWF1 matrices whose palettes differ in kind (one of them
// not a run of consecutive exponents), kFormPalRun those that all are runs.
enum ExpertForm { kFormBf16 = 0, kFormPal = 2, kFormPalRun = 3, kFormMx4 = 4, kFormFp8 = 5 };
constexpr bool form_is_pal(int f) { return f == kFormPal || f == kFormPalRun; }

// One UWF1 expert (device table).
struct ExpertEntry {
  const uint8_t* sm;
  const uint8_t* pidx;
  const uint32_t* vflags;
  const uint32_t* vrank;
  const uint8_t* vexp;
  PalView pal;
};

// a matrix's palette as the kernels take it (api.cpp)
void palette_view(const uw_matrix* m, PalView* out);

// All experts of one projection: expert e's W_e[N][K].
struct ExpertsView {
  int form;
  int count;
  int64_t n, k;
  const uint8_t* w;        // BF16 rows, packed MXFP4 elements or E4M3 bytes of expert 0
  const uint8_t* scale;    // MXFP4: scales of expert 0, mx4_scale_stride(k) bytes a row;
                           // FP8: floats, one per 128 x 128 block, row-major
  int64_t w_stride;        // bytes from one expert's weights to the next
  int64_t scale_stride;
  const ExpertEntry* table;   // UWF1
};

typedef __attribute__((address_space(3))) char lds_char;

// A load the compiler knows to be from global memory.  Pointers read from the
// device table have no address space of their own, and flat loads would
// count with the LDS reads: every wait for one would wait for all.
template <typename T>
__device__ __forceinline__ T gload(const void* p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) T*>(reinterpret_cast<uintptr_t>(p));
}
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4_t;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2_t;
__device__ __forceinline__ uint4 gload16(const void* p) {
  const u32x4_t v = gload<u32x4_t>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 gload8(const void* p) {
  const u32x2_t v = gload<u32x2_t>(p);
  return make_uint2(v.x, v.y);
}

// An offset past the end of every buffer resource here, also with a row's and a K
// tail's own kOutside added: such a load reads zeros, such a store is dropped.
// (Twice this is below 2^32; x beyond this many bytes goes by pointers.)
constexpr uint32_t kOutside = 0x7FFF0000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t byte) {
  const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)byte, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// Tiles in LDS: rows of 128 bytes, 16-byte piece c of row r at c ^ (r / 2 % 8)
__device__ __forceinline__ uint32_t piece_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ ((row >> 1) & 7)) << 4)); }

// A block barrier without a fence: a fence would wait for everything that is on
// its way to LDS.  The caller has waited for what must have landed.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

__host__ __device__ constexpr int64_t mx4_scale_stride(int64_t k) { return (k + 127) / 128 * 4; }

// Ragged rows: expert e's are slots [offsets[e], offsets[e + 1]); slot s
// multiplies row rows[s] of x, or row s when rows is NULL.  offsets NULL: one
// expert with all `slots` rows.
struct RaggedRows {
  const int32_t* offsets;
  const int32_t* rows;
  int64_t slots;      // capacity: offsets are clamped to it, and to their predecessors
  int64_t x_rows;     // rows of x; a row index outside selects a row of zeros
};

// A block's share: `count` slots from `first`, all of expert `expert`;
// count 0: nothing to do.
struct Share {
  int expert;
  int64_t first;
  int count;
};

// A lane's four experts of the 256 from e0: their slots' bounds o, their numbers of
// chunks c; returns the chunks up to and with this lane's.  Every wave of a
// block does this by itself, without a barrier.  Bounds are the running maximum of
// the offsets clamped to [0, slots], so that whatever the array holds, the experts'
// slots are disjoint and inside the capacity (and max_chunks holds); high: the
// last bound of the experts before e0, 0 at first, and afterwards that of the 256.
__device__ __forceinline__ int four_experts(const RaggedRows& r, int experts, int e0, int chunk, int32_t& high,
                                            int32_t (&o)[5], int (&c)[4]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int e = e0 + 4 * lane + i;
    o[i] = r.offsets[e < experts ? e : experts];
  }
  // all five are loaded before the first is touched (left to itself the compiler
  // loads and waits one by one, a microsecond each at the start of every block)
  asm volatile("" : "+v"(o[0]), "+v"(o[1]), "+v"(o[2]), "+v"(o[3]), "+v"(o[4]));
#pragma unroll
  for (int i = 0; i < 5; ++i) o[i] = o[i] < 0 ? 0 : (int64_t)o[i] < r.slots ? o[i] : (int32_t)r.slots;
  // (a plan ascends, so the maximum is taken, and its code laid, out of the way)
  bool down = o[0] < high;
#pragma unroll
  for (int i = 1; i < 5; ++i) down |= o[i] < o[i - 1];
  if (__builtin_expect(__ballot(down) != 0, 0)) {
#pragma unroll
    for (int i = 1; i < 5; ++i) o[i] = max(o[i], o[i - 1]);
    int32_t top = max(o[4], high);   // of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t up = __shfl_up(top, d);
      top = lane >= d ? max(top, up) : top;
    }
    const int32_t up = __shfl_up(top, 1), before = lane ? up : high;
#pragma unroll
    for (int i = 0; i < 5; ++i) o[i] = max(o[i], before);
  }
  high = __builtin_amdgcn_readlane(o[4], 63);
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = (int)(((int64_t)o[i + 1] - o[i] + chunk - 1) / chunk);
    sum += c[i];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(sum, d);
    sum += lane >= d ? up : 0;
  }
  return sum;
}

// Chunk `j` of the experts' slots cut into chunks of at most `chunk`: expert
// e has ceil(rows_e / chunk).
__device__ __forceinline__ Share find_share(const RaggedRows& r, int experts, int64_t j, int chunk) {
  Share out{0, 0, 0};
  if (!r.offsets) {
    const int64_t first = j * chunk;
    if (first < r.slots) {
      out.first = first;
      out.count = (int)(r.slots - first < chunk ? r.slots - first : chunk);
    }
    return out;
  }
  const int lane = threadIdx.x & 63;
  int64_t before = 0;   // chunks of the experts before this round's
  int32_t high = 0;
  for (int e0 = 0; e0 < experts; e0 += 256) {
    int32_t o[5];
    int c[4];
    const int sum = four_experts(r, experts, e0, chunk, high, o, c), mine = c[0] + c[1] + c[2] + c[3];
    const int64_t lo = before + sum - mine;
    const uint64_t hit = __ballot(j >= lo && j < lo + mine);
    if (hit) {
      int at = (int)(j - lo), e = 0;
      int32_t b = o[0], n = o[1];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const bool go = e == i && at >= c[i];
        at -= go ? c[i] : 0;
        e = go ? i + 1 : e;
        b = go ? o[i + 1] : b;
        n = go ? o[i + 2] : n;
      }
      const int src = __ffsll((unsigned long long)hit) - 1;
      out.expert = __builtin_amdgcn_readlane(e0 + 4 * lane + e, src);
      const int32_t begin = __builtin_amdgcn_readlane(b, src), end = __builtin_amdgcn_readlane(n, src);
      out.first = (int64_t)begin + (int64_t)__builtin_amdgcn_readlane(at, src) * chunk;
      out.count = (int)(end - out.first < chunk ? end - out.first : chunk);
      return out;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return out;
}

// Tile `l` of a grid of `chunks` row chunks times `ntiles` column tiles: bands
// of eight column tiles, within a band the row chunks in turn, each over the
// band's columns.  The 32 blocks an XCD runs at once then cover about 4 x 8
// tiles, 12 panels of x and weights to keep in its L2 instead of 33.
__device__ __forceinline__ void tile_of(uint32_t l, uint32_t chunks, uint32_t ntiles, int& chunk, int& nt) {
  constexpr uint32_t kBand = 8;
  const uint32_t band = l / (kBand * chunks), in = l - band * kBand * chunks;
  const uint32_t width = ntiles - band * kBand < kBand ? ntiles - band * kBand : kBand;
  const uint32_t m = in / width;
  chunk = __builtin_amdgcn_readfirstlane((int)m);
  nt = __builtin_amdgcn_readfirstlane((int)(band * kBand + in - m * width));
}

// A chunk (see find_share) and a column tile of ntiles, dealt so that each XCD works
// on one contiguous run of the list of them: entry `turn` of XCD `xcd`'s eighth of the list that
// really exists (its length follows from the offsets); blocks go to the XCDs
// round robin, so block b is on XCD b % 8.  What it returns is in scalar registers:
// buffer resources built from it then need no loop over a wave's lanes (a
// division done in vector registers would leave it there).  The list runs over experts, then column
// tiles, then an expert's row chunks, so neighbours share weights and x in
// one L2.  Returns the column tile, or -1: nothing to do.
__device__ __forceinline__ int find_tile(const RaggedRows& r, int experts, int xcd, int64_t turn, int ntiles, int chunk,
                                         Share& out) {
  out = Share{0, 0, 0};
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  int32_t o[5] = {}, high = 0;
  int c[4] = {}, sum = 0;
  if (!r.offsets) {
    total = (r.slots + chunk - 1) / chunk;
  } else {
    for (int e0 = 0; e0 < experts; e0 += 256) {
      sum = four_experts(r, experts, e0, chunk, high, o, c);
      total += __builtin_amdgcn_readlane(sum, 63);
    }
  }
  const int64_t tiles = total * ntiles, share = (tiles + 7) / 8;
  const int64_t at = xcd * share + turn;
  if (turn >= share || at >= tiles) return -1;
  if (!r.offsets) {
    int m, nt;
    tile_of((uint32_t)at, (uint32_t)total, (uint32_t)ntiles, m, nt);   // (at < 2^31: the grid is)
    out.first = m * (int64_t)chunk;
    out.count = (int)(r.slots - out.first < chunk ? r.slots - out.first : chunk);
    return nt;
  }
  int64_t before = 0;   // chunks of the experts before this round's
  high = 0;
  for (int e0 = 0; e0 < experts; e0 += 256) {
    if (experts > 256) sum = four_experts(r, experts, e0, chunk, high, o, c);   // (else as it was)
    const int mine = c[0] + c[1] + c[2] + c[3];
    const int64_t lo = (before + sum - mine) * ntiles, hi = (before + sum) * ntiles;
    const uint64_t hit = __ballot(at >= lo && at < hi);
    if (hit) {
      int64_t left = at - lo;   // in tiles of this lane's four experts
      int e = 0, n = c[0];
      int32_t b = o[0], end = o[1];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const bool go = e == i && left >= (int64_t)c[i] * ntiles;
        left -= go ? (int64_t)c[i] * ntiles : 0;
        e = go ? i + 1 : e;
        n = go ? c[i + 1] : n;
        b = go ? o[i + 1] : b;
        end = go ? o[i + 2] : end;
      }
      const int src = __ffsll((unsigned long long)hit) - 1;
      out.expert = __builtin_amdgcn_readlane(e0 + 4 * lane + e, src);
      const int chunks = __builtin_amdgcn_readlane(n, src);
      const int l = __builtin_amdgcn_readlane((int)left, src);
      const int32_t begin = __builtin_amdgcn_readlane(b, src), stop = __builtin_amdgcn_readlane(end, src);
      int m, nt;
      tile_of((uint32_t)l, (uint32_t)chunks, (uint32_t)ntiles, m, nt);
      out.first = (int64_t)begin + (int64_t)m * chunk;
      out.count = (int)(stop - out.first < chunk ? stop - out.first : chunk);
      return nt;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return -1;
}

// Chunks that slots rows over `experts` experts can make at most: every
// expert with rows adds less than one chunk beyond its share.
inline int64_t max_chunks(int64_t slots, int experts, int chunk, bool ragged) {
  if (!ragged) return (slots + chunk - 1) / chunk;
  const int64_t with_rows = slots < experts ? slots : experts;
  const int64_t c = slots / chunk + with_rows;
  return c < slots ? c : slots;
}

// ---- MXFP4 --------------------------------------------------------------------
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

// an E8M0 scale as the float whose exponent field it is (byte 0: the field of
// 2^-127, which the scaled conversions read as such)
__device__ __forceinline__ float e8m0_float(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// 8 elements (one dword) times their block's scale -> 8 BF16, exact unless
// the product overflows BF16 (scale bytes 253 and up)
__device__ __forceinline__ uint4 mx4_unpack8(uint32_t q, float scale) {
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
  return o;
}

// float -> BF16, to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) float f2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf16x2_t));
}

// g / (1 + exp(-g)) as g e^2 / (1 + e^2) with e = exp(g / 2): exp(-g) itself would
// overflow below -88.7, where the value, -2.6e-37 there, is a normal BF16 number
// still, while e is normal down to -174 (the value leaves BF16 at -100).  Beyond
// 2^43, g > 59, e^2 / (1 + e^2) is 1 in FP32.  The products' order keeps every
// partial one in range.  The exponential's argument is off by half a unit, 2^-18 of
// the value at |g| = 88; the reciprocal instruction is within one unit in the last place.
__device__ __forceinline__ float silu(float g) {
  const float e = __builtin_amdgcn_exp2f(fminf(g * 0.72134752f, 43.0f));
  return g * (e * __builtin_amdgcn_rcpf(__builtin_fmaf(e, e, 1.0f))) * e;
}

// ---- launchers ----------------------------------------------------------------
// A launch holds fewer than 2^32 threads.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (int64_t)(UINT32_MAX / (unsigned)threads); }

// y = W x (FP32) or, gated, h = silu(W x) * (U x) (BF16; u is then the second
// projection) over ragged rows
struct ExpertsCall {
  ExpertsView w, u;
  bool gated;
  RaggedRows r;
  const uint16_t* x;
  void* y;
  bool check;   // refuse what a launch would, launch nothing
};
hipError_t launch_experts(const ExpertsCall& c, hipStream_t s);
hipError_t launch_experts_rows(const ExpertsCall& c, hipStream_t s);
// rows of a tile: 64, 128 or 256; spread: blocks start along K at different places
hipError_t launch_experts_tile(const ExpertsCall& c, int rows, bool spread, hipStream_t s);

hipError_t launch_quantize_mx4(const void* src, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* elem,
                               uint8_t* scale, hipStream_t s);
hipError_t launch_dequantize_mx4(const uint8_t* elem, const uint8_t* scale, int64_t rows, int64_t cols, uint16_t* out,
                                 int64_t ld, hipStream_t s);
// both operands in MXFP4 (rows contiguous, scales mx4_scale_stride(k) a row)
hipError_t launch_mx4_tile(const uint8_t* we, const uint8_t* ws, int64_t n, int64_t k, const uint8_t* xe,
                           const uint8_t* xs, int64_t batch, float* y, hipStream_t s);
// x -> the BF16 values its MXFP4 form stands for
hipError_t launch_round_mx4(const uint16_t* x, int64_t rows, int64_t cols, uint16_t* out, hipStream_t s);

struct RouteCall {
  const void* logits;   // NULL: ids are given
  bool bf16;
  int64_t tokens, ld;
  int experts, topk, scoring;
  const float* bias;
  bool on_score;        // the bias is added to the logit's sigmoid, not to the logit
  int32_t* ids;
  const int32_t* ids_in;
  float* weights;
  int32_t *offsets, *rows, *slots;
  int32_t* hist;        // [blocks][experts], unless one block does it all
};
int route_blocks(int64_t tokens, int topk);   // 1: no workspace
hipError_t launch_route(const RouteCall& c, hipStream_t s);

// A layer for at most kLayerTokens tokens (route.h): the choice, the plan and the gated
// product h [tokens * topk][n] by slot (c.r is not used), then the down product with the weighted sum.
hipError_t launch_layer_gated(const ExpertsCall& c, const RouteCall& r, hipStream_t s);
hipError_t launch_layer_gated_fp8(const ExpertsCall& c, const RouteCall& r, hipStream_t s);
hipError_t launch_layer_down(const ExpertsView& d, const RouteCall& r, const uint16_t* h, uint16_t* out, hipStream_t s);

// out[t] = sum over j of weights[t][j] d[slots[t][j]], in the order of j
hipError_t launch_combine(const float* d, const int32_t* slots, const float* weights, int64_t tokens, int topk,
                          int64_t n, int64_t d_rows, uint16_t* out, hipStream_t s);

}  // namespace uw

// A set of experts (host object; the weights stay the caller's).
struct uw_experts {
  uw::ExpertsView v{};
  int device = 0;
  const uw_matrix** ms = nullptr;       // UWF1: the matrices, and their indices when the table was made
  const uint8_t** pidx = nullptr;
  uw::ExpertEntry* table = nullptr;     // device
  uw_allocator alloc{};
};
