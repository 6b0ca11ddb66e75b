// route.hip -- a router's choice of experts and the plan that groups rows by
// expert, and the weighted sum that undoes the grouping.
//
// Choice.  key[e] = logit[e] (+ bias[e]), or sigmoid(logit[e]) + bias[e], in FP32;
// NaN and -inf, of the logit too, are never chosen.  The topk largest keys, larger first, equal keys by the lower index;
// a token with fewer selectable experts gets id -1 and weight 0 for the rest.
// Weights come from the logits without the bias: softmax over every selectable
// expert, softmax over the chosen, or sigmoids divided by their sum over the
// chosen, computed as a softmax of log sigmoids so that no logit is too low.
//
// Sixteen lanes hold a token's keys (64 lanes beyond 256 experts); each of the
// topk rounds takes the largest key by lane-local maxima and a butterfly of
// lane permutes, then the lowest index that has it the same way, so nothing
// leaves registers.  16001 tokens, 160 experts, 6 choices: 8.5 us (12 with key,
// index and logit searched in one pass, twice the instructions); a bias on the
// sigmoids costs 2 us more there.
//
// Plan.  A stable counting sort of the (token, choice) pairs by expert.  Up to 64
// pairs one wave does everything, without a barrier, up to 1024 one block;
// beyond, each block counts its tokens' experts, and a second launch places
// its pairs behind the counts of all blocks before it.  No atomics decide an
// order: the rank of a pair among its wave's equals comes from ballots, the
// waves' counts are added in wave order.
#include "experts.h"

namespace uw {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kOneBlockPairs = 1024, kOneWavePairs = 64;

// larger floats have larger keys; 0 = not selectable
__device__ __forceinline__ uint32_t order_key(float v) {
  v += 0.0f;   // -0 ties with 0
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const uint32_t k = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return (v != v || v == -__builtin_inff()) ? 0u : k;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// butterflies over the L lanes of a token: after each step a lane and its
// partner agree
template <int L, typename F>
__device__ __forceinline__ void butterfly(F&& f) {
  f([](uint32_t v) { return dpp<0xB1>(v); });    // quad: 1 0 3 2
  f([](uint32_t v) { return dpp<0x4E>(v); });    // quad: 2 3 0 1
  f([](uint32_t v) { return dpp<0x141>(v); });   // half row mirrored
  f([](uint32_t v) { return dpp<0x140>(v); });   // row mirrored
  if constexpr (L == 64) {
    f([](uint32_t v) { return (uint32_t)__shfl_xor((int)v, 16); });
    f([](uint32_t v) { return (uint32_t)__shfl_xor((int)v, 32); });
  }
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
  butterfly<L>([&](auto from) { v = fmaxf(v, __builtin_bit_cast(float, from(__builtin_bit_cast(uint32_t, v)))); });
  return v;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
  butterfly<L>([&](auto from) { v += __builtin_bit_cast(float, from(__builtin_bit_cast(uint32_t, v))); });
  return v;
}

// exp(v - top) with equals giving 1, infinities included
__device__ __forceinline__ float exp_from(float v, float top) { return v == top ? 1.0f : expf(v - top); }

__device__ __forceinline__ float logit_at(const RouteCall& c, int64_t at) {
  return c.bf16 ? __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(c.logits)[at] << 16)
                : static_cast<const float*>(c.logits)[at];
}

// One token on L lanes (l: this lane's place): lane j < topk returns choice j
// (-1: none) and its weight.  live: the token exists.
template <int L, int NV>
__device__ __forceinline__ void choose(const RouteCall& c, int64_t t, bool live, int l, int& id, float& weight) {
  float v[NV];
  uint32_t key[NV];
  // all loads first, absent keys' from the row's first place (a load under a
  // condition waits for itself: twelve in a row took most of the kernel's time)
  const int64_t row = (live ? t : 0) * c.ld;
  if (c.bf16) {
    uint16_t u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) u[i] = static_cast<const uint16_t*>(c.logits)[row + (i * L + l < c.experts ? i * L + l : 0)];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __builtin_bit_cast(float, (uint32_t)u[i] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = static_cast<const float*>(c.logits)[row + (i * L + l < c.experts ? i * L + l : 0)];
  }
  float bias[NV] = {};
  if (c.bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = c.bias[i * L + l < c.experts ? i * L + l : 0];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = live && i * L + l < c.experts;
    key[i] = in ? order_key(v[i] + bias[i]) : 0u;
  }
  if (c.on_score) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = live && i * L + l < c.experts && order_key(v[i]);
      key[i] = in ? order_key(1.0f / (1.0f + expf(-v[i])) + bias[i]) : 0u;
    }
  }
  float top = -__builtin_inff(), sum = 0.0f;
  if (c.scoring == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, key[i] ? v[i] : -__builtin_inff());
    top = group_max<L>(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += key[i] ? exp_from(v[i], top) : 0.0f;
  }
  id = -1;
  for (int j = 0; j < c.topk; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, key[i]);
    butterfly<L>([&](auto from) { best = max(best, from(best)); });
    if (best == 0) best = 0xFFFFFFFFu;   // nothing left: no key equals this (a positive NaN's, and NaN has key 0)
    // the lowest index that has it
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(i * L + l) : at;
    uint32_t e = at;
    butterfly<L>([&](auto from) { e = min(e, from(e)); });
    id = l == j ? (int)e : id;
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = e == (uint32_t)(i * L + l) ? 0u : key[i];
  }
  float mine = -__builtin_inff();   // lane j: the logit of choice j
  if (id >= 0) mine = logit_at(c, t * c.ld + id);
  const bool chosen = id >= 0;
  if (c.scoring == 2) mine = fminf(mine, 0.0f) - log1pf(expf(-__builtin_fabsf(mine)));   // log sigmoid
  if (c.scoring != 0) {
    top = group_max<L>(chosen ? mine : -__builtin_inff());
    sum = chosen ? exp_from(mine, top) : 0.0f;
  }
  sum = group_sum<L>(sum);
  weight = chosen ? exp_from(mine, top) / sum : 0.0f;
}

// The block's tokens [t0, t1): ids and weights to memory, and expert(pair)
// for each of their pairs through `each` (pair counted from t0's first).
template <int L, int NV, int NT = kThreads, typename F>
__device__ __forceinline__ void choose_range(const RouteCall& c, int64_t t0, int64_t t1, F&& each) {
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  for (int64_t t = t0; t < t1; t += NT / L) {
    const int64_t mine = t + group;
    const bool live = mine < t1;
    if (__ballot(live) == 0) break;
    int id;
    float w;
    choose<L, NV>(c, mine, live, l, id, w);
    if (live && l < c.topk) {
      c.ids[mine * c.topk + l] = id;
      c.weights[mine * c.topk + l] = w;
      each((mine - t0) * c.topk + l, id);
    }
  }
}

__device__ __forceinline__ int valid_id(int id, int experts) { return (unsigned)id < (unsigned)experts ? id : -1; }

// rank of this lane among the wave's lower lanes with the same expert, and
// how many lanes share it; absent lanes pass -1
__device__ __forceinline__ void wave_rank(int e, int& rank, int& same) {
  static_assert(kMaxExperts <= 1 << 10, "ten bits tell experts apart");
  uint64_t mask = __ballot(e >= 0);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    mask &= ((e >> b) & 1) ? set : ~set;
  }
  const uint64_t below = (1ull << (threadIdx.x & 63)) - 1ull;
  rank = __popcll(mask & below);
  same = __popcll(mask);
}

// exclusive prefix over the block's kThreads values; total in every thread
__device__ __forceinline__ int block_prefix(int v, int* wsum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(s, d);
    s += lane >= d ? up : 0;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
  __syncthreads();
  return before + s - v;
}

struct PlanLds {
  uint16_t cnt[kWaves][kMaxExperts];   // a chunk's pairs per wave and expert
  int32_t next[kMaxExperts];           // the next slot of each expert
  int wsum[kWaves];
};

// Place up to 1024 pairs: this thread's pair has expert e (-1: none or
// absent); next[] advances by the chunk's counts.  slot = -1 for none.
__device__ __forceinline__ int place_chunk(PlanLds& s, int experts, int e) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = lane; i < experts; i += 64) s.cnt[wave][i] = 0;
  int rank, same;
  wave_rank(e, rank, same);
  __syncthreads();
  if (e >= 0 && rank == 0) s.cnt[wave][e] = (uint16_t)same;
  __syncthreads();
  int slot = -1;
  if (e >= 0) {
    slot = s.next[e] + rank;
    for (int w = 0; w < wave; ++w) slot += s.cnt[w][e];
  }
  __syncthreads();
  if (threadIdx.x < experts) {
    int add = 0;
    for (int w = 0; w < kWaves; ++w) add += s.cnt[w][threadIdx.x];
    s.next[threadIdx.x] += add;
  }
  __syncthreads();
  return slot;
}

// What the wave's lanes wrote to LDS before, its lanes read after.  LDS serves a
// wave in order, so nothing is waited for, but the compiler has to keep the order: a
// wave barrier alone holds back no memory access.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Everything in one wave (tokens * topk <= 64).
template <int L, int NV>
__global__ __launch_bounds__(64) void k_route_wave(RouteCall c) {
  __shared__ int32_t ids[64], first[kMaxExperts];
  const int pairs = (int)(c.tokens * c.topk), lane = threadIdx.x;
  const int per = (c.experts + 63) / 64;   // experts of a lane, consecutive
  for (int i = lane; i < c.experts; i += 64) first[i] = 0;
  if (c.logits) {
    choose_range<L, NV, 64>(c, 0, c.tokens, [&](int64_t p, int id) { ids[p] = id; });
  } else if (lane < pairs) {
    ids[lane] = valid_id(c.ids_in[lane], c.experts);
  }
  wave_fence();
  const int e = lane < pairs ? ids[lane] : -1;
  int rank, same;
  wave_rank(e, rank, same);
  if (e >= 0 && rank == 0) first[e] = same;
  wave_fence();
  int mine = 0;
  for (int i = 0; i < per; ++i) mine += lane * per + i < c.experts ? first[lane * per + i] : 0;
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(sum, d);
    sum += lane >= d ? up : 0;
  }
  int at = sum - mine;
  for (int i = 0; i < per; ++i) {
    const int x = lane * per + i;
    if (x >= c.experts) break;
    const int n = first[x];
    first[x] = at;
    c.offsets[x] = at;
    at += n;
  }
  if (lane == 63) c.offsets[c.experts] = sum;
  wave_fence();
  if (lane < pairs) {
    const int slot = e >= 0 ? first[e] + rank : -1;
    c.slots[lane] = slot;
    if (slot >= 0) c.rows[slot] = lane / c.topk;
  }
}

// Everything in one block (tokens * topk <= 1024).
template <int L, int NV>
__global__ __launch_bounds__(kThreads) void k_route_one(RouteCall c) {
  __shared__ PlanLds s;
  __shared__ int32_t ids[kOneBlockPairs];
  __shared__ int32_t count[kMaxExperts];
  const int pairs = (int)(c.tokens * c.topk), tid = threadIdx.x;
  count[tid] = 0;
  __syncthreads();
  if (c.logits) {
    choose_range<L, NV>(c, 0, c.tokens, [&](int64_t p, int id) { ids[p] = id; });
  } else if (tid < pairs) {
    ids[tid] = valid_id(c.ids_in[tid], c.experts);
  }
  __syncthreads();
  const int e = tid < pairs ? ids[tid] : -1;
  if (e >= 0) atomicAdd(&count[e], 1);   // a sum: the order does not matter
  __syncthreads();
  int total;
  const int first = block_prefix(tid < c.experts ? count[tid] : 0, s.wsum, total);
  if (tid < c.experts) {
    s.next[tid] = first;
    c.offsets[tid] = first;
  }
  if (tid == 0) c.offsets[c.experts] = total;
  __syncthreads();
  const int slot = place_chunk(s, c.experts, e);
  if (tid < pairs) {
    c.slots[tid] = slot;
    if (slot >= 0) c.rows[slot] = tid / c.topk;
  }
}

// Block b's tokens: [b per, (b + 1) per).
template <int L, int NV>
__global__ __launch_bounds__(kThreads) void k_route_count(RouteCall c, int64_t per) {
  __shared__ int32_t count[kMaxExperts];
  count[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * per, t1 = t0 + per < c.tokens ? t0 + per : c.tokens;
  if (c.logits) {
    choose_range<L, NV>(c, t0, t1, [&](int64_t, int id) {
      if (id >= 0) atomicAdd(&count[id], 1);
    });
  } else {
    for (int64_t p = t0 * c.topk + threadIdx.x; p < t1 * c.topk; p += kThreads) {
      const int id = valid_id(c.ids_in[p], c.experts);
      if (id >= 0) atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  if (threadIdx.x < c.experts) c.hist[(int64_t)blockIdx.x * c.experts + threadIdx.x] = count[threadIdx.x];
}

__global__ __launch_bounds__(kThreads) void k_route_place(RouteCall c, int64_t per) {
  __shared__ PlanLds s;
  const int tid = threadIdx.x;
  // its expert's pairs in the blocks before this one, and in all: the threads
  // form rows of `experts`, each row adding every rows-th block's counts, 24
  // loads in flight (one row and one load at a time this took 30 us)
  __shared__ int32_t part[2][kThreads];
  const int rows = kThreads / c.experts, row = tid / c.experts, col = tid - row * c.experts;
  constexpr int kDeep = 24;
  const int nb = (int)gridDim.x, me = (int)blockIdx.x;
  int before = 0, all = 0;
  if (row < rows) {
    const int32_t* h = c.hist + col;
    for (int b0 = row; b0 < nb; b0 += kDeep * rows) {
      int v[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) v[i] = b0 + i * rows < nb ? h[(int64_t)(b0 + i * rows) * c.experts] : 0;
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        before += b0 + i * rows < me ? v[i] : 0;
        all += v[i];
      }
    }
  }
  part[0][tid] = before;
  part[1][tid] = all;
  __syncthreads();
  before = all = 0;
  if (tid < c.experts)
    for (int r = 0; r < rows; ++r) {
      before += part[0][r * c.experts + tid];
      all += part[1][r * c.experts + tid];
    }
  int total;
  const int first = block_prefix(all, s.wsum, total);
  if (tid < c.experts) {
    s.next[tid] = first + before;
    if (blockIdx.x == 0) c.offsets[tid] = first;
  }
  if (blockIdx.x == 0 && tid == 0) c.offsets[c.experts] = total;
  __syncthreads();
  const int64_t t0 = blockIdx.x * per, t1 = t0 + per < c.tokens ? t0 + per : c.tokens;
  const int32_t* ids = c.logits ? c.ids : c.ids_in;
  for (int64_t p0 = t0 * c.topk; p0 < t1 * c.topk; p0 += kThreads) {
    const int64_t p = p0 + tid;
    const bool in = p < t1 * c.topk;
    const int slot = place_chunk(s, c.experts, in ? valid_id(ids[p], c.experts) : -1);
    if (in) {
      c.slots[p] = slot;
      if (slot >= 0) c.rows[slot] = (int32_t)(p / c.topk);
    }
  }
}

// no more than 256 blocks: each reads every block's counts
int64_t tokens_per_block(int64_t tokens) {
  const int64_t per = (tokens + 255) / 256;
  return per < 64 ? 64 : per;
}

template <int L, int NV>
hipError_t launch_nv(const RouteCall& c, hipStream_t s) {
  const int blocks = route_blocks(c.tokens, c.topk);
  if (c.tokens * c.topk <= kOneWavePairs) {
    hipLaunchKernelGGL((k_route_wave<L, NV>), dim3(1), dim3(64), 0, s, c);
    return hipGetLastError();
  }
  if (blocks == 1) {
    hipLaunchKernelGGL((k_route_one<L, NV>), dim3(1), dim3(kThreads), 0, s, c);
    return hipGetLastError();
  }
  const int64_t per = tokens_per_block(c.tokens);
  hipLaunchKernelGGL((k_route_count<L, NV>), dim3(blocks), dim3(kThreads), 0, s, c, per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_place, dim3(blocks), dim3(kThreads), 0, s, c, per);
  return hipGetLastError();
}

// 8 outputs a thread
__global__ __launch_bounds__(256) void k_combine(const float* __restrict__ d, const int32_t* __restrict__ slots,
                                                 const float* __restrict__ weights, int64_t tokens, int topk, int64_t n,
                                                 int64_t d_rows, uint16_t* __restrict__ out) {
  const int64_t per = n / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= tokens * per) return;
  const int64_t t = i / per, col = (i - t * per) * 8;
  float a[8] = {};
  for (int j = 0; j < topk; ++j) {
    const int64_t slot = slots[t * topk + j];
    if (slot < 0 || slot >= d_rows) continue;
    const float w = weights[t * topk + j];
    const float4* p = reinterpret_cast<const float4*>(d + slot * n + col);
    const float4 u = p[0], v = p[1];
    a[0] += w * u.x; a[1] += w * u.y; a[2] += w * u.z; a[3] += w * u.w;
    a[4] += w * v.x; a[5] += w * v.y; a[6] += w * v.z; a[7] += w * v.w;
  }
  *reinterpret_cast<uint4*>(out + t * n + col) =
      make_uint4(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(a[4], a[5]), bf16_pair(a[6], a[7]));
}

}  // namespace

int route_blocks(int64_t tokens, int topk) {
  if (tokens * topk <= kOneBlockPairs && tokens <= 256) return 1;
  const int64_t per = tokens_per_block(tokens);
  const int64_t b = (tokens + per - 1) / per;
  return b < 2 ? 2 : (int)b;   // (a second, empty block when the pairs of one are too many for one block's sort)
}

hipError_t launch_route(const RouteCall& c, hipStream_t s) {
  // lanes a token times keys a lane cover the experts
  if (c.experts <= 64) return launch_nv<16, 4>(c, s);
  if (c.experts <= 128) return launch_nv<16, 8>(c, s);
  if (c.experts <= 192) return launch_nv<16, 12>(c, s);
  if (c.experts <= 256) return launch_nv<16, 16>(c, s);
  return launch_nv<64, 16>(c, s);
}

hipError_t launch_combine(const float* d, const int32_t* slots, const float* weights, int64_t tokens, int topk,
                          int64_t n, int64_t d_rows, uint16_t* out, hipStream_t s) {
  const int64_t items = tokens * (n / 8);
  hipLaunchKernelGGL(k_combine, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, d, slots, weights, tokens, topk,
                     n, d_rows, out);
  return hipGetLastError();
}

}  // namespace uw
