// route.h -- a router's choice for one token, shared by the routing kernels and by the
// layer kernels that route for themselves (see route.hip for what it computes).
#pragma once

#include "experts.h"

namespace uw {
namespace {

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
// (-1: none) and, with WEIGHTS, its weight.  live: the token exists.
template <int L, int NV, bool WEIGHTS = true>
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
  if (WEIGHTS && c.scoring == 0) {
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
  if constexpr (!WEIGHTS) return;
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

// What the lanes of a wave wrote to LDS before, its lanes read after.  LDS serves a
// wave in order, so nothing is waited for, but the compiler has to keep the order: a
// wave barrier alone holds back no memory access.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- a few tokens, routed by every block for itself ----------------------------
// kLayerTokens tokens at most.  Each block makes the choice anew (a microsecond, while a launch
// of its own and the wait for it cost several) and finds its expert's rows in it;
// block 0 writes the plan, the same that uw_route_experts writes, and nothing else.
template <int L, int NV>
struct RoutedRows {
  static constexpr int kLanes = L, kKeys = NV;
  RouteCall c;
  int64_t slots, x_rows;
};

struct RoutedLds {
  int32_t pair[kLayerPairs];          // a pair's expert, -1: none
  uint32_t has[kMaxExperts / 32];     // experts that have pairs, a bit each
  int32_t tok[4][kLayerTokens];       // per wave: tokens of its block's expert
};

// The choice of every token, into s; WRITE: ids and weights to memory as well.
template <int L, int NV, bool WRITE>
__device__ __forceinline__ void route_few(const RouteCall& c, RoutedLds& s) {
  const int l = threadIdx.x % L, group = threadIdx.x / L, tokens = (int)c.tokens;
  if (threadIdx.x < kMaxExperts / 32) s.has[threadIdx.x] = 0u;
  s.pair[threadIdx.x] = -1;
  __syncthreads();
  for (int t = group; t - group < tokens; t += 256 / L) {
    const bool live = t < tokens;
    if (__ballot(live) == 0) break;
    int id;
    float w = 0.0f;
    choose<L, NV, WRITE>(c, t, live, l, id, w);
    if (live && l < c.topk) {
      s.pair[t * c.topk + l] = id;
      if (id >= 0) atomicOr(&s.has[id >> 5], 1u << (id & 31));   // (bits: the order does not matter)
      if constexpr (WRITE) {
        c.ids[t * c.topk + l] = id;
        c.weights[t * c.topk + l] = w;
      }
    }
  }
  __syncthreads();
}

// The kernel for a layer's number of experts: lanes a token times keys a lane.
template <typename F>
hipError_t with_routed(const RouteCall& c, F&& f) {
  if (c.experts <= 64) return f(RoutedRows<16, 4>{c, c.tokens * c.topk, c.tokens});
  if (c.experts <= 256) return f(RoutedRows<16, 16>{c, c.tokens * c.topk, c.tokens});
  return f(RoutedRows<64, 16>{c, c.tokens * c.topk, c.tokens});
}
// Blocks: the plan's, then `ntiles` for every expert that can have pairs.
inline int64_t routed_grid(const RouteCall& c, int64_t ntiles) {
  const int64_t pairs = c.tokens * c.topk;
  return 1 + ntiles * (pairs < c.experts ? pairs : c.experts);
}

// The plan of the choice in s.  A pair's slot is the number of pairs before it, by
// expert, then by pair.
__device__ __forceinline__ void plan_few(const RouteCall& c, const RoutedLds& s) {
  const int pairs = (int)c.tokens * c.topk, p = threadIdx.x, e = s.pair[p];
  if (p < pairs) {
    int slot = 0;
    for (int q = 0; q < pairs; ++q) {
      const int f = s.pair[q];
      slot += f >= 0 && (f < e || (f == e && q < p)) ? 1 : 0;
    }
    c.slots[p] = e >= 0 ? slot : -1;
    if (e >= 0) c.rows[slot] = p / c.topk;
  }
  for (int x = p; x <= c.experts; x += 256) {
    int n = 0;
    for (int q = 0; q < pairs; ++q) n += s.pair[q] >= 0 && s.pair[q] < x ? 1 : 0;
    c.offsets[x] = n;
  }
}

// The share of the chunk-th expert that has pairs, by index; count 0: there are not
// that many.  Its tokens in the order of their slots go to s.tok[wave].
__device__ __forceinline__ Share share_few(const RouteCall& c, RoutedLds& s, int chunk) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t word = lane < kMaxExperts / 32 ? s.has[lane] : 0u;
  const int mine = __popc(word);
  int upto = mine;
#pragma unroll
  for (int d = 1; d < kMaxExperts / 32; d <<= 1) {
    const int up = __shfl_up(upto, d);
    upto += lane >= d ? up : 0;
  }
  Share out{0, 0, 0};
  const uint64_t hit = __ballot(chunk >= upto - mine && chunk < upto);
  if (hit == 0) return out;
  const int src = __ffsll((unsigned long long)hit) - 1;
  uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, src);
  for (int i = chunk - __builtin_amdgcn_readlane(upto - mine, src); i > 0; --i) bits &= bits - 1u;
  const int e = 32 * src + __ffs((int)bits) - 1;
  out.expert = e;
  int first = 0, count = 0;
#pragma unroll
  for (int i = 0; i < kLayerPairs / 64; ++i) {
    const int p = 64 * i + lane, f = s.pair[p];
    const uint64_t eq = __ballot(f == e);
    first += __popcll(__ballot(f >= 0 && f < e));
    if (f == e) s.tok[wave][count + __popcll(eq & ((1ull << lane) - 1ull))] = p / c.topk;
    count += __popcll(eq);
  }
  out.first = first;
  out.count = count;   // at most one pair a token
  wave_fence();
  return out;
}

}  // namespace
}  // namespace uw
