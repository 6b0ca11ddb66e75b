// route.h -- a router's choice for one token, shared by the routing kernels and by the
// layer kernels that route for themselves (see route.hip for what it computes).
#pragma once

#include <type_traits>

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

// A token's logits v and keys on L lanes (l: this lane's place), expert i L + l in
// place i; live: the token exists.
template <int L, int NV>
__device__ __forceinline__ void load_keys(const RouteCall& c, int64_t t, bool live, int l, float (&v)[NV],
                                          uint32_t (&key)[NV]) {
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
}

// One token on L lanes: lane j < topk returns choice j (-1: none) and its weight.
template <int L, int NV>
__device__ __forceinline__ void choose(const RouteCall& c, int64_t t, bool live, int l, int& id, float& weight) {
  float v[NV];
  uint32_t key[NV];
  load_keys<L, NV>(c, t, live, l, v, key);
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

// What the lanes of a wave wrote to LDS before, its lanes read after.  LDS serves a
// wave in order, so nothing is waited for, but the compiler has to keep the order: a
// wave barrier alone holds back no memory access.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The same choice on a whole wave, without weights, of Q tokens t, t + 4, .. at once: the
// largest key goes through scalar registers, and ballots find the lowest index that
// has it, so a round is one chain of row maxima instead of two butterflies, and
// the tokens' chains run beside each other.
template <int NV, int Q>
__device__ __forceinline__ void choose_wave(const RouteCall& c, int t, int (&id)[Q]) {
  const int lane = threadIdx.x & 63;
  float v[Q][NV];
  uint32_t key[Q][NV];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    load_keys<64, NV>(c, t + 4 * q, t + 4 * q < c.tokens, lane, v[q], key[q]);
    id[q] = -1;
  }
  for (int j = 0; j < c.topk; ++j) {
    uint32_t best[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      best[q] = key[q][0];
#pragma unroll
      for (int i = 1; i < NV; ++i) best[q] = max(best[q], key[q][i]);
      butterfly<16>([&](auto from) { best[q] = max(best[q], from(best[q])); });
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      auto row = [&](int r) __attribute__((always_inline)) { return (uint32_t)__builtin_amdgcn_readlane((int)best[q], 16 * r); };
      const uint32_t most = max(max(row(0), row(1)), max(row(2), row(3)));
      int e = -1;   // stays so when nothing is left
#pragma unroll
      for (int i = NV - 1; i >= 0; --i) {
        const uint64_t has = __ballot(key[q][i] == most);
        e = has && most ? 64 * i + __ffsll((unsigned long long)has) - 1 : e;
      }
      id[q] = lane == j ? e : id[q];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[q][i] = e == 64 * i + lane ? 0u : key[q][i];
    }
  }
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

// The pairs by expert, and the items they make: an expert and up to C of its tokens.
struct PairsLds {
  int32_t expert[kLayerPairs];                       // by slot, -1 behind the last
  int32_t token[kLayerPairs];
  float weight[kLayerPairs];                         // (where they are needed)
  int32_t item_expert[kLayerPairs + 1];              // (one more, and of the first slots, for reading ahead)
  int32_t item_first[kLayerPairs + 2];               // its first slot; behind the last item the number of slots
};

// The items of the slots in s, which the block's threads have written; returns their
// number.  Every wave counts them all, the first four write.
template <int C>
__device__ __forceinline__ int list_items(PairsLds& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int e[kLayerPairs / 64], prev[kLayerPairs / 64];
#pragma unroll
  for (int i = 0; i < kLayerPairs / 64; ++i) {
    const int at = 64 * i + lane;
    e[i] = s.expert[at];
    prev[i] = s.expert[at ? at - 1 : 0];
  }
  const uint64_t upto = (2ull << lane) - 1ull;   // lanes up to this one
  int items = 0, slots = 0, start = 0;           // start: the first slot of the expert before
#pragma unroll
  for (int i = 0; i < kLayerPairs / 64; ++i) {
    const int at = 64 * i + lane;
    const uint64_t starts = __ballot(e[i] >= 0 && (at == 0 || e[i] != prev[i]));
    const int from = (starts & upto) ? 64 * i + 63 - __builtin_clzll(starts & upto) : start;
    const bool first = e[i] >= 0 && (at - from) % C == 0;
    const uint64_t mask = __ballot(first);
    if (wave == i && first) {
      const int mine = items + __popcll(mask & upto) - 1;
      s.item_expert[mine] = e[i];
      s.item_first[mine] = at;
    }
    items += __popcll(mask);
    slots += __popcll(__ballot(e[i] >= 0));
    start = starts ? 64 * i + 63 - __builtin_clzll(starts) : start;
  }
  if (threadIdx.x == 0) s.item_first[items] = slots;
  __syncthreads();
  return items;
}

struct RoutedLds {
  __attribute__((aligned(16))) int32_t pair[kLayerPairs];   // a pair's expert, -1: none
  PairsLds p;
};

// The choice of every token, sorted by expert, into s; returns the number of experts
// with pairs.  A pair's slot is the number of pairs before it, by expert, then by pair.
// WRITE: ids, weights and the plan to memory as well.
template <int L, int NV, bool WRITE>
__device__ __forceinline__ int route_few(const RouteCall& c, RoutedLds& s) {
  const int p = threadIdx.x, tokens = (int)c.tokens;
  s.pair[p] = s.p.expert[p] = -1;
  __syncthreads();
  if constexpr (WRITE) {
    const int l = threadIdx.x % L, group = threadIdx.x / L;
    for (int t = group; t - group < tokens; t += 256 / L) {
      const bool live = t < tokens;
      if (__ballot(live) == 0) break;
      int id;
      float w;
      choose<L, NV>(c, t, live, l, id, w);
      if (live && l < c.topk) {
        s.pair[t * c.topk + l] = id;
        c.ids[t * c.topk + l] = id;
        c.weights[t * c.topk + l] = w;
      }
    }
  } else {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    auto few = [&](auto Q) __attribute__((always_inline)) {
      int id[decltype(Q)::value];
      choose_wave<L * NV / 64>(c, wave, id);
#pragma unroll
      for (int q = 0; q < decltype(Q)::value; ++q)
        if (lane < c.topk && wave + 4 * q < tokens) s.pair[(wave + 4 * q) * c.topk + lane] = id[q];
    };
    static_assert(kLayerTokens == 16, "four tokens a wave");
    if (tokens > 4) few(std::integral_constant<int, 4>{});
    else few(std::integral_constant<int, 1>{});
  }
  __syncthreads();
  const int pairs = tokens * c.topk, e = s.pair[p];
  const int4* four = reinterpret_cast<const int4*>(s.pair);
  auto before = [](int f, int q, int x, int at) __attribute__((always_inline)) {   // pair q of expert f before pair at of x
    return f >= 0 && (f < x || (f == x && q < at)) ? 1 : 0;
  };
  auto count = [&](int x, int at) __attribute__((always_inline)) {
    int n = 0;
#pragma unroll 4
    for (int q = 0; q < pairs; q += 4) {
      const int4 f = four[q / 4];   // (behind the last pair: -1)
      n += before(f.x, q, x, at) + before(f.y, q + 1, x, at) + before(f.z, q + 2, x, at) + before(f.w, q + 3, x, at);
    }
    return n;
  };
  if (e >= 0) {
    const int slot = count(e, p), t = p / c.topk;
    s.p.expert[slot] = e;
    s.p.token[slot] = t;
    if constexpr (WRITE) {
      c.slots[p] = slot;
      c.rows[slot] = t;
    }
  } else if (WRITE && p < pairs) {
    c.slots[p] = -1;
  }
  if constexpr (WRITE) {
    for (int x = p; x <= c.experts; x += 256) c.offsets[x] = count(x, 0);
  }
  __syncthreads();
  return list_items<kLayerTokens>(s.p);
}

// The kernel for a layer's number of experts: lanes a token times keys a lane.
template <typename F>
hipError_t with_routed(const RouteCall& c, F&& f) {
  if (c.experts <= 64) return f(RoutedRows<16, 4>{c, c.tokens * c.topk, c.tokens});
  if (c.experts <= 128) return f(RoutedRows<16, 8>{c, c.tokens * c.topk, c.tokens});
  if (c.experts <= 192) return f(RoutedRows<16, 12>{c, c.tokens * c.topk, c.tokens});
  if (c.experts <= 256) return f(RoutedRows<16, 16>{c, c.tokens * c.topk, c.tokens});
  return f(RoutedRows<64, 16>{c, c.tokens * c.topk, c.tokens});
}
// Blocks: the plan's, then one for each of `ntiles` tiles of every expert that can have
// pairs, or as many as a CU holds at once (`resident`) on every CU.
inline int64_t routed_grid(const RouteCall& c, int64_t ntiles, int resident) {
  const int64_t pairs = c.tokens * c.topk, tiles = ntiles * (pairs < c.experts ? pairs : c.experts);
  const int64_t most = (int64_t)device_cus() * resident;
  return 1 + (tiles < most ? tiles : most);
}

}  // namespace
}  // namespace uw
