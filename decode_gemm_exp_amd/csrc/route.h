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

// Q tokens t, t + step, .. on L lanes each (l: this lane's place): logits v and keys, expert
// i L + l in place i; a token from `end` on has no keys.
template <int L, int NV, int Q>
__device__ __forceinline__ void load_keys(const RouteCall& c, int64_t t, int64_t step, int64_t end, int l,
                                          float (&v)[Q][NV], uint32_t (&key)[Q][NV]) {
  // all loads first, absent keys' from the row's first place (a load under a
  // condition waits for itself: twelve in a row took most of the kernel's time)
  auto at = [&](int q, int i) __attribute__((always_inline)) {
    return (t + q * step < end ? t + q * step : 0) * c.ld + (i * L + l < c.experts ? i * L + l : 0);
  };
  if (c.bf16) {
    uint16_t u[Q][NV];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i) u[q][i] = static_cast<const uint16_t*>(c.logits)[at(q, i)];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[q][i] = __builtin_bit_cast(float, (uint32_t)u[q][i] << 16);
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[q][i] = static_cast<const float*>(c.logits)[at(q, i)];
  }
  float bias[NV] = {};
  if (c.bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = c.bias[i * L + l < c.experts ? i * L + l : 0];
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = t + q * step < end && i * L + l < c.experts;
      key[q][i] = in ? order_key(v[q][i] + bias[i]) : 0u;
    }
  if (c.on_score) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = t + q * step < end && i * L + l < c.experts && order_key(v[q][i]);
        key[q][i] = in ? order_key(1.0f / (1.0f + expf(-v[q][i])) + bias[i]) : 0u;
      }
  }
}

// One token on L lanes: lane j < topk returns choice j (-1: none) and its weight.
template <int L, int NV>
__device__ __forceinline__ void choose(const RouteCall& c, int64_t t, bool live, int l, int& id, float& weight) {
  float v1[1][NV];
  uint32_t key1[1][NV];
  load_keys<L, NV>(c, t, 1, live ? t + 1 : t, l, v1, key1);
  float(&v)[NV] = v1[0];
  uint32_t(&key)[NV] = key1[0];
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

// The same choice on a whole wave as a set, without order and weights, of Q tokens t, t +
// NW, .. at once: sel[q] has bit i where this lane's expert 64 i + lane is chosen.  The
// smallest key that is chosen is found from its top bit down: of the keys not below the
// bits so far at least as many as are wanted must remain.  A step is a few compares and
// scalar bit counts, the search ends where exactly as many remain, and the tokens' chains
// run beside each other.  A block's time up to its first tile, us: one token, 8 of 64
// experts 2.6, with a round a choice as in choose 3.3; sixteen tokens 4.9, 6 of 160
// experts 7.9.
template <int NV, int NW, int Q>
__device__ __forceinline__ void choose_set(const RouteCall& c, int t, uint32_t (&sel)[Q]) {
  const int lane = threadIdx.x & 63;
  float v[Q][NV];
  uint32_t key[Q][NV], least[Q];   // at least `want` keys are not below least
  int want[Q];
  bool exact[Q], open = false;     // exact: `want` are not, no more
  auto remain = [&](int q, uint32_t from) __attribute__((always_inline)) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) n += __popcll(__ballot(key[q][i] >= from));
    return n;
  };
  load_keys<64, NV>(c, t, NW, c.tokens, lane, v, key);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int live = remain(q, 1u);   // (key 0: never chosen)
    const bool all = live <= c.topk;
    want[q] = all ? live : c.topk;
    least[q] = all ? 1u : 0u;
    exact[q] = all;
    open = open || !all;
  }
  for (int b = 31; b >= 0 && open; --b) {
    open = false;
#pragma unroll
    for (int q = 0; q < Q; ++q) {   // (for a token that has ended more bits change nothing; skipping it costs more)
      const uint32_t from = least[q] | 1u << b;
      const int n = remain(q, from);
      least[q] = n >= want[q] ? from : least[q];
      exact[q] = exact[q] || n == want[q];
      open = open || !exact[q];
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    // above the least key all are chosen, of the equal ones the first
    int left = want[q] - remain(q, least[q] + 1u);
    sel[q] = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint64_t same = __ballot(key[q][i] == least[q]);
      const bool first = __popcll(same & ((1ull << lane) - 1ull)) < left;
      sel[q] |= key[q][i] > least[q] || (key[q][i] == least[q] && first) ? 1u << i : 0u;
      left -= __popcll(same);
    }
  }
}

// ---- a few tokens, routed by every block for itself ----------------------------
// kLayerTokens tokens at most.  Each block makes the choice anew (2.6 to 8 us with all that
// precedes its first tile; a launch of its own takes 5.7 and the wait for it) and finds its
// experts' rows in it; block 0 writes the plan, the same that uw_route_experts writes, and
// nothing else.
template <int L, int NV>
struct RoutedRows {
  RouteCall c;
  int64_t x_rows;
};

// The pairs by expert, and the items they make: an expert and up to C of its tokens.
struct PairsLds {
  int32_t expert[kLayerPairs];                       // by slot, -1 behind the last
  int32_t token[kLayerPairs];
  float weight[kLayerPairs];
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

// What a block of the gated product knows of the choice: the experts that have pairs, by
// index, each with its tokens as bits and its first slot.
struct RoutedLds {
  uint32_t tokens[kMaxExperts];
  int32_t expert[kLayerPairs + 1];
  int32_t first[kLayerPairs + 1];
};

// The choice of every token by a block of NW waves; returns the number of experts with
// pairs.  A pair's slot is the number of pairs before it, by expert, then by token.
template <int L, int NV, int NW>
__device__ __forceinline__ int route_few(const RouteCall& c, RoutedLds& s) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tokens = (int)c.tokens;
  for (int i = threadIdx.x; i < c.experts; i += 64 * NW) s.tokens[i] = 0u;
  auto few = [&](auto Q) __attribute__((always_inline)) {
    uint32_t sel[decltype(Q)::value];
    choose_set<L * NV / 64, NW>(c, wave, sel);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < decltype(Q)::value; ++q)
      for (uint32_t left = sel[q]; left; left &= left - 1u)   // (bits: their order does not matter)
        atomicOr(&s.tokens[64 * (__ffs((int)left) - 1) + lane], 1u << (wave + NW * q));
  };
  if (tokens > NW) few(std::integral_constant<int, kLayerTokens / NW>{});
  else few(std::integral_constant<int, 1>{});
  __syncthreads();
  // every wave by itself: four experts a lane, 256 at a time
  int items = 0, slots = 0;
  for (int e0 = 0; e0 < c.experts; e0 += 256) {
    uint32_t t[4];
    int n = 0;   // pairs, and experts that have some in the upper half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + 4 * lane + i;
      t[i] = e < c.experts ? s.tokens[e] : 0u;
      n += __popc(t[i]) + (t[i] ? 1 << 16 : 0);
    }
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(upto, d);
      upto += lane >= d ? up : 0;
    }
    if (wave == 0) {
      int slot = slots + ((upto - n) & 0xFFFF), item = items + ((upto - n) >> 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t[i]) {
          s.expert[item] = e0 + 4 * lane + i;
          s.first[item++] = slot;
        }
        slot += __popc(t[i]);
      }
    }
    const int all = __builtin_amdgcn_readlane(upto, 63);
    slots += all & 0xFFFF;
    items += all >> 16;
  }
  if (threadIdx.x == 0) s.first[items] = slots;
  __syncthreads();
  return items;
}

// The same choice with its weights and the plan, to memory, by one block.
template <int L, int NV, int NW>
__device__ __forceinline__ void write_few(const RouteCall& c, RoutedLds& s) {
  const int l = threadIdx.x % L, group = threadIdx.x / L, tokens = (int)c.tokens;
  for (int t = group; t - group < tokens; t += 64 * NW / L) {
    const bool live = t < tokens;
    if (__ballot(live) == 0) break;
    int id;
    float w;
    choose<L, NV>(c, t, live, l, id, w);
    if (live && l < c.topk) {
      c.ids[t * c.topk + l] = id;
      c.weights[t * c.topk + l] = w;
    }
  }
  const int items = route_few<L, NV, NW>(c, s);
  // which of a token's choices an expert is, the ids say, which this block has just written
  __threadfence_block();
  __syncthreads();
  for (int p = threadIdx.x; p < tokens * c.topk; p += 64 * NW) {
    const int id = c.ids[p], t = p / c.topk;
    int slot = -1;
    if (id >= 0) {
      int lo = 0, hi = items - 1;   // the expert's item
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.expert[mid] < id) lo = mid + 1;
        else hi = mid;
      }
      slot = s.first[lo] + __popc(s.tokens[id] & ((1u << t) - 1u));
      c.rows[slot] = t;
    }
    c.slots[p] = slot;
  }
  for (int x = threadIdx.x; x <= c.experts; x += 64 * NW) {
    int lo = 0, hi = items;   // the first item from expert x on
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s.expert[mid] < x) lo = mid + 1;
      else hi = mid;
    }
    c.offsets[x] = s.first[lo];
  }
}

// the place of the n-th set bit (n below their number) of sixteen
__device__ __forceinline__ int nth_bit(uint32_t bits, int n) {
  int at = 0;
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const int low = __popc(bits & ((1u << w) - 1u));
    const bool up = n >= low;
    n -= up ? low : 0;
    bits = up ? bits >> w : bits;
    at += up ? w : 0;
  }
  return at;
}

// The kernel for a layer's number of experts: lanes a token times keys a lane.
template <typename F>
hipError_t with_routed(const RouteCall& c, F&& f) {
  if (c.experts <= 64) return f(RoutedRows<16, 4>{c, c.tokens});
  if (c.experts <= 128) return f(RoutedRows<16, 8>{c, c.tokens});
  if (c.experts <= 192) return f(RoutedRows<16, 12>{c, c.tokens});
  if (c.experts <= 256) return f(RoutedRows<16, 16>{c, c.tokens});
  return f(RoutedRows<64, 16>{c, c.tokens});
}
// Blocks: the plan's, then one for each of `ntiles` tiles of every expert that can have
// pairs, or `resident` on every CU where that is fewer.  (us with 4 / 2 / 8 a CU / one a
// tile, BF16, 16 tokens, 64 experts 1408x2048: 112 / 124 / 118 / 141; MXFP4, 160 experts,
// with 2 / one a tile: 56 / 97.  Fewer blocks that all take the same number of tiles leave
// less on its way: layer of one token, two of eight BF16 experts 14336x4096 133 -> 140,
// eight of 64 FP8 experts 20.1 -> 21.5.)
inline int64_t routed_grid(const RouteCall& c, int64_t ntiles, int resident) {
  const int64_t pairs = c.tokens * c.topk, tiles = ntiles * (pairs < c.experts ? pairs : c.experts);
  const int64_t most = (int64_t)device_cus() * resident;
  return 1 + (tiles < most ? tiles : most);
}

}  // namespace
}  // namespace uw
