// experts_api.cpp -- the extern "C" entry points of the mixture-of-experts and
// MXFP4 operators (include/unweight.h): argument checks, the experts' weight
// sets, workspaces.
#include <cstring>
#include <new>
#include <vector>

#include "experts.h"

using namespace uw;

namespace {

uw_status status_of(hipError_t e) {
  if (e == hipSuccess) return UW_OK;
  return e == hipErrorOutOfMemory ? UW_ERR_NOMEM : e == hipErrorNotSupported ? UW_ERR_UNSUPPORTED : UW_ERR_DEVICE;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
uint64_t pad256(uint64_t n) { return (n + 255) / 256 * 256; }

// A shape the expert and MXFP4 kernels take: k in whole blocks of 32.  The
// tile kernels address 256 rows of a matrix, and of the output, with 31-bit byte
// offsets, so k and n stay up to 2^20; every byte count of one matrix is far
// inside 63 bits.
uw_status check_shape(int64_t n, int64_t k) {
  if (n <= 0 || k <= 0) return UW_ERR_INVALID;
  if (k % 32 != 0 || n > (1 << 20) || k > (1 << 20)) return UW_ERR_UNSUPPORTED;
  return UW_OK;
}

uw_status new_set(int32_t count, int64_t n, int64_t k, uw_experts** out) {
  if (!out) return UW_ERR_INVALID;
  *out = nullptr;
  if (count <= 0) return UW_ERR_INVALID;
  const uw_status st = check_shape(n, k);
  if (st != UW_OK) return st;
  if (count > kMaxExperts) return UW_ERR_UNSUPPORTED;
  uw_experts* h = new (std::nothrow) uw_experts();
  if (!h) return UW_ERR_NOMEM;
  h->v.count = count;
  h->v.n = n;
  h->v.k = k;
  if (hipGetDevice(&h->device) != hipSuccess) {
    (void)hipGetLastError();
    h->device = 0;   // no device: the set is host state, calls that use it fail themselves
  }
  *out = h;
  return UW_OK;
}

// the set serves calls on the current device, and a UWF1 set's matrices still
// hold the indices its table names
uw_status check_set(const uw_experts* h) {
  if (!h) return UW_ERR_INVALID;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return UW_ERR_DEVICE;
  if (dev != h->device) return UW_ERR_INVALID;
  if (h->ms)
    for (int i = 0; i < h->v.count; ++i)
      if (h->ms[i]->pidx != h->pidx[i]) return UW_ERR_STATE;
  return UW_OK;
}

struct Ragged {
  const int32_t *offsets, *rows;
  int64_t slots;
  const uint16_t* x;
  int64_t x_rows;
};

uw_status check_rows(const Ragged& r, const void* y) {
  if (r.slots == 0) return UW_OK;
  if (!r.offsets || !r.x || !y || r.slots < 0 || r.x_rows <= 0) return UW_ERR_INVALID;
  if (r.slots > INT32_MAX || r.x_rows > INT32_MAX) return UW_ERR_UNSUPPORTED;
  if (!aligned(r.offsets, 4) || !aligned(r.rows, 4) || !aligned(r.x, 16) || !aligned(y, 16)) return UW_ERR_INVALID;
  // without row indices slot s is row s
  if (!r.rows && r.x_rows < r.slots) return UW_ERR_INVALID;
  return UW_OK;
}

uw_status run_experts(const uw_experts* w, const uw_experts* u, const Ragged& r, void* y, hipStream_t s) {
  ExpertsCall c{};
  c.w = w->v;
  c.gated = u != nullptr;
  c.u = u ? u->v : w->v;
  if (u) {
    if (u->v.count != w->v.count || u->v.n != w->v.n || u->v.k != w->v.k) return UW_ERR_INVALID;
    if (u->v.form != w->v.form) {
      if (!form_is_pal(u->v.form) || !form_is_pal(w->v.form)) return UW_ERR_UNSUPPORTED;
      c.w.form = c.u.form = kFormPal;   // the general lookup serves a run as well
    }
  }
  if (r.slots == 0) return UW_OK;
  c.r = RaggedRows{r.offsets, r.rows, r.slots, r.x_rows};
  c.x = r.x;
  c.y = y;
  return status_of(launch_experts(c, s));
}

// Up to this many rows x's 4-bit values go through the register-fed kernel as
// BF16; beyond, both operands stay in 4 bits.  (The header names this number: the
// two differ where a weight's value overflows BF16.)  Measured (us, register-fed /
// 4-bit tiles, x's conversion included):
//   rows           1            8            16           64            128
//   4096x4096      10.4 / 14.4  10.8 / 15.0  11.3 / 15.4  11.3 / 19.3   16.5 / 19.9
//   14336x4096     11.1 / 16.2  11.3 / 16.8  11.8 / 17.2  28.1 / 20.4   47.3 / 21.8
//   5001x8224                   16.6 / 35.1  16.9 / 35.7  26.2 / 41.9   45.4 / 42.5
//   28672x8192     30.0 / 46.1  34.5 / 47.1  37.3 / 48.1  108.2 / 55.4  123.9 / 55.5
// (14336x4096 at 32 rows 15.4 / 17.9.)  So the register-fed kernel is the right one
// up to this many rows, and could serve more: the border lies between 32 and 128
// rows and moves with the blocks that the tiles make.
constexpr int64_t kMx4RowsMax = 8;

uw_status check_route(int64_t tokens, int32_t experts, int32_t topk) {
  if (tokens < 0 || experts <= 0 || topk <= 0 || topk > experts) return UW_ERR_INVALID;
  if (experts > kMaxExperts || topk > kMaxTopk || tokens > INT32_MAX / topk) return UW_ERR_UNSUPPORTED;
  return UW_OK;
}

uw_status run_route(RouteCall& c, void* ws, size_t ws_bytes, hipStream_t s) {
  // without tokens only the offsets are written
  if (!c.offsets || (c.tokens != 0 && (!c.rows || !c.slots))) return UW_ERR_INVALID;
  size_t need = 0;
  const uw_status st = uw_workspace_size_route(c.tokens, c.experts, c.topk, &need);
  if (st != UW_OK) return st;
  if (need && (!ws || ws_bytes < need)) return UW_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return UW_ERR_INVALID;
  c.hist = static_cast<int32_t*>(ws);
  return status_of(launch_route(c, s));
}

}  // namespace

extern "C" {

uw_status uw_quantize_mx4(const void* src_dev, uw_type src_type, int64_t rows, int64_t cols, int64_t ld,
                          uint8_t* elem_dev, uint8_t* scale_dev, void* stream) {
  if (rows == 0) return UW_OK;
  if (!src_dev || !elem_dev || !scale_dev || rows < 0) return UW_ERR_INVALID;
  if (src_type != UW_TYPE_BF16 && src_type != UW_TYPE_F32) return UW_ERR_INVALID;
  const uw_status st = check_shape(rows, cols);
  if (st != UW_OK) return st;
  if (ld < cols) return UW_ERR_INVALID;
  if (ld % 8 != 0) return UW_ERR_UNSUPPORTED;
  if (!aligned(src_dev, 16) || !aligned(elem_dev, 16) || !aligned(scale_dev, 4)) return UW_ERR_INVALID;
  return status_of(launch_quantize_mx4(src_dev, src_type == UW_TYPE_F32, rows, cols, ld, elem_dev, scale_dev,
                                       static_cast<hipStream_t>(stream)));
}

uw_status uw_dequantize_mx4(const uint8_t* elem_dev, const uint8_t* scale_dev, int64_t rows, int64_t cols,
                            uint16_t* out_dev, int64_t ld, void* stream) {
  if (rows == 0) return UW_OK;
  if (!elem_dev || !scale_dev || !out_dev || rows < 0) return UW_ERR_INVALID;
  const uw_status st = check_shape(rows, cols);
  if (st != UW_OK) return st;
  if (ld < cols) return UW_ERR_INVALID;
  if (ld % 8 != 0) return UW_ERR_UNSUPPORTED;
  if (!aligned(elem_dev, 16) || !aligned(scale_dev, 4) || !aligned(out_dev, 16)) return UW_ERR_INVALID;
  return status_of(
      launch_dequantize_mx4(elem_dev, scale_dev, rows, cols, out_dev, ld, static_cast<hipStream_t>(stream)));
}

uw_status uw_workspace_size_mx4(int64_t n, int64_t k, int64_t batch, uw_activation act, size_t* bytes) {
  if (!bytes || batch < 0 || (act != UW_ACT_BF16 && act != UW_ACT_MX4)) return UW_ERR_INVALID;
  const uw_status st = check_shape(n, k);
  if (st != UW_OK) return st;
  // (refused here rather than at a launch, so that nothing has run yet; tiles are 64 rows of 256 at least)
  if (batch > INT32_MAX || !grid_fits((batch + 63) / 64 * ((n + 255) / 256), 512)) return UW_ERR_UNSUPPORTED;
  const uint64_t b = (uint64_t)batch;
  *bytes = act != UW_ACT_MX4     ? 0
           : batch <= kMx4RowsMax ? pad256(2 * b * (uint64_t)k)
                                  : pad256(b * (uint64_t)(k / 2)) + pad256(b * (uint64_t)mx4_scale_stride(k));
  return UW_OK;
}

uw_status uw_matmul_mx4(const uint8_t* elem_dev, const uint8_t* scale_dev, int64_t n, int64_t k,
                        const uint16_t* x_dev, int64_t batch, float* y_dev, uw_activation act, void* ws_dev,
                        size_t ws_bytes, void* stream) {
  if (batch == 0) return UW_OK;
  if (!elem_dev || !scale_dev || !x_dev || !y_dev) return UW_ERR_INVALID;
  size_t need = 0;
  uw_status st = uw_workspace_size_mx4(n, k, batch, act, &need);
  if (st != UW_OK) return st;
  if (!aligned(elem_dev, 16) || !aligned(scale_dev, 4) || !aligned(x_dev, 16) || !aligned(y_dev, 16) ||
      !aligned(ws_dev, 16))
    return UW_ERR_INVALID;
  if (need && (!ws_dev || ws_bytes < need)) return UW_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (act == UW_ACT_MX4 && batch > kMx4RowsMax) {
    uint8_t* xe = static_cast<uint8_t*>(ws_dev);
    uint8_t* xs = xe + pad256((uint64_t)batch * (uint64_t)(k / 2));
    st = status_of(launch_quantize_mx4(x_dev, false, batch, k, k, xe, xs, s));
    return st != UW_OK ? st : status_of(launch_mx4_tile(elem_dev, scale_dev, n, k, xe, xs, batch, y_dev, s));
  }
  if (act == UW_ACT_MX4) {
    st = status_of(launch_round_mx4(x_dev, batch, k, static_cast<uint16_t*>(ws_dev), s));
    if (st != UW_OK) return st;
    x_dev = static_cast<const uint16_t*>(ws_dev);
  }
  ExpertsCall c{};
  c.w.form = kFormMx4;
  c.w.count = 1;
  c.w.n = n;
  c.w.k = k;
  c.w.w = elem_dev;
  c.w.scale = scale_dev;
  c.u = c.w;
  c.r = RaggedRows{nullptr, nullptr, batch, batch};
  c.x = x_dev;
  c.y = y_dev;
  return status_of(launch_experts(c, s));
}

uw_status uw_experts_bf16(const uint16_t* w_dev, int32_t count, int64_t n, int64_t k, int64_t stride,
                          uw_experts** out) {
  uw_status st = new_set(count, n, k, out);
  if (st != UW_OK) return st;
  uw_experts* h = *out;
  if (stride == 0) stride = n * k;
  if (!w_dev || !aligned(w_dev, 16) || stride < n * k) st = UW_ERR_INVALID;
  else if (stride % 8 != 0 || stride > INT64_MAX / 2 / count) st = UW_ERR_UNSUPPORTED;
  if (st != UW_OK) {
    delete h;
    *out = nullptr;
    return st;
  }
  h->v.form = kFormBf16;
  h->v.w = reinterpret_cast<const uint8_t*>(w_dev);
  h->v.w_stride = 2 * stride;
  return UW_OK;
}

uw_status uw_experts_mx4(const uint8_t* elem_dev, const uint8_t* scale_dev, int32_t count, int64_t n, int64_t k,
                         int64_t elem_stride, int64_t scale_stride, uw_experts** out) {
  uw_status st = new_set(count, n, k, out);
  if (st != UW_OK) return st;
  uw_experts* h = *out;
  const int64_t eb = n * (k / 2), sb = n * mx4_scale_stride(k);
  if (elem_stride == 0) elem_stride = eb;
  if (scale_stride == 0) scale_stride = sb;
  if (!elem_dev || !scale_dev || !aligned(elem_dev, 16) || !aligned(scale_dev, 4) || elem_stride < eb ||
      scale_stride < sb)
    st = UW_ERR_INVALID;
  else if (elem_stride % 16 != 0 || scale_stride % 4 != 0 || elem_stride > INT64_MAX / count ||
           scale_stride > INT64_MAX / count)
    st = UW_ERR_UNSUPPORTED;
  if (st != UW_OK) {
    delete h;
    *out = nullptr;
    return st;
  }
  h->v.form = kFormMx4;
  h->v.w = elem_dev;
  h->v.w_stride = elem_stride;
  h->v.scale = scale_dev;
  h->v.scale_stride = scale_stride;
  return UW_OK;
}

uw_status uw_experts_uwf1(const uw_matrix* const* ms, int32_t count, void* stream, uw_experts** out) try {
  if (!out) return UW_ERR_INVALID;
  *out = nullptr;
  if (!ms || count <= 0) return UW_ERR_INVALID;
  if (count > kMaxExperts) return UW_ERR_UNSUPPORTED;
  for (int i = 0; i < count; ++i)
    if (!ms[i]) return UW_ERR_INVALID;
  for (int i = 0; i < count; ++i) {
    if (ms[i]->fp8 || ms[i]->layout != UW_LAYOUT_NK) return UW_ERR_UNSUPPORTED;
    if (ms[i]->rows != ms[0]->rows || ms[i]->cols != ms[0]->cols || ms[i]->device != ms[0]->device)
      return UW_ERR_INVALID;
    if (!ms[i]->pidx) return UW_ERR_STATE;
  }
  uw_status st = new_set(count, (int64_t)ms[0]->rows, (int64_t)ms[0]->cols, out);
  if (st != UW_OK) return st;
  uw_experts* h = *out;
  *out = nullptr;
  h->v.form = kFormPalRun;
  h->alloc = current_allocator();
  struct Guard {
    uw_experts* h;
    ~Guard() { uw_free_experts(h); }
  } guard{h};
  if (h->device != ms[0]->device) return UW_ERR_INVALID;
  h->ms = new const uw_matrix*[count];
  h->pidx = new const uint8_t*[count];
  std::vector<ExpertEntry> table(count);
  for (int i = 0; i < count; ++i) {
    const uw_matrix* m = ms[i];
    h->ms[i] = m;
    h->pidx[i] = m->pidx;
    ExpertEntry& e = table[i];
    std::memset(&e, 0, sizeof(e));
    e.sm = m->sm;
    e.pidx = m->pidx;
    e.vflags = m->vflags;
    e.vrank = m->vrank;
    e.vexp = m->vexp;
    palette_view(m, &e.pal);
    if (!e.pal.run) h->v.form = kFormPal;
  }
  void* t = nullptr;
  st = alloc_with(h->alloc, &t, sizeof(ExpertEntry) * (size_t)count);
  if (st != UW_OK) return st;
  h->table = static_cast<ExpertEntry*>(t);
  h->v.table = h->table;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipMemcpyAsync(t, table.data(), sizeof(ExpertEntry) * (size_t)count, hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return status_of(e);
  guard.h = nullptr;
  *out = h;
  return UW_OK;
} catch (...) {
  return UW_ERR_NOMEM;
}

void uw_free_experts(uw_experts* h) {
  if (!h) return;
  if (h->table) free_with(h->alloc, h->table);
  delete[] h->ms;
  delete[] h->pidx;
  delete h;
}

uw_status uw_workspace_size_route(int64_t tokens, int32_t experts, int32_t topk, size_t* bytes) {
  if (!bytes) return UW_ERR_INVALID;
  const uw_status st = check_route(tokens, experts, topk);
  if (st != UW_OK) return st;
  const int b = route_blocks(tokens, topk);
  *bytes = b > 1 ? pad256(4 * (uint64_t)b * (uint64_t)experts) : 0;
  return UW_OK;
}

uw_status uw_route_experts(const void* logits_dev, uw_type type, int64_t tokens, int32_t experts, int64_t ld,
                           const float* bias_dev, int32_t topk, uw_scoring scoring, int32_t* ids_dev,
                           float* weights_dev, int32_t* offsets_dev, int32_t* rows_dev, int32_t* slots_dev,
                           void* ws_dev, size_t ws_bytes, void* stream) {
  if (ld < experts || (tokens != 0 && (!logits_dev || !ids_dev || !weights_dev))) return UW_ERR_INVALID;
  if (type != UW_TYPE_BF16 && type != UW_TYPE_F32) return UW_ERR_INVALID;
  if (scoring != UW_SCORE_SOFTMAX && scoring != UW_SCORE_SOFTMAX_TOPK && scoring != UW_SCORE_SIGMOID &&
      scoring != UW_SCORE_SIGMOID_BIASED)
    return UW_ERR_INVALID;
  RouteCall c{};
  c.logits = logits_dev;
  c.bf16 = type == UW_TYPE_BF16;
  c.tokens = tokens;
  c.ld = ld;
  c.experts = experts;
  c.topk = topk;
  c.scoring = (int)(scoring == UW_SCORE_SIGMOID_BIASED ? UW_SCORE_SIGMOID : scoring);
  c.bias = bias_dev;
  c.on_score = scoring == UW_SCORE_SIGMOID_BIASED && bias_dev;   // (the logits' order is their sigmoids')
  c.ids = ids_dev;
  c.weights = weights_dev;
  c.offsets = offsets_dev;
  c.rows = rows_dev;
  c.slots = slots_dev;
  return run_route(c, ws_dev, ws_bytes, static_cast<hipStream_t>(stream));
}

uw_status uw_plan_experts(const int32_t* ids_dev, int64_t tokens, int32_t experts, int32_t topk,
                          int32_t* offsets_dev, int32_t* rows_dev, int32_t* slots_dev, void* ws_dev, size_t ws_bytes,
                          void* stream) {
  if (!ids_dev && tokens != 0) return UW_ERR_INVALID;
  RouteCall c{};
  c.ids_in = ids_dev;
  c.tokens = tokens;
  c.experts = experts;
  c.topk = topk;
  c.offsets = offsets_dev;
  c.rows = rows_dev;
  c.slots = slots_dev;
  return run_route(c, ws_dev, ws_bytes, static_cast<hipStream_t>(stream));
}

uw_status uw_matmul_experts(const uw_experts* w, const int32_t* offsets_dev, const int32_t* rows_dev, int64_t slots,
                            const uint16_t* x_dev, int64_t x_rows, float* y_dev, void* stream) {
  if (!w) return UW_ERR_INVALID;
  const Ragged r{offsets_dev, rows_dev, slots, x_dev, x_rows};
  uw_status st = check_rows(r, y_dev);
  if (st == UW_OK) st = check_set(w);
  return st != UW_OK ? st : run_experts(w, nullptr, r, y_dev, static_cast<hipStream_t>(stream));
}

uw_status uw_matmul_experts_gated(const uw_experts* gate, const uw_experts* up, const int32_t* offsets_dev,
                                  const int32_t* rows_dev, int64_t slots, const uint16_t* x_dev, int64_t x_rows,
                                  uint16_t* h_dev, void* stream) {
  if (!gate || !up) return UW_ERR_INVALID;
  const Ragged r{offsets_dev, rows_dev, slots, x_dev, x_rows};
  uw_status st = check_rows(r, h_dev);
  if (st == UW_OK) st = check_set(gate);
  if (st == UW_OK) st = check_set(up);
  return st != UW_OK ? st : run_experts(gate, up, r, h_dev, static_cast<hipStream_t>(stream));
}

uw_status uw_workspace_size_expert_mlp(const uw_experts* gate, const uw_experts* down, int64_t tokens, int32_t topk,
                                       size_t* bytes) {
  if (!gate || !down || !bytes) return UW_ERR_INVALID;
  if (down->v.k != gate->v.n || down->v.n != gate->v.k || down->v.count != gate->v.count) return UW_ERR_INVALID;
  const uw_status st = check_route(tokens, gate->v.count, topk);
  if (st != UW_OK) return st;
  // (the weighted sum's threads take eight outputs each)
  if (!grid_fits((tokens * (down->v.n / 8) + 255) / 256, 256)) return UW_ERR_UNSUPPORTED;
  const uint64_t pairs = (uint64_t)tokens * (uint64_t)topk;
  *bytes = pad256(2 * pairs * (uint64_t)gate->v.n) + pad256(4 * pairs * (uint64_t)down->v.n);
  return UW_OK;
}

uw_status uw_expert_mlp(const uw_experts* gate, const uw_experts* up, const uw_experts* down, int64_t tokens,
                        int32_t topk, const int32_t* offsets_dev, const int32_t* rows_dev, const int32_t* slots_dev,
                        const float* weights_dev, const uint16_t* x_dev, uint16_t* out_dev, void* ws_dev,
                        size_t ws_bytes, void* stream) {
  if (!up || (tokens != 0 && (!rows_dev || !slots_dev || !weights_dev || !out_dev))) return UW_ERR_INVALID;
  size_t need = 0;
  uw_status st = uw_workspace_size_expert_mlp(gate, down, tokens, topk, &need);
  if (st != UW_OK) return st;
  if (tokens == 0) return UW_OK;
  if (!ws_dev || ws_bytes < need) return UW_ERR_WORKSPACE;
  if (!aligned(ws_dev, 16) || !aligned(slots_dev, 4) || !aligned(weights_dev, 4)) return UW_ERR_INVALID;
  const int64_t pairs = tokens * topk;
  uint16_t* h = static_cast<uint16_t*>(ws_dev);
  float* d = reinterpret_cast<float*>(static_cast<uint8_t*>(ws_dev) + pad256(2 * (uint64_t)pairs * (uint64_t)gate->v.n));
  const Ragged in{offsets_dev, rows_dev, pairs, x_dev, tokens}, mid{offsets_dev, nullptr, pairs, h, pairs};
  st = check_rows(in, out_dev);
  if (st == UW_OK) st = check_set(gate);
  if (st == UW_OK) st = check_set(up);
  if (st == UW_OK) st = check_set(down);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (st == UW_OK) st = run_experts(gate, up, in, h, s);
  if (st == UW_OK) st = run_experts(down, nullptr, mid, d, s);
  if (st == UW_OK) st = status_of(launch_combine(d, slots_dev, weights_dev, tokens, topk, down->v.n, pairs, out_dev, s));
  return st;
}

}  // extern "C"
