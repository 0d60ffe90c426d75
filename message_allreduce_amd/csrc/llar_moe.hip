// llar_moe.hip -- host side of the mixture-of-experts operators declared in
// include/llar.h: argument checks, workspaces, launches.
#include "llar_ffn_host.h"
#include "llar_int8.h"
#include "llar_moe.h"

namespace {

int check_experts(const llar_experts* w) {
  if (!w || w->experts < 0 || w->rows < 0 || w->cols < 0) return LLAR_ERR_ARG;
  if (w->experts > kMoeExperts || w->rows > kMaxDim || w->cols > kMaxLine) return LLAR_ERR_UNSUPPORTED;
  if (w->experts == 0 || w->rows == 0 || w->cols == 0) return LLAR_OK;
  if (!w->data || w->expert_stride < 0 || w->row_stride < 0) return LLAR_ERR_ARG;
  return LLAR_OK;
}

int check_rows(const llar_matrix* m) {
  const int st = check(m);
  if (st != LLAR_OK) return st;
  return m->rows == 0 || row_major(m) ? LLAR_OK : LLAR_ERR_UNSUPPORTED;
}

// The workspace of one pair of launches.
struct Rooms {
  size_t xq, xs, h, hq, hs, partial;
  int64_t xld, hld, hlow, hqld;
  size_t total() const {
    return align256(xq) + align256(xs) + align256(h) + align256(hq) + align256(hs) + align256(partial);
  }
};
Rooms rooms(int64_t m, int64_t n, int64_t k, int64_t outs, int64_t experts, int top_k, int es, bool int8) {
  const int64_t tokens = std::min<int64_t>(m, kMoeTokens), choices = tokens * top_k;
  Rooms r = {};
  // the last tokens of a long batch are fewer and may be shared between more
  for (const int64_t t : {tokens, m % kMoeTokens}) {
    const int parts = moe_parts((int)t, n, outs, experts, top_k, int8 ? 1 : es);
    if (parts > 1) r.partial = std::max(r.partial, (size_t)parts * t * outs * 4);
  }
  if (int8) {
    r.xld = cdiv(k, 16) * 16;
    r.xq = (size_t)tokens * r.xld;
    r.xs = (size_t)tokens * 4;
    r.hld = cdiv(n, 4) * 4;
    r.h = (size_t)choices * r.hld * 4;
    r.hqld = cdiv(n, 16) * 16;
    r.hq = (size_t)choices * r.hqld;
    r.hs = (size_t)choices * 4;
  } else {
    r.hlow = cdiv(n, 16 / es) * (16 / es);
    r.hld = es == 2 ? 2 * r.hlow : r.hlow;  // 16-bit types: two numbers for each
    r.h = (size_t)choices * r.hld * es;
  }
  return r;
}

// Whether both kernels of t tokens stay below 2^32 threads: workgroups of 512 there, for 16 inner columns of a
// choice or an expert, and for 16 or 32 outputs.
bool sizes_fit(int64_t t, int64_t n, int64_t outs, int64_t experts, int top_k) {
  const int64_t slots = std::min(t * top_k, experts);
  return launchable(cdiv(n, 16) * slots, 512) && launchable(cdiv(outs, moe_wide((int)t, outs) ? 32 : 16), 512);
}

}  // namespace

extern "C" {

size_t llar_moe_route_workspace(int64_t m, int64_t experts, int64_t k) {
  if (m < 0 || experts < 0 || k < 0 || m > kMaxDim || experts > kMoeExperts || k > kMaxLine) return 0;
  if (route_small(m, experts, k)) return 0;
  return align256((size_t)route_splits(m, experts, k) * std::min(m, kRouteTokens) * experts * 8);
}

int llar_moe_route(const llar_matrix* x, const llar_matrix* router, int top_k, llar_score score, int normalize,
                   float* weights, int32_t* experts, llar_dtype dtype, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!dtype_ok(dtype) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  if ((score != LLAR_SCORE_SOFTMAX && score != LLAR_SCORE_SIGMOID) || top_k < 0) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check_rows(x));
  LLAR_TRY(check_rows(router));
  if (x->cols != router->cols || top_k > router->rows) return llar::fail(LLAR_ERR_ARG);
  if (router->rows > kMoeExperts || top_k > kMoeTopK) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (x->rows == 0 || top_k == 0) return LLAR_OK;
  if (!weights || !experts || workspace_bytes < llar_moe_route_workspace(x->rows, router->rows, x->cols))
    return llar::fail(LLAR_ERR_ARG);
  RouteArgs a = {};
  a.w = router->data;
  a.xld = row_ld(x);
  a.wld = row_ld(router);
  a.E = (int)router->rows;
  a.K = (int)x->cols;
  a.top_k = top_k;
  a.sigmoid = score == LLAR_SCORE_SIGMOID;
  a.normalize = normalize != 0;
  a.small = route_small(x->rows, a.E, a.K);
  a.splits = route_splits(x->rows, a.E, a.K);
  a.logits = (double*)workspace;
  for (int64_t t = 0; t < x->rows; t += kRouteTokens) {
    a.M = (int)std::min(kRouteTokens, x->rows - t);
    a.x = (const uint8_t*)x->data + t * a.xld * elem_size(dtype);
    a.weights = weights + t * top_k;
    a.experts = experts + t * top_k;
    LLAR_TRY(launch_route(dtype, a, (hipStream_t)stream) == hipSuccess ? LLAR_OK : LLAR_ERR_HIP);
  }
  return LLAR_OK;
}

size_t llar_moe_workspace(int64_t m, int64_t n, int64_t k, int64_t outs, int64_t experts, int top_k, llar_dtype dtype,
                          int int8) {
  if (!dtype_ok(dtype) || m < 0 || n < 0 || k < 0 || outs < 0 || experts < 0 || m > kMaxDim || n > kMaxLine ||
      k > kMaxLine || outs > kMaxDim || experts > kMoeExperts || top_k < 0 || top_k > kMoeTopK)
    return 0;
  return rooms(m, n, k, outs, experts, top_k, elem_size(dtype), int8 != 0).total();
}

int llar_moe_ffn(const llar_matrix* x, const void* expert_ids, int id_bytes, const float* weights, int top_k,
                 const llar_experts* w_gate, const llar_experts* w_up, const llar_experts* w_down,
                 const float* gate_scale, const float* up_scale, const float* down_scale, const llar_matrix* residual,
                 const llar_matrix* out, llar_dtype dtype, llar_act act, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  if ((id_bytes != 4 && id_bytes != 8) || top_k < 0) return llar::fail(LLAR_ERR_ARG);
  if (top_k > kMoeTopK) return llar::fail(LLAR_ERR_UNSUPPORTED);
  const bool int8 = gate_scale || up_scale || down_scale;
  if (int8 && !(gate_scale && up_scale && down_scale)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(int8 ? check(x, kGradient) : check_rows(x));
  for (const llar_experts* w : {w_gate, w_up, w_down}) LLAR_TRY(check_experts(w));
  LLAR_TRY(check(out, kOutput));
  if (w_up->experts != w_gate->experts || w_up->rows != w_gate->rows || w_up->cols != w_gate->cols ||
      w_down->experts != w_gate->experts || w_down->cols != w_gate->rows || x->cols != w_gate->cols ||
      out->rows != x->rows || out->cols != w_down->rows)
    return llar::fail(LLAR_ERR_ARG);
  if (w_up->expert_stride != w_gate->expert_stride || w_up->row_stride != w_gate->row_stride)
    return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (int8 && (x->cols > kMaxInt8K || w_down->cols > kMaxInt8K)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (residual) {
    LLAR_TRY(check_rows(residual));
    if (!same_shape(residual, out)) return llar::fail(LLAR_ERR_ARG);
  }
  if (out->rows == 0 || out->cols == 0) return LLAR_OK;
  if (top_k > 0 && (!expert_ids || !weights)) return llar::fail(LLAR_ERR_ARG);
  const int es = elem_size(dtype);
  const int64_t n = w_gate->rows, k = x->cols;
  for (const int64_t t : {std::min<int64_t>(x->rows, kMoeTokens), x->rows % kMoeTokens})
    if (!sizes_fit(t, n, out->cols, w_gate->experts, top_k)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  const Rooms room = rooms(x->rows, n, k, out->cols, w_gate->experts, top_k, es, int8);
  if (workspace_bytes < room.total()) return llar::fail(LLAR_ERR_ARG);
  const hipStream_t s = (hipStream_t)stream;

  Carve c{(uint8_t*)workspace, workspace_bytes};
  int8_t* const xq = (int8_t*)c.take(room.xq);
  float* const xs = (float*)c.take(room.xs);
  void* const h = c.take(room.h);
  int8_t* const hq = (int8_t*)c.take(room.hq);
  float* const hs = (float*)c.take(room.hs);
  float* const partial = (float*)c.take(room.partial);
  if (!c.ok) return llar::fail(LLAR_ERR_ARG);

  MoeArgs a = {};
  a.w[0] = w_gate->data;
  a.w[1] = w_up->data;
  a.wd = w_down->data;
  a.wscale[0] = gate_scale;
  a.wscale[1] = up_scale;
  a.dscale = down_scale;
  a.w_expert = w_gate->expert_stride;
  a.wld = w_gate->row_stride;
  a.d_expert = w_down->expert_stride;
  a.dld = w_down->row_stride;
  a.K = (int)k;
  a.N = (int)n;
  a.outs = (int)out->cols;
  a.E = (int)w_gate->experts;
  a.top_k = top_k;
  a.id_bytes = id_bytes;
  a.act = act;
  a.outld = row_ld(out);
  a.rld = residual ? row_ld(residual) : 0;
  const int64_t xld = x->rows <= 1 ? k : x->row_stride;
  for (int64_t t = 0; t < x->rows; t += kMoeTokens) {
    a.T = (int)std::min<int64_t>(kMoeTokens, x->rows - t);
    a.ids = (const uint8_t*)expert_ids + t * top_k * id_bytes;
    a.weights = weights + t * top_k;
    a.parts = moe_parts(a.T, n, a.outs, a.E, top_k, int8 ? 1 : es);
    a.partial = partial;
    a.resid = residual ? (const uint8_t*)residual->data + t * a.rld * es : nullptr;
    a.out = (uint8_t*)out->data + t * a.outld * es;
    const void* rows = (const uint8_t*)x->data + t * xld * es;
    // few rows are quantised by the kernels that read them: two launches less (1 token, 8 of
    // 64 experts 4096 x 1024: 16.7 + 10.4 us and 4 for each quantisation, now 17.8 + 11.8)
    const bool x_values = int8 && a.T <= kMoeValuesTokens && k <= kMoeValuesK && row_major(x);
    const bool h_values = int8 && a.T <= kMoeValuesRows && a.T * top_k <= kMoeValuesRows && a.T * top_k * n <= kMoeValuesBytes;
    if (int8 && !x_values) {
      QuantArgs q = {};
      q.x = rows;
      q.xld = xld;
      q.xcs = x->cols <= 1 ? 1 : x->col_stride;
      q.M = a.T;
      q.K = (int)k;
      q.q = xq;
      q.qld = q.qpad = (int)room.xld;
      q.scale = xs;
      if (launch_quantize(dtype, q, Pack8Args{}, s) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
      a.x = xq;
      a.xscale = xs;
      a.xld = room.xld;
    } else {
      a.x = rows;
      a.xld = xld;
    }
    a.h = h;
    a.hld = room.hld;
    a.hlow = room.hlow;
    if (launch_moe_up(dtype, int8, x_values, a, s) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
    if (int8 && !h_values) {
      // rows of choices without an expert are whatever they were, and not read
      QuantArgs q = {};
      q.x = h;
      q.xld = room.hld;
      q.xcs = 1;
      q.M = (int64_t)a.T * top_k;
      q.K = (int)n;
      q.q = hq;
      q.qld = q.qpad = (int)room.hqld;
      q.scale = hs;
      if (launch_quantize(LLAR_FP32, q, Pack8Args{}, s) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
      a.h = hq;
      a.hld = room.hqld;
      a.hscale = hs;
    }
    if (launch_moe_down(dtype, int8, h_values, a, s) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
  }
  return LLAR_OK;
}

}  // extern "C"
