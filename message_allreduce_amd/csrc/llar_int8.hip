// llar_int8.hip -- host side of the 8-bit products declared in include/llar.h.
#include "llar_ffn_host.h"
#include "llar_int8.h"

namespace {

int64_t round16(int64_t v) { return cdiv(v, 16) * 16; }

// A matrix of whole numbers with contiguous rows.
int check8(const llar_matrix* m) {
  const int st = check(m);
  if (st != LLAR_OK) return st;
  if (m->rows == 0 || m->cols == 0) return LLAR_OK;
  return row_major(m) ? LLAR_OK : LLAR_ERR_UNSUPPORTED;
}

Operand operand8(const llar_matrix* m) {
  Operand o;
  o.p = m->data;
  o.rows = m->rows;
  o.k = m->cols;
  o.ld = m->rows <= 1 ? round16(m->cols) : m->row_stride;
  return o;
}

// The tiles, or the kernel for few rows.  That one reads x anew for every 16 or 32
// columns, so it has to give way where the columns are many against the rows, and with
// more than 16 rows also where they are few against k, which only a split of k, the
// tiles', spreads over the card.  The bounds lie between these points, tile and few rows,
// us; at two of them the slower one is taken (8 rows 1536 -> 11008 gated, 16 rows
// 8192 -> 16384):
//   3584 -> 8192          8 rows 11.8,  8.0   16 rows 12.0,  8.8   32 rows 12.8, 11.4
//   8192 -> 3584, gated   8 rows 20.1, 13.4   16 rows 19.6, 15.4   32 rows 20.8, 19.7
//   8192 -> 16384         8 rows 32.2, 27.0   16 rows 32.3, 33.4
//   8192 -> 28672         8 rows 48.2, 46.2   16 rows 48.7, 58.7   17 rows 50.5, 66.6
//   1536 -> 11008, gated  8 rows 12.5, 14.0   16 rows 12.8, 16.0
//   8192 -> 1024                                                   17 rows 12.0, 15.3
// More than 32 rows are always the tiles'.
Shape shape8(int64_t m, int64_t n, int64_t k, bool gated) {
  const int64_t pairs = few_pairs(n, gated);
  const bool few = m <= 8 || (m <= 16 && pairs <= 512) || (m <= kFewRows8 && pairs <= 256 && 64 * pairs >= k);
  if (few && m > 0 && n > 0 && n <= kFewColumns) return Shape{true, kTile64, 1, 1, 0};
  return choose(m, n, k, 1, 1, gated, 1, false, false);
}

// Whether the kernel for few rows quantises them itself.
bool takes_values(const Shape& sh, int64_t m, int64_t k) { return sh.few && m <= kFewValuesRows && k <= kFewValuesK; }

size_t copy8_bytes(int64_t rows, int64_t k) { return align256((size_t)rows * round16(k)); }

QuantArgs quant_args(const llar_matrix* x, int8_t* q, int64_t qld, int qpad, float* scale) {
  QuantArgs a = {};
  a.x = x->data;
  a.xld = x->row_stride;
  a.xcs = x->cols <= 1 ? 1 : x->col_stride;
  a.M = x->rows;
  a.K = (int)x->cols;
  a.q = q;
  a.qld = qld;
  a.qpad = qpad;
  a.scale = scale;
  return a;
}

struct Call8 {
  const llar_matrix* x;
  const float* x_scale;  // null: x is of the results' type
  const llar_matrix* w[2];
  const float* w_scale[2];
  int n_w;
  llar_dtype dtype;
  void* space;
  size_t bytes;
  hipStream_t stream;
};

// The checks that both products share, once the matrices themselves are.
int check_call(const Call8& c, const llar_matrix* out) {
  int st;
  if (!c.x) return LLAR_ERR_ARG;
  if (c.x_scale) {
    if ((st = check8(c.x)) != LLAR_OK) return st;
  } else if ((st = check(c.x, kGradient)) != LLAR_OK) {  // any strides
    return st;
  }
  for (int i = 0; i < c.n_w; i++)
    if ((st = check8(c.w[i])) != LLAR_OK) return st;
  if ((st = check(out, kOutput)) != LLAR_OK) return st;
  if (c.x->cols != c.w[0]->cols || out->rows != c.x->rows || out->cols != c.w[0]->rows) return LLAR_ERR_ARG;
  if (c.x->cols > kMaxInt8K) return LLAR_ERR_UNSUPPORTED;
  if (out->rows > 0 && out->cols > 0)
    for (int i = 0; i < c.n_w; i++)
      if (!c.w_scale[i]) return LLAR_ERR_ARG;
  return LLAR_OK;
}

int run8(const Call8& c, Product& p) {
  const int64_t m = c.x->rows, k = c.x->cols;
  if (m == 0 || p.w[0].rows == 0) return LLAR_OK;
  Carve space{(uint8_t*)c.space, c.bytes};
  const Shape sh = shape8(m, p.w[0].rows, k, p.gated);
  // the tiles read whole aligned chunks; the weights of a pair share their strides
  Pack8Args copies = {};
  copies.dld = round16(k);
  copies.width = (int)k;
  auto copy = [&](Operand& o) {
    const int i = copies.count++;
    copies.src[i] = (const int8_t*)o.p;
    copies.ld[i] = o.ld;
    copies.lines[i] = o.rows;
    copies.dst[i] = (int8_t*)space.take((size_t)o.rows * copies.dld);
    copies.first[i + 1] = copies.first[i] + cdiv(o.rows * (copies.dld / 16), kPack8Threads);
    o.p = copies.dst[i];
    o.ld = copies.dld;
    o.padded = true;
  };
  if (!sh.few && k > 0) {
    bool loose = false;
    for (int i = 0; i < c.n_w; i++) loose = loose || !chunks_whole(p.w[i], 1);
    for (int i = 0; loose && i < c.n_w; i++) copy(p.w[i]);
  }
  const float* x_scale = c.x_scale;
  const bool values = !c.x_scale && row_major(c.x) && takes_values(sh, m, k);
  if (values) {
    p.x[0] = operand8(c.x);
  } else if (c.x_scale) {
    p.x[0] = operand8(c.x);
    if (!sh.few && k > 0 && !chunks_whole(p.x[0], 1)) copy(p.x[0]);
    if (!space.ok) return LLAR_ERR_ARG;
    if (copies.count && launch_pack8(copies, c.stream) != hipSuccess) return LLAR_ERR_HIP;
  } else {
    const int64_t ld = round16(k);
    float* scale = (float*)space.take((size_t)m * 4);
    int8_t* q = (int8_t*)space.take((size_t)m * ld);
    if (!space.ok) return LLAR_ERR_ARG;
    if (launch_quantize(c.dtype, quant_args(c.x, q, ld, (int)ld, scale), copies, c.stream) != hipSuccess)
      return LLAR_ERR_HIP;
    x_scale = scale;
    p.x[0].p = q;
    p.x[0].rows = m;
    p.x[0].k = k;
    p.x[0].ld = ld;
    p.x[0].padded = true;
  }
  if (partial_bytes(sh.splits, m, p.N(), p.gated ? 2 : 1) > space.left) return LLAR_ERR_ARG;
  GemmArgs a = args_of(p, sh.splits, (float*)space.p);
  a.xscale = x_scale;
  for (int i = 0; i < 2; i++) a.wscale[i] = c.w_scale[std::min(i, c.n_w - 1)];
  if (sh.few) return launch_few_int8(c.dtype, p.gated, values, a, c.stream) == hipSuccess ? LLAR_OK : LLAR_ERR_HIP;
  GemmPlan plan = {};
  plan.kind = c.dtype;
  plan.tile = sh.tile;
  plan.groups = sh.groups;
  plan.gated = p.gated;
  if (launch_gemm_int8(plan, a, c.stream) != hipSuccess) return LLAR_ERR_HIP;
  if (sh.splits > 1 && launch_join_int8(c.dtype, p.gated, a, c.stream) != hipSuccess) return LLAR_ERR_HIP;
  return LLAR_OK;
}

// What a call on these inputs needs of its workspace.
size_t needed(const Call8& c, llar_ffn_op op) {
  int layout = c.x_scale ? 0 : LLAR_LAYOUT_X_VALUES;
  if (!c.x_scale && !row_major(c.x)) layout |= LLAR_LAYOUT_X_COLUMNS;
  if (c.x_scale && !chunks_whole(operand8(c.x), 1)) layout |= LLAR_LAYOUT_UNALIGNED;
  for (int i = 0; i < c.n_w; i++)
    if (!chunks_whole(operand8(c.w[i]), 1)) layout |= LLAR_LAYOUT_UNALIGNED;
  return llar_int8_workspace(op, c.x->rows, c.w[0]->rows, c.x->cols, layout);
}

}  // namespace

extern "C" {

int llar_quantize_rows(const llar_matrix* x, const llar_matrix* q, float* scale, llar_dtype dtype, void* stream) {
  if (!dtype_ok(dtype)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(x, kGradient));
  LLAR_TRY(check(q, kOutput));
  if (!same_shape(x, q)) return llar::fail(LLAR_ERR_ARG);
  if (x->rows == 0) return LLAR_OK;
  if (!scale) return llar::fail(LLAR_ERR_ARG);
  const QuantArgs a = quant_args(x, (int8_t*)q->data, q->rows <= 1 ? q->cols : q->row_stride, (int)q->cols, scale);
  LLAR_TRY(launch_quantize(dtype, a, Pack8Args{}, (hipStream_t)stream) == hipSuccess ? LLAR_OK : LLAR_ERR_HIP);
  return LLAR_OK;
}

size_t llar_int8_workspace(llar_ffn_op op, int64_t m, int64_t n, int64_t k, int layout) {
  if ((op != LLAR_OP_LINEAR && op != LLAR_OP_GATED_FFN) || m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim ||
      k > kMaxInt8K || m == 0 || n == 0)
    return 0;
  const bool gated = op == LLAR_OP_GATED_FFN, values = layout & LLAR_LAYOUT_X_VALUES;
  const Shape sh = shape8(m, n, k, gated);
  const bool rows = values && !((layout & LLAR_LAYOUT_X_COLUMNS) == 0 && takes_values(sh, m, k));
  size_t need = rows ? align256((size_t)m * 4) + copy8_bytes(m, k) : 0;
  if (!sh.few && (layout & LLAR_LAYOUT_UNALIGNED))
    need += (values ? 0 : copy8_bytes(m, k)) + (gated ? 2 : 1) * copy8_bytes(n, k);
  return need + partial_bytes(sh.splits, m, n, gated ? 2 : 1);
}

int llar_linear_int8(const llar_matrix* x, const float* x_scale, const llar_matrix* w, const float* w_scale,
                     const void* bias, const llar_matrix* residual, const llar_matrix* out, llar_dtype dtype,
                     llar_act act, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  const Call8 c = {x, x_scale, {w, nullptr}, {w_scale, nullptr}, 1, dtype, workspace, workspace_bytes, (hipStream_t)stream};
  LLAR_TRY(check_call(c, out));
  if (residual) {
    LLAR_TRY(check(residual));
    if (!same_shape(residual, out)) return llar::fail(LLAR_ERR_ARG);
    if (!row_major(residual)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  if (workspace_bytes < needed(c, LLAR_OP_LINEAR)) return llar::fail(LLAR_ERR_ARG);
  Product p;
  p.w[0] = operand8(w);
  p.out[0] = out->data;
  p.outld = row_ld(out);
  p.bias = bias;
  if (residual) {
    p.resid = residual->data;
    p.rld = row_ld(residual);
  }
  p.act = act;
  LLAR_TRY(run8(c, p));
  return LLAR_OK;
}

int llar_gated_ffn_int8(const llar_matrix* x, const float* x_scale, const llar_matrix* w_gate, const llar_matrix* w_up,
                        const float* gate_scale, const float* up_scale, const llar_matrix* out, llar_dtype dtype,
                        llar_act act, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  const Call8 c = {x, x_scale, {w_gate, w_up}, {gate_scale, up_scale}, 2, dtype, workspace, workspace_bytes,
                   (hipStream_t)stream};
  LLAR_TRY(check_call(c, out));
  if (!same_shape(w_gate, w_up)) return llar::fail(LLAR_ERR_ARG);
  Product p;
  p.w[0] = operand8(w_gate);
  p.w[1] = operand8(w_up);
  p.n_w = 2;
  if (p.w[0].ld != p.w[1].ld) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (workspace_bytes < needed(c, LLAR_OP_GATED_FFN)) return llar::fail(LLAR_ERR_ARG);
  p.gated = true;
  p.out[0] = out->data;
  p.outld = row_ld(out);
  p.act = act;
  LLAR_TRY(run8(c, p));
  return LLAR_OK;
}

}  // extern "C"
