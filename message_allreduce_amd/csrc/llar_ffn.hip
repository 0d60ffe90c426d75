// llar_ffn.hip -- host side of the feed-forward operators declared in
// include/llar.h: argument checks, tile and split choice, launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "llar.h"
#include "llar_ffn.h"
#include "llar_internal.h"

using namespace llar_ffn;

namespace {

constexpr int64_t kMaxDim = 1 << 30;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int elem_size(int dtype) { return dtype == LLAR_FP32 ? 4 : 2; }

// A matrix as an operand: rows x k, contiguous along k or along the rows.
struct Operand {
  const void* p = nullptr;
  int64_t rows = 0, k = 0, ld = 0;
  bool by_rows = false;
  Operand t() const {  // the transposed matrix
    Operand o = *this;
    o.rows = k;
    o.k = rows;
    o.by_rows = !by_rows;
    return o;
  }
};

int check(const llar_matrix* m, bool output = false) {
  if (!m) return LLAR_ERR_ARG;
  if (m->rows < 0 || m->cols < 0) return LLAR_ERR_ARG;
  if (m->rows > kMaxDim || m->cols > kMaxDim) return LLAR_ERR_UNSUPPORTED;
  if (m->rows == 0 || m->cols == 0) return LLAR_OK;
  if (!m->data || m->row_stride < 0 || m->col_stride < 0) return LLAR_ERR_ARG;
  if (output) {
    if (m->cols > 1 && m->col_stride != 1) return LLAR_ERR_UNSUPPORTED;
    if (m->rows > 1 && m->row_stride < m->cols) return LLAR_ERR_ARG;
  } else if (m->cols > 1 && m->col_stride != 1 && m->rows > 1 && m->row_stride != 1) {
    return LLAR_ERR_UNSUPPORTED;
  }
  return LLAR_OK;
}
bool row_major(const llar_matrix* m) { return m->cols <= 1 || m->col_stride == 1; }

// Row distance of a row-contiguous matrix; one row has none, so it takes one
// that keeps wide accesses possible.
int64_t row_ld(const llar_matrix* m) { return m->rows <= 1 ? cdiv(m->cols, 8) * 8 : m->row_stride; }

Operand operand(const llar_matrix* m) {
  Operand o;
  o.p = m->data;
  o.rows = m->rows;
  o.k = m->cols;
  o.by_rows = !row_major(m);
  o.ld = o.by_rows ? m->col_stride : row_ld(m);  // by rows: two columns at least
  return o;
}
bool same_shape(const llar_matrix* a, const llar_matrix* b) { return a->rows == b->rows && a->cols == b->cols; }

// Whether every 16-byte chunk of the operand's tiles is whole and aligned, and
// a tile's offsets fit the buffer loads' 31 bits.
bool chunks_whole(const Operand& o, int es) {
  const int ce = 16 / es;
  if (((uintptr_t)o.p & 15) || o.ld % ce) return false;
  if ((o.by_rows ? o.rows : o.k) % ce) return false;
  return o.ld * es < (1ll << 31) / 256;
}
bool vec8(const void* p, int64_t ld, int es) { return !p || (((uintptr_t)p & 15) == 0 && ld * es % 16 == 0); }

struct Shape {
  int tile, splits;
};

// Tile and split over k of a product with `outs` output planes of M x N and
// `kt` k tiles in all.
Shape choose(int64_t M, int64_t N, int64_t kt, int outs, bool gated, bool vec) {
  Shape s{kTile64, 1};
  auto tiles = [&](int t) { return cdiv(M, kTileM[t]) * cdiv(N, kTileN[t] / (gated ? 2 : 1)) * outs; };
  if (vec && tiles(kTile256) >= 192)
    s.tile = kTile256;
  else if (tiles(kTile128) >= 256)
    s.tile = kTile128;
  const int64_t n = tiles(s.tile);
  while (n * s.splits < 256 && s.splits < 16 && kt / (2 * s.splits) >= 4) s.splits *= 2;
  return s;
}
size_t partial_bytes(const Shape& s, int64_t M, int64_t N, int planes) {
  return s.splits <= 1 ? 0 : align256((size_t)s.splits * planes * M * (size_t)(cdiv(N, 8) * 8) * 4);
}
int64_t k_tiles(int64_t K, int es) { return cdiv(K * es, kTileKBytes); }

// The workspace of a product of this shape, whatever its operands' alignment.
size_t product_space(int64_t M, int64_t N, int64_t K, int segs, int outs, bool gated, int es) {
  size_t need = 0;
  for (int vec = 0; vec < 2; vec++) {
    const Shape s = choose(M, N, k_tiles(K, es) * segs, outs, gated, vec);
    need = std::max(need, partial_bytes(s, M, N, gated ? 2 : outs));
  }
  return need;
}

struct Product {
  Operand x[2], w[2];
  int n_x = 1, n_w = 1;  // pairs given
  int segs = 1, batch = 1;
  bool gated = false;
  void* out[2] = {nullptr, nullptr};
  int64_t outld = 0;
  void* z[2] = {nullptr, nullptr};
  int64_t zld = 0;
  const void* bias = nullptr;
  const void* resid = nullptr;
  int64_t rld = 0;
  int act = kActNone;
};

int run_product(const Product& p, int dtype, void* space, size_t space_bytes, hipStream_t s) {
  const int es = elem_size(dtype);
  GemmArgs a = {};
  a.M = (int)p.x[0].rows;
  a.N = (int)p.w[0].rows;
  a.K = (int)p.x[0].k;
  if (a.M == 0 || a.N == 0) return LLAR_OK;
  bool vec = true, vec_out = true;
  for (int i = 0; i < 2; i++) {
    a.x[i] = p.x[std::min(i, p.n_x - 1)].p;
    a.w[i] = p.w[std::min(i, p.n_w - 1)].p;
    a.out[i] = p.out[i];
    a.z[i] = p.z[i];
    vec = vec && (i >= p.n_x || chunks_whole(p.x[i], es)) && (i >= p.n_w || chunks_whole(p.w[i], es));
    vec_out = vec_out && vec8(p.out[i], p.outld, es) && vec8(p.z[i], p.zld, es);
  }
  a.bias = p.bias;
  a.resid = p.resid;
  a.vec_out = vec_out && vec8(p.resid, p.rld, es) && vec8(p.bias, 0, es);
  a.xld = p.x[0].ld;
  a.wld = p.w[0].ld;
  a.outld = p.outld;
  a.zld = p.zld;
  a.rld = p.rld;
  a.segs = p.segs;
  a.batch = p.batch;
  a.act = p.act;
  a.npad = (int)(cdiv(a.N, 8) * 8);
  const Shape sh = choose(a.M, a.N, k_tiles(a.K, es) * p.segs, p.batch, p.gated, vec);
  a.splits = sh.splits;
  if (sh.splits > 1) {
    if (partial_bytes(sh, a.M, a.N, p.gated ? 2 : p.batch) > space_bytes) return LLAR_ERR_ARG;
    a.partial = (float*)space;
  }
  GemmPlan plan;
  plan.kind = dtype;
  plan.tile = sh.tile;
  plan.x_rows = p.x[0].by_rows;
  plan.w_rows = p.w[0].by_rows;
  plan.vec = vec;
  plan.gated = p.gated;
  if (launch_gemm(plan, a, s) != hipSuccess) return LLAR_ERR_HIP;
  if (sh.splits > 1 && launch_join(dtype, p.gated, a, s) != hipSuccess) return LLAR_ERR_HIP;
  return LLAR_OK;
}

bool dtype_ok(int t) { return t == LLAR_FP32 || t == LLAR_FP16 || t == LLAR_BF16; }
bool act_ok(int a) { return a >= LLAR_ACT_NONE && a <= LLAR_ACT_SILU; }
int row_chunks(int64_t M, int64_t N) {
  // about 1024 workgroups of 256 columns, at least 32 rows each
  const int64_t cols = std::max<int64_t>(cdiv(N, 256), 1);
  return (int)std::max<int64_t>(1, std::min(cdiv(1024, cols), M / 32));
}

struct Carve {
  uint8_t* p;
  size_t left;
  bool ok = true;
  void* take(size_t n) {
    n = align256(n);
    if (n > left) {
      ok = false;
      return nullptr;
    }
    void* r = p;
    p += n;
    left -= n;
    return r;
  }
};
bool space_ok(void* w, size_t n) { return n == 0 || (w && ((uintptr_t)w & 255) == 0); }

}  // namespace

#define LLAR_TRY(expr)                       \
  do {                                       \
    const int st_ = (expr);                  \
    if (st_ != LLAR_OK) return llar::fail(st_); \
  } while (0)

extern "C" {

size_t llar_ffn_workspace(llar_ffn_op op, int64_t m, int64_t n, int64_t k, llar_dtype dtype) {
  if (!dtype_ok(dtype) || m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  const int es = elem_size(dtype);
  switch (op) {
    case LLAR_OP_LINEAR: return product_space(m, n, k, 1, 1, false, es);
    case LLAR_OP_GATED_FFN: return product_space(m, n, k, 1, 1, true, es);
    case LLAR_OP_LINEAR_BACKWARD:
      return align256((size_t)m * (cdiv(n, 8) * 8) * es) + align256((size_t)row_chunks(m, n) * n * 4) +
             std::max(product_space(m, k, n, 1, 1, false, es), product_space(n, k, m, 1, 1, false, es));
    case LLAR_OP_GATED_FFN_BACKWARD:
      return 2 * align256((size_t)m * (cdiv(n, 8) * 8) * es) +
             std::max(product_space(m, k, n, 2, 1, false, es), product_space(n, k, m, 1, 2, false, es));
  }
  return 0;
}

int llar_linear(const llar_matrix* x, const llar_matrix* w, const void* bias, const llar_matrix* residual,
                const llar_matrix* out, const llar_matrix* pre, llar_dtype dtype, llar_act act, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(x));
  LLAR_TRY(check(w));
  LLAR_TRY(check(out, true));
  if (x->cols != w->cols || out->rows != x->rows || out->cols != w->rows) return llar::fail(LLAR_ERR_ARG);
  if (residual) {
    LLAR_TRY(check(residual));
    if (!same_shape(residual, out)) return llar::fail(LLAR_ERR_ARG);
    if (!row_major(residual)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  if (pre) {
    LLAR_TRY(check(pre, true));
    if (!same_shape(pre, out)) return llar::fail(LLAR_ERR_ARG);
  }
  Product p;
  p.x[0] = operand(x);
  p.w[0] = operand(w);
  p.out[0] = out->data;
  p.outld = row_ld(out);
  p.bias = bias;
  if (residual) {
    p.resid = residual->data;
    p.rld = row_ld(residual);
  }
  if (pre) {
    p.z[0] = pre->data;
    p.zld = row_ld(pre);
  }
  p.act = act;
  LLAR_TRY(run_product(p, dtype, workspace, workspace_bytes, (hipStream_t)stream));
  return LLAR_OK;
}

int llar_linear_backward(const llar_matrix* dy, const llar_matrix* x, const llar_matrix* w, const llar_matrix* pre,
                         const llar_matrix* dx, const llar_matrix* dw, void* db, llar_dtype dtype, llar_act act,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(dy));
  LLAR_TRY(check(x));
  LLAR_TRY(check(w));
  if (x->cols != w->cols || dy->rows != x->rows || dy->cols != w->rows) return llar::fail(LLAR_ERR_ARG);
  const bool with_act = act != LLAR_ACT_NONE;
  if (with_act) {
    LLAR_TRY(check(pre));
    if (!same_shape(pre, dy)) return llar::fail(LLAR_ERR_ARG);
    if (!row_major(pre)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  if ((with_act || db) && !row_major(dy)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (dx) {
    LLAR_TRY(check(dx, true));
    if (!same_shape(dx, x)) return llar::fail(LLAR_ERR_ARG);
  }
  if (dw) {
    LLAR_TRY(check(dw, true));
    if (!same_shape(dw, w)) return llar::fail(LLAR_ERR_ARG);
  }
  if (workspace_bytes < llar_ffn_workspace(LLAR_OP_LINEAR_BACKWARD, x->rows, w->rows, x->cols, dtype))
    return llar::fail(LLAR_ERR_ARG);
  const int64_t M = dy->rows, N = dy->cols;
  const int es = elem_size(dtype);
  Carve c{(uint8_t*)workspace, workspace_bytes};
  Operand dz = operand(dy);
  if (with_act || db) {
    ActGradArgs a = {};
    a.M = (int)M;
    a.N = (int)N;
    a.act = act;
    a.dy = dy->data;
    a.dyld = row_ld(dy);
    a.chunks = row_chunks(M, N);
    bool vec = vec8(dy->data, a.dyld, es);
    if (with_act) {
      a.z = pre->data;
      a.zld = row_ld(pre);
      a.dzld = cdiv(N, 8) * 8;
      a.dz = c.take((size_t)M * a.dzld * es);
      vec = vec && vec8(a.z, a.zld, es);
      dz.p = a.dz;
      dz.ld = a.dzld;
    }
    if (db) {
      a.db = db;
      a.part = (float*)c.take((size_t)a.chunks * N * 4);
    }
    a.vec = vec;
    if (!c.ok) return llar::fail(LLAR_ERR_ARG);
    if (launch_act_grad(dtype, a, (hipStream_t)stream) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
  }
  if (dx) {
    Product p;
    p.x[0] = dz;
    p.w[0] = operand(w).t();
    p.out[0] = dx->data;
    p.outld = row_ld(dx);
    LLAR_TRY(run_product(p, dtype, c.p, c.left, (hipStream_t)stream));
  }
  if (dw) {
    Product p;
    p.x[0] = dz.t();
    p.w[0] = operand(x).t();
    p.out[0] = dw->data;
    p.outld = row_ld(dw);
    LLAR_TRY(run_product(p, dtype, c.p, c.left, (hipStream_t)stream));
  }
  return LLAR_OK;
}

int llar_gated_ffn(const llar_matrix* x, const llar_matrix* w_gate, const llar_matrix* w_up, const llar_matrix* out,
                   const llar_matrix* gate, const llar_matrix* up, llar_dtype dtype, llar_act act, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(x));
  LLAR_TRY(check(w_gate));
  LLAR_TRY(check(w_up));
  LLAR_TRY(check(out, true));
  if (!same_shape(w_gate, w_up) || x->cols != w_gate->cols || out->rows != x->rows || out->cols != w_gate->rows)
    return llar::fail(LLAR_ERR_ARG);
  if (!gate != !up) return llar::fail(LLAR_ERR_ARG);
  if (gate) {
    LLAR_TRY(check(gate, true));
    LLAR_TRY(check(up, true));
    if (!same_shape(gate, out) || !same_shape(up, out)) return llar::fail(LLAR_ERR_ARG);
    if (gate->rows > 1 && gate->row_stride != up->row_stride) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  Product p;
  p.x[0] = operand(x);
  p.w[0] = operand(w_gate);
  p.w[1] = operand(w_up);
  p.n_w = 2;
  if (p.w[0].by_rows != p.w[1].by_rows || p.w[0].ld != p.w[1].ld) return llar::fail(LLAR_ERR_UNSUPPORTED);
  p.gated = true;
  p.out[0] = out->data;
  p.outld = row_ld(out);
  if (gate) {
    p.z[0] = gate->data;
    p.z[1] = up->data;
    p.zld = row_ld(gate);
  }
  p.act = act;
  LLAR_TRY(run_product(p, dtype, workspace, workspace_bytes, (hipStream_t)stream));
  return LLAR_OK;
}

int llar_gated_ffn_backward(const llar_matrix* dh, const llar_matrix* x, const llar_matrix* w_gate,
                            const llar_matrix* w_up, const llar_matrix* gate, const llar_matrix* up,
                            const llar_matrix* dx, const llar_matrix* dw_gate, const llar_matrix* dw_up,
                            llar_dtype dtype, llar_act act, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(dh));
  LLAR_TRY(check(x));
  LLAR_TRY(check(w_gate));
  LLAR_TRY(check(w_up));
  LLAR_TRY(check(gate));
  LLAR_TRY(check(up));
  if (!same_shape(w_gate, w_up) || x->cols != w_gate->cols || dh->rows != x->rows || dh->cols != w_gate->rows ||
      !same_shape(gate, dh) || !same_shape(up, dh))
    return llar::fail(LLAR_ERR_ARG);
  if (!row_major(dh) || !row_major(gate) || !row_major(up)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (!dw_gate != !dw_up) return llar::fail(LLAR_ERR_ARG);
  if (dx) {
    LLAR_TRY(check(dx, true));
    if (!same_shape(dx, x)) return llar::fail(LLAR_ERR_ARG);
  }
  if (dw_gate) {
    LLAR_TRY(check(dw_gate, true));
    LLAR_TRY(check(dw_up, true));
    if (!same_shape(dw_gate, w_gate) || !same_shape(dw_up, w_gate)) return llar::fail(LLAR_ERR_ARG);
    if (dw_gate->rows > 1 && dw_gate->row_stride != dw_up->row_stride) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  const Operand wg = operand(w_gate), wu = operand(w_up);
  if (wg.by_rows != wu.by_rows || wg.ld != wu.ld) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (workspace_bytes < llar_ffn_workspace(LLAR_OP_GATED_FFN_BACKWARD, x->rows, w_gate->rows, x->cols, dtype))
    return llar::fail(LLAR_ERR_ARG);
  const int es = elem_size(dtype);
  const int64_t M = dh->rows, N = dh->cols;
  Carve c{(uint8_t*)workspace, workspace_bytes};
  GateGradArgs a = {};
  a.M = (int)M;
  a.N = (int)N;
  a.act = act;
  a.dh = dh->data;
  a.dhld = row_ld(dh);
  a.g = gate->data;
  a.gld = row_ld(gate);
  a.u = up->data;
  a.uld = row_ld(up);
  a.dld = cdiv(N, 8) * 8;
  a.dg = c.take((size_t)M * a.dld * es);
  a.du = c.take((size_t)M * a.dld * es);
  a.vec = vec8(a.dh, a.dhld, es) && vec8(a.g, a.gld, es) && vec8(a.u, a.uld, es);
  if (!c.ok) return llar::fail(LLAR_ERR_ARG);
  if (launch_gate_grad(dtype, a, (hipStream_t)stream) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
  Operand dg, du;
  dg.p = a.dg;
  dg.rows = M;
  dg.k = N;
  dg.ld = a.dld;
  du = dg;
  du.p = a.du;
  if (dx) {
    Product p;
    p.x[0] = dg;
    p.x[1] = du;
    p.w[0] = wg.t();
    p.w[1] = wu.t();
    p.n_x = p.n_w = 2;
    p.segs = 2;
    p.out[0] = dx->data;
    p.outld = row_ld(dx);
    LLAR_TRY(run_product(p, dtype, c.p, c.left, (hipStream_t)stream));
  }
  if (dw_gate) {
    Product p;
    p.x[0] = dg.t();
    p.x[1] = du.t();
    p.w[0] = operand(x).t();
    p.n_x = 2;
    p.batch = 2;
    p.out[0] = dw_gate->data;
    p.out[1] = dw_up->data;
    p.outld = row_ld(dw_gate);
    LLAR_TRY(run_product(p, dtype, c.p, c.left, (hipStream_t)stream));
  }
  return LLAR_OK;
}

}  // extern "C"
