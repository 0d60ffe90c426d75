// llar_ffn.hip -- host side of the feed-forward operators declared in
// include/llar.h: backward passes, workspaces, the calls themselves.
#include "llar_ffn_host.h"

namespace {

// Both products of a backward pass of M x N gradients and M x K inputs in one
// launch: the same tile for both, the one with more k first, and only that one
// split.  `on`: it costs less than two launches.
struct PairShape {
  bool on, dw_first;
  int tile, groups, splits;  // of the first
};

// The time n0 workgroups of d0 each and then n1 of d1 take, each of them as one
// of the slots comes free.
double list_time(int64_t n0, double d0, int64_t n1, double d1, int64_t slots) {
  const int64_t late = n0 % slots, early = slots - late;  // slots with a workgroup more, and without
  double t_early = n0 / slots * d0, t_late = t_early + d0, end = late ? t_late : t_early;
  const int64_t skip = std::max<int64_t>(0, n1 / slots - (int64_t)(d0 / d1) - 2);  // rounds that all slots take
  n1 -= skip * slots;
  t_early += skip * d1;
  t_late += skip * d1;
  while (n1 > 0) {
    if (late == 0 || t_early <= t_late) {
      n1 -= early;
      t_early += d1;
      end = std::max(end, t_early);
    } else {
      n1 -= late;
      t_late += d1;
      end = std::max(end, t_late);
    }
  }
  return end;
}

PairShape choose_pair(int64_t M, int64_t N, int64_t K, int segs, int batch, int es) {
  PairShape p{false, false, 0, 1, 1};
  if (M <= kFewRows || N == 0 || K == 0) return p;
  const int64_t ktx = k_tiles(N, es) * segs, ktw = k_tiles(M, es);
  p.dw_first = ktw > ktx;
  const int64_t kt0 = std::max(ktx, ktw), kt1 = std::min(ktx, ktw);
  if (kt0 > 64 * kt1) return p;  // nothing to fill in
  double best = choose(M, K, N, segs, 1, false, es, true, false).cost +
                choose(N, K, M, 1, batch, false, es, false, false).cost;
  each_way(es, [&](const Way& w) {
    const int64_t tm = kTileM[w.tile], tn = kTileN[w.tile];
    const int64_t nx = cdiv(M, tm) * cdiv(K, tn), nw = cdiv(N, tm) * cdiv(K, tn) * batch;
    const int64_t n0 = p.dw_first ? nw : nx, n1 = p.dw_first ? nx : nw;
    for (int splits = 1; splits <= 8 && (splits == 1 || kt0 / splits >= 2 * w.groups); splits *= 2) {
      const double step = (n0 * splits + n1 <= kCus ? w.one : w.full) * w.groups;
      const double t = kLaunch +
                       list_time(n0 * splits, w.turn + step * cdiv(cdiv(kt0, splits), w.groups), n1,
                                 w.turn + step * cdiv(kt1, w.groups), kCus * w.occ) +
                       (p.dw_first ? join_cost(splits, batch, N, K) : join_cost(splits, 1, M, K));
      if (t < best) {
        best = t;
        p = {true, p.dw_first, w.tile, w.groups, splits};
      }
    }
  });
  return p;
}

size_t product_space(int64_t M, int64_t N, int64_t K, int segs, int outs, bool gated, int es, bool x_rows,
                     bool w_rows) {
  return partial_bytes(choose(M, N, K, segs, outs, gated, es, !x_rows, w_rows).splits, M, N, gated ? 2 : outs);
}
size_t pair_space(int64_t M, int64_t N, int64_t K, int segs, int batch, int es) {
  const PairShape p = choose_pair(M, N, K, segs, batch, es);
  if (!p.on) return 0;
  return p.dw_first ? partial_bytes(p.splits, N, K, batch) : partial_bytes(p.splits, M, K, 1);
}

// The products of a backward pass: px (dx) and pw (dw), or one of them.
int run_backward(const Product* px, const Product* pw, int dtype, const Carve& space, hipStream_t s) {
  if (px && pw && !px->x[0].by_rows && pw->w[0].by_rows) {
    const PairShape sh =
        choose_pair(px->M(), px->x[0].k, px->N(), px->segs, pw->batch, elem_size(dtype));
    if (sh.on) {
      const Product& first = sh.dw_first ? *pw : *px;
      if (partial_bytes(sh.splits, first.M(), first.N(), first.batch) > space.left) return LLAR_ERR_ARG;
      PairArgs a = {};
      a.dx = args_of(*px, sh.dw_first ? 1 : sh.splits, (float*)space.p);
      a.dw = args_of(*pw, sh.dw_first ? sh.splits : 1, (float*)space.p);
      a.dw_first = sh.dw_first;
      if (launch_pair(dtype, sh.tile, sh.groups, px->w[0].by_rows, a, s) != hipSuccess) return LLAR_ERR_HIP;
      if (sh.splits > 1 && launch_join(dtype, false, sh.dw_first ? a.dw : a.dx, s) != hipSuccess) return LLAR_ERR_HIP;
      return LLAR_OK;
    }
  }
  for (const Product* p : {px, pw}) {
    const int st = p ? run_product(*p, dtype, space, s) : LLAR_OK;
    if (st != LLAR_OK) return st;
  }
  return LLAR_OK;
}

// Row chunks of the bias gradient's sums, 128 rows at a time: about 512
// workgroups of 64 columns.  Up to 512 rows one chunk does without a second
// launch (333 x 1480 fp16: 4 us of 25).
int row_chunks(int64_t M, int64_t N) {
  if (M <= 512) return 1;
  const int64_t cols = std::max<int64_t>(cdiv(N, 64), 1);
  return (int)std::max<int64_t>(1, std::min(cdiv(512, cols), cdiv(M, 128)));
}

// Whether the workspace holds what a call on these inputs needs.
bool enough(size_t bytes, llar_ffn_op op, const llar_matrix* x, const llar_matrix* w, const llar_matrix* w2,
            const llar_matrix* dy, llar_dtype dtype) {
  const int es = elem_size(dtype);
  int layout = 0;
  for (const llar_matrix* m : {x, w, w2, dy})
    if (m && !chunks_whole(operand(m), es)) layout = LLAR_LAYOUT_UNALIGNED;
  if (!row_major(x)) layout |= LLAR_LAYOUT_X_COLUMNS;
  if (!row_major(w)) layout |= LLAR_LAYOUT_W_COLUMNS;
  if (dy && !row_major(dy)) layout |= LLAR_LAYOUT_DY_COLUMNS;
  return bytes >= llar_ffn_workspace(op, x->rows, w->rows, x->cols, dtype, layout);
}

}  // namespace

extern "C" {

size_t llar_ffn_workspace(llar_ffn_op op, int64_t m, int64_t n, int64_t k, llar_dtype dtype, int layout) {
  if (!dtype_ok(dtype) || m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  const int es = elem_size(dtype);
  const bool copies = layout & LLAR_LAYOUT_UNALIGNED, xr = layout & LLAR_LAYOUT_X_COLUMNS,
             wr = layout & LLAR_LAYOUT_W_COLUMNS, yr = layout & LLAR_LAYOUT_DY_COLUMNS;
  const size_t x = copies ? copy_bytes(m, k, es) : 0, w = copies ? copy_bytes(n, k, es) : 0;
  const size_t dz = align256((size_t)m * (cdiv(n, 8) * 8) * es);
  switch (op) {
    case LLAR_OP_LINEAR: return x + w + product_space(m, n, k, 1, 1, false, es, xr, wr);
    case LLAR_OP_GATED_FFN: return x + 2 * w + product_space(m, n, k, 1, 1, true, es, xr, wr);
    case LLAR_OP_LINEAR_BACKWARD: {
      // the products read dy, or dz, whose rows are contiguous
      size_t products = 0;
      for (const bool by_columns : {false, yr})
        products = std::max({products, product_space(m, k, n, 1, 1, false, es, by_columns, !wr),
                             product_space(n, k, m, 1, 1, false, es, !by_columns, !xr),
                             by_columns || xr ? 0 : pair_space(m, n, k, 1, 1, es)});
      return x + w + (copies ? copy_bytes(m, n, es) : dz) + align256((size_t)row_chunks(m, n) * n * 4) + products;
    }
    case LLAR_OP_GATED_FFN_BACKWARD:
      return x + 2 * w + 2 * dz +
             std::max({product_space(m, k, n, 2, 1, false, es, false, !wr),
                       product_space(n, k, m, 1, 2, false, es, true, !xr),
                       xr ? 0 : pair_space(m, n, k, 2, 2, es)});
  }
  return 0;
}

int llar_linear(const llar_matrix* x, const llar_matrix* w, const void* bias, const llar_matrix* residual,
                const llar_matrix* out, const llar_matrix* pre, llar_dtype dtype, llar_act act, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(x));
  LLAR_TRY(check(w));
  LLAR_TRY(check(out, kOutput));
  if (x->cols != w->cols || out->rows != x->rows || out->cols != w->rows) return llar::fail(LLAR_ERR_ARG);
  if (residual) {
    LLAR_TRY(check(residual));
    if (!same_shape(residual, out)) return llar::fail(LLAR_ERR_ARG);
    if (!row_major(residual)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  if (pre) {
    LLAR_TRY(check(pre, kOutput));
    if (!same_shape(pre, out)) return llar::fail(LLAR_ERR_ARG);
  }
  if (!enough(workspace_bytes, LLAR_OP_LINEAR, x, w, nullptr, nullptr, dtype)) return llar::fail(LLAR_ERR_ARG);
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
  LLAR_TRY(pack_and_run(p, dtype, workspace, workspace_bytes, (hipStream_t)stream));
  return LLAR_OK;
}

int llar_linear_backward(const llar_matrix* dy, const llar_matrix* x, const llar_matrix* w, const llar_matrix* pre,
                         const llar_matrix* dx, const llar_matrix* dw, void* db, llar_dtype dtype, llar_act act,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(dy, kGradient));
  LLAR_TRY(check(x));
  LLAR_TRY(check(w));
  if (x->cols != w->cols || dy->rows != x->rows || dy->cols != w->rows) return llar::fail(LLAR_ERR_ARG);
  const bool with_act = act != LLAR_ACT_NONE;
  if (with_act) {
    LLAR_TRY(check(pre));
    if (!same_shape(pre, dy)) return llar::fail(LLAR_ERR_ARG);
    if (!row_major(pre)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  // dz is a matrix of its own with an activation, or where dy cannot be read as it is
  const bool own = with_act || (!row_major(dy) && (db || !unit_axis(dy)));
  if (own && dy->cols > kMaxLine) return llar::fail(LLAR_ERR_UNSUPPORTED);  // dz's rows
  if (dx) {
    LLAR_TRY(check(dx, kOutput));
    if (!same_shape(dx, x)) return llar::fail(LLAR_ERR_ARG);
  }
  if (dw) {
    LLAR_TRY(check(dw, kOutput));
    if (!same_shape(dw, w)) return llar::fail(LLAR_ERR_ARG);
  }
  if (!enough(workspace_bytes, LLAR_OP_LINEAR_BACKWARD, x, w, nullptr, dy, dtype)) return llar::fail(LLAR_ERR_ARG);
  const int64_t M = dy->rows, N = dy->cols;
  const int es = elem_size(dtype);
  Carve c{(uint8_t*)workspace, workspace_bytes};
  Operand dz = operand(dy);
  if (own || db) {
    ActGradArgs a = {};
    a.M = (int)M;
    a.N = (int)N;
    a.act = act;
    a.dy = dy->data;
    a.dyld = row_ld(dy);
    a.dycs = row_major(dy) ? 1 : dy->col_stride;
    a.chunks = row_chunks(M, N);
    if (with_act) {
      a.z = pre->data;
      a.zld = row_ld(pre);
    }
    if (own) {
      a.dzld = cdiv(N, 8) * 8;
      a.dz = c.take((size_t)M * a.dzld * es);
      dz.p = a.dz;
      dz.ld = a.dzld;
      dz.by_rows = false;
      dz.padded = true;
    }
    if (db) {
      a.db = db;
      a.part = (float*)c.take((size_t)a.chunks * N * 4);
    }
    if (!c.ok) return llar::fail(LLAR_ERR_ARG);
    if (launch_act_grad(dtype, a, (hipStream_t)stream) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
  }
  Product px, pw;
  px.x[0] = dz;
  px.w[0] = operand(w).t();
  pw.x[0] = dz.t();
  pw.w[0] = operand(x).t();
  Packer k(es, &c);
  if (dx) pack(px, es, k);
  if (dw) {
    if (px.x[0].p != dz.p) pw.x[0] = px.x[0].t();  // the copy that dx's product reads
    pack(pw, es, k);
  }
  LLAR_TRY(k.run(dtype, (hipStream_t)stream));
  if (dx) {
    px.out[0] = dx->data;
    px.outld = row_ld(dx);
  }
  if (dw) {
    pw.out[0] = dw->data;
    pw.outld = row_ld(dw);
  }
  LLAR_TRY(run_backward(dx ? &px : nullptr, dw ? &pw : nullptr, dtype, c, (hipStream_t)stream));
  return LLAR_OK;
}

int llar_gated_ffn(const llar_matrix* x, const llar_matrix* w_gate, const llar_matrix* w_up, const llar_matrix* out,
                   const llar_matrix* gate, const llar_matrix* up, llar_dtype dtype, llar_act act, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(x));
  LLAR_TRY(check(w_gate));
  LLAR_TRY(check(w_up));
  LLAR_TRY(check(out, kOutput));
  if (!same_shape(w_gate, w_up) || x->cols != w_gate->cols || out->rows != x->rows || out->cols != w_gate->rows)
    return llar::fail(LLAR_ERR_ARG);
  if (!gate != !up) return llar::fail(LLAR_ERR_ARG);
  if (gate) {
    LLAR_TRY(check(gate, kOutput));
    LLAR_TRY(check(up, kOutput));
    if (!same_shape(gate, out) || !same_shape(up, out)) return llar::fail(LLAR_ERR_ARG);
    if (gate->rows > 1 && gate->row_stride != up->row_stride) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  Product p;
  p.x[0] = operand(x);
  p.w[0] = operand(w_gate);
  p.w[1] = operand(w_up);
  p.n_w = 2;
  if (p.w[0].by_rows != p.w[1].by_rows || p.w[0].ld != p.w[1].ld) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (!enough(workspace_bytes, LLAR_OP_GATED_FFN, x, w_gate, w_up, nullptr, dtype))
    return llar::fail(LLAR_ERR_ARG);
  p.gated = true;
  p.out[0] = out->data;
  p.outld = row_ld(out);
  if (gate) {
    p.z[0] = gate->data;
    p.z[1] = up->data;
    p.zld = row_ld(gate);
  }
  p.act = act;
  LLAR_TRY(pack_and_run(p, dtype, workspace, workspace_bytes, (hipStream_t)stream));
  return LLAR_OK;
}

int llar_gated_ffn_backward(const llar_matrix* dh, const llar_matrix* x, const llar_matrix* w_gate,
                            const llar_matrix* w_up, const llar_matrix* gate, const llar_matrix* up,
                            const llar_matrix* dx, const llar_matrix* dw_gate, const llar_matrix* dw_up,
                            llar_dtype dtype, llar_act act, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !space_ok(workspace, workspace_bytes)) return llar::fail(LLAR_ERR_ARG);
  LLAR_TRY(check(dh, kGradient));
  LLAR_TRY(check(x));
  LLAR_TRY(check(w_gate));
  LLAR_TRY(check(w_up));
  LLAR_TRY(check(gate));
  LLAR_TRY(check(up));
  if (!same_shape(w_gate, w_up) || x->cols != w_gate->cols || dh->rows != x->rows || dh->cols != w_gate->rows ||
      !same_shape(gate, dh) || !same_shape(up, dh))
    return llar::fail(LLAR_ERR_ARG);
  if (!row_major(gate) || !row_major(up)) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (!dw_gate != !dw_up) return llar::fail(LLAR_ERR_ARG);
  if (dx) {
    LLAR_TRY(check(dx, kOutput));
    if (!same_shape(dx, x)) return llar::fail(LLAR_ERR_ARG);
  }
  if (dw_gate) {
    LLAR_TRY(check(dw_gate, kOutput));
    LLAR_TRY(check(dw_up, kOutput));
    if (!same_shape(dw_gate, w_gate) || !same_shape(dw_up, w_gate)) return llar::fail(LLAR_ERR_ARG);
    if (dw_gate->rows > 1 && dw_gate->row_stride != dw_up->row_stride) return llar::fail(LLAR_ERR_UNSUPPORTED);
  }
  const Operand wg = operand(w_gate), wu = operand(w_up);
  if (wg.by_rows != wu.by_rows || wg.ld != wu.ld) return llar::fail(LLAR_ERR_UNSUPPORTED);
  if (!enough(workspace_bytes, LLAR_OP_GATED_FFN_BACKWARD, x, w_gate, w_up, nullptr, dtype))
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
  a.dhcs = row_major(dh) ? 1 : dh->col_stride;
  a.g = gate->data;
  a.gld = row_ld(gate);
  a.u = up->data;
  a.uld = row_ld(up);
  a.dld = cdiv(N, 8) * 8;
  a.dg = c.take((size_t)M * a.dld * es);
  a.du = c.take((size_t)M * a.dld * es);
  if (!c.ok) return llar::fail(LLAR_ERR_ARG);
  if (launch_gate_grad(dtype, a, (hipStream_t)stream) != hipSuccess) return llar::fail(LLAR_ERR_HIP);
  Operand dg, du;
  dg.p = a.dg;
  dg.rows = M;
  dg.k = N;
  dg.ld = a.dld;
  dg.padded = true;
  du = dg;
  du.p = a.du;
  Product px, pw;
  px.x[0] = dg;
  px.x[1] = du;
  px.w[0] = wg.t();
  px.w[1] = wu.t();
  px.n_x = px.n_w = px.segs = 2;
  pw.x[0] = dg.t();
  pw.x[1] = du.t();
  pw.w[0] = operand(x).t();
  pw.n_x = pw.batch = 2;
  Packer k(es, &c);
  if (dx) pack(px, es, k);
  if (dw_gate) pack(pw, es, k);
  LLAR_TRY(k.run(dtype, (hipStream_t)stream));
  if (dx) {
    px.out[0] = dx->data;
    px.outld = row_ld(dx);
  }
  if (dw_gate) {
    pw.out[0] = dw_gate->data;
    pw.out[1] = dw_up->data;
    pw.outld = row_ld(dw_gate);
  }
  LLAR_TRY(run_backward(dx ? &px : nullptr, dw_gate ? &pw : nullptr, dtype, c, (hipStream_t)stream));
  return LLAR_OK;
}

}  // extern "C"
