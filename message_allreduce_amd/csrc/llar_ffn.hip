// llar_ffn.hip -- host side of the feed-forward operators declared in
// include/llar.h: argument checks, tile and split choice, launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "llar.h"
#include "llar_ffn.h"
#include "llar_internal.h"

using namespace llar_ffn;

namespace {

constexpr int64_t kMaxDim = 1 << 30;
// a tile's 256 lines are addressed with 31 bits: lines of less than 8 MiB
constexpr int64_t kMaxLine = (1 << 21) - 8;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int elem_size(int dtype) { return dtype == LLAR_FP32 ? 4 : 2; }

// A matrix as an operand: rows x k, contiguous along k or along the rows.
struct Operand {
  const void* p = nullptr;
  int64_t rows = 0, k = 0, ld = 0;
  bool by_rows = false;
  bool padded = false;  // zeros follow every line up to a whole chunk
  Operand t() const {  // the transposed matrix
    Operand o = *this;
    o.rows = k;
    o.k = rows;
    o.by_rows = !by_rows;
    return o;
  }
};

bool row_major(const llar_matrix* m) { return m->cols <= 1 || m->col_stride == 1; }

bool unit_axis(const llar_matrix* m) {
  return m->cols <= 1 || m->col_stride == 1 || m->rows <= 1 || m->row_stride == 1;
}

enum Use { kInput, kGradient, kOutput };  // a gradient may have any strides
int check(const llar_matrix* m, Use use = kInput) {
  if (!m) return LLAR_ERR_ARG;
  if (m->rows < 0 || m->cols < 0) return LLAR_ERR_ARG;
  if (m->rows > kMaxDim || m->cols > kMaxDim) return LLAR_ERR_UNSUPPORTED;
  if (m->rows == 0 || m->cols == 0) return LLAR_OK;
  if (!m->data || m->row_stride < 0 || m->col_stride < 0) return LLAR_ERR_ARG;
  if (use == kOutput) {
    if (m->cols > 1 && m->col_stride != 1) return LLAR_ERR_UNSUPPORTED;
    if (m->rows > 1 && m->row_stride < m->cols) return LLAR_ERR_ARG;
  } else if (use == kInput && !unit_axis(m)) {
    return LLAR_ERR_UNSUPPORTED;
  }
  if (use != kOutput && (row_major(m) ? m->cols : m->rows) > kMaxLine) return LLAR_ERR_UNSUPPORTED;
  return LLAR_OK;
}

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

// Whether every 16-byte chunk of the operand's lines is whole and aligned, and
// a tile's offsets fit the buffer loads' 31 bits.
bool chunks_whole(const Operand& o, int es) {
  const int ce = 16 / es;
  if (((uintptr_t)o.p & 15) || o.ld % ce) return false;
  if (!o.padded && (o.by_rows ? o.rows : o.k) % ce) return false;
  return o.ld * es < (1ll << 31) / 256;
}

// How a product runs: the kernel for few rows, or tiles; and its split over k.
struct Shape {
  bool few;
  int tile, groups, splits;
  double cost;  // us, by the measured costs below; 0 where there is no choice
};

// What the tiles cost (us): `one` is what a k tile takes a workgroup alone on
// its CU, `full` what it takes `occ` of them together, `turn` the first loads and
// the results.  Measured on MI355X at 32 .. 4096 rows, 600 .. 8192 columns,
// k 336 .. 8192.
struct Way {
  int tile, groups, occ;
  double one, full, turn;
};
template <class F>
void each_way(int es, F f) {
  static constexpr Way ways16[] = {{kTile256, 1, 1, 1.42, 1.42, 4},       {kTile128, 2, 1, 0.55, 0.55, 2.5},
                                   {kTile128, 1, 2, 0.78, 1.08, 2.5},     {kTile64, 1, 2, 0.37, 0.50, 1.5},
                                   {kTile128x64, 2, 1, 0.38, 0.38, 2.3}, {kTile64, 2, 1, 0.24, 0.24, 1.7},
                                   {kTile64, 4, 1, 0.26, 0.26, 2}};
  static constexpr Way ways32[] = {{kTile128, 2, 1, 1.36, 1.36, 2.5}, {kTile128, 1, 2, 1.75, 2.57, 2.5},
                                   {kTile64, 1, 4, 0.78, 1.70, 1.5},  {kTile64, 2, 2, 0.50, 0.82, 1.7},
                                   {kTile64, 4, 1, 0.43, 0.43, 2}};
  if (es == 2) {
    for (const Way& w : ways16) f(w);
  } else {
    for (const Way& w : ways32) f(w);
  }
}
constexpr int kCus = 256;
constexpr double kLaunch = 2;
// a second launch, and the planes it joins, written and read at 4 TB/s
double join_cost(int splits, int planes, int64_t M, int64_t N) {
  return splits > 1 ? 4 + (double)splits * planes * M * N * 8 / 4e6 : 0;
}
int64_t k_tiles(int64_t K, int es) { return cdiv(K, 128 / es); }

// `segs`: products added; `outs`: output planes; `few`: x is k-contiguous, so
// that few rows of it, one matrix fragment, may go the direct way.  Both ways at
// 16 and 17 rows, cold weights, bf16: 2048 x 2048 6.8 and 10.9 us, 8192 x 3584
// 17.2 and 17.0, contiguous along n 10.7 and 10.8, 20.3 and 19.1.
Shape choose(int64_t M, int64_t N, int64_t K, int segs, int outs, bool gated, int es, bool few, bool w_rows) {
  Shape s{false, kTile64, 1, 1, 0};
  if (M == 0 || N == 0) return s;  // nothing to launch
  if (few && M <= kFewRows && N <= kFewColumns && outs == 1) {
    s.few = true;
    if (w_rows) {
      // two workgroups a CU want 512; a split leaves every wave four steps
      const int64_t groups = cdiv(N, 64), steps = cdiv(K, 32) * segs / (8 * 4);
      if (groups < 256) s.splits = (int)std::max<int64_t>(1, std::min<int64_t>({cdiv(512, groups), steps, 16}));
    }
    return s;
  }
  s.cost = -1;
  each_way(es, [&](const Way& w) {
    const int64_t tiles = cdiv(M, kTileM[w.tile]) * cdiv(N, kTileN[w.tile] / (gated ? 2 : 1)) * outs;
    const int64_t kt = k_tiles(K, es) * segs;
    for (int splits = 1; splits <= 16 && (splits == 1 || kt / splits >= 2 * w.groups); splits *= 2) {
      const int64_t wgs = tiles * splits, all = kCus * w.occ, rest = wgs % all;
      double tile = (double)(wgs / all) * w.full;
      if (rest > 0) tile += w.one + (rest > kCus ? (w.full - w.one) * (rest - kCus) / (all - kCus) : 0);
      const double t = kLaunch + cdiv(wgs, all) * w.turn + tile * w.groups * cdiv(cdiv(kt, splits), w.groups) +
                       join_cost(splits, gated ? 2 : outs, M, N);
      if (s.cost < 0 || t < s.cost) s = {false, w.tile, w.groups, splits, t};
    }
  });
  return s;
}

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

size_t partial_bytes(int splits, int64_t M, int64_t N, int planes) {
  return splits <= 1 ? 0 : align256((size_t)splits * planes * M * (size_t)(cdiv(N, 8) * 8) * 4);
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

// An upper bound of the room a copy of rows x k elements in whole chunks takes.
size_t copy_bytes(int64_t rows, int64_t k, int es) {
  return align256((size_t)(std::max(rows * (cdiv(k, 8) * 8), k * (cdiv(rows, 8) * 8))) * es);
}

// Collects operands that the tiled kernel cannot read as they are, and copies
// them in one launch.
struct Packer {
  RepackArgs a = {};
  int es;
  Carve* c;
  Packer(int es_, Carve* c_) : es(es_), c(c_) {}
  void add(Operand& o) {
    const int i = a.count++;
    const int64_t lines = o.by_rows ? o.k : o.rows, width = o.by_rows ? o.rows : o.k;
    a.src[i] = o.p;
    a.ld[i] = o.ld;
    a.lines[i] = lines;
    a.width[i] = width;
    a.dld[i] = cdiv(width, 8) * 8;
    a.dst[i] = c->take((size_t)lines * a.dld[i] * es);
    a.first[i + 1] = a.first[i] + cdiv(lines * (a.dld[i] / 8), 256);
    o.p = a.dst[i];
    o.ld = a.dld[i];
    o.padded = true;
  }
  int run(int dtype, hipStream_t s) {
    if (a.count == 0) return LLAR_OK;
    if (!c->ok) return LLAR_ERR_ARG;
    return launch_repack(dtype, a, s) == hipSuccess ? LLAR_OK : LLAR_ERR_HIP;
  }
};

struct Product {
  Operand x[2], w[2];
  int n_x = 1, n_w = 1;  // operands given
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
  int64_t M() const { return x[0].rows; }
  int64_t N() const { return w[0].rows; }
  Shape shape(int es) const {
    return choose(M(), N(), x[0].k, segs, batch, gated, es, !x[0].by_rows, w[0].by_rows);
  }
};

// Operands that the product's kernel cannot read as they are go to the packer.
void pack(Product& p, int es, Packer& k) {
  if (p.M() == 0 || p.N() == 0 || p.x[0].k == 0 || p.shape(es).few) return;
  // both of a pair change, or neither: they share their strides
  bool x = false, w = false;
  for (int i = 0; i < p.n_x; i++) x = x || !chunks_whole(p.x[i], es);
  for (int i = 0; i < p.n_w; i++) w = w || !chunks_whole(p.w[i], es);
  for (int i = 0; x && i < p.n_x; i++) k.add(p.x[i]);
  for (int i = 0; w && i < p.n_w; i++) k.add(p.w[i]);
}

GemmArgs args_of(const Product& p, int splits, float* partial) {
  GemmArgs a = {};
  a.M = (int)p.M();
  a.N = (int)p.N();
  a.K = (int)p.x[0].k;
  for (int i = 0; i < 2; i++) {
    a.x[i] = p.x[std::min(i, p.n_x - 1)].p;
    a.w[i] = p.w[std::min(i, p.n_w - 1)].p;
    a.out[i] = p.out[i];
    a.z[i] = p.z[i];
  }
  a.bias = p.bias;
  a.resid = p.resid;
  a.xld = p.x[0].ld;
  a.wld = p.w[0].ld;
  a.outld = p.outld;
  a.zld = p.zld;
  a.rld = p.rld;
  a.segs = p.segs;
  a.batch = p.batch;
  a.act = p.act;
  a.npad = (int)(cdiv(a.N, 8) * 8);
  a.splits = splits;
  if (splits > 1) a.partial = partial;
  return a;
}

int run_product(const Product& p, int dtype, const Carve& space, hipStream_t s) {
  if (p.M() == 0 || p.N() == 0) return LLAR_OK;
  const Shape sh = p.shape(elem_size(dtype));
  if (partial_bytes(sh.splits, p.M(), p.N(), p.gated ? 2 : p.batch) > space.left) return LLAR_ERR_ARG;
  const GemmArgs a = args_of(p, sh.splits, (float*)space.p);
  if (sh.few) {
    if (launch_few(dtype, p.w[0].by_rows, p.gated, a, s) != hipSuccess) return LLAR_ERR_HIP;
  } else {
    GemmPlan plan;
    plan.kind = dtype;
    plan.tile = sh.tile;
    plan.groups = sh.groups;
    plan.x_rows = p.x[0].by_rows;
    plan.w_rows = p.w[0].by_rows;
    plan.gated = p.gated;
    if (launch_gemm(plan, a, s) != hipSuccess) return LLAR_ERR_HIP;
  }
  if (sh.splits > 1 && launch_join(dtype, p.gated, a, s) != hipSuccess) return LLAR_ERR_HIP;
  return LLAR_OK;
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

// A product with the whole workspace to itself.
int pack_and_run(Product& p, int dtype, void* space, size_t bytes, hipStream_t s) {
  Carve c{(uint8_t*)space, bytes};
  Packer k(elem_size(dtype), &c);
  pack(p, elem_size(dtype), k);
  const int st = k.run(dtype, s);
  return st != LLAR_OK ? st : run_product(p, dtype, c, s);
}

bool dtype_ok(int t) { return t == LLAR_FP32 || t == LLAR_FP16 || t == LLAR_BF16; }
bool act_ok(int a) { return a >= LLAR_ACT_NONE && a <= LLAR_ACT_SILU; }
// Row chunks of the bias gradient's sums, 128 rows at a time: about 512
// workgroups of 64 columns.  Up to 512 rows one chunk does without a second
// launch (333 x 1480 fp16: 4 us of 25).
int row_chunks(int64_t M, int64_t N) {
  if (M <= 512) return 1;
  const int64_t cols = std::max<int64_t>(cdiv(N, 64), 1);
  return (int)std::max<int64_t>(1, std::min(cdiv(512, cols), cdiv(M, 128)));
}
bool space_ok(void* w, size_t n) { return n == 0 || (w && ((uintptr_t)w & 255) == 0); }

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

#define LLAR_TRY(expr)                       \
  do {                                       \
    const int st_ = (expr);                  \
    if (st_ != LLAR_OK) return llar::fail(st_); \
  } while (0)

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
