// llar_ffn_host.h -- what the host sides of the feed-forward operators share:
// argument checks, operands, choice of kernel, tile and split, copies, launches.
#pragma once
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
  if (es <= 2) {  // 8-bit tiles have as many bytes and matrix instructions, of twice the k
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

size_t partial_bytes(int splits, int64_t M, int64_t N, int planes) {
  return splits <= 1 ? 0 : align256((size_t)splits * planes * M * (size_t)(cdiv(N, 8) * 8) * 4);
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
bool space_ok(void* w, size_t n) { return n == 0 || (w && ((uintptr_t)w & 255) == 0); }

}  // namespace

#define LLAR_TRY(expr)                       \
  do {                                       \
    const int st_ = (expr);                  \
    if (st_ != LLAR_OK) return llar::fail(st_); \
  } while (0)
