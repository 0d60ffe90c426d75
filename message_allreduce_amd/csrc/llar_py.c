/* llar_py.c -- the feed-forward operators' Python entry points: reads torch
 * tensors through their Python attributes, checks them, allocates outputs and
 * workspace with torch, and makes one C call of include/llar.h.  Decoding calls
 * these for every token and layer, where the same work in Python takes longer
 * than the kernel (1 x 512 x 512 fp16: 11.3 us a call with ctypes).  Nothing is
 * kept from one call for the next. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "llar.h"

enum { kMaxDims = 16 };

typedef struct {
  PyObject* obj; /* borrowed */
  void* data;
  PyObject* dtype; /* borrowed from torch's singletons */
  long device;     /* -1: not on a GPU */
  int nd;
  int64_t size[kMaxDims], stride[kMaxDims];
} tensor;

static PyObject *s_dtype, *s_get_device, *s_data_ptr, *s_shape, *s_stride, *s_new_empty, *kw_dtype;
static PyObject *t_types[3], *t_uint8, *t_int8, *t_int32, *t_int64, *f_current_device, *f_raw_stream, *e_llar;

static const char* const kActs[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};

static int read_longs(PyObject* tuple, int64_t* to) {
  if (!tuple) return -1;
  if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > kMaxDims) {
    Py_DECREF(tuple);
    PyErr_SetString(PyExc_ValueError, "a tensor with too many dimensions");
    return -1;
  }
  const int n = (int)PyTuple_GET_SIZE(tuple);
  for (int i = 0; i < n; i++) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  Py_DECREF(tuple);
  return PyErr_Occurred() ? -1 : n;
}

static int read_tensor(PyObject* t, tensor* o) {
  o->obj = t;
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) return -1;
  o->dtype = v;
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(t, s_get_device))) return -1;
  o->device = PyLong_AsLong(v);
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(t, s_data_ptr))) return -1;
  o->data = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  o->nd = read_longs(PyObject_GetAttr(t, s_shape), o->size);
  if (o->nd < 0) return -1;
  if (read_longs(PyObject_CallMethodNoArgs(t, s_stride), o->stride) < 0) return -1;
  return PyErr_Occurred() ? -1 : 0;
}

/* A (..., width) tensor as a matrix that shares its memory. */
static int as_matrix(const tensor* t, llar_matrix* m, const char* what) {
  if (t->nd == 0) {
    PyErr_Format(PyExc_ValueError, "%s needs at least one dimension", what);
    return -1;
  }
  m->data = t->data;
  m->cols = t->size[t->nd - 1];
  m->col_stride = t->stride[t->nd - 1];
  m->rows = 1;
  m->row_stride = 0;
  int empty = 0, loose = 0;
  for (int i = t->nd - 2; i >= 0; i--) {
    if (t->size[i] == 0) empty = 1;
    if (t->size[i] != 1) {
      if (m->rows == 1)
        m->row_stride = t->stride[i];
      else if (t->stride[i] != m->row_stride * m->rows)
        loose = 1;
    }
    m->rows *= t->size[i];
  }
  if (loose && !empty) {
    PyErr_Format(PyExc_ValueError, "%s: the leading dimensions cannot be viewed as one; make it contiguous", what);
    return -1;
  }
  return 0;
}

/* t has x's type and device. */
static int like(const tensor* x, PyObject* obj, tensor* t, const char* what) {
  if (read_tensor(obj, t) < 0) return -1;
  if (t->dtype != x->dtype || t->device != x->device) {
    PyErr_Format(PyExc_ValueError, "%s must have x's type and device", what);
    return -1;
  }
  return 0;
}

/* t has x's shape but for its width. */
static int shaped(const tensor* x, const tensor* t, int64_t width, const char* what) {
  int ok = t->nd == x->nd && t->size[t->nd - 1] == width;
  for (int i = 0; ok && i < x->nd - 1; i++) ok = t->size[i] == x->size[i];
  if (!ok) PyErr_Format(PyExc_ValueError, "%s has the wrong shape: x's, with %lld as the width, is expected", what, (long long)width);
  return ok ? 0 : -1;
}

static int activation_shaped(const tensor* x, PyObject* obj, int64_t width, llar_matrix* m, const char* what) {
  tensor t;
  if (like(x, obj, &t, what) < 0 || t.nd == 0) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s needs at least one dimension", what);
    return -1;
  }
  return shaped(x, &t, width, what) < 0 ? -1 : as_matrix(&t, m, what);
}

static int weight_shaped(const tensor* x, PyObject* obj, int64_t n, int64_t k, llar_matrix* m, const char* what) {
  tensor t;
  if (like(x, obj, &t, what) < 0) return -1;
  if (t.nd != 2 || t.size[1] != k || (n >= 0 && t.size[0] != n)) {
    PyErr_Format(PyExc_ValueError, "%s has the wrong shape, (n, %lld) is expected", what, (long long)k);
    return -1;
  }
  m->data = t.data;
  m->rows = t.size[0];
  m->cols = t.size[1];
  m->row_stride = t.stride[0];
  m->col_stride = t.stride[1];
  return 0;
}

/* What every call starts with.  1: another device is current (the caller
 * changes it and comes back), 0: go on, -1: an error is set. */
typedef struct {
  tensor x;
  llar_matrix xm;
  llar_dtype type;
  llar_act act;
  void* stream;
} call;

/* The library's number of a torch type, -1 with an error if it has none. */
static int type_of(PyObject* dtype) {
  int i;
  for (i = 0; i < 3 && dtype != t_types[i]; i++) {
  }
  if (i < 3) return i;
  PyErr_Format(PyExc_TypeError, "unsupported dtype %R (fp32, fp16, bf16 only)", dtype);
  return -1;
}

static int activation(PyObject* act, call* c) {
  int i;
  const char* name = PyUnicode_Check(act) ? PyUnicode_AsUTF8(act) : NULL;
  for (i = 0; name && i < 5 && strcmp(name, kActs[i]); i++) {
  }
  if (!name || i == 5) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "unknown activation %R (one of none, relu, gelu, gelu_tanh, silu)", act);
    return -1;
  }
  c->act = (llar_act)i;
  return 0;
}

/* The device's current stream, and x as a matrix. */
static int begin_on_device(call* c) {
  if (c->x.device < 0) {
    PyObject* v = PyObject_CallFunction(e_llar, "is", LLAR_ERR_HIP, "no GPU tensor: the operators run only on the HIP device");
    if (v) PyErr_SetObject(e_llar, v);
    Py_XDECREF(v);
    return -1;
  }
  PyObject* v = PyObject_CallNoArgs(f_current_device);
  if (!v) return -1;
  const long now = PyLong_AsLong(v);
  Py_DECREF(v);
  if (now != c->x.device) return 1;
  PyObject* at = PyLong_FromLong(c->x.device);
  v = at ? PyObject_CallOneArg(f_raw_stream, at) : NULL;
  Py_XDECREF(at);
  if (!v) return -1;
  c->stream = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  return as_matrix(&c->x, &c->xm, "x");
}

static int begin(PyObject* x, PyObject* act, call* c) {
  if (read_tensor(x, &c->x) < 0) return -1;
  const int i = type_of(c->x.dtype);
  if (i < 0) return -1;
  c->type = (llar_dtype)i;
  return activation(act, c) < 0 ? -1 : begin_on_device(c);
}

/* A new contiguous tensor of x's type, or the type given, on x's device; its address goes to *data. */
static PyObject* new_typed(const tensor* x, const int64_t* size, int nd, PyObject* dtype, void** data) {
  PyObject* shape = PyTuple_New(nd);
  if (!shape) return NULL;
  for (int i = 0; i < nd; i++) PyTuple_SET_ITEM(shape, i, PyLong_FromLongLong(size[i]));
  PyObject* args[3] = {x->obj, shape, dtype};
  PyObject* t = PyObject_VectorcallMethod(s_new_empty, args, 2 | PY_VECTORCALL_ARGUMENTS_OFFSET, dtype ? kw_dtype : NULL);
  Py_DECREF(shape);
  if (!t) return NULL;
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!v) {
    Py_DECREF(t);
    return NULL;
  }
  *data = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return t;
}
static PyObject* new_tensor(const tensor* x, const int64_t* size, int nd, void** data) {
  return new_typed(x, size, nd, NULL, data);
}

static llar_matrix dense(void* data, int64_t rows, int64_t cols) {
  llar_matrix m = {data, rows, cols, cols, 1};
  return m;
}

/* x's shape with another width, and the matrix of the whole. */
static PyObject* new_activation(const call* c, int64_t width, llar_matrix* m) {
  int64_t size[kMaxDims];
  memcpy(size, c->x.size, sizeof(size));
  size[c->x.nd - 1] = width;
  void* data = NULL;
  PyObject* t = new_tensor(&c->x, size, c->x.nd, &data);
  *m = dense(data, c->xm.rows, width);
  return t;
}
static PyObject* new_weight(const call* c, int64_t n, int64_t k, llar_matrix* m) {
  const int64_t size[2] = {n, k};
  void* data = NULL;
  PyObject* t = new_tensor(&c->x, size, 2, &data);
  *m = dense(data, n, k);
  return t;
}

static int by_rows(const llar_matrix* m) { return m->cols <= 1 || m->col_stride == 1; }
static int loose(const llar_matrix* m, int es) {
  const int rows = by_rows(m);
  const int64_t width = rows ? m->cols : m->rows, line = rows ? (m->rows > 1 ? m->row_stride : 0) : m->col_stride;
  return (((intptr_t)m->data | (width | line) * es) & 15) != 0 || line * es >= 1 << 23;
}

/* Device memory for a call's workspace (None: it needs none). */
static PyObject* room(const call* c, size_t bytes, void** data) {
  *data = NULL;
  if (bytes == 0) Py_RETURN_NONE;
  const int64_t n = (int64_t)bytes;
  return new_typed(&c->x, &n, 1, t_uint8, data);
}

/* The workspace of a call (None: it needs none). */
static PyObject* workspace(const call* c, llar_ffn_op op, const llar_matrix* w, const llar_matrix* w2,
                           const llar_matrix* dy, void** data, size_t* bytes) {
  const int es = c->type == LLAR_FP32 ? 4 : 2;
  int layout = 0;
  if (loose(&c->xm, es) || loose(w, es) || (w2 && loose(w2, es)) || (dy && loose(dy, es)))
    layout |= LLAR_LAYOUT_UNALIGNED;
  if (!by_rows(&c->xm)) layout |= LLAR_LAYOUT_X_COLUMNS;
  if (!by_rows(w)) layout |= LLAR_LAYOUT_W_COLUMNS;
  if (dy && !by_rows(dy)) layout |= LLAR_LAYOUT_DY_COLUMNS;
  *bytes = llar_ffn_workspace(op, c->xm.rows, w->rows, c->xm.cols, c->type, layout);
  return room(c, *bytes, data);
}

static int done(int status, const char* what) {
  if (status >= 0) return 0;
  PyObject* v = PyObject_CallFunction(e_llar, "is", status, what);
  if (v) PyErr_SetObject(e_llar, v);
  Py_XDECREF(v);
  return -1;
}

static int arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected", want);
  return -1;
}

/* (x, weight, bias, residual, activation, save, out) */
static PyObject* py_linear(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 7) < 0) return NULL;
  const int st = begin(a[0], a[4], &c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  llar_matrix w, r, y, z;
  if (weight_shaped(&c.x, a[1], -1, c.xm.cols, &w, "weight") < 0) return NULL;
  const void* bias = NULL;
  if (a[2] != Py_None) {
    tensor b;
    if (like(&c.x, a[2], &b, "bias") < 0) return NULL;
    if (b.nd != 1 || b.size[0] != w.rows || (w.rows > 1 && b.stride[0] != 1)) {
      PyErr_Format(PyExc_ValueError, "bias must be contiguous and of shape (%lld,)", (long long)w.rows);
      return NULL;
    }
    bias = b.data;
  }
  const int has_r = a[3] != Py_None, save = PyObject_IsTrue(a[5]);
  if (save < 0) return NULL;
  if (has_r && activation_shaped(&c.x, a[3], w.rows, &r, "residual") < 0) return NULL;
  PyObject *out = NULL, *pre = NULL, *ws = NULL, *result = NULL;
  if (a[6] != Py_None) {
    if (activation_shaped(&c.x, a[6], w.rows, &y, "out") < 0) return NULL;
    out = a[6];
    Py_INCREF(out);
  } else if (!(out = new_activation(&c, w.rows, &y))) {
    return NULL;
  }
  if (save && !(pre = new_activation(&c, w.rows, &z))) goto end;
  void* space;
  size_t bytes;
  if (!(ws = workspace(&c, LLAR_OP_LINEAR, &w, NULL, NULL, &space, &bytes))) goto end;
  if (done(llar_linear(&c.xm, &w, bias, has_r ? &r : NULL, &y, save ? &z : NULL, c.type, c.act, space, bytes, c.stream),
           "llar_linear") < 0)
    goto end;
  if (save) {
    result = PyTuple_Pack(2, out, pre);
  } else {
    result = out;
    out = NULL;
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(pre);
  Py_XDECREF(ws);
  return result;
}

/* (dy, x, weight, pre, activation, input_grad, weight_grad, bias_grad) */
static PyObject* py_linear_backward(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 8) < 0) return NULL;
  const int st = begin(a[1], a[4], &c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  const int want_x = PyObject_IsTrue(a[5]), want_w = PyObject_IsTrue(a[6]), want_b = PyObject_IsTrue(a[7]);
  if (want_x < 0 || want_w < 0 || want_b < 0) return NULL;
  llar_matrix dy, w, z, dxm, dwm;
  if (weight_shaped(&c.x, a[2], -1, c.xm.cols, &w, "weight") < 0) return NULL;
  if (activation_shaped(&c.x, a[0], w.rows, &dy, "dy") < 0) return NULL;
  const int with_act = c.act != LLAR_ACT_NONE;
  if (with_act) {
    if (a[3] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "pre, the value before the activation, is needed");
      return NULL;
    }
    if (activation_shaped(&c.x, a[3], w.rows, &z, "pre") < 0) return NULL;
  }
  PyObject *dx = NULL, *dw = NULL, *db = NULL, *ws = NULL, *result = NULL;
  void *db_data = NULL, *space;
  size_t bytes;
  if (want_x && !(dx = new_activation(&c, c.xm.cols, &dxm))) goto end;
  if (want_w && !(dw = new_weight(&c, w.rows, w.cols, &dwm))) goto end;
  if (want_b && !(db = new_tensor(&c.x, &w.rows, 1, &db_data))) goto end;
  if (!(ws = workspace(&c, LLAR_OP_LINEAR_BACKWARD, &w, NULL, &dy, &space, &bytes))) goto end;
  if (done(llar_linear_backward(&dy, &c.xm, &w, with_act ? &z : NULL, dx ? &dxm : NULL, dw ? &dwm : NULL, db_data,
                                c.type, c.act, space, bytes, c.stream),
           "llar_linear_backward") < 0)
    goto end;
  result = PyTuple_Pack(3, dx ? dx : Py_None, dw ? dw : Py_None, db ? db : Py_None);
end:
  Py_XDECREF(dx);
  Py_XDECREF(dw);
  Py_XDECREF(db);
  Py_XDECREF(ws);
  return result;
}

/* (x, w_gate, w_up, activation, save, out) */
static PyObject* py_gated_ffn(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 6) < 0) return NULL;
  const int st = begin(a[0], a[3], &c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  const int save = PyObject_IsTrue(a[4]);
  if (save < 0) return NULL;
  llar_matrix wg, wu, h, g, u;
  if (weight_shaped(&c.x, a[1], -1, c.xm.cols, &wg, "w_gate") < 0) return NULL;
  if (weight_shaped(&c.x, a[2], wg.rows, c.xm.cols, &wu, "w_up") < 0) return NULL;
  PyObject *out = NULL, *gate = NULL, *up = NULL, *ws = NULL, *result = NULL;
  void* space;
  size_t bytes;
  if (a[5] != Py_None) {
    if (activation_shaped(&c.x, a[5], wg.rows, &h, "out") < 0) return NULL;
    out = a[5];
    Py_INCREF(out);
  } else if (!(out = new_activation(&c, wg.rows, &h))) {
    return NULL;
  }
  if (save && (!(gate = new_activation(&c, wg.rows, &g)) || !(up = new_activation(&c, wg.rows, &u)))) goto end;
  if (!(ws = workspace(&c, LLAR_OP_GATED_FFN, &wg, &wu, NULL, &space, &bytes))) goto end;
  if (done(llar_gated_ffn(&c.xm, &wg, &wu, &h, save ? &g : NULL, save ? &u : NULL, c.type, c.act, space, bytes,
                          c.stream),
           "llar_gated_ffn") < 0)
    goto end;
  if (save) {
    result = PyTuple_Pack(3, out, gate, up);
  } else {
    result = out;
    out = NULL;
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(gate);
  Py_XDECREF(up);
  Py_XDECREF(ws);
  return result;
}

/* (dh, x, w_gate, w_up, gate, up, activation, input_grad, weight_grad) */
static PyObject* py_gated_ffn_backward(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 9) < 0) return NULL;
  const int st = begin(a[1], a[6], &c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  const int want_x = PyObject_IsTrue(a[7]), want_w = PyObject_IsTrue(a[8]);
  if (want_x < 0 || want_w < 0) return NULL;
  llar_matrix dh, wg, wu, g, u, dxm, dgm, dum;
  if (weight_shaped(&c.x, a[2], -1, c.xm.cols, &wg, "w_gate") < 0) return NULL;
  if (weight_shaped(&c.x, a[3], wg.rows, c.xm.cols, &wu, "w_up") < 0) return NULL;
  if (activation_shaped(&c.x, a[0], wg.rows, &dh, "dh") < 0) return NULL;
  if (activation_shaped(&c.x, a[4], wg.rows, &g, "gate") < 0) return NULL;
  if (activation_shaped(&c.x, a[5], wg.rows, &u, "up") < 0) return NULL;
  PyObject *dx = NULL, *dg = NULL, *du = NULL, *ws = NULL, *result = NULL;
  void* space;
  size_t bytes;
  if (want_x && !(dx = new_activation(&c, c.xm.cols, &dxm))) goto end;
  if (want_w && (!(dg = new_weight(&c, wg.rows, wg.cols, &dgm)) || !(du = new_weight(&c, wg.rows, wg.cols, &dum))))
    goto end;
  if (!(ws = workspace(&c, LLAR_OP_GATED_FFN_BACKWARD, &wg, &wu, NULL, &space, &bytes))) goto end;
  if (done(llar_gated_ffn_backward(&dh, &c.xm, &wg, &wu, &g, &u, dx ? &dxm : NULL, dg ? &dgm : NULL, du ? &dum : NULL,
                                   c.type, c.act, space, bytes, c.stream),
           "llar_gated_ffn_backward") < 0)
    goto end;
  result = PyTuple_Pack(3, dx ? dx : Py_None, dg ? dg : Py_None, du ? du : Py_None);
end:
  Py_XDECREF(dx);
  Py_XDECREF(dg);
  Py_XDECREF(du);
  Py_XDECREF(ws);
  return result;
}

/* ---- 8-bit products ---------------------------------------------------------------- */

/* A contiguous binary32 tensor of `count` scales, its leading dimensions x's (lead) or one dimension. */
static const float* scales(const call* c, PyObject* obj, int64_t count, int lead, const char* what) {
  tensor t;
  if (read_tensor(obj, &t) < 0) return NULL;
  if (t.dtype != t_types[0] || t.device != c->x.device) {
    PyErr_Format(PyExc_ValueError, "%s must be float32 and on x's device", what);
    return NULL;
  }
  const int nd = lead ? c->x.nd - 1 : 1;
  int ok = t.nd == nd;
  for (int i = 0; ok && i < nd; i++) ok = t.size[i] == (lead ? c->x.size[i] : count);
  int64_t step = 1;
  for (int i = nd - 1; ok && i >= 0; i--) {
    ok = t.size[i] <= 1 || t.stride[i] == step || count == 0;
    step *= t.size[i];
  }
  if (!ok) {
    PyErr_Format(PyExc_ValueError, lead ? "%s must be contiguous and have x's shape without its width"
                                        : "%s must be contiguous and of shape (%lld,)", what, (long long)count);
    return NULL;
  }
  static const float none = 0.f;
  return t.data ? (const float*)t.data : &none; /* an empty tensor's: never read */
}

static int int8_weight(const call* c, PyObject* obj, int64_t n, llar_matrix* m, const char* what) {
  tensor x = c->x;
  x.dtype = t_int8;
  tensor t;
  if (read_tensor(obj, &t) < 0) return -1;
  if (t.dtype != t_int8 || t.device != c->x.device) {
    PyErr_Format(PyExc_ValueError, "%s must be int8 and on x's device", what);
    return -1;
  }
  return weight_shaped(&x, obj, n, c->xm.cols, m, what);
}

/* x of a call that takes whole numbers with scales, or values: sets c->type to the results' and *xs. */
static int begin_int8(PyObject* x, PyObject* x_scale, PyObject* act, PyObject* dtype, call* c, const float** xs) {
  if (read_tensor(x, &c->x) < 0) return -1;
  int i;
  if (x_scale != Py_None) {
    if (c->x.dtype != t_int8) {
      PyErr_Format(PyExc_TypeError, "x with x_scale must be int8, not %R", c->x.dtype);
      return -1;
    }
    i = dtype == Py_None ? LLAR_BF16 : type_of(dtype);
  } else {
    i = type_of(c->x.dtype);
    if (i >= 0 && dtype != Py_None && dtype != c->x.dtype) {
      PyErr_SetString(PyExc_ValueError, "dtype is x's own where x is not int8");
      return -1;
    }
  }
  if (i < 0) return -1;
  c->type = (llar_dtype)i;
  if (activation(act, c) < 0) return -1;
  const int st = begin_on_device(c);
  if (st != 0) return st;
  *xs = NULL;
  if (x_scale != Py_None && !(*xs = scales(c, x_scale, c->xm.rows, 1, "x_scale"))) return -1;
  return 0;
}

/* The output, given or new, and the workspace. */
static PyObject* int8_out(const call* c, PyObject* given, int64_t width, llar_matrix* m) {
  tensor like_out = c->x;
  like_out.dtype = t_types[c->type];
  if (given != Py_None) {
    if (activation_shaped(&like_out, given, width, m, "out") < 0) return NULL;
    Py_INCREF(given);
    return given;
  }
  int64_t size[kMaxDims];
  memcpy(size, c->x.size, sizeof(size));
  size[c->x.nd - 1] = width;
  void* data = NULL;
  PyObject* t = new_typed(&c->x, size, c->x.nd, t_types[c->type], &data);
  *m = dense(data, c->xm.rows, width);
  return t;
}
static int loose8(const llar_matrix* m) {
  return (((intptr_t)m->data | m->cols | (m->rows > 1 ? m->row_stride : 0)) & 15) != 0 ||
         (m->rows > 1 && m->row_stride >= 1 << 23);
}
static PyObject* int8_room(const call* c, llar_ffn_op op, const float* xs, const llar_matrix* w, const llar_matrix* w2,
                           void** data, size_t* bytes) {
  int layout = xs ? 0 : LLAR_LAYOUT_X_VALUES;
  if (!xs && !by_rows(&c->xm)) layout |= LLAR_LAYOUT_X_COLUMNS;
  if ((xs && loose8(&c->xm)) || loose8(w) || (w2 && loose8(w2))) layout |= LLAR_LAYOUT_UNALIGNED;
  *bytes = llar_int8_workspace(op, c->xm.rows, w->rows, c->xm.cols, layout);
  return room(c, *bytes, data);
}

/* (x) -> (q, scale) */
static PyObject* py_quantize_rows(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 1) < 0) return NULL;
  if (read_tensor(a[0], &c.x) < 0) return NULL;
  const int i = type_of(c.x.dtype);
  if (i < 0) return NULL;
  c.type = (llar_dtype)i;
  const int st = begin_on_device(&c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  void *qd = NULL, *sd = NULL;
  PyObject *q = NULL, *s = NULL, *result = NULL;
  if (!(q = new_typed(&c.x, c.x.size, c.x.nd, t_int8, &qd))) goto end;
  if (!(s = new_typed(&c.x, c.x.size, c.x.nd - 1, t_types[0], &sd))) goto end;
  const llar_matrix qm = dense(qd, c.xm.rows, c.xm.cols);
  if (done(llar_quantize_rows(&c.xm, &qm, (float*)sd, c.type, c.stream), "llar_quantize_rows") < 0) goto end;
  result = PyTuple_Pack(2, q, s);
end:
  Py_XDECREF(q);
  Py_XDECREF(s);
  return result;
}

/* (x, weight, w_scale, x_scale, bias, residual, activation, dtype, out) */
static PyObject* py_linear_int8(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  const float *xs, *ws;
  if (arity(n_args, 9) < 0) return NULL;
  const int st = begin_int8(a[0], a[3], a[6], a[7], &c, &xs);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  llar_matrix w, r, y;
  if (int8_weight(&c, a[1], -1, &w, "weight") < 0) return NULL;
  if (!(ws = scales(&c, a[2], w.rows, 0, "w_scale"))) return NULL;
  tensor like_out = c.x;
  like_out.dtype = t_types[c.type];
  const void* bias = NULL;
  if (a[4] != Py_None) {
    tensor b;
    if (read_tensor(a[4], &b) < 0) return NULL;
    if (b.dtype != like_out.dtype || b.device != c.x.device || b.nd != 1 || b.size[0] != w.rows ||
        (w.rows > 1 && b.stride[0] != 1)) {
      PyErr_Format(PyExc_ValueError, "bias must be contiguous, of shape (%lld,), the output's type and x's device",
                   (long long)w.rows);
      return NULL;
    }
    bias = b.data;
  }
  const int has_r = a[5] != Py_None;
  if (has_r && activation_shaped(&like_out, a[5], w.rows, &r, "residual") < 0) return NULL;
  PyObject *ws_room = NULL, *result = NULL, *out = int8_out(&c, a[8], w.rows, &y);
  void* space;
  size_t bytes;
  if (!out) return NULL;
  if (!(ws_room = int8_room(&c, LLAR_OP_LINEAR, xs, &w, NULL, &space, &bytes))) goto end;
  if (done(llar_linear_int8(&c.xm, xs, &w, ws, bias, has_r ? &r : NULL, &y, c.type, c.act, space, bytes, c.stream),
           "llar_linear_int8") < 0)
    goto end;
  result = out;
  out = NULL;
end:
  Py_XDECREF(out);
  Py_XDECREF(ws_room);
  return result;
}

/* (x, w_gate, w_up, gate_scale, up_scale, x_scale, activation, dtype, out) */
static PyObject* py_gated_ffn_int8(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  const float *xs, *gs, *us;
  if (arity(n_args, 9) < 0) return NULL;
  const int st = begin_int8(a[0], a[5], a[6], a[7], &c, &xs);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  llar_matrix wg, wu, h;
  if (int8_weight(&c, a[1], -1, &wg, "w_gate") < 0) return NULL;
  if (int8_weight(&c, a[2], wg.rows, &wu, "w_up") < 0) return NULL;
  if (!(gs = scales(&c, a[3], wg.rows, 0, "gate_scale"))) return NULL;
  if (!(us = scales(&c, a[4], wg.rows, 0, "up_scale"))) return NULL;
  PyObject *ws_room = NULL, *result = NULL, *out = int8_out(&c, a[8], wg.rows, &h);
  void* space;
  size_t bytes;
  if (!out) return NULL;
  if (!(ws_room = int8_room(&c, LLAR_OP_GATED_FFN, xs, &wg, &wu, &space, &bytes))) goto end;
  if (done(llar_gated_ffn_int8(&c.xm, xs, &wg, &wu, gs, us, &h, c.type, c.act, space, bytes, c.stream),
           "llar_gated_ffn_int8") < 0)
    goto end;
  result = out;
  out = NULL;
end:
  Py_XDECREF(out);
  Py_XDECREF(ws_room);
  return result;
}

/* ---- mixture of experts -------------------------------------------------------------- */

static int contiguous(const tensor* t) {
  int64_t step = 1, count = 1;
  for (int i = 0; i < t->nd; i++) count *= t->size[i];
  for (int i = t->nd - 1; count > 0 && i >= 0; i--) {
    if (t->size[i] > 1 && t->stride[i] != step) return 0;
    step *= t->size[i];
  }
  return 1;
}

/* (x, router, top_k, sigmoid, normalize) -> (weights, experts) */
static PyObject* py_moe_route(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 5) < 0) return NULL;
  if (read_tensor(a[0], &c.x) < 0) return NULL;
  const int i = type_of(c.x.dtype);
  if (i < 0) return NULL;
  c.type = (llar_dtype)i;
  const int st = begin_on_device(&c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  llar_matrix router;
  if (weight_shaped(&c.x, a[1], -1, c.xm.cols, &router, "router") < 0) return NULL;
  const long top_k = PyLong_AsLong(a[2]);
  if (top_k == -1 && PyErr_Occurred()) return NULL;
  if (top_k < 0 || top_k > router.rows) {
    PyErr_Format(PyExc_ValueError, "top_k must be between 0 and the number of experts, %lld", (long long)router.rows);
    return NULL;
  }
  const int sigmoid = PyObject_IsTrue(a[3]), normalize = PyObject_IsTrue(a[4]);
  if (sigmoid < 0 || normalize < 0) return NULL;
  int64_t size[kMaxDims];
  memcpy(size, c.x.size, sizeof(size));
  size[c.x.nd - 1] = top_k;
  void *wd = NULL, *ed = NULL, *space;
  PyObject *w = NULL, *e = NULL, *ws = NULL, *result = NULL;
  const size_t bytes = llar_moe_route_workspace(c.xm.rows, router.rows, c.xm.cols);
  if (!(w = new_typed(&c.x, size, c.x.nd, t_types[0], &wd))) goto end;
  if (!(e = new_typed(&c.x, size, c.x.nd, t_int32, &ed))) goto end;
  if (!(ws = room(&c, bytes, &space))) goto end;
  if (done(llar_moe_route(&c.xm, &router, (int)top_k, sigmoid ? LLAR_SCORE_SIGMOID : LLAR_SCORE_SOFTMAX, normalize,
                          (float*)wd, (int32_t*)ed, c.type, space, bytes, c.stream),
           "llar_moe_route") < 0)
    goto end;
  result = PyTuple_Pack(2, w, e);
end:
  Py_XDECREF(w);
  Py_XDECREF(e);
  Py_XDECREF(ws);
  return result;
}

/* E matrices of x's type or int8; sizes < 0 are any. */
static int expert_weights(const call* c, PyObject* obj, PyObject* dtype, const int64_t* want, llar_experts* m,
                          const char* what) {
  tensor t;
  if (read_tensor(obj, &t) < 0) return -1;
  if (t.dtype != dtype || t.device != c->x.device) {
    PyErr_Format(PyExc_ValueError, "%s must be on x's device and of %s", what,
                 dtype == t_int8 ? "type int8 (it has scales)" : "x's type (without scales)");
    return -1;
  }
  int ok = t.nd == 3;
  for (int i = 0; ok && i < 3; i++) ok = want[i] < 0 || t.size[i] == want[i];
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "%s has the wrong shape: w_gate and w_up are (experts, n, k), w_down (experts, outputs, n)", what);
    return -1;
  }
  if (t.size[2] > 1 && t.stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: the rows of every expert's matrix must be contiguous", what);
    return -1;
  }
  const llar_experts w = {t.data, t.size[0], t.size[1], t.size[2], t.size[0] > 1 ? t.stride[0] : 0,
                          t.size[1] > 1 ? t.stride[1] : 0};
  *m = w;
  return 0;
}

static const float* expert_scales(const call* c, PyObject* obj, int64_t experts, int64_t rows, const char* what) {
  tensor t;
  if (read_tensor(obj, &t) < 0) return NULL;
  if (t.dtype != t_types[0] || t.device != c->x.device || t.nd != 2 || t.size[0] != experts || t.size[1] != rows ||
      !contiguous(&t)) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous, float32, on x's device and of shape (%lld, %lld)", what,
                 (long long)experts, (long long)rows);
    return NULL;
  }
  static const float none = 0.f;
  return t.data ? (const float*)t.data : &none;
}

/* A contiguous tensor with a token's choices: x's shape, with top_k as the width. */
static int choices(const call* c, PyObject* obj, tensor* t, int64_t top_k, const char* what) {
  if (read_tensor(obj, t) < 0) return -1;
  if (t->device != c->x.device || t->nd == 0 || !contiguous(t)) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous and on x's device", what);
    return -1;
  }
  return shaped(&c->x, t, top_k < 0 ? t->size[t->nd - 1] : top_k, what);
}

/* (x, experts, weights, w_gate, w_up, w_down, gate_scale, up_scale, down_scale, activation, residual, out) */
static PyObject* py_moe_ffn(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  call c;
  if (arity(n_args, 12) < 0) return NULL;
  const int st = begin(a[0], a[9], &c);
  if (st < 0) return NULL;
  if (st > 0) Py_RETURN_NOTIMPLEMENTED;
  tensor ids, w;
  if (choices(&c, a[1], &ids, -1, "experts") < 0) return NULL;
  if (ids.dtype != t_int32 && ids.dtype != t_int64) {
    PyErr_Format(PyExc_TypeError, "experts must be int32 or int64, not %R", ids.dtype);
    return NULL;
  }
  const int64_t top_k = ids.size[ids.nd - 1];
  if (choices(&c, a[2], &w, top_k, "weights") < 0) return NULL;
  if (w.dtype != t_types[0]) {
    PyErr_Format(PyExc_TypeError, "weights must be float32, not %R", w.dtype);
    return NULL;
  }
  const int int8 = a[6] != Py_None;
  if (int8 != (a[7] != Py_None) || int8 != (a[8] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "gate_scale, up_scale and down_scale are given together");
    return NULL;
  }
  PyObject* type = int8 ? t_int8 : t_types[c.type];
  llar_experts wg, wu, wd;
  int64_t want[3] = {-1, -1, c.xm.cols};
  if (expert_weights(&c, a[3], type, want, &wg, "w_gate") < 0) return NULL;
  want[0] = wg.experts;
  want[1] = wg.rows;
  if (expert_weights(&c, a[4], type, want, &wu, "w_up") < 0) return NULL;
  want[1] = -1;
  want[2] = wg.rows;
  if (expert_weights(&c, a[5], type, want, &wd, "w_down") < 0) return NULL;
  const float *gs = NULL, *us = NULL, *ds = NULL;
  if (int8 && (!(gs = expert_scales(&c, a[6], wg.experts, wg.rows, "gate_scale")) ||
               !(us = expert_scales(&c, a[7], wg.experts, wg.rows, "up_scale")) ||
               !(ds = expert_scales(&c, a[8], wg.experts, wd.rows, "down_scale"))))
    return NULL;
  llar_matrix r, y;
  const int has_r = a[10] != Py_None;
  if (has_r && activation_shaped(&c.x, a[10], wd.rows, &r, "residual") < 0) return NULL;
  if (top_k > 1 << 20) { /* the library's own limit is far lower; this keeps the number an int */
    PyErr_SetString(PyExc_ValueError, "experts has too many choices a token");
    return NULL;
  }
  PyObject *out = NULL, *ws = NULL, *result = NULL;
  if (a[11] != Py_None) {
    if (activation_shaped(&c.x, a[11], wd.rows, &y, "out") < 0) return NULL;
    out = a[11];
    Py_INCREF(out);
  } else if (!(out = new_activation(&c, wd.rows, &y))) {
    return NULL;
  }
  void* space;
  const size_t bytes = llar_moe_workspace(c.xm.rows, wg.rows, c.xm.cols, wd.rows, wg.experts, (int)top_k, c.type, int8);
  if (!(ws = room(&c, bytes, &space))) goto end;
  if (done(llar_moe_ffn(&c.xm, ids.data, ids.dtype == t_int64 ? 8 : 4, (const float*)w.data, (int)top_k, &wg, &wu, &wd,
                        gs, us, ds, has_r ? &r : NULL, &y, c.type, c.act, space, bytes, c.stream),
           "llar_moe_ffn") < 0)
    goto end;
  result = out;
  out = NULL;
end:
  Py_XDECREF(out);
  Py_XDECREF(ws);
  return result;
}

/* (float32, float16, bfloat16, uint8, int8, int32, int64, current_device(), raw_stream(device), LlarError): once,
 * before any call */
static PyObject* py_setup(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  PyObject** const to[10] = {&t_types[0], &t_types[1], &t_types[2], &t_uint8,          &t_int8,
                             &t_int32,    &t_int64,    &f_current_device, &f_raw_stream, &e_llar};
  if (arity(n_args, 10) < 0) return NULL;
  for (int i = 0; i < 10; i++) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"linear", (PyCFunction)(void (*)(void))py_linear, METH_FASTCALL, NULL},
    {"linear_backward", (PyCFunction)(void (*)(void))py_linear_backward, METH_FASTCALL, NULL},
    {"gated_ffn", (PyCFunction)(void (*)(void))py_gated_ffn, METH_FASTCALL, NULL},
    {"gated_ffn_backward", (PyCFunction)(void (*)(void))py_gated_ffn_backward, METH_FASTCALL, NULL},
    {"quantize_rows", (PyCFunction)(void (*)(void))py_quantize_rows, METH_FASTCALL, NULL},
    {"linear_int8", (PyCFunction)(void (*)(void))py_linear_int8, METH_FASTCALL, NULL},
    {"gated_ffn_int8", (PyCFunction)(void (*)(void))py_gated_ffn_int8, METH_FASTCALL, NULL},
    {"moe_route", (PyCFunction)(void (*)(void))py_moe_route, METH_FASTCALL, NULL},
    {"moe_ffn", (PyCFunction)(void (*)(void))py_moe_ffn, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_llar_py", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__llar_py(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_new_empty = PyUnicode_InternFromString("new_empty");
  if (!s_dtype || !s_get_device || !s_data_ptr || !s_shape || !s_stride || !s_new_empty) return NULL;
  if (!(kw_dtype = PyTuple_Pack(1, s_dtype))) return NULL;
  return PyModule_Create(&module);
}
