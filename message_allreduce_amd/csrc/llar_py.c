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
static PyObject *t_types[3], *t_uint8, *f_current_device, *f_raw_stream, *e_llar;

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

static int begin(PyObject* x, PyObject* act, call* c) {
  if (read_tensor(x, &c->x) < 0) return -1;
  int i;
  for (i = 0; i < 3 && c->x.dtype != t_types[i]; i++) {
  }
  if (i == 3) {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %R (fp32, fp16, bf16 only)", c->x.dtype);
    return -1;
  }
  c->type = (llar_dtype)i;
  const char* name = PyUnicode_Check(act) ? PyUnicode_AsUTF8(act) : NULL;
  for (i = 0; name && i < 5 && strcmp(name, kActs[i]); i++) {
  }
  if (!name || i == 5) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "unknown activation %R (one of none, relu, gelu, gelu_tanh, silu)", act);
    return -1;
  }
  c->act = (llar_act)i;
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

/* A new contiguous tensor of x's type; its address goes to *data. */
static PyObject* new_tensor(const tensor* x, const int64_t* size, int nd, void** data) {
  PyObject* shape = PyTuple_New(nd);
  if (!shape) return NULL;
  for (int i = 0; i < nd; i++) PyTuple_SET_ITEM(shape, i, PyLong_FromLongLong(size[i]));
  PyObject* args[2] = {x->obj, shape};
  PyObject* t = PyObject_VectorcallMethod(s_new_empty, args, 2 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
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
  *data = NULL;
  *bytes = llar_ffn_workspace(op, c->xm.rows, w->rows, c->xm.cols, c->type, layout);
  if (*bytes == 0) Py_RETURN_NONE;
  PyObject* n = PyLong_FromSize_t(*bytes);
  if (!n) return NULL;
  PyObject* args[3] = {c->x.obj, n, t_uint8};
  PyObject* t = PyObject_VectorcallMethod(s_new_empty, args, 2 | PY_VECTORCALL_ARGUMENTS_OFFSET, kw_dtype);
  Py_DECREF(n);
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

/* (float32, float16, bfloat16, uint8, current_device(), raw_stream(device), LlarError): once, before any call */
static PyObject* py_setup(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  if (arity(n_args, 7) < 0) return NULL;
  PyObject** const to[7] = {&t_types[0], &t_types[1], &t_types[2], &t_uint8, &f_current_device, &f_raw_stream, &e_llar};
  for (int i = 0; i < 7; i++) {
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
