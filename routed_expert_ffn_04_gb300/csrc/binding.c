/*
 * CPython module of the entry points around the layer and of its gradient:
 * the tensors' checks and the call in one step. Against the same checks and a
 * ctypes call in Python, a call's time on the host fell from 7.0 to 4.8 us
 * (combine_backward, nine tensors) and from 4.4 to 3.2 (permute_backward): for
 * a few tokens that is the whole call's time, since the kernels take 3 to 5 us.
 *
 * setup() hands over the package's error functions, torch's dtypes and the
 * current stream's lookup. Every function takes (handle, device, ...): the
 * handle's address (or None once closed) and its device's number, tensors as
 * in the package's functions of the same name, and the stream or None.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "../../include/moe.h"

static PyObject *s_dtype, *s_numel, *s_device, *s_contiguous, *s_data_ptr, *s_shape, *s_element_size, *s_cuda_stream;
static PyObject *bad_arg, *bad_status, *current_stream; /* from setup() */
static PyObject *bf16, *f32, *i32, *u8;

static int as_int64(PyObject* v, int64_t* out) { /* steals v */
  if (!v) return 0;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return !(*out == -1 && PyErr_Occurred());
}

/* Pointer of a dense tensor of `numel` elements of `dtype` (numel < 0: any
 * number, dtype NULL: any) on the device; with `optional`, None gives NULL.
 * Raises through bad_arg otherwise. */
static int tensor(PyObject* t, const char* what, const char* name, PyObject* dtype, int64_t numel, int device,
                  int optional, void** out) {
  int64_t v;
  int ok = 0;
  *out = NULL;
  if (t == Py_None && optional) return 1;
  if (t != Py_None) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return 0;
    ok = dtype == NULL || d == dtype;
    Py_DECREF(d);
    if (ok && numel >= 0) {
      if (!as_int64(PyObject_CallMethodNoArgs(t, s_numel), &v)) return 0;
      ok = v == numel;
    }
    if (ok) {
      if (!as_int64(PyObject_CallMethodNoArgs(t, s_device), &v)) return 0;
      ok = v == device;
    }
    if (ok) {
      PyObject* c = PyObject_CallMethodNoArgs(t, s_contiguous);
      if (!c) return 0;
      ok = c == Py_True;
      Py_DECREF(c);
    }
    if (ok) {
      PyObject* p = PyObject_CallMethodNoArgs(t, s_data_ptr);
      if (!p) return 0;
      *out = PyLong_AsVoidPtr(p);
      Py_DECREF(p);
      return !PyErr_Occurred();
    }
  }
  PyObject* r = PyObject_CallFunction(bad_arg, "ssOOLi", what, name, t, dtype ? dtype : Py_None, (long long)numel, device);
  Py_XDECREF(r);
  return 0;
}

/* Sizes that the library refuses later may pass 64 bits here: no tensor has that many elements. */
static int64_t product(int a, int b, int c) {
  int64_t m;
  return __builtin_mul_overflow((int64_t)a * b, (int64_t)c, &m) ? INT64_MAX : m;
}

/* The rows and columns of a tensor [..., cols]. */
static int rows_cols(PyObject* t, const char* what, const char* name, int64_t* rows, int64_t* cols) {
  int64_t n = 0;
  *cols = 0;
  if (t != Py_None) {
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    if (!shape) return 0;
    const Py_ssize_t dims = PyTuple_Check(shape) ? PyTuple_GET_SIZE(shape) : 0;
    if (dims > 0) *cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, dims - 1));
    Py_DECREF(shape);
    if (PyErr_Occurred() || !as_int64(PyObject_CallMethodNoArgs(t, s_numel), &n)) return 0;
  }
  if (*cols <= 0 || *cols > INT32_MAX) {
    PyObject* r = PyObject_CallFunction(bad_arg, "ssOOLi", what, name, t, Py_None, (long long)-1, -1);
    Py_XDECREF(r);
    return 0;
  }
  *rows = n / *cols;
  return 1;
}

static int workspace(PyObject* t, const char* what, int device, void** out, size_t* bytes) {
  int64_t n, e;
  *bytes = 0;
  if (!tensor(t, what, "ws", NULL, -1, device, 1, out)) return 0;
  if (!*out) return 1;
  if (!as_int64(PyObject_CallMethodNoArgs(t, s_numel), &n) || !as_int64(PyObject_CallMethodNoArgs(t, s_element_size), &e))
    return 0;
  *bytes = (size_t)(n * e);
  return 1;
}

static int stream_of(PyObject* s, PyObject* device, void** out) {
  PyObject* v = s == Py_None ? PyObject_CallOneArg(current_stream, device) : PyObject_GetAttr(s, s_cuda_stream);
  if (!v) return 0;
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

static int handle_of(PyObject* h, PyObject* device, moe_handle_t* out, int* dev) {
  *out = h == Py_None ? NULL : (moe_handle_t)PyLong_AsVoidPtr(h);
  *dev = (int)PyLong_AsLong(device);
  return !PyErr_Occurred();
}

/* A ctypes structure's moe_config_t (a copy: the structure may change later). */
static int config_of(PyObject* c, moe_config_t* out) {
  Py_buffer b;
  if (PyObject_GetBuffer(c, &b, PyBUF_SIMPLE) != 0) return 0;
  const int ok = b.len == (Py_ssize_t)sizeof(moe_config_t);
  if (ok) *out = *(const moe_config_t*)b.buf;
  PyBuffer_Release(&b);
  if (!ok) PyErr_SetString(PyExc_TypeError, "a Config is wanted");
  return ok;
}

static PyObject* done(int st, const char* what) {
  if (st != MOE_OK) {
    PyObject* r = PyObject_CallFunction(bad_status, "is", (int)st, what);
    Py_XDECREF(r);
    if (!r) return NULL;
  }
  Py_RETURN_NONE;
}

/* The library's call with the interpreter's lock free: a launch waits when the device's queue is full. */
#define CALL(expr, what)     \
  do {                       \
    int st_;                 \
    Py_BEGIN_ALLOW_THREADS   \
    st_ = (expr);            \
    Py_END_ALLOW_THREADS     \
    return done(st_, (what)); \
  } while (0)

static int count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
  return 0;
}

/* The residual stream's type by a tensor's dtype. */
static int residual_type(PyObject* t, const char* what, PyObject** dtype, moe_residual_t* rt) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  *dtype = d == f32 ? f32 : bf16; /* another one fails at its own check */
  *rt = d == f32 ? MOE_RES_F32 : MOE_RES_BF16;
  Py_DECREF(d);
  return 1;
}

/* handle, device, x, weight, eps, residual, h_out, out, q, q_scale, rstd, stream */
static PyObject* add_rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_add_rmsnorm";
  moe_handle_t h;
  int dev;
  int64_t rows, H;
  void *x, *w, *res, *ho, *out, *q, *qs, *rstd, *st;
  PyObject* rd = bf16;
  moe_residual_t rt = MOE_RES_BF16;
  if (!count_is(n, 12) || !handle_of(a[0], a[1], &h, &dev) || !rows_cols(a[2], what, "x", &rows, &H)) return NULL;
  const double eps = PyFloat_AsDouble(a[4]);
  if (PyErr_Occurred()) return NULL;
  if (a[5] != Py_None || a[6] != Py_None)
    if (!residual_type(a[5] != Py_None ? a[5] : a[6], what, &rd, &rt)) return NULL;
  if (!tensor(a[2], what, "x", bf16, rows * H, dev, 0, &x) || !tensor(a[3], what, "weight", bf16, H, dev, 0, &w) ||
      !tensor(a[5], what, "residual", rd, rows * H, dev, 1, &res) ||
      !tensor(a[6], what, "h_out", rd, rows * H, dev, 1, &ho) || !tensor(a[7], what, "out", bf16, rows * H, dev, 1, &out) ||
      !tensor(a[8], what, "q", u8, rows * H, dev, 1, &q) ||
      !tensor(a[9], what, "q_scale", u8, rows * H / 32, dev, 1, &qs) ||
      !tensor(a[10], what, "rstd", f32, rows, dev, 1, &rstd) || !stream_of(a[11], a[1], &st))
    return NULL;
  CALL(moe_add_rmsnorm(h, rows, (int)H, rt, x, res, w, (float)eps, ho, out, q, qs, rstd, st), what);
}

/* handle, device, dout, h_res, weight, rstd, dh, ws, dh_in, dx, dweight, stream */
static PyObject* add_rmsnorm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_add_rmsnorm_backward";
  moe_handle_t h;
  int dev;
  int64_t rows, H;
  void *dout, *hr, *w, *rstd, *dh, *ws, *di, *dx, *dw, *st;
  size_t ws_bytes;
  PyObject* rd = bf16;
  moe_residual_t rt = MOE_RES_BF16;
  if (!count_is(n, 12) || !handle_of(a[0], a[1], &h, &dev) || !rows_cols(a[3], what, "h_res", &rows, &H) ||
      !residual_type(a[3], what, &rd, &rt))
    return NULL;
  const int64_t m = rows * H;
  if (!tensor(a[2], what, "dout", bf16, m, dev, 0, &dout) || !tensor(a[3], what, "h_res", rd, m, dev, 0, &hr) ||
      !tensor(a[4], what, "weight", bf16, H, dev, 0, &w) || !tensor(a[5], what, "rstd", f32, rows, dev, 0, &rstd) ||
      !tensor(a[6], what, "dh", rd, m, dev, 0, &dh) || !workspace(a[7], what, dev, &ws, &ws_bytes) ||
      !tensor(a[8], what, "dh_in", rd, m, dev, 1, &di) || !tensor(a[9], what, "dx", bf16, m, dev, 1, &dx) ||
      !tensor(a[10], what, "dweight", f32, H, dev, 1, &dw) || !stream_of(a[11], a[1], &st))
    return NULL;
  CALL(moe_add_rmsnorm_backward(h, rows, (int)H, rt, dout, di, hr, w, rstd, dh, dx, dw, ws, ws_bytes, st), what);
}

/* handle, device, cfg, dout, y_perm, topk_w, flat_to_perm, dy_perm, dtopk_w, topk_idx, logits, dlogits, stream */
static PyObject* combine_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_combine_backward";
  moe_handle_t h;
  int dev;
  moe_config_t c;
  void *dout, *y, *w, *f2p, *dy, *dw, *idx, *l, *dl, *st;
  if (!count_is(n, 13) || !handle_of(a[0], a[1], &h, &dev) || !config_of(a[2], &c)) return NULL;
  const int64_t T = c.T, TK = T * c.K, TKH = product(c.T, c.K, c.H);
  if (!tensor(a[3], what, "dout", bf16, T * c.H, dev, 0, &dout) || !tensor(a[4], what, "y_perm", f32, TKH, dev, 0, &y) ||
      !tensor(a[5], what, "topk_w", f32, TK, dev, 0, &w) || !tensor(a[6], what, "flat_to_perm", i32, TK, dev, 0, &f2p) ||
      !tensor(a[7], what, "dy_perm", bf16, TKH, dev, 0, &dy) || !tensor(a[8], what, "dtopk_w", f32, TK, dev, 0, &dw) ||
      !tensor(a[9], what, "topk_idx", i32, TK, dev, 1, &idx) || !tensor(a[10], what, "logits", f32, T * c.E, dev, 1, &l) ||
      !tensor(a[11], what, "dlogits", f32, T * c.E, dev, 1, &dl) || !stream_of(a[12], a[1], &st))
    return NULL;
  CALL(moe_combine_backward(h, &c, dout, y, w, f2p, idx, l, dy, dw, dl, st), what);
}

/* handle, device, cfg, logits, topk_idx, dtopk_w, dlogits, stream */
static PyObject* route_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_route_backward";
  moe_handle_t h;
  int dev;
  moe_config_t c;
  void *l, *idx, *dw, *dl, *st;
  if (!count_is(n, 8) || !handle_of(a[0], a[1], &h, &dev) || !config_of(a[2], &c)) return NULL;
  const int64_t T = c.T, TK = T * c.K;
  if (!tensor(a[3], what, "logits", f32, T * c.E, dev, 0, &l) || !tensor(a[4], what, "topk_idx", i32, TK, dev, 0, &idx) ||
      !tensor(a[5], what, "dtopk_w", f32, TK, dev, 0, &dw) || !tensor(a[6], what, "dlogits", f32, T * c.E, dev, 0, &dl) ||
      !stream_of(a[7], a[1], &st))
    return NULL;
  CALL(moe_route_backward(h, &c, l, idx, dw, dl, st), what);
}

/* handle, device, cfg, dx_perm, flat_to_perm, dx, dx_add, stream */
static PyObject* permute_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_permute_backward";
  moe_handle_t h;
  int dev;
  moe_config_t c;
  void *dxp, *f2p, *dx, *add, *st;
  if (!count_is(n, 8) || !handle_of(a[0], a[1], &h, &dev) || !config_of(a[2], &c)) return NULL;
  const int64_t T = c.T, TK = T * c.K;
  if (!tensor(a[3], what, "dx_perm", bf16, product(c.T, c.K, c.H), dev, 0, &dxp) ||
      !tensor(a[4], what, "flat_to_perm", i32, TK, dev, 0, &f2p) || !tensor(a[5], what, "dx", bf16, T * c.H, dev, 0, &dx) ||
      !tensor(a[6], what, "dx_add", bf16, T * c.H, dev, 1, &add) || !stream_of(a[7], a[1], &st))
    return NULL;
  CALL(moe_permute_backward(h, &c, dxp, f2p, add, dx, st), what);
}

/* handle, device, a, dy, offsets, w_gate, w_up, w_down, da, dw_gate, dw_up, dw_down, ws, num_groups, H, I, dtype, stream */
static PyObject* grouped_swiglu_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_grouped_swiglu_backward";
  moe_handle_t h;
  int dev;
  int64_t rows, cols;
  void *in, *dy, *off, *w[3], *da, *dw[3], *ws, *st;
  size_t ws_bytes;
  if (!count_is(n, 18) || !handle_of(a[0], a[1], &h, &dev) || !rows_cols(a[2], what, "a", &rows, &cols)) return NULL;
  const long G = PyLong_AsLong(a[13]), H = PyLong_AsLong(a[14]), I = PyLong_AsLong(a[15]), dt = PyLong_AsLong(a[16]);
  if (PyErr_Occurred()) return NULL;
  if (G < 0 || H < 0 || I < 0 || G >= INT32_MAX || H > INT32_MAX || I > INT32_MAX || cols != H || rows > INT32_MAX)
    return done(MOE_ERR_INVALID_ARG, what);
  const int64_t m = product((int)G, (int)H, (int)I);
  if (!tensor(a[2], what, "a", bf16, rows * H, dev, 0, &in) || !tensor(a[3], what, "dy", bf16, rows * H, dev, 0, &dy) ||
      !tensor(a[4], what, "offsets", i32, G + 1, dev, G == 1, &off) || !tensor(a[5], what, "w_gate", bf16, m, dev, 0, &w[0]) ||
      !tensor(a[6], what, "w_up", bf16, m, dev, 0, &w[1]) || !tensor(a[7], what, "w_down", bf16, m, dev, 0, &w[2]) ||
      !tensor(a[8], what, "da", bf16, rows * H, dev, 1, &da) || !tensor(a[9], what, "dw_gate", bf16, m, dev, 1, &dw[0]) ||
      !tensor(a[10], what, "dw_up", bf16, m, dev, 1, &dw[1]) || !tensor(a[11], what, "dw_down", bf16, m, dev, 1, &dw[2]) ||
      !workspace(a[12], what, dev, &ws, &ws_bytes) || !stream_of(a[17], a[1], &st))
    return NULL;
  CALL(moe_grouped_swiglu_backward(h, (int)G, (int)rows, (int)H, (int)I, (moe_dtype_t)dt, in, dy, off, w[0], w[1],
                                          w[2], da, dw[0], dw[1], dw[2], ws, ws_bytes, st), what);
}

/* bad_arg, bad_status, current_stream, bfloat16, float32, int32, uint8 */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  PyObject** to[] = {&bad_arg, &bad_status, &current_stream, &bf16, &f32, &i32, &u8};
  if (!count_is(n, 7)) return NULL;
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(setup), FAST(add_rmsnorm), FAST(add_rmsnorm_backward), FAST(combine_backward),
                                FAST(route_backward), FAST(permute_backward), FAST(grouped_swiglu_backward),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_numel = PyUnicode_InternFromString("numel");
  s_device = PyUnicode_InternFromString("get_device");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_element_size = PyUnicode_InternFromString("element_size");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_dtype || !s_numel || !s_device || !s_contiguous || !s_data_ptr || !s_shape || !s_element_size || !s_cuda_stream)
    return NULL;
  return PyModule_Create(&module);
}
