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

/* Type of a plain operand by its tensor's dtype. */
static int float_type(PyObject* t, PyObject** dtype, moe_float_t* ft) {
  PyObject* d = t == Py_None ? NULL : PyObject_GetAttr(t, s_dtype);
  if (!d && t != Py_None) return 0;
  *dtype = d == f32 ? f32 : bf16; /* another one fails at its own check */
  *ft = d == f32 ? MOE_FLOAT_F32 : MOE_FLOAT_BF16;
  Py_XDECREF(d);
  return 1;
}
static int64_t blocks_of(int64_t n) { return n / 128 + (n % 128 != 0); }
/* `n` integers of the arguments, each in [0, 2^31). */
static int ints_of(PyObject* const* a, int n, int* out, const char* what) {
  for (int i = 0; i < n; ++i) {
    const long v = PyLong_AsLong(a[i]);
    if (PyErr_Occurred()) return 0;
    if (v < 0 || v >= INT32_MAX) {
      PyObject* r = done(MOE_ERR_INVALID_ARG, what);
      Py_XDECREF(r);
      return 0;
    }
    out[i] = (int)v;
  }
  return 1;
}
/* The rows of a tensor [rows, cols], which the call's `cols` has to be. */
static int rows_of(PyObject* t, const char* what, const char* name, int cols, int* rows) {
  int64_t r, c;
  if (!rows_cols(t, what, name, &r, &c)) return 0;
  if (c != cols || r > INT32_MAX) {
    PyObject* v = done(MOE_ERR_INVALID_ARG, what);
    Py_XDECREF(v);
    return 0;
  }
  *rows = (int)r;
  return 1;
}

/* The sequences of a batch: offsets [B+1] or None. */
static int sequences(PyObject* t, const char* what, int device, void** out, int* num) {
  int64_t n;
  *num = 1;
  if (!tensor(t, what, "seq_offsets", i32, -1, device, 1, out)) return 0;
  if (!*out) return t == Py_None ? 1 : (done(MOE_ERR_INVALID_ARG, what), 0);
  if (!as_int64(PyObject_CallMethodNoArgs(t, s_numel), &n)) return 0;
  *num = n - 1 > INT32_MAX ? INT32_MAX : (int)(n - 1);
  return 1;
}

/* handle, device, cfg, logits, topk_idx, counts, prob, loss, ws, coef, score, seq_offsets, stream */
static PyObject* balance_loss(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_balance_loss";
  moe_handle_t h;
  int dev, B, score;
  moe_config_t c;
  void *l, *idx, *cnt, *prob, *loss, *ws, *seq, *st;
  size_t ws_bytes;
  if (!count_is(n, 13) || !handle_of(a[0], a[1], &h, &dev) || !config_of(a[2], &c)) return NULL;
  const double coef = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred() || !ints_of(a + 10, 1, &score, what) || !sequences(a[11], what, dev, &seq, &B)) return NULL;
  const int64_t T = c.T, BE = product(B, c.E, 1);
  if (!tensor(a[3], what, "logits", f32, T * c.E, dev, 0, &l) || !tensor(a[4], what, "topk_idx", i32, T * c.K, dev, 0, &idx) ||
      !tensor(a[5], what, "counts", i32, BE, dev, 0, &cnt) || !tensor(a[6], what, "prob", f32, BE, dev, 0, &prob) ||
      !tensor(a[7], what, "loss", f32, B, dev, 0, &loss) || !workspace(a[8], what, dev, &ws, &ws_bytes) ||
      !stream_of(a[12], a[1], &st))
    return NULL;
  CALL(moe_balance_loss(h, &c, (moe_score_t)score, (float)coef, l, idx, seq, B, cnt, prob, loss, ws, ws_bytes, st), what);
}

/* handle, device, cfg, logits, counts, dloss, dlogits, coef, score, seq_offsets, dlogits_add, stream */
static PyObject* balance_loss_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_balance_loss_backward";
  moe_handle_t h;
  int dev, B, score;
  moe_config_t c;
  void *l, *cnt, *dloss, *dl, *seq, *add, *st;
  if (!count_is(n, 12) || !handle_of(a[0], a[1], &h, &dev) || !config_of(a[2], &c)) return NULL;
  const double coef = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred() || !ints_of(a + 8, 1, &score, what) || !sequences(a[9], what, dev, &seq, &B)) return NULL;
  const int64_t T = c.T;
  if (!tensor(a[3], what, "logits", f32, T * c.E, dev, 0, &l) ||
      !tensor(a[4], what, "counts", i32, product(B, c.E, 1), dev, 0, &cnt) ||
      !tensor(a[5], what, "dloss", f32, B, dev, 0, &dloss) || !tensor(a[6], what, "dlogits", f32, T * c.E, dev, 0, &dl) ||
      !tensor(a[10], what, "dlogits_add", f32, T * c.E, dev, 1, &add) || !stream_of(a[11], a[1], &st))
    return NULL;
  CALL(moe_balance_loss_backward(h, &c, (moe_score_t)score, (float)coef, l, cnt, seq, B, dloss, add, dl, st), what);
}

/* handle, device, x, q, scale, squares, rows (of a matrix), stream */
static PyObject* quantize_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_quantize_fp8";
  moe_handle_t h;
  int dev, rows;
  int64_t all, cols;
  void *x, *q, *sc, *st;
  PyObject* dt;
  moe_float_t ft;
  if (!count_is(n, 8) || !handle_of(a[0], a[1], &h, &dev) || !rows_cols(a[2], what, "x", &all, &cols) ||
      !float_type(a[2], &dt, &ft) || !ints_of(a + 6, 1, &rows, what))
    return NULL;
  const int squares = PyObject_IsTrue(a[5]);
  if (squares < 0) return NULL;
  const int64_t batch = rows ? all / rows : 0;
  const int64_t m = squares ? batch * blocks_of(rows) * blocks_of(cols) : all * blocks_of(cols);
  if (!tensor(a[2], what, "x", dt, all * cols, dev, 0, &x) || !tensor(a[3], what, "q", u8, all * cols, dev, 0, &q) ||
      !tensor(a[4], what, "scale", f32, m, dev, 0, &sc) || !stream_of(a[7], a[1], &st))
    return NULL;
  CALL(moe_quantize_fp8(h, x, ft, batch, rows, (int)cols, squares, q, sc, st), what);
}

/* handle, device, x, offsets, q, scale, num_groups, stream */
static PyObject* quantize_fp8_columns(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_quantize_fp8_columns";
  moe_handle_t h;
  int dev, G;
  int64_t rows, cols, padded;
  void *x, *off, *q, *sc, *st;
  PyObject* dt;
  moe_float_t ft;
  if (!count_is(n, 8) || !handle_of(a[0], a[1], &h, &dev) || !rows_cols(a[2], what, "x", &rows, &cols) ||
      !float_type(a[2], &dt, &ft) || !ints_of(a + 6, 1, &G, what))
    return NULL;
  if (rows > INT32_MAX || moe_fp8_padded_rows((int)rows, G, &padded) != MOE_OK) return done(MOE_ERR_INVALID_ARG, what);
  if (!tensor(a[2], what, "x", dt, rows * cols, dev, 0, &x) || !tensor(a[3], what, "offsets", i32, (int64_t)G + 1, dev, G == 1, &off) ||
      !tensor(a[4], what, "q", u8, padded * cols, dev, 0, &q) || !tensor(a[5], what, "scale", f32, padded / 128 * cols, dev, 0, &sc) ||
      !stream_of(a[7], a[1], &st))
    return NULL;
  CALL(moe_quantize_fp8_columns(h, x, ft, G, (int)rows, (int)cols, off, q, sc, st), what);
}

/* handle, device, a, a_scale, offsets, w, w_scale, out, num_groups, N, K, transposed, stream */
static PyObject* grouped_gemm_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_grouped_gemm_fp8";
  moe_handle_t h;
  int dev, v[3], rows;
  void *in, *as, *off, *w, *ws, *out, *st;
  PyObject* dt;
  moe_float_t ft;
  if (!count_is(n, 13) || !handle_of(a[0], a[1], &h, &dev) || !ints_of(a + 8, 3, v, what)) return NULL;
  const int G = v[0], N = v[1], K = v[2], transposed = PyObject_IsTrue(a[11]);
  if (transposed < 0 || !rows_of(a[2], what, "a", K, &rows) || !float_type(a[7], &dt, &ft)) return NULL;
  if (!tensor(a[2], what, "a", u8, (int64_t)rows * K, dev, 0, &in) ||
      !tensor(a[3], what, "a_scale", f32, rows * blocks_of(K), dev, 0, &as) ||
      !tensor(a[4], what, "offsets", i32, (int64_t)G + 1, dev, G == 1, &off) || !tensor(a[5], what, "w", u8, product(G, N, K), dev, 0, &w) ||
      !tensor(a[6], what, "w_scale", f32, product(G, (int)blocks_of(N), (int)blocks_of(K)), dev, 0, &ws) ||
      !tensor(a[7], what, "out", dt, (int64_t)rows * N, dev, 0, &out) || !stream_of(a[12], a[1], &st))
    return NULL;
  CALL(moe_grouped_gemm_fp8(h, G, rows, N, K, transposed, in, as, off, w, ws, ft, out, st), what);
}

/* handle, device, a, a_scale, offsets, w_gate, s_gate, w_up, s_up, q, scale, num_groups, H, I, stream */
static PyObject* grouped_gate_up_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_grouped_gate_up_fp8";
  moe_handle_t h;
  int dev, v[3], rows;
  void *in, *as, *off, *wg, *sg, *wu, *su, *q, *sc, *st;
  if (!count_is(n, 15) || !handle_of(a[0], a[1], &h, &dev) || !ints_of(a + 11, 3, v, what)) return NULL;
  const int G = v[0], H = v[1], I = v[2];
  const int64_t m = product(G, H, I), ms = product(G, (int)blocks_of(H), (int)blocks_of(I));
  if (!rows_of(a[2], what, "a", H, &rows)) return NULL;
  if (!tensor(a[2], what, "a", u8, (int64_t)rows * H, dev, 0, &in) ||
      !tensor(a[3], what, "a_scale", f32, rows * blocks_of(H), dev, 0, &as) ||
      !tensor(a[4], what, "offsets", i32, (int64_t)G + 1, dev, G == 1, &off) || !tensor(a[5], what, "w_gate", u8, m, dev, 0, &wg) ||
      !tensor(a[6], what, "s_gate", f32, ms, dev, 0, &sg) || !tensor(a[7], what, "w_up", u8, m, dev, 0, &wu) ||
      !tensor(a[8], what, "s_up", f32, ms, dev, 0, &su) || !tensor(a[9], what, "q", u8, (int64_t)rows * I, dev, 0, &q) ||
      !tensor(a[10], what, "scale", f32, rows * blocks_of(I), dev, 0, &sc) || !stream_of(a[14], a[1], &st))
    return NULL;
  CALL(moe_grouped_gate_up_fp8(h, G, rows, H, I, in, as, off, wg, sg, wu, su, q, sc, st), what);
}

/* handle, device, dy, dy_scale, a, a_scale, offsets, dw, rows, num_groups, N, K, stream */
static PyObject* grouped_weight_grad_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char what[] = "moe_grouped_weight_grad_fp8";
  moe_handle_t h;
  int dev, v[4];
  int64_t P;
  void *dy, *ds, *in, *as, *off, *dw, *st;
  PyObject* dt;
  moe_float_t ft;
  if (!count_is(n, 13) || !handle_of(a[0], a[1], &h, &dev) || !ints_of(a + 8, 4, v, what) || !float_type(a[7], &dt, &ft))
    return NULL;
  const int rows = v[0], G = v[1], N = v[2], K = v[3];
  if (moe_fp8_padded_rows(rows, G, &P) != MOE_OK) return done(MOE_ERR_INVALID_ARG, what);
  if (!tensor(a[2], what, "dy", u8, P * N, dev, 0, &dy) || !tensor(a[3], what, "dy_scale", f32, P / 128 * N, dev, 0, &ds) ||
      !tensor(a[4], what, "a", u8, P * K, dev, 0, &in) || !tensor(a[5], what, "a_scale", f32, P / 128 * K, dev, 0, &as) ||
      !tensor(a[6], what, "offsets", i32, (int64_t)G + 1, dev, G == 1, &off) || !tensor(a[7], what, "dw", dt, product(G, N, K), dev, 0, &dw) ||
      !stream_of(a[12], a[1], &st))
    return NULL;
  CALL(moe_grouped_weight_grad_fp8(h, G, rows, N, K, dy, ds, in, as, off, ft, dw, st), what);
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
                                FAST(balance_loss), FAST(balance_loss_backward), FAST(quantize_fp8),
                                FAST(quantize_fp8_columns), FAST(grouped_gemm_fp8), FAST(grouped_gate_up_fp8),
                                FAST(grouped_weight_grad_fp8), {NULL, NULL, 0, NULL}};
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
