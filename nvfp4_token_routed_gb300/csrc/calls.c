/* calls.c -- the routed-row calls of the binding in their ordinary form, as a CPython
 * extension: new outputs, the current stream, every row.  A call of a few microseconds of GPU
 * time otherwise waits for the interpreter: sort_routes and dispatch of 16 tokens take 10.5 us
 * here, 20 interpreted; what is left is allocation (1.2 us each) and launch (2 us).
 *
 * Each function takes the positional arguments of its namesake in experts.py (mx_raw: of
 * MxTensor) and returns its result, or None where the call is not an ordinary one: other types, shapes, devices or
 * layouts than expected, or a status other than MOE_OK.  experts.py then goes its own way,
 * which makes every check and raises every error; so nothing here reports one. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

#include "moe_nvfp4.h"

typedef moe_status (*sort_fn)(int32_t, int32_t, int32_t, const void*, int32_t, int32_t*, int32_t*,
                              int32_t*, void*, size_t, moe_stream_t);
typedef size_t (*sort_ws_fn)(int32_t, int32_t, int32_t);
typedef moe_status (*dispatch_fn)(const moe_rows*, int32_t, const int32_t*, void*, int64_t,
                                  moe_stream_t);
typedef moe_status (*combine_fn)(const moe_rows*, int32_t, int32_t, const int32_t*, const float*,
                                 void*, int64_t, moe_stream_t);
typedef moe_status (*combine_grad_fn)(const moe_rows*, int32_t, int32_t, const int32_t*,
                                      const float*, const void*, int64_t, void*, int64_t, float*,
                                      moe_stream_t);
typedef moe_status (*checkpoint_fn)(const moe_rows*, uint8_t*, uint8_t*, const int32_t*,
                                    moe_stream_t);
typedef moe_status (*restore_fn)(const uint8_t*, const uint8_t*, const moe_rows*, const int32_t*,
                                 moe_stream_t);
typedef moe_status (*act_fn)(const moe_rows*, int32_t, float, void*, int64_t, uint8_t*, uint8_t*,
                             const int32_t*, moe_stream_t);
typedef moe_status (*act_grad_fn)(const uint8_t*, const uint8_t*, int32_t, float, const moe_rows*,
                                  void*, int64_t, const int32_t*, moe_stream_t);
typedef moe_status (*quantize_fn)(const moe_rows*, const moe_mx*, const int32_t*, moe_stream_t);
typedef moe_status (*product_fn)(const moe_mx*, const moe_mx*, int32_t, const int32_t*, int32_t,
                                 void*, int64_t, moe_stream_t);

/* Set once by attach() and kept. */
static struct {
  PyObject *tensor, *empty, *get_device, *get_stream; /* torch.Tensor, functions; empty: of
                                                         (size, stride, type), current device */
  PyObject *f32, *bf16, *f16, *u8, *i32, *i64;        /* torch types */
  PyObject *mx, *kept, *plan;                         /* MxTensor, Checkpoint, RoutePlan */
  void* fn[11];
} g;
enum { SORT, DISPATCH, COMBINE, COMBINE_GRAD, CHECKPOINT, RESTORE, ACT, ACT_GRAD, QUANTIZE, PRODUCT,
       SORT_WS };

static PyObject *s_dtype, *s_shape, *s_stride, *s_device_of, *s_data_ptr, *s_contiguous;
static PyObject *s_raw, *s_codes, *s_scales, *s_buf, *s_cut, *s_device, *s_rows, *s_cols, *s_act;
static PyObject *s_halves, *s_limit, *s_c, *empty_tuple;

/* None, with any error of a failed look-up cleared. */
static PyObject* not_ordinary(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

static int call_long(PyObject* t, PyObject* name, int64_t* v) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return 0;
  *v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *v != -1 || !PyErr_Occurred();
}
static int address(PyObject* t, void** p) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return 0;
  *p = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *p || !PyErr_Occurred();
}
/* The sizes of a tuple of `n` integers. */
static int sizes(PyObject* tuple, int n, int64_t* v) {
  if (!tuple) return 0;
  int ok = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n;
  for (int i = 0; ok && i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    ok = v[i] != -1 || !PyErr_Occurred();
  }
  Py_DECREF(tuple);
  return ok;
}
/* The current device, and whether a tensor lies on it (-1: the CPU). */
static int on_device(PyObject* t, int64_t* dev) {
  int64_t d;
  if (!PyObject_TypeCheck(t, (PyTypeObject*)g.tensor) || !call_long(t, s_device_of, &d) || d < 0)
    return 0;
  if (*dev < 0) {
    PyObject* r = PyObject_CallNoArgs(g.get_device);
    if (!r) return 0;
    *dev = PyLong_AsLongLong(r);
    Py_DECREF(r);
  }
  return d == *dev;
}
static int stream_of(int64_t dev, moe_stream_t* s) {
  PyObject* d = PyLong_FromLongLong(dev);
  PyObject* r = d ? PyObject_CallOneArg(g.get_stream, d) : NULL;
  Py_XDECREF(d);
  if (!r) return 0;
  *s = (moe_stream_t)PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *s || !PyErr_Occurred();
}

static int float_type(PyObject* dtype) {
  return dtype == g.f32 ? MOE_DTYPE_F32 : dtype == g.bf16 ? MOE_DTYPE_BF16
         : dtype == g.f16 ? MOE_DTYPE_F16 : -1;
}
static PyObject* type_object(int dtype) {
  return dtype == MOE_DTYPE_F32 ? g.f32 : dtype == MOE_DTYPE_BF16 ? g.bf16 : g.f16;
}

/* Rows of a 2-D tensor on the current device: contiguous each, not overlapping. */
static int rows_of(PyObject* t, int64_t* dev, moe_rows* m) {
  int64_t sh[2], st[2];
  void* p;
  if (!on_device(t, dev)) return 0;
  PyObject* dt = PyObject_GetAttr(t, s_dtype);
  if (!dt) return 0;
  m->dtype = float_type(dt);
  Py_DECREF(dt);
  if (m->dtype < 0 || !sizes(PyObject_GetAttr(t, s_shape), 2, sh) ||
      !sizes(PyObject_CallMethodNoArgs(t, s_stride), 2, st) || !address(t, &p))
    return 0;
  if (sh[0] < 1 || sh[1] < 1 || sh[0] > INT32_MAX || sh[1] > INT32_MAX ||
      (st[1] != 1 && sh[1] > 1) || (st[0] < sh[1] && sh[0] > 1))
    return 0;
  m->data = p;
  m->ld = sh[0] > 1 ? st[0] : sh[1];
  m->rows = (int32_t)sh[0];
  m->cols = (int32_t)sh[1];
  return 1;
}
/* A contiguous tensor of one of two types (0 or 1 in *which) and of a shape of up to 3 sizes. */
static int arg_of(PyObject* t, int64_t* dev, PyObject* type0, PyObject* type1, int n,
                  const int64_t* shape, void** p, int* which) {
  int64_t sh[3];
  if (!on_device(t, dev)) return 0;
  PyObject* dt = PyObject_GetAttr(t, s_dtype);
  if (!dt) return 0;
  Py_DECREF(dt);
  if (dt != type0 && dt != type1) return 0;
  if (which) *which = dt == type1;
  if (!sizes(PyObject_GetAttr(t, s_shape), n, sh)) return 0;
  for (int i = 0; i < n; ++i)
    if (sh[i] != shape[i]) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_contiguous);
  if (!c) return 0;
  Py_DECREF(c);
  return c == Py_True && address(t, p);
}

/* A new tensor on the current device and its address. */
static PyObject* new_tensor(int n, const int64_t* shape, PyObject* type, void** p) {
  PyObject* size = n == 1 ? Py_BuildValue("(L)", shape[0]) : Py_BuildValue("(LL)", shape[0], shape[1]);
  PyObject* stride = n == 1 ? Py_BuildValue("(i)", 1) : Py_BuildValue("(Li)", shape[1], 1);
  PyObject* args[3] = {size, stride, type};
  PyObject* t = size && stride ? PyObject_Vectorcall(g.empty, args, 3, NULL) : NULL;
  Py_XDECREF(size);
  Py_XDECREF(stride);
  if (t && !address(t, p)) Py_CLEAR(t);
  return t;
}
/* Codes and scales of an MxTensor or Checkpoint, cut from one new buffer. */
static PyObject* new_buffer(int64_t codes, int64_t scales, uint8_t** p, int64_t* at) {
  void* q;
  *at = (codes + 255) & ~(int64_t)255;
  const int64_t n = *at + scales;
  PyObject* t = new_tensor(1, &n, g.u8, &q);
  *p = (uint8_t*)q;
  return t;
}
static int set_steal(PyObject* o, PyObject* name, PyObject* v) {
  if (!v) return 0;
  const int ok = PyObject_SetAttr(o, name, v) == 0;
  Py_DECREF(v);
  return ok;
}
static int set_held(PyObject* o, PyObject* buf, int64_t codes, int64_t at, int64_t dev) {
  return PyObject_SetAttr(o, s_codes, Py_None) == 0 && PyObject_SetAttr(o, s_scales, Py_None) == 0 &&
         PyObject_SetAttr(o, s_buf, buf) == 0 &&
         set_steal(o, s_cut, Py_BuildValue("(LL)", codes, at)) &&
         set_steal(o, s_device, PyLong_FromLongLong(dev));
}
static PyObject* new_object(PyObject* cls) {
  PyTypeObject* t = (PyTypeObject*)cls;
  return t->tp_new(t, empty_tuple, NULL);
}

static int held_device(PyObject* o, int64_t* dev) {
  PyObject* d = PyObject_GetAttr(o, s_device);
  if (!d) return 0;
  const int64_t v = PyLong_AsLongLong(d);
  Py_DECREF(d);
  if (v < 0) return 0;
  if (*dev < 0) {
    PyObject* r = PyObject_CallNoArgs(g.get_device);
    if (!r) return 0;
    *dev = PyLong_AsLongLong(r);
    Py_DECREF(r);
  }
  return v == *dev;
}
/* Whether codes and scales still lie where they did (0.1 us): the tensors of a caller may have
 * been given other storage, a buffer is the object's own. */
static int still_at(PyObject* o, const void* codes, const void* scales) {
  PyObject* buf = PyObject_GetAttr(o, s_buf);
  if (!buf) return 0;
  const int own = buf != Py_None;
  Py_DECREF(buf);
  if (own) return 1;
  PyObject *c = PyObject_GetAttr(o, s_codes), *s = c ? PyObject_GetAttr(o, s_scales) : NULL;
  void *p, *q;
  const int ok = s && address(c, &p) && address(s, &q) && p == codes && q == scales;
  Py_XDECREF(c);
  Py_XDECREF(s);
  return ok;
}
static int mx_of(PyObject* o, int64_t* dev, moe_mx* m) {
  if ((PyObject*)Py_TYPE(o) != g.mx || !held_device(o, dev)) return 0;
  PyObject* raw = PyObject_GetAttr(o, s_raw);
  if (!raw) return 0;
  const int ok = PyBytes_Check(raw) && PyBytes_GET_SIZE(raw) == sizeof(*m);
  if (ok) memcpy(m, PyBytes_AS_STRING(raw), sizeof(*m));
  Py_DECREF(raw);
  return ok && still_at(o, m->codes, m->scales);
}
typedef struct {
  void *codes, *scales;
  int64_t rows, cols, halves;
  int act;   /* -1: none */
  double limit;
} Kept;
static int attr_long(PyObject* o, PyObject* name, int64_t* v) {
  PyObject* r = PyObject_GetAttr(o, name);
  if (!r) return 0;
  *v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *v != -1 || !PyErr_Occurred();
}
static int act_of(PyObject* act) {
  if (!PyUnicode_Check(act)) return -1;
  if (PyUnicode_CompareWithASCIIString(act, "swiglu") == 0) return MOE_ACT_SWIGLU;
  return PyUnicode_CompareWithASCIIString(act, "relu2") == 0 ? MOE_ACT_RELU2 : -1;
}
static int kept_of(PyObject* o, int64_t* dev, Kept* k) {
  if ((PyObject*)Py_TYPE(o) != g.kept || !held_device(o, dev) || !attr_long(o, s_rows, &k->rows) ||
      !attr_long(o, s_cols, &k->cols) || !attr_long(o, s_halves, &k->halves))
    return 0;
  PyObject* c = PyObject_GetAttr(o, s_c);
  if (!c) return 0;
  int ok = PyTuple_Check(c) && PyTuple_GET_SIZE(c) == 2;
  if (ok) {
    k->codes = PyLong_AsVoidPtr(PyTuple_GET_ITEM(c, 0));
    k->scales = PyLong_AsVoidPtr(PyTuple_GET_ITEM(c, 1));
    ok = k->codes && k->scales && still_at(o, k->codes, k->scales);
  }
  Py_DECREF(c);
  PyObject* act = ok ? PyObject_GetAttr(o, s_act) : NULL;
  if (!act) return 0;
  k->act = act_of(act);
  Py_DECREF(act);
  PyObject* l = PyObject_GetAttr(o, s_limit);
  if (!l) return 0;
  k->limit = PyFloat_AsDouble(l);
  Py_DECREF(l);
  return !PyErr_Occurred();
}
/* A new Checkpoint of `rows` rows of `cols` values a half. */
static PyObject* new_kept(int64_t rows, int64_t cols, int halves, PyObject* type, PyObject* act,
                          double limit, int64_t dev, uint8_t** codes, uint8_t** scales) {
  const int64_t blocks = rows * halves * ((cols + 31) / 32);
  int64_t at;
  uint8_t* p;
  PyObject* buf = new_buffer(32 * blocks, blocks, &p, &at);
  PyObject* k = buf ? new_object(g.kept) : NULL;
  if (k && !(set_held(k, buf, 32 * blocks, at, dev) && set_steal(k, s_rows, PyLong_FromLongLong(rows)) &&
             set_steal(k, s_cols, PyLong_FromLongLong(cols)) && PyObject_SetAttr(k, s_dtype, type) == 0 &&
             PyObject_SetAttr(k, s_act, act) == 0 && set_steal(k, s_halves, PyLong_FromLong(halves)) &&
             set_steal(k, s_limit, PyFloat_FromDouble(limit)) &&
             set_steal(k, s_c, Py_BuildValue("(NN)", PyLong_FromVoidPtr(p), PyLong_FromVoidPtr(p + at)))))
    Py_CLEAR(k);
  Py_XDECREF(buf);
  *codes = p;
  *scales = k ? p + at : NULL;
  return k;
}

/* Row numbers [T][K] of a plan, its last tensor. */
static int inv_of(PyObject* plan, int64_t T, int64_t* dev, void** inv, int64_t* K) {
  int64_t sh[2];
  if ((PyObject*)Py_TYPE(plan) != g.plan || PyTuple_GET_SIZE(plan) != 3) return 0;
  PyObject* t = PyTuple_GET_ITEM(plan, 2);
  if (!PyObject_TypeCheck(t, (PyTypeObject*)g.tensor) ||
      !sizes(PyObject_GetAttr(t, s_shape), 2, sh) || (T >= 0 && sh[0] != T))
    return 0;
  *K = sh[1];
  return arg_of(t, dev, g.i32, g.i32, 2, sh, inv, NULL);
}
static int plan_tokens(PyObject* plan, int64_t* T) {
  int64_t sh[2];
  if ((PyObject*)Py_TYPE(plan) != g.plan || PyTuple_GET_SIZE(plan) != 3 ||
      !sizes(PyObject_GetAttr(PyTuple_GET_ITEM(plan, 2), s_shape), 2, sh))
    return 0;
  *T = sh[0];
  return 1;
}
/* The caller's matrix of this shape and type, or a new one. */
static PyObject* matrix_out(PyObject* given, int64_t rows, int64_t cols, int dtype, int64_t* dev,
                            void** p, int64_t* ld) {
  if (given == Py_None) {
    const int64_t sh[2] = {rows, cols};
    *ld = cols;
    return new_tensor(2, sh, type_object(dtype), p);
  }
  moe_rows m;
  if (!rows_of(given, dev, &m) || m.rows != rows || m.cols != cols || m.dtype != dtype) return NULL;
  *p = (void*)m.data;
  *ld = m.ld;
  Py_INCREF(given);
  return given;
}
/* topk_w, or NULL for None. */
static int weights_of(PyObject* w, int64_t T, int64_t K, int64_t* dev, void** p) {
  const int64_t sh[2] = {T, K};
  *p = NULL;
  return w == Py_None || arg_of(w, dev, g.f32, g.f32, 2, sh, p, NULL);
}

#define CALL(NAME, TYPE) ((TYPE)g.fn[NAME])
/* `status` of an entry point, called without the interpreter's lock: a launch waits where the
 * stream's queue is full, and what the queue waits for may need another Python thread.  (0.1 us.)
 * The arguments are plain values; their tensors are the caller's, or new and held here. */
#define LAUNCH(status, NAME, TYPE, ...)       \
  do {                                        \
    const TYPE entry = CALL(NAME, TYPE);      \
    Py_BEGIN_ALLOW_THREADS                    \
    status = entry(__VA_ARGS__);              \
    Py_END_ALLOW_THREADS                      \
  } while (0)
#define ORDINARY(cond) \
  if (!(cond)) return not_ordinary()

/* sort_routes(topk_ids, E) */
static PyObject* sort_routes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, sh[2];
  void *ids, *po, *pp, *pi, *pw = NULL;
  int is64;
  moe_stream_t s;
  ORDINARY(n == 2 && PyObject_TypeCheck(a[0], (PyTypeObject*)g.tensor) && PyLong_Check(a[1]));
  const int64_t E = PyLong_AsLongLong(a[1]);
  ORDINARY(E >= 1 && E <= 1024 && sizes(PyObject_GetAttr(a[0], s_shape), 2, sh));
  ORDINARY(sh[0] >= 1 && sh[0] <= INT32_MAX && sh[1] >= 1 && sh[1] <= 32 &&
           arg_of(a[0], &dev, g.i32, g.i64, 2, sh, &ids, &is64) && stream_of(dev, &s));
  const int64_t ws = (int64_t)CALL(SORT_WS, sort_ws_fn)((int32_t)sh[0], (int32_t)sh[1], (int32_t)E);
  ORDINARY(ws > 0);
  // a workspace only where the sort needs more than the status that nobody reads here
  const int64_t no = E + 1, np = sh[0] * sh[1], nw = np > 32768 ? ws : 0;
  PyObject* offsets = new_tensor(1, &no, g.i32, &po);
  PyObject* perm = offsets ? new_tensor(1, &np, g.i32, &pp) : NULL;
  PyObject* inv = perm ? new_tensor(2, sh, g.i32, &pi) : NULL;
  PyObject* work = inv && nw ? new_tensor(1, &nw, g.u8, &pw) : NULL;
  PyObject* plan = NULL;
  moe_status st = MOE_ERR_CUDA;
  if (inv && (work || !nw))
    LAUNCH(st, SORT, sort_fn, (int32_t)sh[0], (int32_t)sh[1], (int32_t)E, ids, is64, po, pp, pi, pw,
           (size_t)nw, s);
  if (st == MOE_OK) {
    PyObject* items = Py_BuildValue("((OOO))", offsets, perm, inv);
    if (items) plan = PyTuple_Type.tp_new((PyTypeObject*)g.plan, items, NULL);
    Py_XDECREF(items);
  }
  Py_XDECREF(offsets);
  Py_XDECREF(perm);
  Py_XDECREF(inv);
  Py_XDECREF(work); /* its memory is used next by work behind this on the stream */
  return plan ? plan : not_ordinary();
}

/* dispatch(x, plan, rows) */
static PyObject* dispatch(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, K, ld;
  moe_rows x;
  void *inv, *p;
  moe_stream_t s;
  ORDINARY(n == 3 && rows_of(a[0], &dev, &x) && inv_of(a[1], x.rows, &dev, &inv, &K) &&
           stream_of(dev, &s));
  PyObject* out = matrix_out(a[2], x.rows * K, x.cols, x.dtype, &dev, &p, &ld);
  moe_status st = MOE_OK;
  if (out) LAUNCH(st, DISPATCH, dispatch_fn, &x, (int32_t)K, inv, p, ld, s);
  if (st != MOE_OK) Py_CLEAR(out);
  return out ? out : not_ordinary();
}

/* combine(rows, plan, topk_w) */
static PyObject* combine(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, T, K, ld;
  moe_rows x;
  void *inv, *w, *p;
  moe_stream_t s;
  ORDINARY(n == 3 && rows_of(a[0], &dev, &x) && plan_tokens(a[1], &T) &&
           inv_of(a[1], T, &dev, &inv, &K) && weights_of(a[2], T, K, &dev, &w) &&
           stream_of(dev, &s));
  PyObject* out = matrix_out(Py_None, T, x.cols, x.dtype, &dev, &p, &ld);
  moe_status st = MOE_OK;
  if (out) LAUNCH(st, COMBINE, combine_fn, &x, (int32_t)T, (int32_t)K, inv, w, p, ld, s);
  if (st != MOE_OK) Py_CLEAR(out);
  return out ? out : not_ordinary();
}

/* combine_grad(rows, plan, topk_w, dout, drows) */
static PyObject* combine_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, T, K, ld;
  moe_rows x, d;
  void *inv, *w, *p, *pw;
  moe_stream_t s;
  ORDINARY(n == 5 && rows_of(a[0], &dev, &x) && plan_tokens(a[1], &T) &&
           inv_of(a[1], T, &dev, &inv, &K) && weights_of(a[2], T, K, &dev, &w) &&
           rows_of(a[3], &dev, &d) && d.rows == T && d.cols == x.cols && d.dtype == x.dtype &&
           x.rows == T * K && stream_of(dev, &s));
  const int64_t sh[2] = {T, K};
  PyObject* drows = matrix_out(a[4], x.rows, x.cols, x.dtype, &dev, &p, &ld);
  PyObject* dw = drows ? new_tensor(2, sh, g.f32, &pw) : NULL;
  PyObject* r = NULL;
  moe_status st = MOE_ERR_CUDA;
  if (dw)
    LAUNCH(st, COMBINE_GRAD, combine_grad_fn, &x, (int32_t)T, (int32_t)K, inv, w, d.data, d.ld, p,
           ld, pw, s);
  if (st == MOE_OK) r = PyTuple_Pack(2, drows, dw);
  Py_XDECREF(drows);
  Py_XDECREF(dw);
  return r ? r : not_ordinary();
}

/* checkpoint(x) */
static PyObject* checkpoint(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1;
  moe_rows x;
  uint8_t *codes, *scales;
  moe_stream_t s;
  ORDINARY(n == 1 && rows_of(a[0], &dev, &x) && stream_of(dev, &s));
  PyObject* k = new_kept(x.rows, x.cols, 1, type_object(x.dtype), Py_None, 0.0, dev, &codes, &scales);
  moe_status st = MOE_OK;
  if (k) LAUNCH(st, CHECKPOINT, checkpoint_fn, &x, codes, scales, NULL, s);
  if (st != MOE_OK) Py_CLEAR(k);
  return k ? k : not_ordinary();
}

/* restore(kept), of the type that was kept */
static PyObject* restore(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1;
  Kept k;
  void* p;
  moe_stream_t s;
  ORDINARY(n == 1 && kept_of(a[0], &dev, &k) && k.act < 0 && k.halves == 1 && k.rows >= 1 &&
           k.rows <= INT32_MAX && k.cols <= INT32_MAX && stream_of(dev, &s));
  PyObject* act = PyObject_GetAttr(a[0], s_act); /* None, or nothing that act_of knows */
  ORDINARY(act);
  Py_DECREF(act);
  ORDINARY(act == Py_None);
  PyObject* dt = PyObject_GetAttr(a[0], s_dtype);
  ORDINARY(dt);
  const int type = float_type(dt);
  Py_DECREF(dt);
  ORDINARY(type >= 0);
  const int64_t sh[2] = {k.rows, k.cols};
  PyObject* out = new_tensor(2, sh, type_object(type), &p);
  if (out) {
    const moe_rows m = {p, k.cols, (int32_t)k.rows, (int32_t)k.cols, type};
    moe_status st;
    LAUNCH(st, RESTORE, restore_fn, k.codes, k.scales, &m, NULL, s);
    if (st != MOE_OK) Py_CLEAR(out);
  }
  return out ? out : not_ordinary();
}

/* expert_act(h, act, swiglu_limit, checkpoint) */
static PyObject* expert_act(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1;
  moe_rows h;
  uint8_t *codes = NULL, *scales = NULL;
  void* p;
  moe_stream_t s;
  ORDINARY(n == 4 && rows_of(a[0], &dev, &h) && stream_of(dev, &s));
  const int act = act_of(a[1]), halves = act == MOE_ACT_SWIGLU ? 2 : 1;
  const double limit = PyFloat_AsDouble(a[2]);
  const int keep = PyObject_IsTrue(a[3]);
  ORDINARY(act >= 0 && !PyErr_Occurred() && keep >= 0 && h.cols % halves == 0 &&
           (limit == 0.0 || (float)limit != 0.0f));
  const int64_t sh[2] = {h.rows, h.cols / halves};
  PyObject* y = new_tensor(2, sh, type_object(h.dtype), &p);
  PyObject* k = y && keep ? new_kept(sh[0], sh[1], halves, type_object(h.dtype), a[1], limit, dev,
                                     &codes, &scales)
                          : NULL;
  PyObject* r = NULL;
  moe_status st = MOE_ERR_CUDA;
  if (y && (k || !keep))
    LAUNCH(st, ACT, act_fn, &h, act, (float)limit, p, sh[1], codes, scales, NULL, s);
  if (st == MOE_OK && !keep) Py_INCREF(r = y);
  if (st == MOE_OK && keep) r = PyTuple_Pack(2, y, k);
  Py_XDECREF(y);
  Py_XDECREF(k);
  return r ? r : not_ordinary();
}

/* expert_act_grad(kept, dy) */
static PyObject* expert_act_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1;
  Kept k;
  moe_rows dy;
  void* p;
  moe_stream_t s;
  ORDINARY(n == 2 && kept_of(a[0], &dev, &k) && k.act >= 0 && rows_of(a[1], &dev, &dy) &&
           dy.rows == k.rows && dy.cols == k.cols && stream_of(dev, &s));
  const int64_t sh[2] = {dy.rows, dy.cols * k.halves};
  PyObject* dh = new_tensor(2, sh, type_object(dy.dtype), &p);
  moe_status st = MOE_OK;
  if (dh)
    LAUNCH(st, ACT_GRAD, act_grad_fn, k.codes, k.scales, k.act, (float)k.limit, &dy, p, sh[1], NULL,
           s);
  if (st != MOE_OK) Py_CLEAR(dh);
  return dh ? dh : not_ordinary();
}

/* mx_quantize(x), x a matrix */
static PyObject* mx_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, at;
  moe_rows x;
  uint8_t* p;
  moe_stream_t s;
  ORDINARY(n == 1 && rows_of(a[0], &dev, &x) && stream_of(dev, &s));
  const int64_t dp = ((int64_t)x.cols + 255) & ~(int64_t)255, codes = x.rows * dp / 2;
  PyObject* buf = new_buffer(codes, (((int64_t)x.rows + 1) & ~(int64_t)1) * dp / 32, &p, &at);
  PyObject* q = NULL;
  if (buf) {
    moe_mx m;
    memset(&m, 0, sizeof(m));
    m.codes = p;
    m.scales = p + at;
    m.rows = x.rows;
    m.cols = x.cols;
    moe_status st;
    LAUNCH(st, QUANTIZE, quantize_fn, &x, &m, NULL, s);
    if (st == MOE_OK && (q = new_object(g.mx)) &&
        !(set_held(q, buf, codes, at, dev) &&
          set_steal(q, s_shape, Py_BuildValue("(ii)", x.rows, x.cols)) &&
          set_steal(q, s_raw, PyBytes_FromStringAndSize((const char*)&m, sizeof(m)))))
      Py_CLEAR(q);
    Py_DECREF(buf);
  }
  return q ? q : not_ordinary();
}

/* The moe_mx of an MxTensor of these codes, scales and shape, as bytes. */
static PyObject* mx_raw(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, sh[3];
  void *codes, *scales;
  ORDINARY(n == 3 && PyTuple_Check(a[2]));
  const int dims = (int)PyTuple_GET_SIZE(a[2]);
  ORDINARY(dims == 2 || dims == 3);
  Py_INCREF(a[2]);
  ORDINARY(sizes(a[2], dims, sh)); /* takes the reference */
  const int64_t cols = sh[dims - 1], e = dims == 3 ? sh[0] : 1, each = sh[dims - 2];
  ORDINARY(cols >= 1 && cols <= INT32_MAX && e >= 1 && e <= INT32_MAX && each >= 1 &&
           each <= INT32_MAX / e);
  const int64_t rows = e * each, dp = (cols + 255) & ~(int64_t)255;
  const int64_t c[2] = {rows, dp / 2}, s[3] = {dp / 256, (rows + 1) & ~(int64_t)1, 8};
  ORDINARY(arg_of(a[0], &dev, g.u8, g.u8, 2, c, &codes, NULL) &&
           arg_of(a[1], &dev, g.u8, g.u8, 3, s, &scales, NULL));
  moe_mx m;
  memset(&m, 0, sizeof(m));
  m.codes = codes;
  m.scales = scales;
  m.rows = (int32_t)rows;
  m.cols = (int32_t)cols;
  PyObject* raw = PyBytes_FromStringAndSize((const char*)&m, sizeof(m));
  return raw ? raw : not_ordinary();
}

/* mx_product(x, w, offsets, dtype) */
static PyObject* mx_product(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, sx[2], sw[3];
  moe_mx x, w;
  void *off = NULL, *p;
  moe_stream_t s;
  ORDINARY(n == 4 && mx_of(a[0], &dev, &x) && mx_of(a[1], &dev, &w) && stream_of(dev, &s));
  const int type = float_type(a[3]);
  ORDINARY(type >= 0 && sizes(PyObject_GetAttr(a[0], s_shape), 2, sx));
  int64_t E = 1, N = w.rows;
  PyObject* shape = PyObject_GetAttr(a[1], s_shape);
  ORDINARY(shape);
  if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 3) {
    ORDINARY(sizes(shape, 3, sw)); /* takes the reference */
    E = sw[0];
    N = sw[1];
  } else {
    Py_DECREF(shape);
  }
  const int64_t groups = E + 1;
  ORDINARY(a[2] == Py_None ? E == 1 : arg_of(a[2], &dev, g.i32, g.i32, 1, &groups, &off, NULL));
  const int64_t sh[2] = {sx[0], N};
  ORDINARY(sx[0] >= 1);
  PyObject* out = new_tensor(2, sh, a[3], &p);
  moe_status st = MOE_OK;
  if (out) LAUNCH(st, PRODUCT, product_fn, &x, &w, (int32_t)E, off, type, p, N, s);
  if (st != MOE_OK) Py_CLEAR(out);
  return out ? out : not_ordinary();
}

/* attach((Tensor, empty, current device, current stream), (f32, bf16, f16, u8, i32, i64),
 *        (MxTensor, Checkpoint, RoutePlan), eleven entry points' addresses) */
static PyObject* attach(PyObject* self, PyObject* args) {
  PyObject* o[13];
  unsigned long long fn[11];
  if (!PyArg_ParseTuple(args, "(OOOO)(OOOOOO)(OOO)(KKKKKKKKKKK)", &o[0], &o[1], &o[2], &o[3], &o[4],
                        &o[5], &o[6], &o[7], &o[8], &o[9], &o[10], &o[11], &o[12], &fn[0], &fn[1],
                        &fn[2], &fn[3], &fn[4], &fn[5], &fn[6], &fn[7], &fn[8], &fn[9], &fn[10]))
    return NULL;
  PyObject** slot[13] = {&g.tensor, &g.empty, &g.get_device, &g.get_stream, &g.f32, &g.bf16, &g.f16,
                         &g.u8, &g.i32, &g.i64, &g.mx, &g.kept, &g.plan};
  if (!PyType_Check(o[0]) || !PyType_Check(o[10]) || !PyType_Check(o[11]) || !PyType_Check(o[12])) {
    PyErr_SetString(PyExc_TypeError, "attach: expected types");
    return NULL;
  }
  for (int i = 0; i < 13; ++i) {
    Py_INCREF(o[i]);
    Py_XSETREF(*slot[i], o[i]);
  }
  for (int i = 0; i < 11; ++i) g.fn[i] = (void*)(uintptr_t)fn[i];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"attach", attach, METH_VARARGS, NULL},
                                FAST(sort_routes),
                                FAST(dispatch),
                                FAST(combine),
                                FAST(combine_grad),
                                FAST(checkpoint),
                                FAST(restore),
                                FAST(expert_act),
                                FAST(expert_act_grad),
                                FAST(mx_quantize),
                                FAST(mx_raw),
                                FAST(mx_product),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
  struct {
    PyObject** name;
    const char* text;
  } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"},
               {&s_device_of, "get_device"}, {&s_data_ptr, "data_ptr"},
               {&s_contiguous, "is_contiguous"}, {&s_raw, "raw"}, {&s_codes, "_codes"},
               {&s_scales, "_scales"}, {&s_buf, "_buf"}, {&s_cut, "_cut"}, {&s_device, "device"},
               {&s_rows, "rows"}, {&s_cols, "cols"}, {&s_act, "act"}, {&s_halves, "halves"},
               {&s_limit, "swiglu_limit"}, {&s_c, "c"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].name = PyUnicode_InternFromString(names[i].text))) return NULL;
  if (!(empty_tuple = PyTuple_New(0))) return NULL;
  return PyModule_Create(&module);
}
