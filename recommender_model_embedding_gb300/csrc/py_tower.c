/* Python side of the expert-tower calls: tensors' attributes are checked and handed to the C entry
 * points of libemb.so.
 *
 * The kernels behind a small call run for a few microseconds, so the host's share of the call is
 * what a caller waits for: read from Python with ctypes, the arguments of one call cost about as
 * much as its launch.  The attributes are the public ones (dtype, shape, stride(), data_ptr(),
 * ...), so any object that has them serves.  Every check comes before the library is called: a
 * mismatch raises ValueError, a status of the library the package's EmbError. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdlib.h>

#include "emb.h"

static PyObject *s_dtype, *s_shape, *s_stride, *s_is_cuda, *s_data_ptr, *s_numel, *s_is_contiguous,
    *s_get_device, *s_cuda_stream, *s_element_size;
static PyObject *t_f32, *t_bf16, *t_i32, *t_i64; /* torch's dtypes */
static PyObject *f_raw_stream, *f_check, *f_workspace;

static const char* kPackage = "recommender_model_embedding_gb300";

/* torch's dtypes and the package's helpers, on the first call (the package imports without torch) */
static int setup(void) {
  PyObject *torch, *c, *pkg;
  if (f_check) return 1;
  torch = PyImport_ImportModule("torch");
  pkg = PyImport_ImportModule(kPackage);
  if (!torch || !pkg) return 0;
  t_f32 = PyObject_GetAttrString(torch, "float32");
  t_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  t_i32 = PyObject_GetAttrString(torch, "int32");
  t_i64 = PyObject_GetAttrString(torch, "int64");
  c = PyObject_GetAttrString(torch, "_C");
  f_raw_stream = c ? PyObject_GetAttrString(c, "_cuda_getCurrentRawStream") : NULL;
  if (!f_raw_stream) {
    PyErr_Clear();
    f_raw_stream = PyObject_GetAttrString(pkg, "_current_stream");
  }
  f_workspace = PyObject_GetAttrString(pkg, "_new_workspace");
  f_check = PyObject_GetAttrString(pkg, "_check");
  Py_XDECREF(c);
  Py_DECREF(torch);
  Py_DECREF(pkg);
  if (t_f32 && t_bf16 && t_i32 && t_i64 && f_raw_stream && f_workspace && f_check) return 1;
  Py_CLEAR(f_check);
  return 0;
}

/* ---- attributes (0: an exception is set) ---- */

static int truth(PyObject* o, int* v) { /* takes the reference */
  if (!o) return 0;
  *v = o == Py_True ? 1 : o == Py_False ? 0 : PyObject_IsTrue(o);
  Py_DECREF(o);
  return *v >= 0;
}

static int number(PyObject* o, int64_t* v) { /* takes the reference */
  if (!o) return 0;
  *v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return !(*v == -1 && PyErr_Occurred());
}

static int address(PyObject* t, void** p) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!o) return 0;
  *p = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return !(!*p && PyErr_Occurred());
}

static int is_cuda(PyObject* t, const char* name) {
  int v;
  if (!truth(PyObject_GetAttr(t, s_is_cuda), &v)) return 0;
  if (!v) PyErr_Format(PyExc_ValueError, "%s: expected a CUDA tensor", name);
  return v;
}

/* two entries of a shape or of strides */
static int pair(PyObject* o, const char* name, int64_t* a, int64_t* b) { /* takes the reference */
  if (!o) return 0;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) {
    Py_DECREF(o);
    PyErr_Format(PyExc_ValueError, "%s: expected a matrix", name);
    return 0;
  }
  *a = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0));
  *b = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1));
  Py_DECREF(o);
  return !PyErr_Occurred();
}

/* EMB_F32 or EMB_BF16 of a matrix, its dtype (borrowed: torch's own) and its size */
static int matrix(PyObject* t, const char* name, int32_t* code, PyObject** dtype, int64_t* n, int64_t* d) {
  PyObject* o = PyObject_GetAttr(t, s_dtype);
  if (!o) return 0;
  *dtype = o == t_f32 ? t_f32 : o == t_bf16 ? t_bf16 : NULL;
  if (!*dtype) {
    PyErr_Format(PyExc_ValueError, "%s: expected float32 or bfloat16, got %S", name, o);
    Py_DECREF(o);
    return 0;
  }
  Py_DECREF(o);
  *code = *dtype == t_bf16 ? EMB_BF16 : EMB_F32;
  return pair(PyObject_GetAttr(t, s_shape), name, n, d);
}

static int has_dtype(PyObject* t, PyObject* dtype, const char* name) {
  PyObject* o = PyObject_GetAttr(t, s_dtype);
  int ok;
  if (!o) return 0;
  ok = o == dtype;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s: expected dtype %S, got %S", name, dtype, o);
  Py_DECREF(o);
  return ok;
}

/* a CUDA matrix [n, d] of dtype whose rows may lie any number of elements apart */
static int rows(PyObject* t, PyObject* dtype, int64_t n, int64_t d, const char* name, void** p, int64_t* ld) {
  int64_t a, b, step, inner;
  if (!has_dtype(t, dtype, name) || !is_cuda(t, name)) return 0;
  if (!pair(PyObject_GetAttr(t, s_shape), name, &a, &b)) return 0;
  if (a != n || b != d) {
    PyErr_Format(PyExc_ValueError, "%s: (%lld, %lld), expected (%lld, %lld)", name, (long long)a,
                 (long long)b, (long long)n, (long long)d);
    return 0;
  }
  if (!pair(PyObject_CallMethodNoArgs(t, s_stride), name, &step, &inner)) return 0;
  if (inner != 1 && d > 1) {
    PyErr_Format(PyExc_ValueError, "%s: the elements of a row must be adjacent", name);
    return 0;
  }
  *ld = n > 1 ? step : d;
  return address(t, p);
}

static int opt_rows(PyObject* t, PyObject* dtype, int64_t n, int64_t d, const char* name, void** p,
                    int64_t* ld) {
  *p = NULL, *ld = 0;
  return t == Py_None || rows(t, dtype, n, d, name, p, ld);
}

/* a contiguous CUDA tensor of dtype and at least n elements (`exact`: of n) */
static int flat(PyObject* t, PyObject* dtype, int64_t n, int exact, const char* name, void** p) {
  int64_t m;
  int dense;
  if (t == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s: expected a CUDA tensor", name);
    return 0;
  }
  if (!has_dtype(t, dtype, name) || !is_cuda(t, name)) return 0;
  if (!number(PyObject_CallMethodNoArgs(t, s_numel), &m)) return 0;
  if (!truth(PyObject_CallMethodNoArgs(t, s_is_contiguous), &dense)) return 0;
  if (!dense) {
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous CUDA tensor", name);
    return 0;
  }
  if (m < n || (exact && m != n)) {
    PyErr_Format(PyExc_ValueError, "%s: %lld elements, %s%lld needed", name, (long long)m,
                 exact ? "" : "at least ", (long long)n);
    return 0;
  }
  return address(t, p);
}

static int vec(PyObject* t, int64_t d, const char* name, void** p) { /* optional float32 [d] */
  *p = NULL;
  return t == Py_None || flat(t, t_f32, d, 1, name, p);
}

/* the call's stream: the given one, or the current one of the tensor's device */
static int on(PyObject* stream, PyObject* like, void** s) {
  PyObject *o, *dev;
  if (stream != Py_None) {
    o = PyObject_GetAttr(stream, s_cuda_stream);
  } else {
    dev = PyObject_CallMethodNoArgs(like, s_get_device);
    if (!dev) return 0;
    o = PyObject_CallOneArg(f_raw_stream, dev);
    Py_DECREF(dev);
  }
  if (!o) return 0;
  *s = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return !(!*s && PyErr_Occurred());
}

/* The workspace of a call that needs `need` bytes: the caller's (any contiguous CUDA tensor of
 * enough bytes), or one from torch's allocator on the call's stream, whose memory is reused in
 * that stream's order.  *keep: a reference to drop after the call. */
static int workspace(int64_t need, PyObject* ws, PyObject* stream, PyObject* like, PyObject** keep,
                     void** p, int64_t* have) {
  int64_t m, size;
  int dense;
  *keep = NULL, *p = NULL, *have = 0;
  if (need <= 0) return 1;
  if (ws == Py_None) {
    PyObject* n = PyLong_FromLongLong(need);
    if (!n) return 0;
    *keep = PyObject_CallFunctionObjArgs(f_workspace, n, stream, like, NULL);
    Py_DECREF(n);
    *have = need;
    if (*keep && address(*keep, p)) return 1;
    Py_CLEAR(*keep);
    return 0;
  }
  if (!is_cuda(ws, "workspace")) return 0;
  if (!number(PyObject_CallMethodNoArgs(ws, s_numel), &m)) return 0;
  if (!number(PyObject_CallMethodNoArgs(ws, s_element_size), &size)) return 0;
  if (!truth(PyObject_CallMethodNoArgs(ws, s_is_contiguous), &dense)) return 0;
  *have = m * size;
  if (!dense || *have < need) {
    PyErr_Format(PyExc_ValueError, "workspace: %lld bytes%s, at least %lld contiguous ones needed",
                 (long long)*have, dense ? "" : " apart", (long long)need);
    return 0;
  }
  return address(ws, p);
}

static PyObject* done(emb_status st, const char* call) {
  if (st != EMB_OK) return PyObject_CallFunction(f_check, "si", call, (int)st); /* raises */
  Py_RETURN_NONE;
}

static int args_are(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return got == want && setup();
}

/* experts of a row: k of a pos with n * k places */
static int slots(PyObject* pos, int64_t n, int64_t* k, void** p) {
  int64_t m;
  if (!number(PyObject_CallMethodNoArgs(pos, s_numel), &m)) return 0;
  if (n == 0 ? m != 0 : (m == 0 || m % n)) {
    PyErr_Format(PyExc_ValueError, "pos: %lld elements, expected a multiple of %lld rows", (long long)m,
                 (long long)n);
    return 0;
  }
  *k = n ? m / n : 1;
  if (*k > INT32_MAX) *k = INT32_MAX; /* refused by the library */
  return flat(pos, t_i32, m, 0, "pos", p);
}

static int fits_int(int64_t v, const char* name) {
  if (v >= 0 && v <= INT32_MAX) return 1;
  PyErr_Format(PyExc_ValueError, "%s: %lld is out of range", name, (long long)v);
  return 0;
}

/* ---- the calls ---- */

/* (ids, num_experts, order, pos, offsets, workspace, stream) */
static PyObject* py_sort(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  int64_t n, k, E, S, have;
  void *ids, *order, *pos, *off, *ws, *s;
  PyObject* keep;
  emb_status st;
  if (!args_are(na, 7)) return NULL;
  if (!pair(PyObject_GetAttr(a[0], s_shape), "ids", &n, &k)) return NULL;
  E = PyLong_AsLongLong(a[1]);
  if (E == -1 && PyErr_Occurred()) return NULL;
  if (!fits_int(k, "ids") || !fits_int(E, "num_experts")) return NULL;
  S = n * k;
  if (!flat(a[0], t_i64, S, 0, "ids", &ids) || !flat(a[2], t_i32, S, 0, "order", &order) ||
      !flat(a[3], t_i32, S, 0, "pos", &pos) || !flat(a[4], t_i32, E + 1, 0, "offsets", &off) ||
      !workspace(emb_expert_sort_workspace(n, (int32_t)k, (int32_t)E), a[5], a[6], a[0], &keep, &ws, &have))
    return NULL;
  if (!on(a[6], a[0], &s)) {
    Py_XDECREF(keep);
    return NULL;
  }
  Py_BEGIN_ALLOW_THREADS;
  st = emb_expert_sort(ids, n, (int32_t)k, (int32_t)E, order, pos, off, ws, have, s);
  Py_END_ALLOW_THREADS;
  Py_XDECREF(keep);
  return done(st, "emb_expert_sort");
}

/* (x, pos, xs, stream) */
static PyObject* py_dispatch(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  int64_t n, d, k, xl, ol;
  int32_t code;
  PyObject* t;
  void *x, *pos, *xs, *s;
  emb_status st;
  if (!args_are(na, 4) || !matrix(a[0], "x", &code, &t, &n, &d) || !fits_int(d, "x") ||
      !slots(a[1], n, &k, &pos) || !rows(a[0], t, n, d, "x", &x, &xl) ||
      !rows(a[2], t, n * k, d, "xs", &xs, &ol) || !on(a[3], a[0], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_expert_dispatch(x, xl, pos, n, (int32_t)k, (int32_t)d, code, xs, ol, s);
  Py_END_ALLOW_THREADS;
  return done(st, "emb_expert_dispatch");
}

/* (dxs, pos, dx, stream) */
static PyObject* py_dispatch_backward(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  int64_t n, d, k, il, ol;
  int32_t code;
  PyObject* t;
  void *in, *pos, *out, *s;
  emb_status st;
  if (!args_are(na, 4) || !matrix(a[2], "dx", &code, &t, &n, &d) || !fits_int(d, "dx") ||
      !slots(a[1], n, &k, &pos) || !rows(a[0], t, n * k, d, "dxs", &in, &il) ||
      !rows(a[2], t, n, d, "dx", &out, &ol) || !on(a[3], a[2], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_expert_dispatch_backward(in, il, pos, n, (int32_t)k, (int32_t)d, code, out, ol, s);
  Py_END_ALLOW_THREADS;
  return done(st, "emb_expert_dispatch_backward");
}

/* (ys, pos, w, out, stream) */
static PyObject* py_combine(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  int64_t n, d, k, il, ol;
  int32_t code;
  PyObject* t;
  void *in, *pos, *w, *out, *s;
  emb_status st;
  if (!args_are(na, 5) || !matrix(a[3], "out", &code, &t, &n, &d) || !fits_int(d, "out") ||
      !slots(a[1], n, &k, &pos) || !rows(a[0], t, n * k, d, "ys", &in, &il) ||
      !flat(a[2], t_f32, n * k, 0, "w", &w) || !rows(a[3], t, n, d, "out", &out, &ol) ||
      !on(a[4], a[3], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_expert_combine(in, il, pos, w, n, (int32_t)k, (int32_t)d, code, out, ol, s);
  Py_END_ALLOW_THREADS;
  return done(st, "emb_expert_combine");
}

/* (dout, ys, pos, w, dys, dw, stream) */
static PyObject* py_combine_backward(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  int64_t n, d, k, gl, yl, ol;
  int32_t code;
  PyObject* t;
  void *g, *y, *pos, *w, *out, *dw, *s;
  emb_status st;
  if (!args_are(na, 7) || !matrix(a[0], "dout", &code, &t, &n, &d) || !fits_int(d, "dout") ||
      !slots(a[2], n, &k, &pos) || !rows(a[0], t, n, d, "dout", &g, &gl) ||
      !rows(a[1], t, n * k, d, "ys", &y, &yl) || !flat(a[3], t_f32, n * k, 0, "w", &w) ||
      !rows(a[4], t, n * k, d, "dys", &out, &ol) || !flat(a[5], t_f32, n * k, 0, "dw", &dw) ||
      !on(a[6], a[0], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_expert_combine_backward(g, gl, y, yl, pos, w, n, (int32_t)k, (int32_t)d, code, out, ol, dw, s);
  Py_END_ALLOW_THREADS;
  return done(st, "emb_expert_combine_backward");
}

/* sizes and types of a gated-norm call: from the stream's matrix x, and the block's matrices y or,
 * without them, b (h or its gradient) */
static int norm_sizes(emb_norm* p, PyObject* x, const char* xname, PyObject* y, PyObject* b,
                      const char* bname, PyObject** xt, PyObject** bt) {
  int64_t d, m;
  PyObject* block = y != Py_None ? y : b;
  if (!matrix(x, xname, &p->x_dtype, xt, &p->n, &d) || !fits_int(d, xname)) return 0;
  p->dim = (int32_t)d;
  p->dtype = p->x_dtype, *bt = *xt;
  return block == Py_None || matrix(block, y != Py_None ? "y" : bname, &p->dtype, bt, &m, &m);
}

static int norm_gate(emb_norm* p, PyObject* gate, PyObject* bt) {
  int64_t n, cols;
  void* q;
  if (gate == Py_None) return 1;
  if (!pair(PyObject_GetAttr(gate, s_shape), "gate", &n, &cols)) return 0;
  if (cols != 1 && cols != p->dim) {
    PyErr_Format(PyExc_ValueError, "gate: %lld columns, expected 1 or %d", (long long)cols, (int)p->dim);
    return 0;
  }
  p->gate_cols = (int32_t)cols;
  if (!rows(gate, bt, p->n, cols, "gate", &q, &p->gate_ld)) return 0;
  p->d_gate = q;
  return 1;
}

static int norm_vecs(emb_norm* p, PyObject* w_post, PyObject* res_scale, PyObject* w_pre) {
  void *a, *b, *c;
  if (!vec(w_post, p->dim, "w_post", &a) || !vec(res_scale, p->dim, "res_scale", &b) ||
      !vec(w_pre, p->dim, "w_pre", &c))
    return 0;
  p->d_w_post = a, p->d_res_scale = b, p->d_w_pre = c;
  return 1;
}

/* (x, y, x_out, h, gate, w_post, res_scale, w_pre, eps, stream) */
static PyObject* py_norm(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  emb_norm p = {0};
  PyObject *xt, *bt;
  void *x, *y, *s;
  emb_status st;
  if (!args_are(na, 10) || !norm_sizes(&p, a[0], "x", a[1], a[3], "h", &xt, &bt) ||
      !rows(a[0], xt, p.n, p.dim, "x", &x, &p.x_ld) || !opt_rows(a[1], bt, p.n, p.dim, "y", &y, &p.y_ld) ||
      !opt_rows(a[2], xt, p.n, p.dim, "x_out", &p.d_x_out, &p.x_out_ld) ||
      !opt_rows(a[3], bt, p.n, p.dim, "h", &p.d_h, &p.h_ld) || !norm_gate(&p, a[4], bt) ||
      !norm_vecs(&p, a[5], a[6], a[7]))
    return NULL;
  p.d_x = x, p.d_y = y;
  p.eps = (float)PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred() || !on(a[9], a[0], &s)) return NULL;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_gated_norm(&p, s);
  Py_END_ALLOW_THREADS;
  return done(st, "emb_gated_norm");
}

/* (dx_out, dh, x_out, y, dx, dy, gate, w_post, res_scale, w_pre, dgate, dw_post, dres_scale, dw_pre,
 *  eps, workspace, stream) */
static PyObject* py_norm_backward(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  emb_norm p = {0};
  PyObject *xt, *bt, *keep;
  void *t, *h, *y, *dgate, *u, *v, *w, *ws, *s;
  int64_t have;
  emb_status st;
  if (!args_are(na, 17) || !norm_sizes(&p, a[2], "x_out", a[3], a[1], "dh", &xt, &bt) ||
      !rows(a[2], xt, p.n, p.dim, "x_out", &p.d_x_out, &p.x_out_ld) ||
      !opt_rows(a[0], xt, p.n, p.dim, "dx_out", &t, &p.dx_out_ld) ||
      !opt_rows(a[1], bt, p.n, p.dim, "dh", &h, &p.dh_ld) ||
      !opt_rows(a[3], bt, p.n, p.dim, "y", &y, &p.y_ld) ||
      !opt_rows(a[4], xt, p.n, p.dim, "dx", &p.d_dx, &p.dx_ld) ||
      !opt_rows(a[5], bt, p.n, p.dim, "dy", &p.d_dy, &p.dy_ld) || !norm_gate(&p, a[6], bt) ||
      !opt_rows(a[10], bt, p.n, p.gate_cols ? p.gate_cols : p.dim, "dgate", &dgate, &p.dgate_ld) ||
      !norm_vecs(&p, a[7], a[8], a[9]) || !vec(a[11], p.dim, "dw_post", &u) ||
      !vec(a[12], p.dim, "dres_scale", &v) || !vec(a[13], p.dim, "dw_pre", &w))
    return NULL;
  p.d_dx_out = t, p.d_dh = h, p.d_y = y, p.d_dgate = dgate;
  p.d_dw_post = u, p.d_dres_scale = v, p.d_dw_pre = w;
  p.eps = (float)PyFloat_AsDouble(a[14]);
  if (PyErr_Occurred() ||
      !workspace(a[15] == Py_None && emb_gated_norm_backward_one_launch(p.n, p.dim)
                     ? 0
                     : emb_gated_norm_backward_workspace(p.n, p.dim),
                 a[15], a[16], a[2], &keep, &ws, &have))
    return NULL;
  if (!on(a[16], a[2], &s)) {
    Py_XDECREF(keep);
    return NULL;
  }
  Py_BEGIN_ALLOW_THREADS;
  st = emb_gated_norm_backward(&p, ws, have, s);
  Py_END_ALLOW_THREADS;
  Py_XDECREF(keep);
  return done(st, "emb_gated_norm_backward");
}

static int dense_tensor(PyObject* t, const char* name, PyObject** dtype, int64_t* n, void** p) {
  PyObject* o = PyObject_GetAttr(t, s_dtype);
  int dense;
  if (!o) return 0;
  *dtype = o == t_f32 ? t_f32 : o == t_bf16 ? t_bf16 : NULL;
  if (!*dtype) PyErr_Format(PyExc_ValueError, "%s: expected float32 or bfloat16, got %S", name, o);
  Py_DECREF(o);
  if (!*dtype || !is_cuda(t, name)) return 0;
  if (!truth(PyObject_CallMethodNoArgs(t, s_is_contiguous), &dense)) return 0;
  if (!dense) {
    PyErr_Format(PyExc_ValueError, "%s: expected contiguous CUDA tensors", name);
    return 0;
  }
  return number(PyObject_CallMethodNoArgs(t, s_numel), n) && address(t, p);
}

/* (grads, max_norm, norm, out, workspace, stream) */
static PyObject* py_clip(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  PyObject *grads = NULL, *out = NULL, *keep = NULL, *res = NULL, *t, *u;
  emb_tensor* list = NULL;
  Py_ssize_t count, i;
  int64_t total = 0, m, have;
  double max_norm;
  void *norm, *ws, *s, *p;
  emb_status st;
  if (!args_are(na, 6)) return NULL;
  grads = PySequence_Fast(a[0], "grads: expected a list of tensors");
  if (!grads) goto end;
  count = PySequence_Fast_GET_SIZE(grads);
  if (a[3] != Py_None) {
    out = PySequence_Fast(a[3], "out: expected a list of tensors");
    if (!out) goto end;
    if (PySequence_Fast_GET_SIZE(out) != count) {
      PyErr_Format(PyExc_ValueError, "out: %zd tensors for %zd gradients", PySequence_Fast_GET_SIZE(out), count);
      goto end;
    }
  }
  max_norm = PyFloat_AsDouble(a[1]);
  if (max_norm == -1.0 && PyErr_Occurred()) goto end;
  list = calloc(count ? (size_t)count : 1, sizeof(emb_tensor));
  if (!list) {
    PyErr_NoMemory();
    goto end;
  }
  for (i = 0; i < count; ++i) {
    if (!dense_tensor(PySequence_Fast_GET_ITEM(grads, i), "grads", &t, &list[i].numel, &p)) goto end;
    list[i].dtype = t == t_bf16 ? EMB_BF16 : EMB_F32;
    list[i].d_src = list[i].d_out = p;
    total += list[i].numel;
    if (out) {
      if (!dense_tensor(PySequence_Fast_GET_ITEM(out, i), "out", &u, &m, &p)) goto end;
      if (u != t || m != list[i].numel) {
        PyErr_Format(PyExc_ValueError, "out: tensor %zd is not of its gradient's type and size", i);
        goto end;
      }
      list[i].d_out = p;
    }
  }
  if (!flat(a[2], t_f32, 1, 0, "norm", &norm)) goto end;
  /* short lists take one launch and no workspace */
  if (!workspace(total <= EMB_CLIP_ONE_LAUNCH && count <= 256 ? 0 : emb_clip_grads_workspace(count), a[4],
                 a[5], a[2], &keep, &ws, &have) ||
      !on(a[5], a[2], &s))
    goto end;
  Py_BEGIN_ALLOW_THREADS;
  st = emb_clip_grads(list, count, (float)max_norm, norm, ws, have, s);
  Py_END_ALLOW_THREADS;
  res = done(st, "emb_clip_grads");
end:
  free(list);
  Py_XDECREF(keep);
  Py_XDECREF(grads);
  Py_XDECREF(out);
  return res;
}

static PyMethodDef methods[] = {
    {"sort", (PyCFunction)(void (*)(void))py_sort, METH_FASTCALL, NULL},
    {"dispatch", (PyCFunction)(void (*)(void))py_dispatch, METH_FASTCALL, NULL},
    {"dispatch_backward", (PyCFunction)(void (*)(void))py_dispatch_backward, METH_FASTCALL, NULL},
    {"combine", (PyCFunction)(void (*)(void))py_combine, METH_FASTCALL, NULL},
    {"combine_backward", (PyCFunction)(void (*)(void))py_combine_backward, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL, NULL},
    {"norm_backward", (PyCFunction)(void (*)(void))py_norm_backward, METH_FASTCALL, NULL},
    {"clip", (PyCFunction)(void (*)(void))py_clip, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tower", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tower(void) {
  struct {
    PyObject** to;
    const char* text;
  } names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},
               {&s_stride, "stride"},     {&s_is_cuda, "is_cuda"},
               {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
               {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"},
               {&s_cuda_stream, "cuda_stream"},     {&s_element_size, "element_size"}};
  size_t i;
  for (i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].text))) return NULL;
  return PyModule_Create(&module);
}
