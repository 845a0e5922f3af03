// Python side of the expert-tower calls: tensors are checked and their addresses handed to the C
// entry points of libemb.so.
//
// The kernels behind a small call run for a few microseconds, so the host's share of the call is
// what a caller waits for.  Read from Python with ctypes, the arguments of one call cost about
// as much as its launch; read from the tensor object itself they cost next to nothing.  Objects
// that are not torch's own tensors are read through the same public attributes (dtype, shape,
// stride(), data_ptr(), ...).  Every check comes before the library is called: a mismatch raises
// ValueError, a status of the library the package's EmbError.  A call's tensors, its workspace and
// its stream are on one device, and that device is the current one while the library is called.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdlib>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <string>
#include <vector>

#include "emb.h"

namespace {

enum Kind { F32, BF16, I32, I64, OTHER };
const char* const kKindNames[] = {"float32", "bfloat16", "int32", "int64", "another type (float16, say)"};
constexpr const char* kPackage = "recommender_model_embedding_gb300";

// A Python exception is set; unwinds to the call's guard.
struct Raised : std::exception {};

template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Raised();
}

struct Ref {  // an owned reference
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {
    if (!o) throw Raised();
  }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_DECREF(o); }
};

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v;
}

// What the checks read of a tensor.
struct Seen {
  Kind kind = OTHER;
  int64_t dims = 0, numel = 0, size[2] = {0, 0}, step[2] = {0, 0};
  bool cuda = false, dense = false;
  int device = -1;
  void* p = nullptr;
};

// The one device of a call: that of the first tensor seen.
struct Device {
  int index = -1;
  c10::cuda::OptionalCUDAGuard guard;
  void same(int other, const char* name) {
    if (other < 0) return;  // an object that does not say
    if (index < 0) index = other;
    if (other != index) refuse("%s: on cuda:%d, the call's first tensor is on cuda:%d", name, other, index);
  }
  // makes it current until the call returns (where there is none, the library's call says so)
  void enter() {
    const int devices = c10::cuda::device_count();
    if (index < 0 || devices == 0 || (devices == 1 && index == 0)) return;
    if (c10::cuda::current_device() != index) guard.set_index((c10::DeviceIndex)index);
  }
};

Seen see_object(PyObject* o) {  // through attributes
  Seen s;
  const Ref dtype(PyObject_GetAttrString(o, "dtype"));
  const Ref name(PyObject_Str(dtype.o));
  const char* text = PyUnicode_AsUTF8(name.o);
  if (!text) throw Raised();
  for (int k = F32; k < OTHER; ++k)
    if (std::string("torch.") + kKindNames[k] == text) s.kind = (Kind)k;
  const Ref cuda(PyObject_GetAttrString(o, "is_cuda"));
  s.cuda = truth(cuda.o);
  if (s.cuda && PyObject_HasAttrString(o, "device")) {
    const Ref device(PyObject_GetAttrString(o, "device"));
    const Ref name(PyObject_Str(device.o));  // cuda:N
    const char* text = PyUnicode_AsUTF8(name.o);
    if (!text) throw Raised();
    if (const char* colon = std::strchr(text, ':')) s.device = std::atoi(colon + 1);
  }
  const Ref shape(PyObject_GetAttrString(o, "shape"));
  const Ref step(PyObject_CallMethod(o, "stride", nullptr));
  s.dims = PySequence_Size(shape.o);
  if (s.dims < 0) throw Raised();
  if (s.dims == 2)
    for (int i = 0; i < 2; ++i) {
      const Ref a(PySequence_GetItem(shape.o, i)), b(PySequence_GetItem(step.o, i));
      s.size[i] = number(a.o), s.step[i] = number(b.o);
    }
  const Ref numel(PyObject_CallMethod(o, "numel", nullptr)), dense(PyObject_CallMethod(o, "is_contiguous", nullptr));
  s.numel = number(numel.o), s.dense = truth(dense.o);
  const Ref p(PyObject_CallMethod(o, "data_ptr", nullptr));
  s.p = PyLong_AsVoidPtr(p.o);
  if (!s.p && PyErr_Occurred()) throw Raised();
  return s;
}

Seen see(PyObject* o, const char* name, Device& dev) {
  if (o == Py_None) refuse("%s: expected a CUDA tensor", name);
  if (!THPVariable_CheckExact(o)) {
    const Seen s = see_object(o);
    if (s.cuda) dev.same(s.device, name);
    return s;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  Seen s;
  if (t.layout() != c10::kStrided) refuse("%s: expected a dense tensor", name);
  switch (t.scalar_type()) {
    case at::kFloat: s.kind = F32; break;
    case at::kBFloat16: s.kind = BF16; break;
    case at::kInt: s.kind = I32; break;
    case at::kLong: s.kind = I64; break;
    default: break;
  }
  s.dims = t.dim(), s.numel = t.numel();
  s.cuda = t.is_cuda(), s.dense = t.is_contiguous();
  if (s.dims == 2)
    for (int i = 0; i < 2; ++i) s.size[i] = t.size(i), s.step[i] = t.stride(i);
  if (s.cuda) s.device = t.get_device(), s.p = t.data_ptr(), dev.same(s.device, name);
  return s;
}

// EMB_F32 or EMB_BF16 of a matrix
int32_t code_of(const Seen& s, const char* name) {
  if (s.kind != F32 && s.kind != BF16) refuse("%s: expected float32 or bfloat16, got %s", name, kKindNames[s.kind]);
  if (s.dims != 2) refuse("%s: expected a matrix", name);
  return s.kind == BF16 ? EMB_BF16 : EMB_F32;
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};

// a CUDA matrix [n, d] of the kind whose rows may lie any number of elements apart
Rows rows(const Seen& s, Kind kind, int64_t n, int64_t d, const char* name) {
  if (s.kind != kind) refuse("%s: expected dtype %s, got %s", name, kKindNames[kind], kKindNames[s.kind]);
  if (!s.cuda) refuse("%s: expected a CUDA tensor", name);
  if (s.dims != 2) refuse("%s: expected a matrix", name);
  if (s.size[0] != n || s.size[1] != d)
    refuse("%s: (%lld, %lld), expected (%lld, %lld)", name, (long long)s.size[0], (long long)s.size[1],
           (long long)n, (long long)d);
  if (s.step[1] != 1 && d > 1) refuse("%s: the elements of a row must be adjacent", name);
  return {s.p, n > 1 ? s.step[0] : d};
}

Rows rows(PyObject* o, Kind kind, int64_t n, int64_t d, const char* name, Device& dev) {
  return rows(see(o, name, dev), kind, n, d, name);
}

Rows opt_rows(PyObject* o, Kind kind, int64_t n, int64_t d, const char* name, Device& dev) {
  return o == Py_None ? Rows{} : rows(o, kind, n, d, name, dev);
}

// a contiguous CUDA tensor of the kind and at least n elements (`exact`: of n)
void* flat(const Seen& s, Kind kind, int64_t n, bool exact, const char* name) {
  if (s.kind != kind) refuse("%s: expected dtype %s, got %s", name, kKindNames[kind], kKindNames[s.kind]);
  if (!s.cuda || !s.dense) refuse("%s: expected a contiguous CUDA tensor", name);
  if (s.numel < n || (exact && s.numel != n))
    refuse("%s: %lld elements, %s%lld needed", name, (long long)s.numel, exact ? "" : "at least ", (long long)n);
  return s.p;
}

void* flat(PyObject* o, Kind kind, int64_t n, const char* name, Device& dev) {
  return flat(see(o, name, dev), kind, n, false, name);
}

// a value for each slot of n rows of k: as flat(), and a matrix has to be k wide (one of another width
// would be read and written as if its rows were k long)
void* by_slot(const Seen& s, Kind kind, int64_t n, int64_t k, const char* name) {
  if (s.dims == 2 && s.size[0] > 1 && s.size[1] > 1 && s.size[1] != k)
    refuse("%s: (%lld, %lld), expected (%lld, %lld)", name, (long long)s.size[0], (long long)s.size[1],
           (long long)n, (long long)k);
  return flat(s, kind, n * k, false, name);
}

void* by_slot(PyObject* o, Kind kind, int64_t n, int64_t k, const char* name, Device& dev) {
  return by_slot(see(o, name, dev), kind, n, k, name);
}

void* vec(PyObject* o, int64_t d, const char* name, Device& dev) {  // optional float32 [d]
  return o == Py_None ? nullptr : flat(see(o, name, dev), F32, d, true, name);
}

int32_t fits_int(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) refuse("%s: %lld is out of range", name, (long long)v);
  return (int32_t)v;
}

// the call's stream: the given one, or the current one of the call's device
void* stream_of(PyObject* stream, Device& dev) {
  if (stream == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
  if (PyObject_HasAttrString(stream, "device_index")) {
    const Ref index(PyObject_GetAttrString(stream, "device_index"));
    dev.same((int)number(index.o), "stream");
  }
  const Ref o(PyObject_GetAttrString(stream, "cuda_stream"));
  void* s = PyLong_AsVoidPtr(o.o);
  if (!s && PyErr_Occurred()) throw Raised();
  return s;
}

// The workspace of a call: the caller's (any contiguous CUDA tensor of enough bytes, checked at
// once), or one that take() gets from torch's allocator for the call's stream, given back after
// the call and reused in that stream's order.
struct Workspace {
  void* p = nullptr;
  int64_t bytes = 0;
  bool mine = false;
  Workspace(int64_t need, PyObject* ws, Device& dev) {
    if (need <= 0) return;
    bytes = need;
    mine = ws == Py_None;
    if (mine) return;
    const Seen s = see(ws, "workspace", dev);
    if (!s.cuda || !s.dense) refuse("workspace: expected a contiguous CUDA tensor");
    const Ref size(PyObject_CallMethod(ws, "element_size", nullptr));
    p = s.p, bytes = s.numel * number(size.o);
    if (bytes < need) refuse("workspace: %lld bytes, at least %lld needed", (long long)bytes, (long long)need);
  }
  void take(void* stream) {
    if (mine) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream((size_t)bytes, (cudaStream_t)stream);
  }
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  ~Workspace() {
    if (mine && p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

// A tensor that a call has written is new to autograd, as after torch's own operations in place: a
// backward that saved what it held before says so.
void wrote(PyObject* o) {
  if (o == Py_None || !THPVariable_Check(o)) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();  // (those have no versions)
}

// the library's call without the interpreter's lock; its status as an exception.  `outs`: what it
// writes
template <typename F>
PyObject* call(const char* name, std::initializer_list<PyObject*> outs, F f) {
  emb_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st != EMB_OK) {
    const Ref pkg(PyImport_ImportModule(kPackage));
    const Ref raised(PyObject_CallMethod(pkg.o, "_check", "si", name, (int)st));  // raises
  }
  for (PyObject* o : outs) wrote(o);
  Py_RETURN_NONE;
}

template <typename F>
PyObject* guard(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) {
      PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
      return nullptr;
    }
    return f();
  } catch (const Raised&) {
  } catch (...) {  // torch's own exceptions keep their types (OutOfMemoryError)
    if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// experts of a row: k of a pos with n * k places
struct Places {
  int32_t k;
  const int32_t* p;
};
Places places(PyObject* pos, int64_t n, Device& dev) {
  const Seen s = see(pos, "pos", dev);
  if (n == 0 ? s.numel != 0 : (s.numel == 0 || s.numel % n))
    refuse("pos: %lld elements, expected a multiple of %lld rows", (long long)s.numel, (long long)n);
  const int64_t k = n ? s.numel / n : 1;
  return {fits_int(k, "pos"), static_cast<const int32_t*>(by_slot(s, I32, n, k, "pos"))};
}

// (ids, num_experts, order, pos, offsets, workspace, stream)
PyObject* py_sort(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 7, [&]() -> PyObject* {
    Device dev;
    const Seen ids = see(a[0], "ids", dev);
    if (ids.dims != 2) refuse("ids: expected a matrix [n, k]");
    const int64_t n = ids.size[0], S = ids.numel;
    const int32_t k = fits_int(ids.size[1], "ids"), E = fits_int(number(a[1]), "num_experts");
    const auto* p = static_cast<const int64_t*>(flat(ids, I64, S, false, "ids"));
    auto* order = static_cast<int32_t*>(flat(a[2], I32, S, "order", dev));
    auto* pos = static_cast<int32_t*>(by_slot(a[3], I32, n, k, "pos", dev));
    auto* offsets = static_cast<int32_t*>(flat(a[4], I32, (int64_t)E + 1, "offsets", dev));
    dev.enter();
    Workspace ws(emb_expert_sort_workspace(n, k, E), a[5], dev);
    void* s = stream_of(a[6], dev);
    ws.take(s);
    return call("emb_expert_sort", {a[2], a[3], a[4]}, [&] {
      return emb_expert_sort(p, n, k, E, order, pos, offsets, ws.p, ws.bytes, s);
    });
  });
}

// (x, pos, xs, stream)
PyObject* py_dispatch(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 4, [&]() -> PyObject* {
    Device dev;
    const Seen m = see(a[0], "x", dev);
    const int32_t code = code_of(m, "x"), d = fits_int(m.size[1], "x");
    const int64_t n = m.size[0];
    const Places pos = places(a[1], n, dev);
    const Rows x = rows(m, m.kind, n, d, "x"), xs = rows(a[2], m.kind, n * pos.k, d, "xs", dev);
    dev.enter();
    void* s = stream_of(a[3], dev);
    return call("emb_expert_dispatch", {a[2]},
                [&] { return emb_expert_dispatch(x.p, x.ld, pos.p, n, pos.k, d, code, xs.p, xs.ld, s); });
  });
}

// (dxs, pos, dx, stream)
PyObject* py_dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 4, [&]() -> PyObject* {
    Device dev;
    const Seen m = see(a[2], "dx", dev);
    const int32_t code = code_of(m, "dx"), d = fits_int(m.size[1], "dx");
    const int64_t n = m.size[0];
    const Places pos = places(a[1], n, dev);
    const Rows in = rows(a[0], m.kind, n * pos.k, d, "dxs", dev), out = rows(m, m.kind, n, d, "dx");
    dev.enter();
    void* s = stream_of(a[3], dev);
    return call("emb_expert_dispatch_backward", {a[2]}, [&] {
      return emb_expert_dispatch_backward(in.p, in.ld, pos.p, n, pos.k, d, code, out.p, out.ld, s);
    });
  });
}

// (ys, pos, w, out, stream)
PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 5, [&]() -> PyObject* {
    Device dev;
    const Seen m = see(a[3], "out", dev);
    const int32_t code = code_of(m, "out"), d = fits_int(m.size[1], "out");
    const int64_t n = m.size[0];
    const Places pos = places(a[1], n, dev);
    const Rows in = rows(a[0], m.kind, n * pos.k, d, "ys", dev), out = rows(m, m.kind, n, d, "out");
    const auto* w = static_cast<const float*>(by_slot(a[2], F32, n, pos.k, "w", dev));
    dev.enter();
    void* s = stream_of(a[4], dev);
    return call("emb_expert_combine", {a[3]}, [&] {
      return emb_expert_combine(in.p, in.ld, pos.p, w, n, pos.k, d, code, out.p, out.ld, s);
    });
  });
}

// (dout, ys, pos, w, dys, dw, stream)
PyObject* py_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 7, [&]() -> PyObject* {
    Device dev;
    const Seen m = see(a[0], "dout", dev);
    const int32_t code = code_of(m, "dout"), d = fits_int(m.size[1], "dout");
    const int64_t n = m.size[0];
    const Places pos = places(a[2], n, dev);
    const int64_t S = n * pos.k;
    const Rows g = rows(m, m.kind, n, d, "dout"), y = rows(a[1], m.kind, S, d, "ys", dev),
               dys = rows(a[4], m.kind, S, d, "dys", dev);
    const auto* w = static_cast<const float*>(by_slot(a[3], F32, n, pos.k, "w", dev));
    auto* dw = static_cast<float*>(by_slot(a[5], F32, n, pos.k, "dw", dev));
    dev.enter();
    void* s = stream_of(a[6], dev);
    return call("emb_expert_combine_backward", {a[4], a[5]}, [&] {
      return emb_expert_combine_backward(g.p, g.ld, y.p, y.ld, pos.p, w, n, pos.k, d, code, dys.p, dys.ld, dw, s);
    });
  });
}

// Sizes and types of a gated-norm call: from the stream's matrix, and the block's matrices y or,
// without them, `other` (h or its gradient).
struct NormCall {
  Device dev;
  emb_norm p{};
  Seen x;
  Kind xt, bt;
  int64_t n, d;
  NormCall(PyObject* xo, const char* xname, PyObject* y, PyObject* other, const char* oname, PyObject* gate)
      : x(see(xo, xname, dev)) {
    p.x_dtype = p.dtype = code_of(x, xname);
    p.n = n = x.size[0];
    p.dim = fits_int(d = x.size[1], xname);
    xt = bt = x.kind;
    if (y != Py_None || other != Py_None) {
      const char* name = y != Py_None ? "y" : oname;
      const Seen b = see(y != Py_None ? y : other, name, dev);
      p.dtype = code_of(b, name), bt = b.kind;
    }
    const Rows r = opt_rows(y, bt, n, d, "y", dev);
    p.d_y = r.p, p.y_ld = r.ld;
    if (gate == Py_None) return;
    const Seen g = see(gate, "gate", dev);
    if (g.dims != 2 || (g.size[1] != 1 && g.size[1] != d))
      refuse("gate: expected (%lld, 1) or (%lld, %lld)", (long long)n, (long long)n, (long long)d);
    p.gate_cols = (int32_t)g.size[1];
    const Rows q = rows(g, bt, n, p.gate_cols, "gate");
    p.d_gate = q.p, p.gate_ld = q.ld;
  }
  void vectors(PyObject* w_post, PyObject* res_scale, PyObject* w_pre, PyObject* eps) {
    p.d_w_post = static_cast<const float*>(vec(w_post, d, "w_post", dev));
    p.d_res_scale = static_cast<const float*>(vec(res_scale, d, "res_scale", dev));
    p.d_w_pre = static_cast<const float*>(vec(w_pre, d, "w_pre", dev));
    p.eps = (float)PyFloat_AsDouble(eps);
    if (PyErr_Occurred()) throw Raised();
  }
};

// (x, y, x_out, h, gate, w_post, res_scale, w_pre, eps, stream)
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 10, [&]() -> PyObject* {
    NormCall c(a[0], "x", a[1], a[3], "h", a[4]);
    emb_norm& p = c.p;
    Device& dev = c.dev;
    const Rows x = rows(c.x, c.xt, c.n, c.d, "x"), o = opt_rows(a[2], c.xt, c.n, c.d, "x_out", dev),
               h = opt_rows(a[3], c.bt, c.n, c.d, "h", dev);
    p.d_x = x.p, p.x_ld = x.ld, p.d_x_out = o.p, p.x_out_ld = o.ld, p.d_h = h.p, p.h_ld = h.ld;
    c.vectors(a[5], a[6], a[7], a[8]);
    dev.enter();
    void* s = stream_of(a[9], dev);
    return call("emb_gated_norm", {a[1] != Py_None ? a[2] : Py_None, a[3]}, [&] { return emb_gated_norm(&p, s); });
  });
}

// (dx_out, dh, x_out, y, dx, dy, gate, w_post, res_scale, w_pre, dgate, dw_post, dres_scale, dw_pre,
//  eps, workspace, stream)
PyObject* py_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 17, [&]() -> PyObject* {
    NormCall c(a[2], "x_out", a[3], a[1], "dh", a[6]);
    emb_norm& p = c.p;
    Device& dev = c.dev;
    const int64_t n = c.n, d = c.d;
    const Rows x = rows(c.x, c.xt, n, d, "x_out"), t = opt_rows(a[0], c.xt, n, d, "dx_out", dev),
               h = opt_rows(a[1], c.bt, n, d, "dh", dev), dx = opt_rows(a[4], c.xt, n, d, "dx", dev),
               dy = opt_rows(a[5], c.bt, n, d, "dy", dev),
               dg = opt_rows(a[10], c.bt, n, p.gate_cols ? p.gate_cols : d, "dgate", dev);
    p.d_x_out = x.p, p.x_out_ld = x.ld, p.d_dx_out = t.p, p.dx_out_ld = t.ld, p.d_dh = h.p, p.dh_ld = h.ld;
    p.d_dx = dx.p, p.dx_ld = dx.ld, p.d_dy = dy.p, p.dy_ld = dy.ld, p.d_dgate = dg.p, p.dgate_ld = dg.ld;
    c.vectors(a[7], a[8], a[9], a[14]);
    p.d_dw_post = static_cast<float*>(vec(a[11], d, "dw_post", dev));
    p.d_dres_scale = static_cast<float*>(vec(a[12], d, "dres_scale", dev));
    p.d_dw_pre = static_cast<float*>(vec(a[13], d, "dw_pre", dev));
    dev.enter();
    Workspace ws(emb_gated_norm_backward_workspace(p.n, p.dim), a[15], dev);
    void* s = stream_of(a[16], dev);
    ws.take(s);
    return call("emb_gated_norm_backward", {a[4], a[5], a[10], a[11], a[12], a[13]},
                [&] { return emb_gated_norm_backward(&p, ws.p, ws.bytes, s); });
  });
}

// (grads, max_norm, norm, out, workspace, stream)
PyObject* py_clip(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guard(na, 6, [&]() -> PyObject* {
    Device dev;
    const Ref grads(PySequence_Fast(a[0], "grads: expected a list of tensors"));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(grads.o);
    const bool apart = a[3] != Py_None;
    const Ref out(apart ? PySequence_Fast(a[3], "out: expected a list of tensors") : Py_NewRef(Py_None));
    if (apart && PySequence_Fast_GET_SIZE(out.o) != count)
      refuse("out: %zd tensors for %zd gradients", PySequence_Fast_GET_SIZE(out.o), count);
    const double max_norm = PyFloat_AsDouble(a[1]);
    if (max_norm == -1.0 && PyErr_Occurred()) throw Raised();
    std::vector<emb_tensor> list((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const Seen g = see(PySequence_Fast_GET_ITEM(grads.o, i), "grads", dev);
      if ((g.kind != F32 && g.kind != BF16) || !g.cuda || !g.dense)
        refuse("grads: expected contiguous CUDA tensors, float32 or bfloat16");
      emb_tensor& t = list[(size_t)i];
      t.dtype = g.kind == BF16 ? EMB_BF16 : EMB_F32;
      t.d_src = t.d_out = g.p;
      t.numel = g.numel;
      if (!apart) continue;
      const Seen o = see(PySequence_Fast_GET_ITEM(out.o, i), "out", dev);
      if (o.kind != g.kind || o.numel != g.numel || !o.cuda || !o.dense)
        refuse("out: expected a contiguous CUDA tensor of each gradient's type and size");
      t.d_out = o.p;
    }
    const Seen norm = see(a[2], "norm", dev);
    auto* np = static_cast<float*>(flat(norm, F32, 1, false, "norm"));
    dev.enter();
    Workspace ws(emb_clip_grads_workspace(count), a[4], dev);
    void* s = stream_of(a[5], dev);
    ws.take(s);
    PyObject* done = call("emb_clip_grads", {a[2]}, [&] {
      return emb_clip_grads(list.data(), count, (float)max_norm, np, ws.p, ws.bytes, s);
    });
    for (Py_ssize_t i = 0; i < count; ++i) wrote(PySequence_Fast_GET_ITEM(apart ? out.o : grads.o, i));
    return done;
  });
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"sort", fast(py_sort), METH_FASTCALL, nullptr},
                         {"dispatch", fast(py_dispatch), METH_FASTCALL, nullptr},
                         {"dispatch_backward", fast(py_dispatch_backward), METH_FASTCALL, nullptr},
                         {"combine", fast(py_combine), METH_FASTCALL, nullptr},
                         {"combine_backward", fast(py_combine_backward), METH_FASTCALL, nullptr},
                         {"norm", fast(py_norm), METH_FASTCALL, nullptr},
                         {"norm_backward", fast(py_norm_backward), METH_FASTCALL, nullptr},
                         {"clip", fast(py_clip), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tower", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `torch_version`: the torch whose tensors this module reads in place
PyMODINIT_FUNC PyInit__tower(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", EMB_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
