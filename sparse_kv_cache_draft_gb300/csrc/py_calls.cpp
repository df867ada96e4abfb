// Python calls on rows, drafted trees and bounded caches that need no context: arguments are checked and passed to the C ABI.
//
// A small call's time is the host's. With the checks in Python and the arguments through ctypes, a call on one row
// took 10.2 us on a Grace core (5.2 of checks, 1.8 for its Rotary, 1.1 of ctypes, 2.1 in the launch) where its
// kernel takes 4.6. Here tensors are read as C++ objects and keywords are compared as interned pointers: 3.5 us
// (0.5 for its Rotary, 2.1 in the launch), so that calls back to back are bound by their kernels.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <structmember.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <exception>
#include <initializer_list>

#include "okv.h"

namespace {

struct Raised {};  // thrown once a Python exception is set

PyObject* g_error = nullptr;  // binding.OkvError

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Raised{};
}

// Runs f; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// ---- arguments -------------------------------------------------------------------------------------------------

// Parameters of a call in order; `positional` of them may come without a name.
template <int N>
struct Signature {
  const char* fn;
  int positional;
  uint32_t required;  // bit i: parameter i has to be given
  const char* names[N];
  PyObject* keys[N];

  bool intern() {
    for (int i = 0; i < N; ++i)
      if (!(keys[i] = PyUnicode_InternFromString(names[i]))) return false;
    return true;
  }

  int find(PyObject* key) const {
    for (int i = 0; i < N; ++i)
      if (keys[i] == key) return i;
    for (int i = 0; i < N; ++i)
      if (PyUnicode_Compare(keys[i], key) == 0) return i;
    if (PyErr_Occurred()) throw Raised{};
    raise(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, key);
  }

  // out[i]: the argument of parameter i, null where it was not given
  void bind(PyObject* const* args, Py_ssize_t n, PyObject* kwnames, PyObject** out) const {
    for (int i = 0; i < N; ++i) out[i] = nullptr;
    if (n > positional) raise(PyExc_TypeError, "%s() takes at most %d positional arguments (%zd given)", fn, positional, n);
    for (Py_ssize_t i = 0; i < n; ++i) out[i] = args[i];
    const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < nk; ++k) {
      const int i = find(PyTuple_GET_ITEM(kwnames, k));
      if (out[i]) raise(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, names[i]);
      out[i] = args[n + k];
    }
    for (int i = 0; i < N; ++i)
      if ((required >> i & 1) && !out[i]) raise(PyExc_TypeError, "%s() missing required argument: '%s'", fn, names[i]);
  }
};

bool given(PyObject* o) { return o && o != Py_None; }

int32_t as_i32(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v != (int32_t)v) raise(PyExc_ValueError, "%s: %ld is outside 32 bits", name, v);
  return (int32_t)v;
}

int32_t count(int64_t n, const char* name) {
  if (n != (int32_t)n) raise(PyExc_ValueError, "%s: %lld rows or requests are outside 32 bits", name, (long long)n);
  return (int32_t)n;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a CUDA tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// Raises ValueError: `what`, followed by the tensor's type, shape, strides and device.
[[noreturn]] void refuse(PyObject* t, const char* name, PyObject* what) {
  PyObject* dtype = what ? PyObject_GetAttrString(t, "dtype") : nullptr;
  PyObject* shape = dtype ? PyObject_GetAttrString(t, "shape") : nullptr;
  PyObject* device = shape ? PyObject_GetAttrString(t, "device") : nullptr;
  PyObject* stride = device ? PyObject_CallMethod(t, "stride", nullptr) : nullptr;
  if (stride) PyErr_Format(PyExc_ValueError, "%s: expected %U, got %S %S strides %S on %S", name, what, dtype, shape, stride, device);
  Py_XDECREF(what);
  Py_XDECREF(dtype);
  Py_XDECREF(shape);
  Py_XDECREF(device);
  Py_XDECREF(stride);
  throw Raised{};
}

// A tensor of a storage type: its okv dtype and device.
int32_t storage(PyObject* o, const char* name, int* dev) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) raise(PyExc_TypeError, "%s: expected a CUDA tensor", name);
  *dev = (int)t.get_device();
  if (t.scalar_type() == at::kFloat) return OKV_F32;
  if (t.scalar_type() == at::kBFloat16) return OKV_BF16;
  refuse(o, name, PyUnicode_FromString("float32 or bfloat16"));
}

struct Types {
  at::ScalarType one, other;
  const char* names;
};
const Types kInt{at::kInt, at::kInt, "torch.int32"}, kBits{at::kLong, at::kUInt64, "torch.int64 or torch.uint64"},
    kF32{at::kFloat, at::kFloat, "torch.float32"}, kBf16{at::kBFloat16, at::kBFloat16, "torch.bfloat16"};

// The address of a contiguous tensor of this shape and type on device `dev`.
void* address(PyObject* o, const char* name, std::initializer_list<int64_t> shape, const Types& types, int dev) {
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType st = t.scalar_type();
  if ((st != types.one && st != types.other) || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() ||
      t.sizes() != at::IntArrayRef(shape)) {
    PyObject* want = PyTuple_New((Py_ssize_t)shape.size());
    if (!want) throw Raised{};
    Py_ssize_t i = 0;
    for (const int64_t n : shape) PyTuple_SET_ITEM(want, i++, PyLong_FromLongLong(n));
    PyObject* what = PyUnicode_FromFormat("contiguous %s %S on cuda:%d", types.names, want, dev);
    Py_DECREF(want);
    refuse(o, name, what);
  }
  return t.data_ptr();
}

void* optional(PyObject* o, const char* name, std::initializer_list<int64_t> shape, const Types& types, int dev) {
  return given(o) ? address(o, name, shape, types, dev) : nullptr;
}

// Elements between the rows of t [...][width], whose leading dims are one run of rows.
int64_t row_stride(PyObject* o, int64_t width) {
  const at::Tensor& t = tensor(o, "qkv");
  const int64_t nd = t.dim();
  if (nd >= 1 && t.size(nd - 1) == width && t.is_contiguous()) return width;
  if (nd < 1 || t.size(nd - 1) != width || (t.stride(nd - 1) != 1 && width > 1))
    refuse(o, "qkv", PyUnicode_FromFormat("rows of %lld adjacent elements", (long long)width));
  int64_t step = 0, run = 0;  // between rows, of the dims seen so far from the last one
  bool seen = false;
  for (int64_t i = nd - 2; i >= 0; --i) {
    const int64_t n = t.size(i), s = t.stride(i);
    if (n == 1) continue;
    if (!seen) {
      seen = true;
      step = s;
      run = s * n;
    } else if (s != run) {
      refuse(o, "qkv", PyUnicode_FromString("rows at one distance"));
    } else {
      run *= n;
    }
  }
  return seen ? step : width;
}

int64_t width(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  int64_t w;
  if (__builtin_mul_overflow(q_heads + 2 * kv_heads, head_dim, &w)) raise(PyExc_ValueError, "q_heads, kv_heads, head_dim: a row past 64 bits");
  return w;
}

// Device `dev` current while it lives, and the stream of a call.
struct Launch {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;

  Launch(int dev, PyObject* s) {
    if (!given(s)) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else if (PyLong_Check(s)) {
      stream = PyLong_AsVoidPtr(s);
    } else {
      PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
      if (!h) throw Raised{};
      stream = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
    }
    if (PyErr_Occurred()) throw Raised{};
    if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
  }
};

// Runs the C call without the interpreter's lock: a launch waits where its stream's queue is full.
template <typename F>
PyObject* launch(const char* fn, F call) {
  okv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  if (st == OKV_OK) Py_RETURN_NONE;
  PyObject* msg = PyUnicode_FromFormat("%s failed (shape, alignment or size outside its limits, or a CUDA error)", fn);
  PyObject* e = msg ? PyObject_CallFunction(g_error, "iN", (int)st, msg) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// ---- Rotary ----------------------------------------------------------------------------------------------------

struct Rotary {
  PyObject_HEAD
  PyObject* tensors;  // (inv_freq, q_weight, k_weight), kept alive
  float eps;
  int32_t interleaved;
};

PyTypeObject* rotary_type();

Signature<5> rotary_sig{"Rotary", 5, 0, {"inv_freq", "q_weight", "k_weight", "eps", "interleaved"}, {}};

const at::Tensor& vector(PyObject* o, int i) {
  const at::Tensor& t = tensor(o, rotary_sig.names[i]);
  if (!t.is_cuda() || t.dim() != 1 || !t.is_contiguous()) refuse(o, rotary_sig.names[i], PyUnicode_FromString("a contiguous CUDA vector"));
  if (i == 0 && t.scalar_type() != at::kFloat) refuse(o, "inv_freq", PyUnicode_FromString("float32"));
  return t;
}

PyObject* rotary_new(PyObject*, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[5];
    rotary_sig.bind(args, PyVectorcall_NARGS(nargsf), kwnames, a);
    for (int i = 0; i < 3; ++i)
      if (given(a[i])) vector(a[i], i);
    const double eps = a[3] ? PyFloat_AsDouble(a[3]) : 1e-6;
    if (eps == -1 && PyErr_Occurred()) throw Raised{};
    const int interleaved = a[4] ? PyObject_IsTrue(a[4]) : 0;
    if (interleaved < 0) throw Raised{};
    PyObject* none = Py_None;
    PyObject* kept = PyTuple_Pack(3, a[0] ? a[0] : none, a[1] ? a[1] : none, a[2] ? a[2] : none);
    if (!kept) throw Raised{};
    Rotary* self = PyObject_GC_New(Rotary, rotary_type());
    if (!self) {
      Py_DECREF(kept);
      throw Raised{};
    }
    self->tensors = kept;
    self->eps = (float)eps;
    self->interleaved = interleaved;
    PyObject_GC_Track(self);
    return (PyObject*)self;
  });
}

int rotary_traverse(PyObject* o, visitproc visit, void* arg) {
  Py_VISIT(((Rotary*)o)->tensors);
  return 0;
}

int rotary_clear(PyObject* o) {
  Py_CLEAR(((Rotary*)o)->tensors);
  return 0;
}

void rotary_dealloc(PyObject* o) {
  PyObject_GC_UnTrack(o);
  rotary_clear(o);
  PyObject_GC_Del(o);
}

// The okv_rotary of tensors that fit rows of this type, device and head_dim, wherever the tensors are by now.
okv_rotary rotary_for(PyObject* o, at::ScalarType dtype, int dev, int32_t head_dim) {
  if (!Py_IS_TYPE(o, rotary_type())) raise(PyExc_TypeError, "rotary: expected a Rotary, got %s", Py_TYPE(o)->tp_name);
  const Rotary* self = (const Rotary*)o;
  if (!self->tensors) raise(PyExc_ValueError, "rotary: its tensors are gone");
  okv_rotary r{};
  const void* ptr[3] = {};
  for (int i = 0; i < 3; ++i) {
    PyObject* t = PyTuple_GET_ITEM(self->tensors, i);
    if (t == Py_None) continue;
    const at::Tensor& w = vector(t, i);
    if (w.get_device() != dev || (i && (w.scalar_type() != dtype || w.numel() != head_dim)))
      refuse(t, rotary_sig.names[i], i ? PyUnicode_FromFormat("[%d] of the rows' type on cuda:%d", head_dim, dev)
                                       : PyUnicode_FromFormat("a vector on the rows' device cuda:%d", dev));
    if (i == 0) r.rotary_dim = count(2 * w.numel(), "inv_freq");
    ptr[i] = w.data_ptr();
  }
  r.inv_freq = (const float*)ptr[0];
  r.q_weight = ptr[1];
  r.k_weight = ptr[2];
  r.eps = self->eps;
  r.interleaved = self->interleaved;
  return r;
}

PyObject* rotary_check(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) raise(PyExc_TypeError, "_check() takes 2 arguments (%zd given)", n);
    const at::Tensor& t = tensor(args[0], "qkv");
    const okv_rotary r = rotary_for(self, t.scalar_type(), (int)t.get_device(), as_i32(args[1], "head_dim"));
    return PyBytes_FromStringAndSize((const char*)&r, sizeof r);
  });
}

PyMethodDef rotary_methods[] = {
    {"_check", (PyCFunction)(void*)rotary_check, METH_FASTCALL,
     "_check($self, qkv, head_dim, /)\n--\n\nThe okv_rotary, as bytes, of tensors that fit rows like qkv."},
    {}};
PyMemberDef rotary_members[] = {{"tensors", T_OBJECT, offsetof(Rotary, tensors), READONLY, "(inv_freq, q_weight, k_weight)"}, {}};

PyTypeObject* rotary_type() {
  static PyTypeObject type = [] {
    PyTypeObject t{PyVarObject_HEAD_INIT(nullptr, 0)};
    t.tp_name = "sparse_kv_cache_draft_gb300._calls.Rotary";
    t.tp_basicsize = sizeof(Rotary);
    t.tp_dealloc = rotary_dealloc;
    t.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC | Py_TPFLAGS_DISALLOW_INSTANTIATION;
    t.tp_doc =
        "Rotary(inv_freq=None, q_weight=None, k_weight=None, eps=1e-06, interleaved=False)\n--\n\n"
        "okv_rotary: inv_freq [rotary_dim / 2] float32 (None: no rotation), q_weight and k_weight [head_dim] of\n"
        "the rows' dtype (None: no norm). Keeps the tensors; read at each call.";
    t.tp_traverse = rotary_traverse;
    t.tp_clear = rotary_clear;
    t.tp_methods = rotary_methods;
    t.tp_members = rotary_members;
    t.tp_vectorcall = rotary_new;
    return t;
  }();
  return &type;
}

// ---- calls -----------------------------------------------------------------------------------------------------

Signature<10> rows_sig{"norm_rope", 5, 0b0111100011,
                       {"qkv", "positions", "q", "k", "v", "q_heads", "kv_heads", "head_dim", "rotary", "stream"}, {}};

PyObject* norm_rope(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[10];
    rows_sig.bind(args, nargs, kwnames, a);
    int dev;
    const int32_t dt = storage(a[0], "qkv", &dev);
    const at::Tensor& qkv = THPVariable_Unpack(a[0]);
    if (qkv.dim() != 2) refuse(a[0], "qkv", PyUnicode_FromString("rows [n][...]"));
    const Types& st = dt == OKV_F32 ? kF32 : kBf16;
    const int64_t n = qkv.size(0), hq = as_i32(a[5], "q_heads"), hkv = as_i32(a[6], "kv_heads"), d = as_i32(a[7], "head_dim");
    const int32_t rows = count(n, "qkv");
    const int64_t stride = row_stride(a[0], width(hq, hkv, d));
    void* pos = address(a[1], "positions", {n}, kInt, dev);
    const okv_rotary rot = rotary_for(a[8], qkv.scalar_type(), dev, (int32_t)d);
    void* q = optional(a[2], "q", {n, hq, d}, st, dev);
    void* k = optional(a[3], "k", {n, hkv, d}, st, dev);
    void* v = optional(a[4], "v", {n, hkv, d}, st, dev);
    void* x = qkv.data_ptr();
    Launch at(dev, a[9]);
    return launch("okv_norm_rope", [&] {
      return okv_norm_rope(rows, (int32_t)hq, (int32_t)hkv, (int32_t)d, dt, x, stride, (const int32_t*)pos, &rot, q, k, v, at.stream);
    });
  });
}

Signature<13> append_sig{"append_qkv_static", 6, 0b0111111011111,
                         {"qkv", "lengths", "counts", "pool", "slot_block", "q", "q_heads", "kv_heads", "head_dim", "block_size", "slots", "rotary", "stream"}, {}};

PyObject* append_qkv_static(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[13];
    append_sig.bind(args, nargs, kwnames, a);
    int dev;
    const int32_t dt = storage(a[0], "qkv", &dev);
    const at::Tensor& qkv = THPVariable_Unpack(a[0]);
    if (qkv.dim() != 3) refuse(a[0], "qkv", PyUnicode_FromString("rows [R][T][...]"));
    const Types& st = dt == OKV_F32 ? kF32 : kBf16;
    const int64_t R = qkv.size(0), T = qkv.size(1), hq = as_i32(a[6], "q_heads"), hkv = as_i32(a[7], "kv_heads"),
                  d = as_i32(a[8], "head_dim"), bs = as_i32(a[9], "block_size"), kb = as_i32(a[10], "slots");
    const int32_t r = count(R, "qkv"), t = count(T, "qkv");
    const int64_t stride = row_stride(a[0], width(hq, hkv, d));
    void* lengths = address(a[1], "lengths", {R}, kInt, dev);
    void* counts = optional(a[2], "counts", {R}, kInt, dev);
    const okv_rotary rot = rotary_for(a[11], qkv.scalar_type(), dev, (int32_t)d);
    void* pool = address(a[3], "pool", {R, hkv, kb, 2, bs, d}, st, dev);
    void* slot_block = address(a[4], "slot_block", {R, hkv, kb}, kInt, dev);
    void* q = optional(a[5], "q", {R, T, hq, d}, st, dev);
    void* x = qkv.data_ptr();
    Launch at(dev, a[12]);
    return launch("okv_append_qkv_static", [&] {
      return okv_append_qkv_static(r, t, (int32_t)hq, (int32_t)hkv, (int32_t)d, (int32_t)bs, (int32_t)kb, dt, x, stride,
                                   (const int32_t*)lengths, (const int32_t*)counts, &rot, pool, (const int32_t*)slot_block, q, at.stream);
    });
  });
}

Signature<15> tree_sig{"attend_tree_static", 9, 0b011111111111111,
                       {"pool", "slot_block", "lengths", "counts", "q", "k", "v", "mask", "out", "q_heads", "kv_heads", "head_dim", "block_size", "slots", "stream"}, {}};

PyObject* attend_tree_static(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[15];
    tree_sig.bind(args, nargs, kwnames, a);
    int dev;
    const int32_t dt = storage(a[0], "pool", &dev);
    const at::Tensor& qt = tensor(a[4], "q");
    if (qt.dim() != 4) refuse(a[4], "q", PyUnicode_FromString("drafted tokens [R][T][q_heads][head_dim]"));
    const Types& st = dt == OKV_F32 ? kF32 : kBf16;
    const int64_t R = qt.size(0), T = qt.size(1), hq = as_i32(a[9], "q_heads"), hkv = as_i32(a[10], "kv_heads"),
                  d = as_i32(a[11], "head_dim"), bs = as_i32(a[12], "block_size"), kb = as_i32(a[13], "slots");
    const int32_t r = count(R, "q"), t = count(T, "q");
    void* pool = address(a[0], "pool", {R, hkv, kb, 2, bs, d}, st, dev);
    void* slot_block = address(a[1], "slot_block", {R, hkv, kb}, kInt, dev);
    void* lengths = address(a[2], "lengths", {R}, kInt, dev);
    void* counts = optional(a[3], "counts", {R}, kInt, dev);
    void* q = address(a[4], "q", {R, T, hq, d}, st, dev);
    void* k = address(a[5], "k", {R, T, hkv, d}, st, dev);
    void* v = address(a[6], "v", {R, T, hkv, d}, st, dev);
    void* mask = address(a[7], "mask", {R, T}, kBits, dev);
    void* out = address(a[8], "out", {R, T, hq, d}, st, dev);
    Launch at(dev, a[14]);
    return launch("okv_attend_tree_static", [&] {
      return okv_attend_tree_static(r, t, (int32_t)hq, (int32_t)hkv, (int32_t)d, (int32_t)bs, (int32_t)kb, dt, pool,
                                    (const int32_t*)slot_block, (const int32_t*)lengths, (const int32_t*)counts, q, k, v,
                                    (const uint64_t*)mask, out, at.stream);
    });
  });
}

Signature<17> chunk_sig{"attend_chunk_static", 9, 0b00011111000111111,
                        {"pool", "slot_block", "lengths", "counts", "q", "out", "lse", "weight", "weight_out", "q_heads", "kv_heads", "head_dim", "block_size",
                         "slots", "window", "sinks", "stream"}, {}};

PyObject* attend_chunk_static(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[17];
    chunk_sig.bind(args, nargs, kwnames, a);
    int dev;
    const int32_t dt = storage(a[0], "pool", &dev);
    const at::Tensor& qt = tensor(a[4], "q");
    if (qt.dim() != 4) refuse(a[4], "q", PyUnicode_FromString("new tokens [R][T][q_heads][head_dim]"));
    const Types& st = dt == OKV_F32 ? kF32 : kBf16;
    const int64_t R = qt.size(0), T = qt.size(1), hq = as_i32(a[9], "q_heads"), hkv = as_i32(a[10], "kv_heads"),
                  d = as_i32(a[11], "head_dim"), bs = as_i32(a[12], "block_size"), kb = as_i32(a[13], "slots");
    const int32_t window = given(a[14]) ? as_i32(a[14], "window") : 0, sinks = given(a[15]) ? as_i32(a[15], "sinks") : 0;
    const int32_t r = count(R, "q"), t = count(T, "q");
    void* pool = address(a[0], "pool", {R, hkv, kb, 2, bs, d}, st, dev);
    void* slot_block = address(a[1], "slot_block", {R, hkv, kb}, kInt, dev);
    void* lengths = address(a[2], "lengths", {R}, kInt, dev);
    void* counts = optional(a[3], "counts", {R}, kInt, dev);
    void* q = address(a[4], "q", {R, T, hq, d}, st, dev);
    void* out = address(a[5], "out", {R, T, hq, d}, st, dev);
    void* lse = optional(a[6], "lse", {R, T, hq}, kF32, dev);
    void* weight = optional(a[7], "weight", {R, hkv, kb}, kF32, dev);
    void* weight_out = given(a[8]) ? address(a[8], "weight_out", {R, hkv, kb}, kF32, dev) : weight;
    if (weight_out && !lse) raise(PyExc_ValueError, "lse: the weights need it");
    Launch at(dev, a[16]);
    return launch("okv_attend_chunk_static", [&] {
      return okv_attend_chunk_static(r, t, (int32_t)hq, (int32_t)hkv, (int32_t)d, (int32_t)bs, (int32_t)kb, dt, pool, (const int32_t*)slot_block,
                                     (const int32_t*)lengths, (const int32_t*)counts, window, sinks, q, out, (float*)lse, (const float*)weight,
                                     (float*)weight_out, at.stream);
    });
  });
}

Signature<13> evict_sig{"evict_static", 6, 0b0001111001111,
                        {"slot_block", "weight", "lengths", "counts", "slot_block_out", "weight_out", "n_new", "kv_heads", "block_size", "slots", "sinks",
                         "recent", "stream"}, {}};

PyObject* evict_static(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    PyObject* a[13];
    evict_sig.bind(args, nargs, kwnames, a);
    const at::Tensor& sb = tensor(a[0], "slot_block");
    if (!sb.is_cuda()) raise(PyExc_TypeError, "slot_block: expected a CUDA tensor");
    if (sb.dim() != 3) refuse(a[0], "slot_block", PyUnicode_FromString("slot tables [R][kv_heads][slots]"));
    const int dev = (int)sb.get_device();
    const int32_t n_new = as_i32(a[6], "n_new"), hkv = as_i32(a[7], "kv_heads"), bs = as_i32(a[8], "block_size"), kb = as_i32(a[9], "slots");
    const int32_t sinks = given(a[10]) ? as_i32(a[10], "sinks") : 0, recent = given(a[11]) ? as_i32(a[11], "recent") : 0;
    const int64_t R = sb.size(0);
    const int32_t r = count(R, "slot_block");
    void* slot_block = address(a[0], "slot_block", {R, hkv, kb}, kInt, dev);
    void* weight = address(a[1], "weight", {R, hkv, kb}, kF32, dev);
    void* lengths = address(a[2], "lengths", {R}, kInt, dev);
    void* counts = optional(a[3], "counts", {R}, kInt, dev);
    void* slot_block_out = given(a[4]) ? address(a[4], "slot_block_out", {R, hkv, kb}, kInt, dev) : slot_block;
    void* weight_out = given(a[5]) ? address(a[5], "weight_out", {R, hkv, kb}, kF32, dev) : weight;
    Launch at(dev, a[12]);
    return launch("okv_evict_static", [&] {
      return okv_evict_static(r, n_new, hkv, bs, kb, (const int32_t*)lengths, (const int32_t*)counts, sinks, recent, (const int32_t*)slot_block,
                              (const float*)weight, (int32_t*)slot_block_out, (float*)weight_out, at.stream);
    });
  });
}

PyObject* py_row_stride(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) raise(PyExc_TypeError, "_row_stride() takes 2 arguments (%zd given)", n);
    return PyLong_FromLongLong(row_stride(args[0], as_i32(args[1], "width")));
  });
}

PyMethodDef methods[] = {
    {"norm_rope", (PyCFunction)(void*)norm_rope, METH_FASTCALL | METH_KEYWORDS,
     "norm_rope($module, qkv, positions, q=None, k=None, v=None, *, q_heads, kv_heads, head_dim, rotary, stream=None)\n--\n\n"
     "okv_norm_rope: norms and rotates rows qkv [n][(q_heads + 2 kv_heads) head_dim] (rows may be strided) at\n"
     "positions [n] int32 into q [n][q_heads][head_dim], k and v [n][kv_heads][head_dim] (any may be None).\n"
     "Rows with a negative position are not written."},
    {"append_qkv_static", (PyCFunction)(void*)append_qkv_static, METH_FASTCALL | METH_KEYWORDS,
     "append_qkv_static($module, qkv, lengths, counts, pool, slot_block, q=None, *, q_heads, kv_heads, head_dim, block_size, slots, rotary, stream=None)\n--\n\n"
     "okv_append_qkv_static: rows qkv [R][T][(q_heads + 2 kv_heads) head_dim] at positions lengths[r] + t, normed\n"
     "and rotated; queries into q [R][T][q_heads][head_dim] (or None), keys and values into the resident slots of\n"
     "pool [R][kv_heads][slots][2][block_size][head_dim]; counts [R] int32 or None."},
    {"attend_tree_static", (PyCFunction)(void*)attend_tree_static, METH_FASTCALL | METH_KEYWORDS,
     "attend_tree_static($module, pool, slot_block, lengths, counts, q, k, v, mask, out, *, q_heads, kv_heads, head_dim, block_size, slots, stream=None)\n--\n\n"
     "okv_attend_tree_static: drafted tokens q, out [R][T][q_heads][head_dim], k, v [R][T][kv_heads][head_dim], mask\n"
     "[R][T] int64 or uint64 (bit j: drafted token j is attended), counts [R] int32 or None, over a pool of\n"
     "attend_static's layout."},
    {"attend_chunk_static", (PyCFunction)(void*)attend_chunk_static, METH_FASTCALL | METH_KEYWORDS,
     "attend_chunk_static($module, pool, slot_block, lengths, counts, q, out, lse=None, weight=None, weight_out=None, *, q_heads, kv_heads, head_dim, block_size, slots, window=0, sinks=0, stream=None)\n--\n\n"
     "okv_attend_chunk_static: new tokens q, out [R][T][q_heads][head_dim] at positions lengths[r] + t, over the resident\n"
     "tokens at their positions and before (and less than window before, or among the first sinks); lse [R][T][q_heads]\n"
     "float32; weight [R][kv_heads][slots] float32 has what each slot draws added to it, in place or into weight_out\n"
     "(which alone starts from zero); counts [R] int32 or None; over a pool of attend_static's layout."},
    {"evict_static", (PyCFunction)(void*)evict_static, METH_FASTCALL | METH_KEYWORDS,
     "evict_static($module, slot_block, weight, lengths, counts, slot_block_out=None, weight_out=None, *, n_new, kv_heads, block_size, slots, sinks=0, recent=0, stream=None)\n--\n\n"
     "okv_evict_static: slots of slot_block [R][kv_heads][slots] int32 for the blocks that the next counts[r] tokens begin (None:\n"
     "n_new each), empty ones, then those of least weight [R][kv_heads][slots] float32, but not of the first sinks or the last\n"
     "recent tokens; in place, or into slot_block_out and weight_out."},
    {"_row_stride", (PyCFunction)(void*)py_row_stride, METH_FASTCALL,
     "_row_stride($module, t, width, /)\n--\n\nElements between the rows of t [...][width], whose leading dims are one run of rows."},
    {}};

PyModuleDef module_def{PyModuleDef_HEAD_INIT, "_calls", "Calls on rows, drafted trees and bounded caches that need no context.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  if (!rotary_sig.intern() || !rows_sig.intern() || !append_sig.intern() || !tree_sig.intern() || !chunk_sig.intern() || !evict_sig.intern()) return nullptr;
  PyObject* binding = PyImport_ImportModule("sparse_kv_cache_draft_gb300.binding");
  if (!binding) return nullptr;
  g_error = PyObject_GetAttrString(binding, "OkvError");
  Py_DECREF(binding);
  if (!g_error || PyType_Ready(rotary_type()) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module_def);
  if (!m) return nullptr;
  if (PyModule_AddObjectRef(m, "Rotary", (PyObject*)rotary_type()) < 0 || PyModule_AddStringConstant(m, "built_for", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
