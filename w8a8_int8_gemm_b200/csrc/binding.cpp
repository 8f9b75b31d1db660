// binding.cpp -- the calls whose smallest cases are bound by the host, from
// torch tensors to the C ABI: w8a8_qk_norm_rope, w8a8_attention and
// w8a8_linear_glu(_fp8).  Marshalling only, as in the Python module that wraps
// it: layouts are checked, outputs that the caller did not pass are allocated,
// and the library is called on the current stream.  (Through Python and ctypes
// the checks and allocations of a call took 6 to 9 us, more than the library
// and the kernel of a single token need.)
//
// A function returns its output, or the status of a call that the library
// refused as an int; a tensor that is not as it should be raises here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <limits>
#include <optional>

#include "../../include/w8a8.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Raised {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Raised{};
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void check(const Tensor& t, const char* name, ScalarType type, int64_t dims) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %R, got %R", name, torch::getTHPDtype(type),
                 torch::getTHPDtype(t.scalar_type()));
    throw Raised{};
  }
  if (t.dim() != dims) {
    PyErr_Format(PyExc_ValueError, "%s must have %lld dimensions, got %lld", name, static_cast<long long>(dims),
                 static_cast<long long>(t.dim()));
    throw Raised{};
  }
}

void check_shape(const Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() == shape) return;
  PyObject* want = PyTuple_New(static_cast<Py_ssize_t>(shape.size()));
  PyObject* got = PyTuple_New(static_cast<Py_ssize_t>(shape.size()));
  if (want != nullptr && got != nullptr) {
    for (size_t i = 0; i < shape.size(); ++i) {
      PyTuple_SET_ITEM(want, static_cast<Py_ssize_t>(i), PyLong_FromLongLong(shape[i]));
      PyTuple_SET_ITEM(got, static_cast<Py_ssize_t>(i), PyLong_FromLongLong(t.size(static_cast<int64_t>(i))));
    }
    PyErr_Format(PyExc_ValueError, "%s must have shape %R, got %R", name, want, got);
  }
  Py_XDECREF(want);
  Py_XDECREF(got);
  throw Raised{};
}

// The devices of a call's tensors, which have to be one.
struct Device {
  int index = -1;
  void add(const Tensor& t, const char* name) {
    const int i = t.get_device();
    if (index < 0) index = i;
    if (i != index) fail(PyExc_ValueError, "tensors are on different devices: %s is not on the first one's", name);
  }
};

// A contiguous tensor of a type and shape.
const Tensor& contiguous(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, Device& dev) {
  const Tensor& t = tensor(o, name);
  check(t, name, type, static_cast<int64_t>(shape.size()));
  check_shape(t, name, shape);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  dev.add(t, name);
  return t;
}

// Its data, or null for None.
template <class T>
T* optional(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, Device& dev) {
  return o == Py_None ? nullptr : static_cast<T*>(contiguous(o, name, type, shape, dev).data_ptr());
}

// A table's data.  One without entries has no address of its own, and null would say that there is no table: it gets
// one that is never read.
const float* table(PyObject* o, const char* name, at::IntArrayRef shape, Device& dev) {
  const float* data = optional<const float>(o, name, ScalarType::Float, shape, dev);
  return data != nullptr ? data : reinterpret_cast<const float*>(uintptr_t{16});
}

// A bf16 [tokens, heads, head_dim] view: its sizes and strides in elements.
struct Heads {
  void* data;
  int64_t rows, heads, dim, ld, hs;
};

Heads view(const Tensor& t) {
  Heads h{t.data_ptr(), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
  // (the stride of a dimension of one is free)
  if (h.heads <= 1) h.hs = h.dim;
  if (h.rows <= 1) h.ld = h.dim;
  return h;
}

const Tensor& heads(PyObject* o, const char* name, Device& dev) {
  const Tensor& t = tensor(o, name);
  check(t, name, ScalarType::BFloat16, 3);
  if (t.numel() > 0 && t.stride(2) != 1) {
    fail(PyExc_ValueError, "%s must be contiguous in its last dimension", name);
  }
  dev.add(t, name);
  return t;
}

// The stream of a call: a handle, or None for the current one.
struct Stream {
  std::optional<c10::cuda::CUDAStream> given;
  explicit Stream(PyObject* o, int device) {
    if (o == Py_None) return;
    void* handle = PyLong_AsVoidPtr(o);
    if (handle == nullptr && PyErr_Occurred()) throw Raised{};
    given = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle),
                                             static_cast<c10::DeviceIndex>(device));
  }
  w8a8_stream_t handle(int device) const {
    return reinterpret_cast<w8a8_stream_t>(
        given ? given->stream()
              : c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
  }
  // A new tensor that belongs to the stream of the call: memory of another stream could be handed out again by that
  // stream before this one's kernels are done with it.
  Tensor empty(at::IntArrayRef shape, const at::TensorOptions& options) const {
    if (!given) return at::empty(shape, options);
    const c10::cuda::CUDAStreamGuard guard(*given);
    return at::empty(shape, options);
  }
};

// The caller's tensor, or a new one, and the object to return.
struct Output {
  PyObject* object;  // borrowed from the caller, or null: `made` is new
  Tensor made;
  Heads h;
  PyObject* take() {
    return object != nullptr ? Py_NewRef(object) : THPVariable_Wrap(std::move(made));
  }
};

Output heads_out(PyObject* o, const char* name, const Tensor& like, const Stream& stream, Device& dev) {
  if (o == Py_None) {
    Output r{nullptr, stream.empty(like.sizes(), like.options()), {}};
    r.h = view(r.made);
    return r;
  }
  const Tensor& t = heads(o, name, dev);
  check_shape(t, name, like.sizes());
  return {o, Tensor(), view(t)};
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}

int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}

// (what does not fit is no valid argument either)
int32_t narrow(int64_t x) {
  constexpr int64_t lo = std::numeric_limits<int32_t>::min(), hi = std::numeric_limits<int32_t>::max();
  return static_cast<int32_t>(x < lo ? lo : x > hi ? hi : x);
}

// The library call, on the tensors' device and without the interpreter's lock.
template <class F>
w8a8_status call(int device, F&& f) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  w8a8_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

#define W8A8_ARGS(count)                                                                         \
  if (n != (count)) {                                                                            \
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", static_cast<int>(count), n); \
    return nullptr;                                                                              \
  }

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  W8A8_ARGS(12)
  try {
    Device dev;
    const Tensor& q = heads(a[0], "q", dev);
    const Tensor& k = heads(a[1], "k", dev);
    const Heads hq = view(q), hk = view(k);
    if (hk.dim != hq.dim) fail(PyExc_ValueError, "%s must have the head dimension of q", "k");
    if (hk.rows != hq.rows) fail(PyExc_ValueError, "%s must have the tokens of q", "k");
    w8a8_qk_desc d{};
    d.q_weight = optional<void>(a[2], "q_weight", ScalarType::BFloat16, {hq.dim}, dev);
    d.k_weight = optional<void>(a[3], "k_weight", ScalarType::BFloat16, {hq.dim}, dev);
    if ((a[4] == Py_None) != (a[5] == Py_None)) fail(PyExc_ValueError, "%s come together", "cos and sin");
    if (a[4] != Py_None) {
      const Tensor& cos = tensor(a[4], "cos");
      check(cos, "cos", ScalarType::Float, 2);
      d.table_rows = cos.size(0);
      d.rot_dim = narrow(2 * cos.size(1));
      d.cos = table(a[4], "cos", cos.sizes(), dev);
      d.sin = table(a[5], "sin", cos.sizes(), dev);
    }
    d.positions = optional<const int32_t>(a[6], "positions", ScalarType::Int, {hq.rows}, dev);
    d.eps = static_cast<float>(number(a[7]));
    d.layout = narrow(integer(a[8]));
    const Stream stream(a[11], dev.index);
    Output q_out = heads_out(a[9], "q_out", q, stream, dev);
    Output k_out = heads_out(a[10], "k_out", k, stream, dev);
    d.q = hq.data;
    d.k = hk.data;
    d.q_out = q_out.h.data;
    d.k_out = k_out.h.data;
    d.M = hq.rows;
    d.ldq = hq.ld;
    d.hsq = hq.hs;
    d.ldk = hk.ld;
    d.hsk = hk.hs;
    d.ldq_out = q_out.h.ld;
    d.hsq_out = q_out.h.hs;
    d.ldk_out = k_out.h.ld;
    d.hsk_out = k_out.h.hs;
    d.heads_q = narrow(hq.heads);
    d.heads_k = narrow(hk.heads);
    d.head_dim = narrow(hq.dim);
    const w8a8_stream_t s = stream.handle(dev.index);
    const w8a8_status st = call(dev.index, [&] { return w8a8_qk_norm_rope(&d, s); });
    if (st != W8A8_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) return nullptr;
    PyTuple_SET_ITEM(r, 0, q_out.take());
    PyTuple_SET_ITEM(r, 1, k_out.take());
    return r;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  W8A8_ARGS(15)
  try {
    Device dev;
    const Tensor& q = heads(a[0], "q", dev);
    const Tensor& k = heads(a[1], "k", dev);
    const Tensor& v = heads(a[2], "v", dev);
    const Heads hq = view(q), hk = view(k), hv = view(v);
    if (hk.dim != hq.dim) fail(PyExc_ValueError, "%s must have the head dimension of q", "k");
    check_shape(v, "v", k.sizes());
    w8a8_attention_desc d{};
    d.scale = static_cast<float>(a[3] == Py_None ? std::pow(static_cast<double>(hq.dim), -0.5) : number(a[3]));
    d.cap = static_cast<float>(number(a[4]));
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0) return nullptr;
    d.causal = causal;
    int64_t docs = 1;
    if (a[8] != Py_None) {
      docs = integer(a[8]);
    } else if (a[6] != Py_None || a[7] != Py_None) {
      docs = tensor(a[6] != Py_None ? a[6] : a[7], a[6] != Py_None ? "cu_q" : "cu_k").size(0) - 1;
    }
    d.docs = narrow(docs);
    d.cu_q = optional<const int32_t>(a[6], "cu_q", ScalarType::Int, {docs + 1}, dev);
    d.cu_k = optional<const int32_t>(a[7], "cu_k", ScalarType::Int, {docs + 1}, dev);
    d.prefix = optional<const int32_t>(a[9], "prefix", ScalarType::Int, {docs}, dev);
    d.slopes = optional<const float>(a[10], "slopes", ScalarType::Float, {hq.heads}, dev);
    d.lse = optional<float>(a[12], "lse", ScalarType::Float, {hq.rows, hq.heads}, dev);
    d.kernel = narrow(integer(a[13]));
    const Stream stream(a[14], dev.index);
    Output out = heads_out(a[11], "out", q, stream, dev);
    d.q = hq.data;
    d.k = hk.data;
    d.v = hv.data;
    d.out = out.h.data;
    d.tokens_q = hq.rows;
    d.tokens_k = hk.rows;
    d.ldq = hq.ld;
    d.hsq = hq.hs;
    d.ldk = hk.ld;
    d.hsk = hk.hs;
    d.ldv = hv.ld;
    d.hsv = hv.hs;
    d.ldo = out.h.ld;
    d.hso = out.h.hs;
    d.heads_q = narrow(hq.heads);
    d.heads_k = narrow(hk.heads);
    d.head_dim = narrow(hq.dim);
    const w8a8_stream_t s = stream.handle(dev.index);
    const w8a8_status st = call(dev.index, [&] { return w8a8_attention(&d, s); });
    return st != W8A8_OK ? PyLong_FromLong(st) : out.take();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* linear_glu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  W8A8_ARGS(10)
  try {
    Device dev;
    const bool fp8 = a[8] == Py_True;
    const ScalarType code = fp8 ? ScalarType::Byte : ScalarType::Char;
    const Tensor& x = tensor(a[0], "x");
    check(x, "x", ScalarType::BFloat16, 2);
    const int64_t M = x.size(0), K = x.size(1);
    contiguous(a[0], "x", ScalarType::BFloat16, x.sizes(), dev);
    const Tensor& wq = tensor(a[1], "wq");
    check(wq, "wq", code, 2);
    const int64_t rows = wq.size(0), N = rows / 2;
    if (rows % 2 != 0) fail(PyExc_ValueError, "%s must have an even number of rows (gate, then up)", "wq");
    if (wq.size(1) != K) fail(PyExc_ValueError, "inner dimensions of x and %s differ", "wq");
    contiguous(a[1], "wq", code, wq.sizes(), dev);
    const Tensor& scale_w = contiguous(a[2], "scale_w", ScalarType::Float, {rows}, dev);
    const void* bias = optional<void>(a[3], "bias", ScalarType::BFloat16, {rows}, dev);
    const int32_t act = narrow(integer(a[5]));
    const Stream stream(a[9], dev.index);
    Tensor out_made, ws_q, ws_s;  // held until the kernels are launched
    void* out = a[4] == Py_None ? (out_made = stream.empty({M, N}, x.options())).data_ptr()
                                : contiguous(a[4], "out", ScalarType::BFloat16, {M, N}, dev).data_ptr();
    void* codes;
    float* scales;
    if (a[6] == Py_None && a[7] == Py_None) {
      // one allocation for both: the codes, then the scales (16-byte aligned)
      const int64_t at = (M * K + 15) / 16 * 16;
      ws_q = stream.empty({at + 4 * M}, wq.options());
      codes = ws_q.data_ptr();
      scales = reinterpret_cast<float*>(static_cast<char*>(codes) + at);
    } else {
      codes = a[6] == Py_None ? (ws_q = stream.empty({M, K}, wq.options())).data_ptr()
                              : contiguous(a[6], "ws_xq", code, {M, K}, dev).data_ptr();
      scales = static_cast<float*>(
          a[7] == Py_None ? (ws_s = stream.empty({M}, scale_w.options())).data_ptr()
                          : contiguous(a[7], "ws_scale_a", ScalarType::Float, {M}, dev).data_ptr());
    }
    const void* xp = x.data_ptr();
    const void* w = wq.data_ptr();
    const float* sw = static_cast<const float*>(scale_w.data_ptr());
    const w8a8_stream_t s = stream.handle(dev.index);
    const w8a8_status st = call(dev.index, [&] {
      return fp8 ? w8a8_linear_glu_fp8(xp, static_cast<const uint8_t*>(w), sw, bias, out, static_cast<uint8_t*>(codes),
                                       scales, M, N, K, act, s)
                 : w8a8_linear_glu(xp, static_cast<const int8_t*>(w), sw, bias, out, static_cast<int8_t*>(codes),
                                   scales, M, N, K, act, s);
    });
    if (st != W8A8_OK) return PyLong_FromLong(st);
    return a[4] == Py_None ? THPVariable_Wrap(std::move(out_made)) : Py_NewRef(a[4]);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyCFunction function(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {  // (METH_FASTCALL's is another type)
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"qk_norm_rope", function(qk_norm_rope), METH_FASTCALL, nullptr},
    {"attention", function(attention), METH_FASTCALL, nullptr},
    {"linear_glu", function(linear_glu), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
