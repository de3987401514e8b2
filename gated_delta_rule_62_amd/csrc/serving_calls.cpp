// The serving operators' calls from Python (serving.py): a dozen tensors each, with a dtype,
// shape, device and layout to compare, then the C function.  Through Python and ctypes that
// is 3-4 microseconds of a small call's 7, from here 1.  Host code only.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/kda.h"

namespace {

// A Python exception on its way out of a function below; no type: one is set already.
struct Raise {
  PyObject* type;
  std::string text;
};
[[noreturn]] void fail(const std::string& text) { throw Raise{PyExc_ValueError, text}; }

using Shape = std::initializer_list<int64_t>;

const at::Tensor& unpack(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) throw Raise{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

const at::Tensor& with_dims(const char* name, PyObject* o, int64_t dims, const char* what) {
  const at::Tensor& t = unpack(name, o);
  if (t.dim() != dims) fail(what);
  return t;
}

int gpu_of(const at::Tensor& t) {
  if (!t.is_cuda()) fail("every tensor must live on the same GPU");
  return t.get_device();
}

// The tensor of this dtype, shape and device.
const at::Tensor& checked(const char* name, PyObject* o, at::ScalarType dtype, Shape shape,
                          int dev) {
  const at::Tensor& t = unpack(name, o);
  if (t.scalar_type() != dtype || t.sizes() != at::IntArrayRef(shape)) {
    std::ostringstream s;
    s << name << " must be " << dtype << " " << at::IntArrayRef(shape) << ", got "
      << t.scalar_type() << " " << t.sizes();
    fail(s.str());
  }
  if (!t.is_cuda() || t.get_device() != dev) fail("every tensor must live on the same GPU");
  return t;
}

// Address of a contiguous tensor.
template <class T = void>
T* tensor(const char* name, PyObject* o, at::ScalarType dtype, Shape shape, int dev) {
  const at::Tensor& t = checked(name, o, dtype, shape, dev);
  if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}

// The same, or null for None.
template <class T = void>
T* optional(const char* name, PyObject* o, at::ScalarType dtype, Shape shape, int dev) {
  return o == Py_None ? nullptr : tensor<T>(name, o, dtype, shape, dev);
}

// Address and row stride in elements of a bf16 tensor [..., heads, D] whose tokens lie one
// fixed row stride apart.
struct Rows {
  void* at;
  int64_t row;
};
Rows rows(const char* name, PyObject* o, Shape shape, int dev) {
  const at::Tensor& t = checked(name, o, at::kBFloat16, shape, dev);
  const int64_t dims = t.dim(), heads = t.size(dims - 2), D = t.size(dims - 1);
  int64_t row = heads * D;
  if (!t.is_contiguous()) {
    bool ok = (t.stride(dims - 1) == 1 || D == 1) && (t.stride(dims - 2) == D || heads == 1);
    if (dims == 3) {
      if (t.size(0) > 1) row = t.stride(0);
    } else {
      const int64_t B = t.size(0), T = t.size(1);
      if (T > 1) row = t.stride(1);
      else if (B > 1) row = t.stride(0);
      ok = ok && (B == 1 || T == 1 || t.stride(0) == T * row);
    }
    if (!ok)
      fail(std::string(name) + " must have contiguous heads, its tokens one row stride apart");
  }
  return Rows{t.data_ptr(), row};
}

// A state tensor [n, H, D, D], bf16 or fp32, or null for None where that may be.
struct State {
  void* at;
  int dtype;
  int64_t n;
};
State state_of(const char* name, PyObject* o, int64_t n, int64_t H, int64_t D, int dev) {
  const at::Tensor& t = unpack(name, o);
  const at::ScalarType d = t.scalar_type();
  if (d != at::kBFloat16 && d != at::kFloat)
    throw Raise{PyExc_TypeError,
                std::string("state tensors must be bfloat16 or float32, got ") + c10::toString(d)};
  return State{tensor(name, o, d, {n, H, D, D}, dev),
               d == at::kFloat ? KDA_DTYPE_FP32 : KDA_DTYPE_BF16, n};
}
State optional_state(const char* name, PyObject* o, int64_t n, int64_t H, int64_t D, int dev) {
  return o == Py_None ? State{nullptr, 0, 0} : state_of(name, o, n, H, D, dev);
}
State pool_of(PyObject* o, int64_t H, int64_t D, int dev) {
  const at::Tensor& t = with_dims("state", o, 4, "state must be [slots,H,D,D]");
  return state_of("state", o, t.size(0), H, D, dev);
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return static_cast<float>(x);
}
int64_t integer(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  const long long x = i ? PyLong_AsLongLong(i) : -1;
  Py_XDECREF(i);
  if (x == -1 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return x;
}
template <class F>
F function(PyObject* address) {
  void* p = PyLong_AsVoidPtr(address);
  if (p == nullptr) throw Raise{PyExc_TypeError, "expected a function's address"};
  return reinterpret_cast<F>(p);
}

// None: torch's current stream of the device; a torch stream; a raw one.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream(dev).stream();
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (raw == nullptr) {
    PyErr_Clear();
    raw = PyNumber_Index(o);
  }
  void* s = raw ? PyLong_AsVoidPtr(raw) : nullptr;
  Py_XDECREF(raw);
  if (PyErr_Occurred()) throw Raise{nullptr, ""};
  return s;
}

// Makes dev current for the library, which goes by the current device.
struct Device {
  int before, dev;
  explicit Device(int d) : before(c10::hip::current_device()), dev(d) {
    if (before != dev) c10::hip::set_device(static_cast<c10::DeviceIndex>(dev));
  }
  ~Device() {
    if (before != dev) (void)c10::hip::SetDevice(static_cast<c10::DeviceIndex>(before));
  }
};

// The caller's workspace; missing one that is wanted, `want` says how large.
struct Workspace {
  void* at = nullptr;
  int64_t bytes = 0, want = 0;
};
Workspace workspace_of(PyObject* o, int64_t need, int dev) {
  Workspace w;
  if (o == Py_None) {
    w.want = need > 0 ? need : 0;  // a negative one is a status that the call will return
    return w;
  }
  const at::Tensor& t = unpack("workspace", o);
  if (t.scalar_type() != at::kByte || t.dim() != 1) fail("workspace must be a 1-d uint8 tensor");
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    fail("workspace must be contiguous and live on the same GPU");
  w.at = t.data_ptr();
  w.bytes = t.numel();
  return w;
}

// Runs f, a whole call: its status, or the bytes of the workspace it wants.  C++ exceptions
// become Python's.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) throw Raise{PyExc_TypeError, "wrong number of arguments"};
    return PyLong_FromLongLong(f());
  } catch (const Raise& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <class F>
int64_t without_gil(F f) {
  PyThreadState* s = PyEval_SaveThread();
  const int64_t st = f();
  PyEval_RestoreThread(s);
  return st;
}

const auto bf16 = at::kBFloat16, fp32 = at::kFloat, int64 = at::kLong;

PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_step)>(a[0]);
    const at::Tensor& tq = with_dims("q", a[1], 3, "q must be [N,H,D]");
    const int64_t N = tq.size(0), H = tq.size(1), D = tq.size(2);
    const int dev = gpu_of(tq);
    const void *q = tensor("q", a[1], bf16, {N, H, D}, dev),
               *k = tensor("k", a[2], bf16, {N, H, D}, dev),
               *v = tensor("v", a[3], bf16, {N, H, D}, dev),
               *g = tensor("g", a[4], bf16, {N, H, D}, dev),
               *beta = tensor("beta", a[5], bf16, {N, H}, dev);
    const float scale = number(a[6]);
    void* out = tensor("out", a[7], bf16, {N, H, D}, dev);
    const float *A_log = tensor<float>("A_log", a[8], fp32, {H}, dev),
                *dt_bias = tensor<float>("dt_bias", a[9], fp32, {H, D}, dev);
    const float lower_bound = number(a[10]);
    const State s = pool_of(a[11], H, D, dev);
    const int64_t *in = optional<int64_t>("slot_in", a[12], int64, {N}, dev),
                  *to = optional<int64_t>("slot_out", a[13], int64, {N}, dev);
    void* stream = stream_of(a[14], dev);
    Device current(dev);
    return without_gil([&] {
      return fn(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, s.at, s.dtype, s.n, in,
                to, N, H, D, stream);
    });
  });
}

PyObject* la_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_la_step)>(a[0]);
    const at::Tensor &tq = with_dims("q", a[1], 3, "q and v must be [N,heads,D]"),
                     &tv = with_dims("v", a[3], 3, "q and v must be [N,heads,D]");
    const int64_t N = tv.size(0), H = tv.size(1), D = tv.size(2), Hk = tq.size(1);
    const int dev = gpu_of(tq);
    const Rows q = rows("q", a[1], {N, Hk, D}, dev), k = rows("k", a[2], {N, Hk, D}, dev),
               v = rows("v", a[3], {N, H, D}, dev);
    const float* g = optional<float>("g", a[4], fp32, {N, H}, dev);
    const float scale = number(a[5]);
    void* out = tensor("out", a[6], bf16, {N, H, D}, dev);
    const State s = pool_of(a[7], H, D, dev);
    const float* decay = optional<float>("decay", a[8], fp32, {H}, dev);
    const int64_t *in = optional<int64_t>("slot_in", a[9], int64, {N}, dev),
                  *to = optional<int64_t>("slot_out", a[10], int64, {N}, dev);
    void* stream = stream_of(a[11], dev);
    Device current(dev);
    return without_gil([&] {
      return fn(q.at, q.row, k.at, k.row, v.at, v.row, g, decay, scale, out, s.at, s.dtype, s.n,
                in, to, N, H, Hk, D, stream);
    });
  });
}

PyObject* la_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_la_fwd)>(a[0]);
    const auto ws_bytes = function<decltype(&kda_la_workspace_bytes)>(a[1]);
    const at::Tensor &tq = with_dims("q", a[2], 4, "q and v must be [B,T,heads,D]"),
                     &tv = with_dims("v", a[4], 4, "q and v must be [B,T,heads,D]");
    const int64_t B = tv.size(0), T = tv.size(1), H = tv.size(2), D = tv.size(3), Hk = tq.size(2);
    const int dev = gpu_of(tq);
    const Rows q = rows("q", a[2], {B, T, Hk, D}, dev), k = rows("k", a[3], {B, T, Hk, D}, dev),
               v = rows("v", a[4], {B, T, H, D}, dev);
    const float* g = optional<float>("g", a[5], fp32, {B, T, H}, dev);
    const float scale = number(a[6]);
    void* out = tensor("out", a[7], bf16, {B, T, H, D}, dev);
    const float* decay = optional<float>("decay", a[8], fp32, {H}, dev);
    const int64_t N = a[11] == Py_None ? B : unpack("cu_seqlens", a[11]).numel() - 1;
    const State first = optional_state("initial_state", a[9], N, H, D, dev),
                last = optional_state("final_state", a[10], N, H, D, dev);
    const int64_t* cu = optional<int64_t>("cu_seqlens", a[11], int64, {N + 1}, dev);
    const int64_t segment = integer(a[12]);
    void* stream = stream_of(a[14], dev);
    Device current(dev);
    const Workspace w = workspace_of(a[13], ws_bytes(B * T, N, H, D, segment), dev);
    if (w.want) return w.want;
    return without_gil([&] {
      return fn(q.at, q.row, k.at, k.row, v.at, v.row, g, decay, scale, out, first.at,
                first.dtype, last.at, last.dtype, cu, N, B, T, H, Hk, D, segment, w.at, w.bytes,
                stream);
    });
  });
}

PyObject* attn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_attn_fwd)>(a[0]);
    const auto ws_bytes = function<decltype(&kda_attn_workspace_bytes)>(a[1]);
    const at::Tensor &tq = with_dims("q", a[2], 4, "q and k must be [B,T,heads,D]"),
                     &tk = with_dims("k", a[3], 4, "q and k must be [B,T,heads,D]");
    const int64_t Bq = tq.size(0), Tq = tq.size(1), Hq = tq.size(2), D = tq.size(3),
                  Bk = tk.size(0), Tk = tk.size(1), Hk = tk.size(2);
    const int dev = gpu_of(tq);
    const Rows q = rows("q", a[2], {Bq, Tq, Hq, D}, dev), k = rows("k", a[3], {Bk, Tk, Hk, D}, dev),
               v = rows("v", a[4], {Bk, Tk, Hk, D}, dev);
    const float scale = number(a[5]);
    void* out = tensor("out", a[6], bf16, {Bq, Tq, Hq, D}, dev);
    float* lse = optional<float>("lse", a[7], fp32, {Bq, Tq, Hq}, dev);
    const int64_t N = a[8] == Py_None ? Bq : unpack("cu_seqlens_q", a[8]).numel() - 1;
    const int64_t *cu_q = optional<int64_t>("cu_seqlens_q", a[8], int64, {N + 1}, dev),
                  *cu_k = optional<int64_t>("cu_seqlens_k", a[9], int64, {N + 1}, dev),
                  *k_lens = optional<int64_t>("k_lens", a[10], int64, {N}, dev);
    const int64_t splits = integer(a[11]);
    void* stream = stream_of(a[13], dev);
    Device current(dev);
    const Workspace w =
        workspace_of(a[12], ws_bytes(N, Bq, Tq, Bk, Tk, Hq, Hk, D, splits), dev);
    if (w.want) return w.want;
    return without_gil([&] {
      return fn(q.at, q.row, k.at, k.row, v.at, v.row, scale, out, lse, cu_q, cu_k, k_lens, N, Bq,
                Tq, Bk, Tk, Hq, Hk, D, splits, w.at, w.bytes, stream);
    });
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"step", fast(step), METH_FASTCALL, "kda_step: its address and arguments -> status."},
    {"la_step", fast(la_step), METH_FASTCALL, "kda_la_step: its address and arguments -> status."},
    {"la_fwd", fast(la_fwd), METH_FASTCALL,
     "kda_la_fwd: its and its workspace function's address, arguments -> status, or the bytes "
     "of the workspace it wants."},
    {"attn_fwd", fast(attn_fwd), METH_FASTCALL, "The same for kda_attn_fwd."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving_calls(void) { return PyModule_Create(&module); }
