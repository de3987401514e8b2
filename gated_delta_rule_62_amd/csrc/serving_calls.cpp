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

// Address and row stride of a bf16 tensor [..., W] whose rows lie one stride apart.
Rows flat_rows(const char* name, PyObject* o, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = unpack(name, o);
  if (t.scalar_type() != bf16 || t.sizes() != shape) {
    std::ostringstream s;
    s << name << " must be " << bf16 << " " << shape << ", got " << t.scalar_type() << " "
      << t.sizes();
    fail(s.str());
  }
  if (!t.is_cuda() || t.get_device() != dev) fail("every tensor must live on the same GPU");
  const int64_t dims = t.dim(), W = t.size(dims - 1);
  int64_t row = W;
  if (!t.is_contiguous()) {
    bool ok = t.stride(dims - 1) == 1 || W == 1;
    int64_t rows = 1;  // of the dimensions behind this one
    for (int64_t d = dims - 2; d >= 0; --d) {
      if (t.size(d) == 1) continue;
      if (rows == 1) row = t.stride(d);
      ok = ok && t.stride(d) == rows * row;
      rows *= t.size(d);
    }
    if (!ok) fail(std::string(name) + " must have its rows one stride apart");
  }
  return Rows{t.data_ptr(), row};
}
// Address of a contiguous tensor of one of two dtypes.
void* either(const char* name, PyObject* o, at::IntArrayRef shape, int dev, int* dtype) {
  const at::Tensor& t = unpack(name, o);
  const at::ScalarType d = t.scalar_type();
  if ((d != bf16 && d != fp32) || t.sizes() != shape) {
    std::ostringstream s;
    s << name << " must be " << bf16 << " or " << fp32 << " " << shape << ", got " << d << " "
      << t.sizes();
    fail(s.str());
  }
  if (!t.is_cuda() || t.get_device() != dev) fail("every tensor must live on the same GPU");
  if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
  *dtype = d == fp32 ? KDA_DTYPE_FP32 : KDA_DTYPE_BF16;
  return t.data_ptr();
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raise{nullptr, ""};
  return x != 0;
}

PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_norm)>(a[0]);
    const at::Tensor& tx = unpack("x", a[1]);
    if (tx.dim() < 1) fail("x must be [..,W]");
    const at::IntArrayRef shape = tx.sizes();
    const int64_t W = shape.back();
    int64_t R = 1;
    for (size_t d = 0; d + 1 < shape.size(); ++d) R *= shape[d];
    const int dev = gpu_of(tx);
    const Rows x = flat_rows("x", a[1], shape, dev);
    void* out = nullptr;
    if (a[2] != Py_None) {
      const at::Tensor& t = unpack("out", a[2]);
      if (t.scalar_type() != bf16) fail("out must be bfloat16");
      int dtype;
      out = either("out", a[2], shape, dev, &dtype);
    }
    int wd = KDA_DTYPE_BF16, pd = KDA_DTYPE_BF16, rd = KDA_DTYPE_BF16, hd = KDA_DTYPE_BF16;
    const void *w = nullptr, *post = nullptr, *res = nullptr;
    void* res_out = nullptr;
    int64_t group = W;
    if (a[3] != Py_None) w = either("weight", a[3], {W}, dev, &wd);
    const float eps = number(a[4]);
    if (a[5] != Py_None) {
      group = with_dims("post_weight", a[5], 1, "post_weight must be [G]").numel();
      post = either("post_weight", a[5], {group}, dev, &pd);
      if (w == nullptr) wd = pd;
      else if (wd != pd) fail("weight and post_weight must have one dtype");
    }
    Rows gate{nullptr, W};
    if (a[6] != Py_None) gate = flat_rows("gate", a[6], shape, dev);
    const char* act = PyUnicode_Check(a[7]) ? PyUnicode_AsUTF8(a[7]) : "";
    if (act == nullptr) throw Raise{nullptr, ""};
    const std::string kind = act;
    if (kind != "sigmoid" && kind != "silu") fail("gate_fn must be 'sigmoid' or 'silu'");
    if (a[8] != Py_None) res = either("residual", a[8], shape, dev, &rd);
    if (a[9] != Py_None) res_out = either("residual_out", a[9], shape, dev, &hd);
    if (res && res_out && rd != hd) fail("residual and residual_out must have one dtype");
    if (!res != !res_out) fail("residual and residual_out come together");
    const float alpha = number(a[10]);
    void* stream = stream_of(a[11], dev);
    Device current(dev);
    return without_gil([&] {
      return fn(x.at, x.row, gate.at, gate.row,
                kind == "silu" ? KDA_GATE_SILU : KDA_GATE_SIGMOID, post, group, w, wd, eps, res,
                res_out, rd, alpha, out, R, W, stream);
    });
  });
}

PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_rope)>(a[0]);
    const at::Tensor& tq = with_dims("q", a[1], 4, "q must be [B,T,heads,D]");
    const int64_t B = tq.size(0), T = tq.size(1), Hq = tq.size(2), D = tq.size(3);
    const int dev = gpu_of(tq);
    const Rows q = rows("q", a[1], {B, T, Hq, D}, dev);
    const double* freqs;
    const int64_t half = with_dims("freqs", a[3], 1, "freqs must be [rot/2]").numel();
    freqs = tensor<double>("freqs", a[3], at::kDouble, {half}, dev);
    const Rows q_out = rows("q_out", a[4], {B, T, Hq, D}, dev);
    Rows k{nullptr, 0}, k_out{nullptr, 0};
    int64_t Hk = 0;
    if ((a[2] == Py_None) != (a[5] == Py_None)) fail("k and k_out come together");
    if (a[2] != Py_None) {
      Hk = with_dims("k", a[2], 4, "k must be [B,T,heads,D]").size(2);
      if (Hk < 1) fail("k must have heads");
      k = rows("k", a[2], {B, T, Hk, D}, dev);
      k_out = rows("k_out", a[5], {B, T, Hk, D}, dev);
    }
    const int64_t N = a[8] == Py_None ? B : unpack("cu_seqlens", a[8]).numel() - 1;
    const int64_t *pos = optional<int64_t>("positions", a[6], int64, {B, T}, dev),
                  *off = optional<int64_t>("offsets", a[7], int64, {N}, dev),
                  *cu = optional<int64_t>("cu_seqlens", a[8], int64, {N + 1}, dev);
    const bool inter = truth(a[9]);
    const float amplitude = number(a[10]);
    const bool inverse = truth(a[11]);
    void* stream = stream_of(a[12], dev);
    Device current(dev);
    return without_gil([&] {
      return fn(q.at, q.row, q_out.at, q_out.row, k.at, k.row, k_out.at, k_out.row, freqs,
                2 * half, amplitude, inter, inverse, pos, off, cu, N, B, T, Hq, Hk, D, stream);
    });
  });
}

// The tensors k4, ks, v4, vs from o on, [slots, Hk, cap, D / 2] the first.
struct Caches {
  void *k4, *ks, *v4, *vs;
  int64_t slots, cap;
};
Caches caches(PyObject* const* o, int64_t Hk, int64_t D, int dev) {
  const at::Tensor& t = with_dims("k4", o[0], 4, "k4 must be [slots,Hk,capacity,D/2]");
  const int64_t S = t.size(0), cap = t.size(2), tiles = cap / 32;
  return Caches{tensor("k4", o[0], at::kByte, {S, Hk, cap, D / 2}, dev),
                tensor("ks", o[1], at::kByte, {S, Hk, tiles, D / 32, 32}, dev),
                tensor("v4", o[2], at::kByte, {S, Hk, tiles, 16 * D}, dev),
                tensor("vs", o[3], at::kByte, {S, Hk, tiles, D / 32, 32}, dev),
                S,
                cap};
}

PyObject* put4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_cache4_put)>(a[0]);
    const at::Tensor& tk = with_dims("k", a[1], 4, "k must be [B,T,heads,D]");
    const int64_t B = tk.size(0), T = tk.size(1), Hk = tk.size(2), D = tk.size(3);
    const int dev = gpu_of(tk);
    const Rows k = rows("k", a[1], {B, T, Hk, D}, dev), v = rows("v", a[2], {B, T, Hk, D}, dev);
    const Caches c = caches(a + 3, Hk, D, dev);
    const int64_t N = a[8] == Py_None ? B : unpack("cu_seqlens", a[8]).numel() - 1;
    const int64_t *off = optional<int64_t>("offsets", a[7], int64, {N}, dev),
                  *cu = optional<int64_t>("cu_seqlens", a[8], int64, {N + 1}, dev),
                  *slots = optional<int64_t>("slots", a[9], int64, {N}, dev);
    if ((a[10] == Py_None) != (a[11] == Py_None)) fail("k_out and v_out come together");
    void *k_out = optional("k_out", a[10], bf16, {B, T, Hk, D}, dev),
         *v_out = optional("v_out", a[11], bf16, {B, T, Hk, D}, dev);
    void* stream = stream_of(a[12], dev);
    Device current(dev);
    return without_gil([&] {
      return fn(k.at, k.row, v.at, v.row, c.k4, c.ks, c.v4, c.vs, c.slots, c.cap, k_out, v_out,
                off, slots, cu, N, B, T, Hk, D, stream);
    });
  });
}

PyObject* attn4_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> int64_t {
    const auto fn = function<decltype(&kda_attn4_fwd)>(a[0]);
    const auto ws_bytes = function<decltype(&kda_attn4_workspace_bytes)>(a[1]);
    const at::Tensor &tq = with_dims("q", a[2], 4, "q must be [B,T,heads,D]"),
                     &tk = with_dims("k4", a[3], 4, "k4 must be [slots,Hk,capacity,D/2]");
    const int64_t Bq = tq.size(0), Tq = tq.size(1), Hq = tq.size(2), D = tq.size(3),
                  Hk = tk.size(1);
    const int dev = gpu_of(tq);
    const Rows q = rows("q", a[2], {Bq, Tq, Hq, D}, dev);
    const Caches c = caches(a + 3, Hk, D, dev);
    const float scale = number(a[7]);
    void* out = tensor("out", a[8], bf16, {Bq, Tq, Hq, D}, dev);
    float* lse = optional<float>("lse", a[9], fp32, {Bq, Tq, Hq}, dev);
    const int64_t N = a[11] == Py_None ? Bq : unpack("cu_seqlens_q", a[11]).numel() - 1;
    const int64_t *k_lens = optional<int64_t>("k_lens", a[10], int64, {N}, dev),
                  *cu = optional<int64_t>("cu_seqlens_q", a[11], int64, {N + 1}, dev),
                  *slots = optional<int64_t>("slots", a[12], int64, {N}, dev);
    const int64_t part = integer(a[13]);
    void* stream = stream_of(a[15], dev);
    Device current(dev);
    const Workspace w =
        workspace_of(a[14], ws_bytes(N, Bq, Tq, c.cap, Hq, Hk, D, part), dev);
    if (w.want) return w.want;
    return without_gil([&] {
      return fn(q.at, q.row, c.k4, c.ks, c.v4, c.vs, c.slots, c.cap, scale, out, lse, cu, k_lens,
                slots, N, Bq, Tq, Hq, Hk, D, part, w.at, w.bytes, stream);
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
    {"norm", fast(norm), METH_FASTCALL, "kda_norm: its address and arguments -> status."},
    {"rope", fast(rope), METH_FASTCALL, "kda_rope: its address and arguments -> status."},
    {"put4", fast(put4), METH_FASTCALL, "kda_cache4_put: its address and arguments -> status."},
    {"attn4_fwd", fast(attn4_fwd), METH_FASTCALL, "As attn_fwd for kda_attn4_fwd."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving_calls(void) { return PyModule_Create(&module); }
