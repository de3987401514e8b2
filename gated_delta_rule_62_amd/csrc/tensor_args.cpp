// Argument checks of the serving operators' Python bindings: a dozen tensors a call, each
// with a dtype, shape, device and layout to compare, which costs 4 of a small call's 10
// microseconds from Python and 1 from here.  Host code only; no GPU call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

namespace {

// dtype codes: as KDA_DTYPE_* in include/kda.h, and int64 offsets
bool dtype_of(long code, at::ScalarType* out) {
  switch (code) {
    case 0: *out = at::kBFloat16; return true;
    case 1: *out = at::kFloat; return true;
    case 2: *out = at::kLong; return true;
  }
  return false;
}

// A Python exception on its way out of a function below.
struct Raise {
  PyObject* type;
  std::string text;
};
[[noreturn]] void fail(const std::string& text) { throw Raise{PyExc_ValueError, text}; }

// Runs f, whose C++ exceptions become Python's.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raise& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The tensor of a call's (name, tensor, dtype, shape, device) arguments, once its dtype,
// shape and device are right.
const at::Tensor& checked(PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !PyUnicode_Check(a[0]) || !PyTuple_Check(a[3]))
    throw Raise{PyExc_TypeError, "expected name, tensor, dtype, shape, device"};
  if (!THPVariable_Check(a[1]))
    throw Raise{PyExc_TypeError, std::string(PyUnicode_AsUTF8(a[0])) + " must be a tensor"};
  const at::Tensor& t = THPVariable_Unpack(a[1]);
  at::ScalarType dtype;
  if (!dtype_of(PyLong_AsLong(a[2]), &dtype)) throw Raise{PyExc_TypeError, "unknown dtype code"};
  const Py_ssize_t dims = PyTuple_GET_SIZE(a[3]);
  bool same = t.scalar_type() == dtype && t.dim() == dims;
  for (Py_ssize_t i = 0; same && i < dims; ++i)
    same = t.size(i) == PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], i));
  if (!same) {
    std::ostringstream s;
    s << PyUnicode_AsUTF8(a[0]) << " must be " << dtype << " [";
    for (Py_ssize_t i = 0; i < dims; ++i)
      s << (i ? ", " : "") << PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], i));
    s << "], got " << t.scalar_type() << " " << t.sizes();
    fail(s.str());
  }
  if (!t.is_cuda() || t.get_device() != PyLong_AsLong(a[4]))
    fail("every tensor must live on the same GPU");
  return t;
}

// tensor(name, t, dtype, shape, device) -> address of a contiguous tensor.
PyObject* tensor(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    const at::Tensor& t = checked(a, n);
    if (!t.is_contiguous()) fail(std::string(PyUnicode_AsUTF8(a[0])) + " must be contiguous");
    return PyLong_FromVoidPtr(t.data_ptr());
  });
}

// optional(...) -> the same, or None for None.
PyObject* optional(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n > 1 && a[1] == Py_None) Py_RETURN_NONE;
  return tensor(self, a, n);
}

// rows(name, t, dtype, shape, device) -> (address, row stride in elements) of a tensor
// [..., heads, D] whose tokens lie one fixed row stride apart.
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    const at::Tensor& t = checked(a, n);
    const int64_t dims = t.dim();
    if (dims != 3 && dims != 4) throw Raise{PyExc_TypeError, "expected 3 or 4 dimensions"};
    const int64_t heads = t.size(dims - 2), D = t.size(dims - 1);
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
        fail(std::string(PyUnicode_AsUTF8(a[0])) +
             " must have contiguous heads, its tokens one row stride apart");
    }
    return Py_BuildValue("(NL)", PyLong_FromVoidPtr(t.data_ptr()), (long long)row);
  });
}

PyMethodDef methods[] = {
    {"tensor", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tensor)),
     METH_FASTCALL, "Address of a contiguous tensor of this dtype, shape and device."},
    {"optional", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(optional)),
     METH_FASTCALL, "The same, or None for None."},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL,
     "Address and row stride of a tensor whose tokens lie one row stride apart."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
