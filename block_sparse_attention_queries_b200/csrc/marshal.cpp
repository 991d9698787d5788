// Checks and addresses of torch tensors for the binding's calls on paths where
// a step is bound by the host (single tokens): one call for all tensors of a
// library call instead of several attribute look-ups each.
//
//   tensors(index, t, dtype, shape, name, t, dtype, shape, name, ...)
//       every t a contiguous tensor of that dtype and shape on CUDA device
//       `index`: their addresses, a tuple of int (None for None)
//   tokens(index, t, shape, name)
//       t a bf16 tensor [(B,) T, H, d] of that shape on CUDA device `index`, its
//       last dimension contiguous: the bytes of an ab_tokens
//
// Anything else raises ValueError.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <sstream>

#include "ab.h"

namespace {

// Whole numbers in every place of a shape.
bool is_shape(PyObject* shape) {
  if (!PyTuple_Check(shape)) return false;
  for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(shape); ++k)
    if (!PyLong_Check(PyTuple_GET_ITEM(shape, k))) return false;
  return true;
}

bool same_shape(const at::Tensor& t, PyObject* shape) {
  const auto sizes = t.sizes();
  if (Py_ssize_t(sizes.size()) != PyTuple_GET_SIZE(shape)) return false;
  for (size_t k = 0; k < sizes.size(); ++k)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, Py_ssize_t(k))) != sizes[k]) return false;
  return true;
}

PyObject* refuse(PyObject* obj, const char* want, at::ScalarType type, PyObject* shape, long index, PyObject* name) {
  std::ostringstream s;
  PyObject* text = PyObject_Str(shape);
  s << PyUnicode_AsUTF8(name) << ": expected " << want << " " << at::toString(type) << " "
    << (text ? PyUnicode_AsUTF8(text) : "?") << " on cuda:" << index << ", got ";
  Py_XDECREF(text);
  if (THPVariable_Check(obj)) {
    const at::Tensor& t = THPVariable_Unpack(obj);
    s << at::toString(t.scalar_type()) << " " << t.sizes() << ", strides " << t.strides() << ", on " << t.device();
  } else {
    s << Py_TYPE(obj)->tp_name;
  }
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  return nullptr;
}

bool on_device(const at::Tensor& t, long index) { return t.is_cuda() && t.device().index() == index; }

PyObject* tensors(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 1 || (n - 1) % 4 != 0 || !PyLong_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "tensors(index, (tensor, dtype, shape, name) ...)");
    return nullptr;
  }
  try {
    const long index = PyLong_AsLong(args[0]);
    const Py_ssize_t count = (n - 1) / 4;
    PyObject* out = PyTuple_New(count);
    if (!out) return nullptr;
    for (Py_ssize_t k = 0; k < count; ++k) {
      PyObject* const* a = args + 1 + 4 * k;
      PyObject* item = nullptr;
      if (!THPDtype_Check(a[1]) || !is_shape(a[2]) || !PyUnicode_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "tensors: dtype, shape tuple and name expected");
      } else if (a[0] == Py_None) {
        Py_INCREF(Py_None);
        item = Py_None;
      } else {
        const at::ScalarType type = reinterpret_cast<THPDtype*>(a[1])->scalar_type;
        if (!THPVariable_Check(a[0])) {
          refuse(a[0], "contiguous", type, a[2], index, a[3]);
        } else {
          const at::Tensor& t = THPVariable_Unpack(a[0]);
          if (t.scalar_type() != type || !on_device(t, index) || !t.is_contiguous() || !same_shape(t, a[2]))
            refuse(a[0], "contiguous", type, a[2], index, a[3]);
          else
            item = PyLong_FromVoidPtr(t.data_ptr());
        }
      }
      if (!item) {
        Py_DECREF(out);
        return nullptr;
      }
      PyTuple_SET_ITEM(out, k, item);
    }
    return out;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !PyLong_Check(args[0]) || !is_shape(args[2]) || !PyUnicode_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "tokens(index, tensor, shape, name)");
    return nullptr;
  }
  try {
    const long index = PyLong_AsLong(args[0]);
    if (!THPVariable_Check(args[1])) return refuse(args[1], "strided", at::kBFloat16, args[2], index, args[3]);
    const at::Tensor& t = THPVariable_Unpack(args[1]);
    const auto st = t.strides();
    const size_t dims = st.size();
    if (t.scalar_type() != at::kBFloat16 || !on_device(t, index) || !same_shape(t, args[2]) || dims < 3 || dims > 4 ||
        st[dims - 1] != 1)
      return refuse(args[1], "contiguous heads of", at::kBFloat16, args[2], index, args[3]);
    const ab_tokens x{t.data_ptr(), dims == 4 ? st[0] : 0, st[dims - 3], st[dims - 2]};
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&x), sizeof x);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"tensors", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(tensors)), METH_FASTCALL, nullptr},
    {"tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(tokens)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// The torch whose headers this was built with, for the build and for the binding.
const char kTorch[] = "AB_TORCH=" AB_TORCH ";";

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", kTorch) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
