// marshal.cpp -- what the Python binding reads off torch tensors, in one native call each: a decode step's kernels
// run for a few microseconds, and a tensor's shape, strides, dtype and pointer cost one microsecond of
// Python attribute reads (0.1 here).  Built where torch's headers are found; the binding falls back to Python
// reads without it, with the same checks and the same errors.
#include <torch/csrc/autograd/python_variable.h>

#include <Python.h>

#include <cstring>

#include "../../include/qnre.h"

namespace {

// qnre_dtype_t, then 3 = int32, 4 = int64; -1 for the rest.
int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return QNRE_DTYPE_BF16;
    case at::kHalf: return QNRE_DTYPE_FP16;
    case at::kFloat: return QNRE_DTYPE_FP32;
    case at::kInt: return 3;
    case at::kLong: return 4;
    default: return -1;
  }
}

// view4(tensor) -> the bytes of its qnre_tensor4_t, or None where it is no rank-4 tensor of a known float type.
PyObject* view4(PyObject*, PyObject* obj) {
  if (!THPVariable_Check(obj)) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(obj);
  const int code = code_of(t);
  if (t.dim() != 4 || code < 0 || code > QNRE_DTYPE_FP32) Py_RETURN_NONE;
  qnre_tensor4_t v;
  std::memset(&v, 0, sizeof(v));
  v.data = t.data_ptr();
  for (int i = 0; i < 4; ++i) {
    v.shape[i] = t.size(i);
    v.stride[i] = t.stride(i);
  }
  v.dtype = code;
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&v), sizeof(v));
}

// pointer(tensor, code, *shape) -> its address, or None unless it is contiguous, of that type and (where given) shape.
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 2 || !THPVariable_Check(args[0])) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  if (code_of(t) != PyLong_AsLong(args[1]) || !t.is_contiguous()) Py_RETURN_NONE;
  if (n > 2) {
    if (t.dim() != n - 2) Py_RETURN_NONE;
    for (Py_ssize_t i = 0; i < n - 2; ++i)
      if (t.size(i) != PyLong_AsLongLong(args[2 + i])) Py_RETURN_NONE;
  }
  return PyLong_FromVoidPtr(t.data_ptr());
}

// sizes(tensor) -> its shape as a plain tuple.
PyObject* sizes(PyObject*, PyObject* obj) {
  if (!THPVariable_Check(obj)) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(obj);
  PyObject* r = PyTuple_New(t.dim());
  if (r == nullptr) return nullptr;
  for (int64_t i = 0; i < t.dim(); ++i) PyTuple_SET_ITEM(r, i, PyLong_FromLongLong(t.size(i)));
  return r;
}

// type_code(tensor) -> as code_of.
PyObject* type_code(PyObject*, PyObject* obj) {
  return PyLong_FromLong(THPVariable_Check(obj) ? code_of(THPVariable_Unpack(obj)) : -1);
}

PyMethodDef methods[] = {{"view4", view4, METH_O, nullptr},
                         {"pointer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointer)), METH_FASTCALL,
                          nullptr},
                         {"sizes", sizes, METH_O, nullptr},
                         {"type_code", type_code, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
