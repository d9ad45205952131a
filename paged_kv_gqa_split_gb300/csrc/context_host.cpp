// A look at all tensors of a Python call in one step: 0.3 us for six, where an attribute at a time took 4.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

constexpr Py_ssize_t kMost = 16;

bool scalar_type(char c, at::ScalarType* t) {
  switch (c) {
    case 'b': *t = at::kBFloat16; return true;
    case 'f': *t = at::kFloat; return true;
    case 'i': *t = at::kInt; return true;
    case 'u': *t = at::kByte; return true;
    default: return false;
  }
}

// gather(spec, *tensors): (GPU index, addresses, then the sizes of each) if tensor i is a contiguous CUDA tensor of type
// spec[2 i] with spec[2 i + 1] dimensions, all on one GPU; None otherwise.
PyObject* gather(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  const Py_ssize_t n = count - 1;
  if (n < 1 || n > kMost || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != 2 * n) {
    PyErr_SetString(PyExc_TypeError, "gather(spec, *tensors)");
    return nullptr;
  }
  const char* spec = PyBytes_AS_STRING(args[0]);
  const at::Tensor* t[kMost];
  Py_ssize_t dims = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    at::ScalarType type;
    if (!scalar_type(spec[2 * i], &type) || !THPVariable_Check(args[1 + i])) Py_RETURN_NONE;
    t[i] = &THPVariable_Unpack(args[1 + i]);
    if (!t[i]->is_cuda() || t[i]->layout() != at::kStrided || t[i]->scalar_type() != type || t[i]->dim() != spec[2 * i + 1] - '0' ||
        !t[i]->is_contiguous() || t[i]->get_device() != t[0]->get_device())
      Py_RETURN_NONE;
    dims += t[i]->dim();
  }
  PyObject* got = PyTuple_New(1 + n + dims);
  if (got == nullptr) return nullptr;
  Py_ssize_t at = 0;
  PyTuple_SET_ITEM(got, at++, PyLong_FromLong(t[0]->get_device()));
  for (Py_ssize_t i = 0; i < n; ++i) PyTuple_SET_ITEM(got, at++, PyLong_FromVoidPtr(t[i]->data_ptr()));
  for (Py_ssize_t i = 0; i < n; ++i)
    for (const int64_t size : t[i]->sizes()) PyTuple_SET_ITEM(got, at++, PyLong_FromLongLong(size));
  return got;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gather)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_context_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__context_host() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
