// Argument checks of the Python binding's block operators in one native call: the addresses of a
// call's tensors, or None if any of them is not what the call's sizes say (the binding then finds
// out which, and says so). Checked one attribute at a time from Python, eight tensors cost 4 us,
// half of a small call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// ptrs(tensors, counts, kinds, device): tuples of tensors (or None, or addresses) and of their
// numbers of elements, their types (a string of b bfloat16, f float32, i int32, u uint8), and the
// current device.
PyObject* ptrs(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  Py_ssize_t kinds = 0;
  if (nargs != 4 || !PyTuple_Check(args[0]) || !PyTuple_Check(args[1])) Py_RETURN_NONE;
  const char* kind = PyUnicode_AsUTF8AndSize(args[2], &kinds);
  const long device = PyLong_AsLong(args[3]);
  if (!kind || PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PyTuple_GET_SIZE(args[0]);
  if (PyTuple_GET_SIZE(args[1]) != n || kinds != n) Py_RETURN_NONE;
  PyObject* out = PyTuple_New(n);
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(args[0], i);
    PyObject* address = nullptr;
    if (o == Py_None || PyLong_Check(o)) {
      Py_INCREF(o);
      address = o;
    } else if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      const at::ScalarType type = kind[i] == 'b'   ? at::kBFloat16
                                  : kind[i] == 'f' ? at::kFloat
                                  : kind[i] == 'i' ? at::kInt
                                                   : at::kByte;
      const long long count = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], i));
      try {
        if (t.defined() && t.is_cuda() && t.get_device() == device && t.scalar_type() == type &&
            t.numel() == count && t.is_contiguous())
          address = PyLong_FromVoidPtr(t.data_ptr());
      } catch (...) {  // a tensor without storage: the binding's own checks name it
      }
    }
    if (!address) {
      Py_DECREF(out);
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    PyTuple_SET_ITEM(out, i, address);
  }
  return out;
}

PyMethodDef methods[] = {
    {"ptrs", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(ptrs)), METH_FASTCALL,
     "Device addresses of a call's tensors, or None if one of them does not fit."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
