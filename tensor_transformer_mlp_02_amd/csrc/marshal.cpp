// Checks and device addresses of a call's tensors for the Python binding.
//
// A call of this library passes 5 to 18 tensors; looking at each from Python
// (device, contiguity, size, type, address) takes longer than the launch.
// addresses(items, device) does it here, on the same items as the binding's
// own loop: tuples (tensor | int | None, bytes | None, name[, type name]).
// It returns the list of addresses, or None where any item does not pass:
// the binding's loop then finds the item and words the error.
#include <torch/csrc/autograd/python_variable.h>

namespace {

struct Owned {  // dropped on every way out, exceptions included
  PyObject* p;
  ~Owned() { Py_XDECREF(p); }
};

bool type_is(const at::Tensor& t, PyObject* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return PyUnicode_CompareWithASCIIString(name, "float32") == 0;
    case at::kInt: return PyUnicode_CompareWithASCIIString(name, "int32") == 0;
    case at::kBFloat16: return PyUnicode_CompareWithASCIIString(name, "bfloat16") == 0;
    default: return false;
  }
}

PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses(list, device)");
    return nullptr;
  }
  PyObject* items = args[0];
  const long device = PyLong_AsLong(args[1]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PyList_GET_SIZE(items);
  Owned list{PyList_New(n)};
  if (!list.p) return nullptr;
  PyObject* out = list.p;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* it = PyList_GET_ITEM(items, i);
    bool fine = PyTuple_Check(it) && PyTuple_GET_SIZE(it) >= 3;
    PyObject* value = nullptr;
    if (fine) {
      PyObject* t = PyTuple_GET_ITEM(it, 0);
      if (t == Py_None || PyLong_Check(t)) {
        Py_INCREF(t);
        value = t;
      } else if (THPVariable_Check(t)) {
        const at::Tensor& x = THPVariable_Unpack(t);
        PyObject* nb = PyTuple_GET_ITEM(it, 1);
        PyObject* type = PyTuple_GET_SIZE(it) > 3 ? PyTuple_GET_ITEM(it, 3) : Py_None;
        fine = x.is_cuda() && x.get_device() == device && x.is_contiguous() &&
               (type == Py_None || (PyUnicode_Check(type) && type_is(x, type)));
        if (fine && nb != Py_None) {
          const long long need = PyLong_AsLongLong(nb);
          if (need == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            fine = false;
          } else {
            fine = (long long)x.nbytes() >= need;
          }
        }
        if (fine) value = PyLong_FromVoidPtr(x.data_ptr());
      } else {
        fine = false;
      }
    }
    if (!fine || !value) {
      Py_XDECREF(value);
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    PyList_SET_ITEM(out, i, value);
  }
  list.p = nullptr;
  return out;
}

// x.data_ptr() and the like may throw (a tensor without storage): the
// binding's loop meets the same and words it
PyObject* addresses_safe(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return addresses(self, args, nargs);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(addresses_safe)),
     METH_FASTCALL, "addresses(items, device) -> list of addresses, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
