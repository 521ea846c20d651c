// Calls of the library from the Python binding.
//
// A call passes 5 to 18 tensors; looking at each from Python (device,
// contiguity, size, type, address) takes longer than the launch.  Here it is
// done in one step, on the same items as the binding's own loop: tuples
// (tensor | int | None, bytes | None, name[, type name]).
//   addresses(items, device) -> the list of addresses
//   call(name, function, args, stream) -> the int result of the entry point
//       `name` at the address `function`; `args` is a tuple of items and of
//       plain ints / None, one for each of its arguments but the last, the
//       stream; stream None: the current one
//   setup(device, stream): torch's functions for the current device and for
//       a device's current raw stream
//   torch_version: the torch whose headers it was built with
// The first two return None where an item does not pass, call also where no
// item is a tensor (nothing shows that the GPU is in use): the binding's own
// loop then does the work, or finds the item and words the error.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "../../include/tpmlp_block.h"
#include "../../include/tpmlp_fp8g.h"

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

// The address that an item stands for; false: it does not pass (or an error
// is set).
bool address_of(PyObject* it, long device, uintptr_t& out) {
  if (!PyTuple_Check(it) || PyTuple_GET_SIZE(it) < 3) return false;
  PyObject* t = PyTuple_GET_ITEM(it, 0);
  if (t == Py_None) {
    out = 0;
    return true;
  }
  if (PyLong_Check(t)) {
    out = (uintptr_t)PyLong_AsUnsignedLongLong(t);
    return !PyErr_Occurred();
  }
  if (!THPVariable_Check(t)) return false;
  const at::Tensor& x = THPVariable_Unpack(t);
  PyObject* nb = PyTuple_GET_ITEM(it, 1);
  PyObject* type = PyTuple_GET_SIZE(it) > 3 ? PyTuple_GET_ITEM(it, 3) : Py_None;
  if (!x.is_cuda() || x.get_device() != device || !x.is_contiguous()) return false;
  if (type != Py_None && !(PyUnicode_Check(type) && type_is(x, type))) return false;
  if (nb != Py_None) {
    const long long need = PyLong_AsLongLong(nb);
    if (need == -1 && PyErr_Occurred()) return false;
    if ((long long)x.nbytes() < need) return false;
  }
  out = reinterpret_cast<uintptr_t>(x.data_ptr());
  return true;
}

PyObject* refused() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses(list, device)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[1]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PyList_GET_SIZE(args[0]);
  Owned list{PyList_New(n)};
  if (!list.p) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    uintptr_t a = 0;
    PyObject* it = PyList_GET_ITEM(args[0], i);
    if (!address_of(it, device, a)) return refused();
    PyObject* value = nullptr;
    if (PyTuple_GET_ITEM(it, 0) == Py_None) {
      Py_INCREF(Py_None);
      value = Py_None;
    } else {
      value = PyLong_FromUnsignedLongLong(a);
    }
    if (!value) return nullptr;
    PyList_SET_ITEM(list.p, i, value);
  }
  PyObject* out = list.p;
  list.p = nullptr;
  return out;
}

// An entry point is called as the function that its header declares: each slot
// becomes an argument of the declared type, a pointer or an integer.
constexpr int SLOTS = 24;
template <typename A>
A argument(uintptr_t v) {
  if constexpr (std::is_pointer_v<A>) return reinterpret_cast<A>(v);
  else return static_cast<A>(v);
}
template <typename F> struct Declared;
template <typename... A>
struct Declared<int(A...)> {
  static_assert(sizeof...(A) <= SLOTS);
  static constexpr int COUNT = sizeof...(A);
  template <size_t... I>
  static int spread(int (*f)(A...), const uintptr_t* v, std::index_sequence<I...>) {
    return f(argument<A>(v[I])...);
  }
  static int call(uintptr_t f, const uintptr_t* v) {
    return spread(reinterpret_cast<int (*)(A...)>(f), v, std::index_sequence_for<A...>{});
  }
};
struct Entry {
  const char* name;
  int count;  // arguments
  int (*call)(uintptr_t function, const uintptr_t* slots);
};
#define ENTRY(f) {#f, Declared<decltype(f)>::COUNT, &Declared<decltype(f)>::call}
constexpr Entry entries[] = {ENTRY(tp_block_norm_fwd), ENTRY(tp_block_norm_bwd), ENTRY(tp_moe_route_fwd),
                             ENTRY(tp_moe_route_bwd), ENTRY(tp_moe_route_tables), ENTRY(tp_adamw_step),
                             ENTRY(tp_fp8g_quantize), ENTRY(tp_fp8g_gemm), ENTRY(tp_fp8g_glu_fwd),
                             ENTRY(tp_fp8g_glu_bwd)};
#undef ENTRY
const Entry* entry_of(PyObject* name) {
  if (PyUnicode_Check(name))
    for (const Entry& e : entries)
      if (PyUnicode_CompareWithASCIIString(name, e.name) == 0) return &e;
  return nullptr;
}

PyObject* current_device = nullptr;
PyObject* current_stream = nullptr;

PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2 || !PyCallable_Check(args[0]) || !PyCallable_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "setup(device function, stream function)");
    return nullptr;
  }
  for (int i = 0; i < 2; ++i) {
    PyObject*& to = i == 0 ? current_device : current_stream;
    Py_INCREF(args[i]);
    Py_XDECREF(to);
    to = args[i];
  }
  Py_RETURN_NONE;
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4 || !PyTuple_Check(args[2]) || !current_device) {
    PyErr_SetString(PyExc_TypeError, "call(name, function, tuple, stream), after setup()");
    return nullptr;
  }
  const Entry* entry = entry_of(args[0]);
  if (!entry) return PyErr_Format(PyExc_TypeError, "%R is no entry point", args[0]);
  const uintptr_t fn = (uintptr_t)PyLong_AsUnsignedLongLong(args[1]);
  if (PyErr_Occurred()) return nullptr;
  PyObject* list = args[2];
  const Py_ssize_t n = PyTuple_GET_SIZE(list);
  if (n + 1 != entry->count)
    return PyErr_Format(PyExc_TypeError, "%s takes %d arguments before the stream, got %zd", entry->name,
                        entry->count - 1, n);
  long device = -1;
  PyObject* device_object = nullptr;
  uintptr_t v[SLOTS] = {0};
  Owned holder{nullptr};
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* it = PyTuple_GET_ITEM(list, i);
    if (it == Py_None) continue;
    if (PyLong_Check(it)) {
      int over = 0;
      const long long x = PyLong_AsLongLongAndOverflow(it, &over);
      v[i] = over > 0 ? (uintptr_t)PyLong_AsUnsignedLongLong(it) : (uintptr_t)x;
      if (over < 0 || PyErr_Occurred()) return refused();
      continue;
    }
    if (!PyTuple_Check(it) || PyTuple_GET_SIZE(it) < 3) return refused();
    if (!device_object && THPVariable_Check(PyTuple_GET_ITEM(it, 0))) {
      // a GPU tensor: torch is set up for the GPU
      if (!THPVariable_Unpack(PyTuple_GET_ITEM(it, 0)).is_cuda()) return refused();
      holder.p = device_object = PyObject_CallNoArgs(current_device);
      if (!device_object) return refused();
      device = PyLong_AsLong(device_object);
    }
    if (!address_of(it, device, v[i])) return refused();
  }
  if (!device_object) return refused();
  if (args[3] == Py_None) {
    Owned s{PyObject_CallOneArg(current_stream, device_object)};
    if (!s.p) return refused();
    v[n] = (uintptr_t)PyLong_AsUnsignedLongLong(s.p);
  } else {
    v[n] = (uintptr_t)PyLong_AsUnsignedLongLong(args[3]);
  }
  if (PyErr_Occurred()) return refused();
  int rc;
  Py_BEGIN_ALLOW_THREADS  // a full queue makes a launch wait
  rc = entry->call(fn, v);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// x.data_ptr() and the like may throw (a tensor without storage): the
// binding's loop meets the same and words it
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return F(self, args, nargs);
  } catch (...) {
    return refused();
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<F>));
}

PyMethodDef methods[] = {
    {"addresses", method<addresses>(), METH_FASTCALL, "addresses(items, device)"},
    {"call", method<call>(), METH_FASTCALL, "call(name, function, args, stream)"},
    {"setup", method<setup>(), METH_FASTCALL, "setup(device function, stream function)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
