// Python calls of the C ABI's entry points that take (plan, device pointers..., stream):
// the operands are checked against what the plan says and the entry point is called,
// without a Python frame between. A small product takes the GPU 2.6 us, and the host
// 2.0 for checking its operands one by one in Python and the call through ctypes; here
// both are 0.33 (a norm with seven operands: 3.3 and 0.37).
//
//   Call(entry point's address, plan handle, index of the main operand, specs)
//
// specs: one (dtype, shape, row stride or None) an operand; None: a vector. The call takes the
// operands and the stream (None: the current one) and returns the entry point's
// status, or -1 where an operand is not what the specs say or is no tensor: the
// caller then goes through the checks in Python, which name the operand.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

constexpr int kMost = 8;   // operands of an entry point

struct Spec {
  c10::ScalarType type;
  int dims;
  int64_t shape[2];
  int64_t ld;              // 0: a vector
};

struct Call {
  PyObject_HEAD
  vectorcallfunc vector;
  void* fn;
  void* plan;
  int count, main;
  Spec specs[kMost];
};

PyObject* current_device;  // torch._C._cuda_getDevice
PyObject* current_stream;  // torch._C._cuda_getCurrentRawStream

// The operand's address; false where the slow path has to look at it.
bool address(PyObject* o, const Spec& s, int device, void*& p) {
  if (o == Py_None) {
    p = nullptr;
    return true;
  }
  if (!THPVariable_CheckExact(o)) return false;
  c10::TensorImpl* t = THPVariable_Unpack(o).unsafeGetTensorImpl();
  if (!t->is_cuda() || t->device().index() != device || t->dtype() != c10::scalarTypeToTypeMeta(s.type) ||
      t->dim() != s.dims)
    return false;
  const auto size = t->sizes(), stride = t->strides();
  for (int d = 0; d < s.dims; d++)
    if (size[d] != s.shape[d]) return false;
  if (s.ld == 0) {
    if (s.shape[0] > 1 && stride[0] != 1) return false;
  } else {
    if (stride[0] != s.ld && s.shape[0] > 1 && s.shape[1] > 0) return false;
    if (stride[1] != 1 && s.shape[1] > 1) return false;
  }
  p = t->mutable_data();
  return true;
}

int32_t enter(void* fn, void* h, void* const* a, int n, void* s) {
  typedef void* P;
  switch (n) {
    case 4: return reinterpret_cast<int32_t (*)(P, P, P, P, P, P)>(fn)(h, a[0], a[1], a[2], a[3], s);
    case 5: return reinterpret_cast<int32_t (*)(P, P, P, P, P, P, P)>(fn)(h, a[0], a[1], a[2], a[3], a[4], s);
    default:
      return reinterpret_cast<int32_t (*)(P, P, P, P, P, P, P, P, P, P)>(fn)(h, a[0], a[1], a[2], a[3], a[4], a[5],
                                                                             a[6], a[7], s);
  }
}

PyObject* call(PyObject* self, PyObject* const* args, size_t nargsf, PyObject* names) {
  const Call* c = reinterpret_cast<const Call*>(self);
  if (PyVectorcall_NARGS(nargsf) != c->count + 1 || names) {
    PyErr_SetString(PyExc_TypeError, "expected the operands and a stream");
    return nullptr;
  }
  try {
    if (!THPVariable_CheckExact(args[c->main])) return PyLong_FromLong(-1);
    const c10::TensorImpl* main = THPVariable_Unpack(args[c->main]).unsafeGetTensorImpl();
    if (!main->is_cuda()) return PyLong_FromLong(-1);
    const int device = main->device().index();
    void* p[kMost];
    for (int i = 0; i < c->count; i++)
      if (!address(args[i], c->specs[i], device, p[i])) return PyLong_FromLong(-1);
    PyObject* now = PyObject_CallNoArgs(current_device);
    if (!now) return nullptr;
    const long on = PyLong_AsLong(now);
    PyObject* where = nullptr;                       // the stream, owned
    if (on == device && args[c->count] == Py_None) where = PyObject_CallOneArg(current_stream, now);
    else if (on == device && PyLong_CheckExact(args[c->count])) where = Py_NewRef(args[c->count]);
    Py_DECREF(now);
    if (!where) return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1);
    void* stream = PyLong_AsVoidPtr(where);
    Py_DECREF(where);
    if (PyErr_Occurred()) return nullptr;
    int32_t status;
    Py_BEGIN_ALLOW_THREADS
    status = enter(c->fn, c->plan, p, c->count, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
  } catch (const std::exception& e) {                // a tensor without storage or strides
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

int init(PyObject* self, PyObject* args, PyObject*) {
  Call* c = reinterpret_cast<Call*>(self);
  PyObject *fn, *plan, *specs;
  if (!PyArg_ParseTuple(args, "OOiO!", &fn, &plan, &c->main, &PyTuple_Type, &specs)) return -1;
  c->fn = PyLong_AsVoidPtr(fn);
  c->plan = PyLong_AsVoidPtr(plan);
  if (PyErr_Occurred()) return -1;
  const Py_ssize_t n = PyTuple_GET_SIZE(specs);
  if ((n != 4 && n != 5 && n != 8) || c->main < 0 || c->main >= n || !c->fn || !c->plan) {
    PyErr_SetString(PyExc_ValueError, "an entry point with 4, 5 or 8 operands and a plan is expected");
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; i++) {
    Spec& s = c->specs[i];
    PyObject *type, *shape, *ld;
    if (!PyArg_ParseTuple(PyTuple_GET_ITEM(specs, i), "OO!O", &type, &PyTuple_Type, &shape, &ld)) return -1;
    if (!THPDtype_Check(type)) {
      PyErr_SetString(PyExc_TypeError, "a spec begins with a dtype");
      return -1;
    }
    s.type = reinterpret_cast<THPDtype*>(type)->scalar_type;
    s.dims = (int)PyTuple_GET_SIZE(shape);
    s.ld = ld == Py_None ? 0 : PyLong_AsLongLong(ld);
    if (!PyErr_Occurred() && (s.dims != (s.ld == 0 ? 1 : 2) || s.ld < 0))
      PyErr_SetString(PyExc_ValueError, "a matrix has two dimensions and a row stride, a vector one and None");
    for (int d = 0; d < s.dims && !PyErr_Occurred(); d++) s.shape[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
    if (PyErr_Occurred()) return -1;
  }
  c->count = (int)n;
  c->vector = call;
  return 0;
}

PyTypeObject type = {PyVarObject_HEAD_INIT(nullptr, 0)};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nmcall", nullptr, -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nmcall(void) {
  type.tp_name = "_nmcall.Call";
  type.tp_basicsize = sizeof(Call);
  type.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_VECTORCALL;
  type.tp_vectorcall_offset = offsetof(Call, vector);
  type.tp_call = PyVectorcall_Call;
  type.tp_new = PyType_GenericNew;
  type.tp_init = init;
  if (PyType_Ready(&type) < 0) return nullptr;
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (!torch_c) return nullptr;
  current_device = PyObject_GetAttrString(torch_c, "_cuda_getDevice");
  current_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  Py_DECREF(torch_c);
  if (!current_device || !current_stream) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  if (PyModule_AddObjectRef(m, "Call", reinterpret_cast<PyObject*>(&type)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
