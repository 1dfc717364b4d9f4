// pytensor.cpp -- what the torch helpers have to know of a tensor (pointer,
// sizes, strides, type, device), read from torch's own tensor object: through
// Python's attributes and methods each of them costs 30 to 60 ns, five or more to
// a tensor, which was most of a small call's time on the host.
//
// Built against torch's headers into the module _pytensor; without it, or with another
// torch than the one whose headers it was built with (SIMAR_TORCH, the version that
// torch's Python side gives), the package takes the same checks in Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

#include <exception>

namespace {

// Errors of torch (a tensor without storage, say) are Python errors.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* usage(const char* text) {
  PyErr_SetString(PyExc_TypeError, text);
  return nullptr;
}

const at::Tensor* tensor_of(PyObject* o, PyObject* what) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%S must be a tensor", what);
  return nullptr;
}

// the library's code of a float type, 0 for any other type
int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return 1;
    case at::kHalf: return 2;
    case at::kBFloat16: return 3;
    default: return 0;
  }
}
// those float types, as dtypes
PyObject* floats() {
  static PyObject* types = Py_BuildValue("(OOO)", (PyObject*)torch::getTHPDtype(at::kFloat),
                                         (PyObject*)torch::getTHPDtype(at::kHalf), (PyObject*)torch::getTHPDtype(at::kBFloat16));
  return types;
}
PyObject* dtype_of(const at::Tensor& t) { return (PyObject*)torch::getTHPDtype(t.scalar_type()); }
unsigned long long address(const at::Tensor& t) { return (unsigned long long)(uintptr_t)t.data_ptr(); }

// A 2-D device tensor with contiguous rows: the elements from row to row, or -1
// and an error.
long long row_step(const at::Tensor& t, PyObject* what) {
  if (t.dim() != 2 || !t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%S must be a 2-D device tensor", what);
    return -1;
  }
  if (t.stride(1) != 1 && t.size(1) > 1) {
    PyErr_Format(PyExc_ValueError, "%S's rows must be contiguous", what);
    return -1;
  }
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

struct Rows {
  unsigned long long at;
  long long step, rows, cols;
  int code;
  long device;
};
// ... of one of the float types and, where `like` is not None, of the shape, type
// and device that this tuple of rows() says
bool read_rows(PyObject* const* a, Rows& r) {
  const at::Tensor* t = tensor_of(a[0], a[1]);
  if (!t || (r.step = row_step(*t, a[1])) < 0) return false;
  r.rows = t->size(0);
  r.cols = t->size(1);
  r.device = t->get_device();
  if ((r.code = code_of(*t)) == 0) {
    PyErr_Format(PyExc_ValueError, "unsupported dtype %S", dtype_of(*t));
    return false;
  }
  if (a[2] != Py_None) {
    if (!PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 6) return usage("like: a tuple that rows() returned");
    const bool same = PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], 2)) == r.rows &&
                      PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], 3)) == r.cols &&
                      PyLong_AsLong(PyTuple_GET_ITEM(a[2], 4)) == r.code &&
                      PyLong_AsLong(PyTuple_GET_ITEM(a[2], 5)) == r.device;
    if (PyErr_Occurred()) return false;
    if (!same) {
      PyErr_Format(PyExc_ValueError, "%S must have the first tensor's shape, dtype and device", a[1]);
      return false;
    }
  }
  r.at = address(*t);
  return true;
}

// rows(tensor, what, like): (pointer, row stride, rows, columns, type code, device
// index)
PyObject* rows(PyObject* const* a, Py_ssize_t n) {
  Rows r;
  if (n != 3) return usage("rows(tensor, what, like)");
  return read_rows(a, r) ? Py_BuildValue("(KLLLil)", r.at, r.step, r.rows, r.cols, r.code, r.device) : nullptr;
}
// like(tensor, what, like): the first two of rows()'s; of None, None and the
// columns
PyObject* like(PyObject* const* a, Py_ssize_t n) {
  Rows r;
  if (n != 3 || !PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 6)
    return usage("like(tensor, what, a tuple that rows() returned)");
  if (a[0] == Py_None) return Py_BuildValue("(OO)", Py_None, PyTuple_GET_ITEM(a[2], 3));
  return read_rows(a, r) ? Py_BuildValue("(KL)", r.at, r.step) : nullptr;
}

// raw(tensor, what, dtype): (pointer, bytes from row to row, rows, bytes of a row,
// device index) of a tensor of any type; dtype: the one it must have, or None.
PyObject* raw(PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return usage("raw(tensor, what, dtype)");
  const at::Tensor* t = tensor_of(a[0], a[1]);
  if (!t) return nullptr;
  const long long step = row_step(*t, a[1]);
  if (step < 0) return nullptr;
  if (a[2] != Py_None && a[2] != dtype_of(*t))
    return PyErr_Format(PyExc_ValueError, "%S must be of type %S", a[1], a[2]);
  const long long e = (long long)t->element_size();
  return Py_BuildValue("(KLLLl)", address(*t), step * e, (long long)t->size(0), (long long)t->size(1) * e,
                       (long)t->get_device());
}

// Whether a tensor is contiguous, on that device, of that shape and one of those
// types; an error that says what it must be where not.
bool fits(const at::Tensor& t, PyObject* what, PyObject* types, long device, const long long* shape, int dims) {
  bool ok = t.dim() == dims && t.get_device() == device && t.is_contiguous();
  for (int i = 0; ok && i < dims; i++) ok = t.size(i) == shape[i];
  bool type = false;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(types); i++) type = type || PyTuple_GET_ITEM(types, i) == dtype_of(t);
  if (ok && type) return true;
  PyObject* sizes = PyTuple_New(dims);
  for (int i = 0; sizes && i < dims; i++) {
    PyObject* d = PyLong_FromLongLong(shape[i]);
    if (!d) Py_CLEAR(sizes);
    else PyTuple_SET_ITEM(sizes, i, d);
  }
  if (sizes)
    PyErr_Format(PyExc_ValueError, "%S must be a contiguous tensor %R of one of %R on cuda:%ld", what, sizes, types, device);
  Py_XDECREF(sizes);
  return false;
}

// pointer(tensor, what, types, device index, *shape): the data pointer of such a
// tensor (None for None)
constexpr int kDims = 4;
PyObject* pointer(PyObject* const* a, Py_ssize_t n) {
  if (n < 4 || n > 4 + kDims || !PyTuple_Check(a[2])) return usage("pointer(tensor, what, types, device, *shape)");
  if (a[0] == Py_None) Py_RETURN_NONE;
  long long shape[kDims];
  for (Py_ssize_t i = 4; i < n; i++) shape[i - 4] = PyLong_AsLongLong(a[i]);
  const long device = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* t = tensor_of(a[0], a[1]);
  if (!t || !fits(*t, a[1], a[2], device, shape, (int)n - 4)) return nullptr;
  return PyLong_FromUnsignedLongLong(address(*t));
}

// gain(tensor, columns, device index): (pointer, type code) of that many floats; of
// None, None and fp32's code
PyObject* gain(PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return usage("gain(tensor, columns, device)");
  if (a[0] == Py_None) return Py_BuildValue("(Oi)", Py_None, 1);
  const long long shape[1] = {PyLong_AsLongLong(a[1])};
  const long device = PyLong_AsLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  static PyObject* what = PyUnicode_InternFromString("gain");
  const at::Tensor* t = tensor_of(a[0], what);
  if (!t || !fits(*t, what, floats(), device, shape, 1)) return nullptr;
  return Py_BuildValue("(Ki)", address(*t), code_of(*t));
}

// slots(ids, teacher, ids' types, rows, device index): (ids pointer, teacher
// pointer, the teacher's type code, topk) of [rows, topk] tensors
PyObject* slots(PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !PyTuple_Check(a[2])) return usage("slots(ids, teacher, types, rows, device)");
  static PyObject *ids_s = PyUnicode_InternFromString("ids"), *teacher_s = PyUnicode_InternFromString("teacher");
  const at::Tensor *ids = tensor_of(a[0], ids_s), *teacher = ids ? tensor_of(a[1], teacher_s) : nullptr;
  if (!teacher) return nullptr;
  if (ids->dim() != 2) return PyErr_Format(PyExc_ValueError, "ids must be [rows, topk]");
  const long long shape[2] = {PyLong_AsLongLong(a[3]), ids->size(1)};
  const long device = PyLong_AsLong(a[4]);
  if (PyErr_Occurred() || !fits(*ids, ids_s, a[2], device, shape, 2) || !fits(*teacher, teacher_s, floats(), device, shape, 2))
    return nullptr;
  return Py_BuildValue("(KKiL)", address(*ids), address(*teacher), code_of(*teacher), shape[1]);
}

// tensors(sequence, what, device index, like): (pointers, counts, type codes), each
// an array of the host in a bytes object, of contiguous tensors on that device;
// like: None, or such a tuple whose counts and types they must have
PyObject* tensors(PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return usage("tensors(sequence, what, device, like)");
  const long device = PyLong_AsLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  // (a tuple of its own: it cannot change while it is read)
  PyObject* seq = PySequence_Tuple(a[0]);
  if (!seq) return nullptr;
  const Py_ssize_t count = PyTuple_GET_SIZE(seq);
  PyObject* made[3] = {PyBytes_FromStringAndSize(nullptr, count * (Py_ssize_t)sizeof(void*)),
                       PyBytes_FromStringAndSize(nullptr, count * (Py_ssize_t)sizeof(int64_t)),
                       PyBytes_FromStringAndSize(nullptr, count * (Py_ssize_t)sizeof(int))};
  bool ok = made[0] && made[1] && made[2];
  try {
    for (Py_ssize_t i = 0; ok && i < count; i++) {
      const at::Tensor* t = tensor_of(PyTuple_GET_ITEM(seq, i), a[1]);
      const int code = t ? code_of(*t) : 0;
      ok = t != nullptr;
      if (ok && (code == 0 || t->get_device() != device || !t->is_contiguous())) {
        PyErr_Format(PyExc_ValueError, "%S[%zd] must be a contiguous tensor of one of the float types on cuda:%ld", a[1], i,
                     device);
        ok = false;
      }
      if (!ok) break;
      ((void**)PyBytes_AS_STRING(made[0]))[i] = t->data_ptr();
      ((int64_t*)PyBytes_AS_STRING(made[1]))[i] = t->numel();
      ((int*)PyBytes_AS_STRING(made[2]))[i] = code;
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    ok = false;
  }
  Py_DECREF(seq);
  if (ok && a[3] != Py_None) {
    int same = PyTuple_Check(a[3]) && PyTuple_GET_SIZE(a[3]) == 3;
    for (int i = 1; same > 0 && i < 3; i++) same = PyObject_RichCompareBool(made[i], PyTuple_GET_ITEM(a[3], i), Py_EQ);
    if (same == 0) PyErr_Format(PyExc_ValueError, "%S must have the gradients' sizes and types", a[1]);
    ok = same > 0;
  }
  if (ok) return Py_BuildValue("(NNN)", made[0], made[1], made[2]);
  for (PyObject* m : made) Py_XDECREF(m);
  return nullptr;
}

#define METHOD(f, doc) {#f, (PyCFunction)(void (*)(void))guarded<f>, METH_FASTCALL, doc}
PyMethodDef methods[] = {
    METHOD(rows, "rows(tensor, what, like): pointer, row stride, rows, columns, type code, device"),
    METHOD(like, "like(tensor, what, like): pointer, row stride"),
    METHOD(raw, "raw(tensor, what, dtype): pointer, row pitch, rows, row bytes, device"),
    METHOD(pointer, "pointer(tensor, what, types, device, *shape): the checked data pointer"),
    METHOD(gain, "gain(tensor, columns, device): pointer, type code"),
    METHOD(slots, "slots(ids, teacher, types, rows, device): pointers, teacher's type code, topk"),
    METHOD(tensors, "tensors(sequence, what, device, like): pointers, counts, type codes"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pytensor", "Tensors' pointers, sizes and types for the Python binding.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pytensor(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", SIMAR_TORCH) < 0) Py_CLEAR(m);
  return m;
}
