/* pycall.c -- the Python object behind prepare_allreduce(), and the direct
 * calls behind the routing and loss helpers (further down).
 *
 * prepare_allreduce() marshals the arguments of one sim_allreduce call
 * once; calling the object it returns makes that C call again.  Through
 * ctypes every such call converts its eight argument objects on the host
 * (measured on MI355X hosts: about a sixth of a small all-reduce's
 * per-call cost); this type holds the arguments as C values and calls the
 * entry point directly.  It adds no logic of its own: every argument is
 * checked by the library, as for any other call.  The entry point's address
 * is taken from the library the package loaded, so a variant build chosen
 * at import time is the one called.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "simar.h"

typedef int (*allreduce_fn)(const void* const*, void* const*, int, size_t, int, int, int, void*);

typedef struct {
  PyObject_HEAD
  allreduce_fn fn;
  const void* in[SIM_MAX_RANKS];
  void* out[SIM_MAX_RANKS];
  int p;
  size_t n;
  int dtype, op, algo;
  void* stream;
} PreparedCall;

/* p device pointers (Python ints) from a sequence of exactly p items */
static int read_ptrs(PyObject* seq, int p, void** dst, const char* what) {
  PyObject* fast = PySequence_Fast(seq, what);
  if (!fast) return -1;
  if (PySequence_Fast_GET_SIZE(fast) != p) {
    PyErr_Format(PyExc_ValueError, "%s: expected %d pointers, got %zd", what, p, PySequence_Fast_GET_SIZE(fast));
    Py_DECREF(fast);
    return -1;
  }
  for (int i = 0; i < p; i++) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(PySequence_Fast_GET_ITEM(fast, i));
    if (v == (unsigned long long)-1 && PyErr_Occurred()) {
      Py_DECREF(fast);
      return -1;
    }
    dst[i] = (void*)(uintptr_t)v;
  }
  Py_DECREF(fast);
  return 0;
}

/* PreparedCall(entry_address, in_ptrs, out_ptrs, p, n, dtype, op, algo, stream) */
static int PreparedCall_init(PreparedCall* self, PyObject* args, PyObject* kw) {
  unsigned long long fn = 0, n = 0, stream = 0;
  PyObject *ins = NULL, *outs = NULL;
  int p = 0, dtype = 0, op = 0, algo = 0;
  if (kw && PyDict_GET_SIZE(kw) != 0) {
    PyErr_SetString(PyExc_TypeError, "PreparedCall takes positional arguments only");
    return -1;
  }
  if (!PyArg_ParseTuple(args, "KOOiKiiiK", &fn, &ins, &outs, &p, &n, &dtype, &op, &algo, &stream)) return -1;
  if (!fn) {
    PyErr_SetString(PyExc_ValueError, "null entry point");
    return -1;
  }
  /* the pointer arrays hold SIM_MAX_RANKS entries; other p values are the
     library's to refuse, with at most that many pointers read here */
  if (p < 0 || p > SIM_MAX_RANKS) {
    PyErr_Format(PyExc_ValueError, "p = %d: at most %d ranks", p, SIM_MAX_RANKS);
    return -1;
  }
  memset(self->in, 0, sizeof self->in);
  memset(self->out, 0, sizeof self->out);
  if (read_ptrs(ins, p, (void**)self->in, "in_ptrs") || read_ptrs(outs, p, self->out, "out_ptrs")) return -1;
  self->fn = (allreduce_fn)(uintptr_t)fn;
  self->p = p;
  self->n = (size_t)n;
  self->dtype = dtype;
  self->op = op;
  self->algo = algo;
  self->stream = (void*)(uintptr_t)stream;
  return 0;
}

/* call() -> the status sim_allreduce returned */
static PyObject* PreparedCall_call(PyObject* obj, PyObject* args, PyObject* kw) {
  PreparedCall* self = (PreparedCall*)obj;
  if (PyTuple_GET_SIZE(args) != 0 || (kw && PyDict_GET_SIZE(kw) != 0)) {
    PyErr_SetString(PyExc_TypeError, "a prepared call takes no arguments");
    return NULL;
  }
  if (!self->fn) {
    PyErr_SetString(PyExc_RuntimeError, "PreparedCall was not initialised");
    return NULL;
  }
  return PyLong_FromLong(self->fn(self->in, self->out, self->p, self->n, self->dtype, self->op, self->algo,
                                  self->stream));
}

static PyTypeObject PreparedCallType = {
    PyVarObject_HEAD_INIT(NULL, 0)
    .tp_name = "_pycall.PreparedCall",
    .tp_basicsize = sizeof(PreparedCall),
    .tp_flags = Py_TPFLAGS_DEFAULT,
    .tp_doc = "one sim_allreduce call with its arguments marshalled once; call it to run it",
    .tp_new = PyType_GenericNew,
    .tp_init = (initproc)PreparedCall_init,
    .tp_call = PreparedCall_call,
};

/* ---- the routing and loss entry points ------------------------------------
 * bind(name, address) sets an entry point once; the function of that name
 * then takes the C function's arguments (pointers as integers or None) and
 * returns its status. */
#define ENTRY(name) static __typeof__(sim_##name)* name##_fn
ENTRY(route);
ENTRY(route_grad);
ENTRY(distill_step);
ENTRY(distill_parts);
ENTRY(distill_join);
ENTRY(distill_grad);

static void* as_pointer(PyObject* o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }
static int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v != (int)v && !PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
  return (int)v;
}
#define P(i) as_pointer(a[i])
#define I(i) as_int(a[i])
#define L(i) ((int64_t)PyLong_AsLongLong(a[i]))
#define Z(i) ((size_t)PyLong_AsUnsignedLongLong(a[i]))
#define F(i) ((float)PyFloat_AsDouble(a[i]))

static int ready(const void* fn, Py_ssize_t n, Py_ssize_t want) {
  if (!fn) PyErr_SetString(PyExc_RuntimeError, "entry point not bound");
  else if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments wanted, %zd given", want, n);
  else return 1;
  return 0;
}
/* The arguments are converted into locals first, so that a failed conversion
 * is seen before the call. */
#define ARGS(...) __VA_ARGS__
#define WRAP(name, count, DECL, CALL)                                                       \
  static PyObject* py_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) {            \
    (void)self;                                                                             \
    if (!ready((const void*)name##_fn, n, count)) return NULL;                              \
    DECL if (PyErr_Occurred()) return NULL;                                                 \
    return PyLong_FromLong(name##_fn(CALL));                                                \
  }

WRAP(route, 15,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); void* keep = P(3); int64_t tokens = L(4); int experts = I(5);
     int topk = I(6); int norm = I(7); void* chosen = P(8); void* w = P(9); void* counts = P(10); void* sums = P(11);
     void* work = P(12); size_t bytes = Z(13); void* s = P(14);
     , ARGS(x, ld, dt, keep, tokens, experts, topk, norm, chosen, w, counts, sums, work, bytes, s))
WRAP(route_grad, 17,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); void* keep = P(3); int64_t tokens = L(4); int experts = I(5);
     int topk = I(6); int norm = I(7); void* chosen = P(8); void* dw = P(9); void* counts = P(10); void* sums = P(11);
     float coef = F(12); void* dx = P(13); int64_t dld = L(14); void* loss = P(15); void* s = P(16);
     , ARGS(x, ld, dt, keep, tokens, experts, topk, norm, chosen, dw, counts, sums, coef, dx, dld, loss, s))
WRAP(distill_step, 18,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); int64_t rows = L(3); int64_t vocab = L(4); void* ids = P(5);
     void* z = P(6); int zdt = I(7); int topk = I(8); float tau = F(9); void* rs = P(10); float coef = F(11);
     void* dx = P(12); int64_t dld = L(13); void* loss = P(14); void* work = P(15); size_t bytes = Z(16); void* s = P(17);
     , ARGS(x, ld, dt, rows, vocab, ids, z, zdt, topk, tau, rs, coef, dx, dld, loss, work, bytes, s))
WRAP(distill_parts, 16,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); int64_t rows = L(3); int64_t cols = L(4); int64_t first = L(5);
     int64_t vocab = L(6); void* ids = P(7); void* z = P(8); int zdt = I(9); int topk = I(10); float tau = F(11);
     void* parts = P(12); void* work = P(13); size_t bytes = Z(14); void* s = P(15);
     , ARGS(x, ld, dt, rows, cols, first, vocab, ids, z, zdt, topk, tau, parts, work, bytes, s))
WRAP(distill_join, 12,
     void* parts = P(0); int nparts = I(1); int64_t rows = L(2); int64_t vocab = L(3); void* ids = P(4); void* z = P(5);
     int zdt = I(6); int topk = I(7); float tau = F(8); void* loss = P(9); void* norm = P(10); void* s = P(11);
     , ARGS(parts, nparts, rows, vocab, ids, z, zdt, topk, tau, loss, norm, s))
WRAP(distill_grad, 18,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); int64_t rows = L(3); int64_t cols = L(4); int64_t first = L(5);
     int64_t vocab = L(6); void* ids = P(7); void* z = P(8); int zdt = I(9); int topk = I(10); float tau = F(11);
     void* norm = P(12); void* rs = P(13); float coef = F(14); void* dx = P(15); int64_t dld = L(16); void* s = P(17);
     , ARGS(x, ld, dt, rows, cols, first, vocab, ids, z, zdt, topk, tau, norm, rs, coef, dx, dld, s))

static PyObject* py_bind(PyObject* self, PyObject* args) {
  (void)self;
  const char* name;
  unsigned long long at;
  if (!PyArg_ParseTuple(args, "sK", &name, &at)) return NULL;
#define SET(entry) \
  if (!strcmp(name, #entry)) { entry##_fn = (__typeof__(sim_##entry)*)(uintptr_t)at; Py_RETURN_NONE; }
  SET(route) SET(route_grad) SET(distill_step) SET(distill_parts) SET(distill_join) SET(distill_grad)
  PyErr_Format(PyExc_ValueError, "no entry point %s", name);
  return NULL;
}

/* ---- tensors -------------------------------------------------------------------
 * What the helpers have to know of a tensor, through its own attributes and
 * methods.  types(...) sets the logit types once: code i + 1 is entry i. */
#define TYPES 3
static PyObject* logit_type[TYPES];
static PyObject *s_dtype, *s_shape, *s_device, *s_contiguous, *s_data_ptr, *s_stride;

static PyObject* py_types(PyObject* self, PyObject* args) {
  (void)self;
  PyObject* t[TYPES];
  if (!PyArg_ParseTuple(args, "OOO", &t[0], &t[1], &t[2])) return NULL;
  for (int i = 0; i < TYPES; i++) {
    Py_INCREF(t[i]);
    Py_XSETREF(logit_type[i], t[i]);
  }
  Py_RETURN_NONE;
}

/* the code of a tensor's type, 0 for any other type, -1 on an error */
static int code_of(PyObject* t) {
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) return -1;
  Py_DECREF(v);  /* types live as long as their module */
  for (int i = 0; i < TYPES; i++)
    if (logit_type[i] == v) return i + 1;
  return 0;
}

/* a method's result as an integer (-1: look for an error) */
static long number(PyObject* t, PyObject* method) {
  PyObject* v = PyObject_CallMethodNoArgs(t, method);
  if (!v) return -1;
  const long n = PyLong_AsLong(v);
  Py_DECREF(v);
  return n;
}

/* whether a 2-tuple of integers was read */
static int pair_of(PyObject* v, long long* a, long long* b) {
  const int two = PyTuple_Check(v) && PyTuple_GET_SIZE(v) == 2;
  if (two) {
    *a = PyLong_AsLongLong(PyTuple_GET_ITEM(v, 0));
    *b = PyLong_AsLongLong(PyTuple_GET_ITEM(v, 1));
  }
  return two && !PyErr_Occurred();
}

/* rows(tensor, what, like): (pointer, row stride, rows, columns, type code,
 * device index) of a 2-D device tensor with contiguous rows; like: None, or
 * the tuple of a tensor whose shape, type and device it must have. */
static PyObject* py_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "rows(tensor, what, like)");
    return NULL;
  }
  long long rows = 0, cols = 0, ld = 0, step = 0;
  PyObject* v = PyObject_GetAttr(a[0], s_shape);
  if (!v) return NULL;
  int ok = pair_of(v, &rows, &cols);
  Py_DECREF(v);
  const long dev = ok ? number(a[0], s_device) : -1;
  if (PyErr_Occurred()) return NULL;
  if (dev < 0) return PyErr_Format(PyExc_ValueError, "%S must be a 2-D device tensor", a[1]);
  if (!(v = PyObject_CallMethodNoArgs(a[0], s_stride))) return NULL;
  ok = pair_of(v, &ld, &step);
  Py_DECREF(v);
  if (PyErr_Occurred()) return NULL;
  if (!ok || (step != 1 && cols > 1)) return PyErr_Format(PyExc_ValueError, "%S's rows must be contiguous", a[1]);
  if (rows <= 1) ld = cols;
  const int code = code_of(a[0]);
  if (code < 0) return NULL;
  if (code == 0) {
    if ((v = PyObject_GetAttr(a[0], s_dtype))) {
      PyErr_Format(PyExc_ValueError, "unsupported dtype %S", v);
      Py_DECREF(v);
    }
    return NULL;
  }
  if (a[2] != Py_None) {
    if (!PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 6) {
      PyErr_SetString(PyExc_TypeError, "like: a tuple that rows() returned");
      return NULL;
    }
    ok = PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], 2)) == rows && PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], 3)) == cols &&
         PyLong_AsLong(PyTuple_GET_ITEM(a[2], 4)) == code && PyLong_AsLong(PyTuple_GET_ITEM(a[2], 5)) == dev;
    if (PyErr_Occurred()) return NULL;
    if (!ok) return PyErr_Format(PyExc_ValueError, "%S must have the logits' shape, dtype and device", a[1]);
  }
  if (!(v = PyObject_CallMethodNoArgs(a[0], s_data_ptr))) return NULL;
  return Py_BuildValue("(NLLLil)", v, ld, rows, cols, code, dev);
}

/* whether a tensor is contiguous, on that device, of that shape and one of
 * those types; -1 on an error */
static int fits(PyObject* t, PyObject* const* types, Py_ssize_t ntypes, long dev, const long long* shape,
                Py_ssize_t dims) {
  int ok = 0;
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) return -1;
  for (Py_ssize_t i = 0; i < ntypes; i++) ok = ok || types[i] == v;
  Py_DECREF(v);
  if (!ok) return 0;
  if (!(v = PyObject_GetAttr(t, s_shape))) return -1;
  ok = PyTuple_Check(v) && PyTuple_GET_SIZE(v) == dims;
  for (Py_ssize_t i = 0; ok && i < dims; i++) ok = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i)) == shape[i];
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (!ok) return 0;
  ok = number(t, s_device) == dev;
  if (PyErr_Occurred()) return -1;
  if (!ok) return 0;
  if (!(v = PyObject_CallMethodNoArgs(t, s_contiguous))) return -1;
  ok = PyObject_IsTrue(v);
  Py_DECREF(v);
  return ok;
}

/* the pointer of a tensor that fits, or an error that says what it must be */
static PyObject* pointer_of(PyObject* t, PyObject* what, PyObject* const* types, Py_ssize_t ntypes, long dev,
                            const long long* shape, Py_ssize_t dims) {
  const int ok = fits(t, types, ntypes, dev, shape, dims);
  if (ok < 0) return NULL;
  if (ok) return PyObject_CallMethodNoArgs(t, s_data_ptr);
  PyObject *of = PyTuple_New(ntypes), *sizes = PyTuple_New(dims);
  for (Py_ssize_t i = 0; of && i < ntypes; i++) {
    Py_INCREF(types[i]);
    PyTuple_SET_ITEM(of, i, types[i]);
  }
  for (Py_ssize_t i = 0; sizes && i < dims; i++) {
    PyObject* d = PyLong_FromLongLong(shape[i]);
    if (!d) Py_CLEAR(sizes);
    else PyTuple_SET_ITEM(sizes, i, d);
  }
  if (of && sizes)
    PyErr_Format(PyExc_ValueError, "%S must be a contiguous tensor %R of one of %R on cuda:%ld", what, sizes, of, dev);
  Py_XDECREF(of);
  Py_XDECREF(sizes);
  return NULL;
}

/* pointer(tensor, what, types, device index, *shape): the data pointer of a
 * contiguous tensor of that shape and device and one of those types (None
 * for None). */
#define DIMS 4
static PyObject* py_pointer(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n < 4 || n > 4 + DIMS || !PyTuple_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "pointer(tensor, what, types, device, *shape)");
    return NULL;
  }
  if (a[0] == Py_None) Py_RETURN_NONE;
  long long shape[DIMS];
  for (Py_ssize_t i = 4; i < n; i++) shape[i - 4] = PyLong_AsLongLong(a[i]);
  const long dev = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return NULL;
  return pointer_of(a[0], a[1], PySequence_Fast_ITEMS(a[2]), PyTuple_GET_SIZE(a[2]), dev, shape, n - 4);
}

/* slots(ids, teacher, ids' types, rows, device index): (ids pointer, teacher
 * pointer, the teacher's type code, topk) of contiguous [rows, topk] tensors. */
static PyObject *s_ids, *s_teacher;
static PyObject* py_slots(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 5 || !PyTuple_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "slots(ids, teacher, types, rows, device)");
    return NULL;
  }
  long long had = 0, shape[2] = {PyLong_AsLongLong(a[3]), 0};
  const long dev = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return NULL;
  PyObject* v = PyObject_GetAttr(a[0], s_shape);
  if (!v) return NULL;
  const int ok = pair_of(v, &had, &shape[1]);
  Py_DECREF(v);
  if (PyErr_Occurred()) return NULL;
  if (!ok) return PyErr_Format(PyExc_ValueError, "ids must be [rows, topk]");
  PyObject* ids = pointer_of(a[0], s_ids, PySequence_Fast_ITEMS(a[2]), PyTuple_GET_SIZE(a[2]), dev, shape, 2);
  if (!ids) return NULL;
  PyObject* teacher = pointer_of(a[1], s_teacher, logit_type, TYPES, dev, shape, 2);
  const int code = teacher ? code_of(a[1]) : -1;
  if (code < 0) {
    Py_DECREF(ids);
    Py_XDECREF(teacher);
    return NULL;
  }
  return Py_BuildValue("(NNiL)", ids, teacher, code, shape[1]);
}

#define METHOD(name, f, doc) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, doc}
static PyMethodDef pycall_methods[] = {
    {"bind", py_bind, METH_VARARGS, "bind(name, address): set an entry point"},
    {"types", py_types, METH_VARARGS, "types(fp32, fp16, bf16): set the logit types"},
    METHOD("rows", py_rows, "rows(tensor, what, like): pointer, row stride, rows, columns, type code, device"),
    METHOD("pointer", py_pointer, "pointer(tensor, what, types, device, *shape): the checked data pointer"),
    METHOD("slots", py_slots, "slots(ids, teacher, types, rows, device): pointers, teacher's type code, topk"),
    METHOD("route", py_route, "sim_route"),
    METHOD("route_grad", py_route_grad, "sim_route_grad"),
    METHOD("distill_step", py_distill_step, "sim_distill_step"),
    METHOD("distill_parts", py_distill_parts, "sim_distill_parts"),
    METHOD("distill_join", py_distill_join, "sim_distill_join"),
    METHOD("distill_grad", py_distill_grad, "sim_distill_grad"),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef pycall_module = {
    PyModuleDef_HEAD_INIT, "_pycall", "Prepared C-ABI calls for the Python binding.", -1, pycall_methods,
};

PyMODINIT_FUNC PyInit__pycall(void) {
  if (PyType_Ready(&PreparedCallType) < 0) return NULL;
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_device = PyUnicode_InternFromString("get_device");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_ids = PyUnicode_InternFromString("ids");
  s_teacher = PyUnicode_InternFromString("teacher");
  if (!s_dtype || !s_shape || !s_device || !s_contiguous || !s_data_ptr || !s_stride || !s_ids || !s_teacher) return NULL;
  PyObject* m = PyModule_Create(&pycall_module);
  if (!m) return NULL;
  Py_INCREF(&PreparedCallType);
  if (PyModule_AddObject(m, "PreparedCall", (PyObject*)&PreparedCallType) < 0) {
    Py_DECREF(&PreparedCallType);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
