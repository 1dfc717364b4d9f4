/* pycall.c -- the Python object behind prepare_allreduce(), and the direct
 * calls behind the helpers that work on one rank's data (further down).
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

/* ---- the entry points that work on one rank's data ------------------------------------
 * bind(name, address) sets an entry point once; the function of that name
 * then takes the C function's arguments (pointers as integers, bytes objects or
 * None) and returns its status. */
#define ENTRY(name) static __typeof__(sim_##name)* name##_fn
ENTRY(route);
ENTRY(route_grad);
ENTRY(distill_step);
ENTRY(distill_parts);
ENTRY(distill_join);
ENTRY(distill_grad);
ENTRY(norm);
ENTRY(norm_grad);
ENTRY(dispatch);
ENTRY(combine);
ENTRY(combine_grad);
ENTRY(clip_work);
ENTRY(clip_norm);
ENTRY(clip);

/* (an array of the host: the bytes object that tensors() made) */
static void* as_pointer(PyObject* o) {
  if (o == Py_None) return NULL;
  return PyBytes_Check(o) ? (void*)PyBytes_AS_STRING(o) : PyLong_AsVoidPtr(o);
}
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

WRAP(norm, 17,
     void* x = P(0); int64_t ld = L(1); int dt = I(2); void* res = P(3); int64_t rld = L(4); int64_t rows = L(5);
     int64_t cols = L(6); void* g = P(7); int gdt = I(8); float eps = F(9); void* sum = P(10); int64_t sld = L(11);
     void* out = P(12); int64_t old = L(13); void* sc = P(14); int group = I(15); void* s = P(16);
     , ARGS(x, ld, dt, res, rld, rows, cols, g, gdt, eps, sum, sld, out, old, sc, group, s))
WRAP(norm_grad, 18,
     void* h = P(0); int64_t ld = L(1); int dt = I(2); int64_t rows = L(3); int64_t cols = L(4); void* g = P(5);
     int gdt = I(6); float eps = F(7); void* dy = P(8); int64_t dyld = L(9); void* ds = P(10); int64_t dsld = L(11);
     void* dx = P(12); int64_t dxld = L(13); void* dg = P(14); void* work = P(15); size_t bytes = Z(16); void* s = P(17);
     , ARGS(h, ld, dt, rows, cols, g, gdt, eps, dy, dyld, ds, dsld, dx, dxld, dg, work, bytes, s))
WRAP(dispatch, 17,
     void* x = P(0); int64_t ld = L(1); int64_t rb = L(2); void* sc = P(3); int64_t groups = L(4); void* chosen = P(5);
     int64_t tokens = L(6); int topk = I(7); int experts = I(8); void* rows = P(9); int64_t rld = L(10);
     void* rsc = P(11); void* place = P(12); void* off = P(13); void* work = P(14); size_t bytes = Z(15); void* s = P(16);
     , ARGS(x, ld, rb, sc, groups, chosen, tokens, topk, experts, rows, rld, rsc, place, off, work, bytes, s))
WRAP(combine, 12,
     void* rows = P(0); int64_t ld = L(1); int dt = I(2); int64_t nrows = L(3); int64_t cols = L(4); void* place = P(5);
     void* w = P(6); int64_t tokens = L(7); int topk = I(8); void* out = P(9); int64_t old = L(10); void* s = P(11);
     , ARGS(rows, ld, dt, nrows, cols, place, w, tokens, topk, out, old, s))
WRAP(combine_grad, 15,
     void* dy = P(0); int64_t dyld = L(1); int dt = I(2); void* rows = P(3); int64_t ld = L(4); int64_t nrows = L(5);
     int64_t cols = L(6); void* place = P(7); void* w = P(8); int64_t tokens = L(9); int topk = I(10);
     void* dr = P(11); int64_t drld = L(12); void* dw = P(13); void* s = P(14);
     , ARGS(dy, dyld, dt, rows, ld, nrows, cols, place, w, tokens, topk, dr, drld, dw, s))
WRAP(clip_norm, 8,
     void* g = P(0); void* c = P(1); void* d = P(2); int n_t = I(3); void* norm = P(4); void* work = P(5);
     size_t bytes = Z(6); void* s = P(7);
     , ARGS(g, c, d, n_t, norm, work, bytes, s))
WRAP(clip, 12,
     void* g = P(0); void* o = P(1); void* c = P(2); void* d = P(3); int n_t = I(4); void* parts = P(5);
     int nparts = I(6); float most = F(7); void* norm = P(8); void* work = P(9); size_t bytes = Z(10); void* s = P(11);
     , ARGS(g, o, c, d, n_t, parts, nparts, most, norm, work, bytes, s))

static PyObject* py_bind(PyObject* self, PyObject* args) {
  (void)self;
  const char* name;
  unsigned long long at;
  if (!PyArg_ParseTuple(args, "sK", &name, &at)) return NULL;
#define SET(entry) \
  if (!strcmp(name, #entry)) { entry##_fn = (__typeof__(sim_##entry)*)(uintptr_t)at; Py_RETURN_NONE; }
  SET(route) SET(route_grad) SET(distill_step) SET(distill_parts) SET(distill_join) SET(distill_grad)
  SET(norm) SET(norm_grad) SET(dispatch) SET(combine) SET(combine_grad) SET(clip_work) SET(clip_norm) SET(clip)
  PyErr_Format(PyExc_ValueError, "no entry point %s", name);
  return NULL;
}

/* clip_work(counts, type codes, number): sim_clip_work's bytes, or its status */
static PyObject* py_clip_work(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!ready((const void*)clip_work_fn, n, 3)) return NULL;
  void *counts = P(0), *types = P(1);
  const int tensors = I(2);
  if (PyErr_Occurred()) return NULL;
  size_t bytes = 0;
  const int rc = clip_work_fn(counts, types, tensors, &bytes);
  return rc ? PyLong_FromLong(rc) : PyLong_FromSize_t(bytes);
}

#define METHOD(name, f, doc) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, doc}
static PyMethodDef pycall_methods[] = {
    {"bind", py_bind, METH_VARARGS, "bind(name, address): set an entry point"},
    METHOD("route", py_route, "sim_route"),
    METHOD("route_grad", py_route_grad, "sim_route_grad"),
    METHOD("distill_step", py_distill_step, "sim_distill_step"),
    METHOD("distill_parts", py_distill_parts, "sim_distill_parts"),
    METHOD("distill_join", py_distill_join, "sim_distill_join"),
    METHOD("distill_grad", py_distill_grad, "sim_distill_grad"),
    METHOD("clip_work", py_clip_work, "clip_work(counts, types, number): sim_clip_work's bytes, or its status"),
    METHOD("norm", py_norm, "sim_norm"),
    METHOD("norm_grad", py_norm_grad, "sim_norm_grad"),
    METHOD("dispatch", py_dispatch, "sim_dispatch"),
    METHOD("combine", py_combine, "sim_combine"),
    METHOD("combine_grad", py_combine_grad, "sim_combine_grad"),
    METHOD("clip_norm", py_clip_norm, "sim_clip_norm"),
    METHOD("clip", py_clip, "sim_clip"),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef pycall_module = {
    PyModuleDef_HEAD_INIT, "_pycall", "Prepared C-ABI calls for the Python binding.", -1, pycall_methods,
};

PyMODINIT_FUNC PyInit__pycall(void) {
  if (PyType_Ready(&PreparedCallType) < 0) return NULL;
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
