// The 4-bit and expert entry points of include/imc.h as functions of a Python
// module: a call of a few tokens is bound by its way through Python, and ctypes
// takes 1.2 us to convert fourteen arguments, this 0.2 (whole calls, us: quantising
// 7.9 / 6.2, the 4-bit product 8.6 / 6.8, routing 9.6 / 7.6).
// Arguments are integers (addresses too; None is a null pointer) in the order of
// the C functions, which check them; the status is returned.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "imc.h"

typedef union {
  void* p;
  int64_t l;
  int i;
  double d;
} Arg;

// Converts the arguments as `kinds` says: p address, l 64-bit integer, i int, d double.
static int take(const char* name, const char* kinds, PyObject* const* a, Py_ssize_t n, Arg* v) {
  if (n != (Py_ssize_t)strlen(kinds)) {
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments (%d given)", name, (int)strlen(kinds),
                 (int)n);
    return -1;
  }
  for (Py_ssize_t j = 0; j < n; ++j) {
    switch (kinds[j]) {
      case 'p':
        v[j].p = a[j] == Py_None ? NULL : (void*)(uintptr_t)PyLong_AsUnsignedLongLong(a[j]);
        break;
      case 'l':
        v[j].l = PyLong_AsLongLong(a[j]);
        break;
      case 'i': {
        const long i = PyLong_AsLong(a[j]);
        v[j].i = (int)i;
        if (i != v[j].i && !PyErr_Occurred())
          PyErr_Format(PyExc_OverflowError, "%s: argument %d is no int", name, (int)j);
        break;
      }
      default:
        v[j].d = PyFloat_AsDouble(a[j]);
    }
    if (PyErr_Occurred()) return -1;
  }
  return 0;
}

#define ENTRY(name, kinds, ...)                                                        \
  static PyObject* call_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) {     \
    Arg v[sizeof(kinds)];                                                              \
    int rc;                                                                            \
    (void)self;                                                                        \
    if (take(#name, kinds, a, n, v)) return NULL;                                      \
    Py_BEGIN_ALLOW_THREADS rc = name(__VA_ARGS__);                                     \
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);                                   \
  }
#define P(j) v[j].p
#define L(j) v[j].l
#define I(j) v[j].i

ENTRY(mxfp4_quantize, "pilllllipp", P(0), I(1), L(2), L(3), L(4), L(5), L(6), I(7), P(8), P(9))
ENTRY(mxfp4_dequantize, "plllipp", P(0), L(1), L(2), L(3), I(4), P(5), P(6))
ENTRY(mxfp4_linear, "pilpppillliplp", P(0), I(1), L(2), P(3), P(4), P(5), I(6), L(7), L(8), L(9), I(10),
      P(11), (size_t)L(12), P(13))
ENTRY(mxfp4_linear_backward, "pppilllppplp", P(0), P(1), P(2), I(3), L(4), L(5), L(6), P(7), P(8),
      P(9), (size_t)L(10), P(11))
ENTRY(moe_route, "pilllplillidppp", P(0), I(1), L(2), L(3), L(4), P(5), L(6), I(7), L(8), L(9), I(10),
      v[11].d, P(12), P(13), P(14))
ENTRY(moe_route_backward, "ppilllpliidpp", P(0), P(1), I(2), L(3), L(4), L(5), P(6), L(7), I(8), I(9),
      v[10].d, P(11), P(12))
ENTRY(moe_layout, "plllpp", P(0), L(1), L(2), L(3), P(4), P(5))
ENTRY(mxfp4_experts_linear, "pillppppillllliplp", P(0), I(1), L(2), L(3), P(4), P(5), P(6), P(7), I(8),
      L(9), L(10), L(11), L(12), L(13), I(14), P(15), (size_t)L(16), P(17))
ENTRY(mxfp4_experts_weight_grad, "ppilpplllllplp", P(0), P(1), I(2), L(3), P(4), P(5), L(6), L(7),
      L(8), L(9), L(10), P(11), (size_t)L(12), P(13))
ENTRY(moe_combine, "piplllpp", P(0), I(1), P(2), L(3), L(4), L(5), P(6), P(7))
ENTRY(moe_combine_f32, "pplllpip", P(0), P(1), L(2), L(3), L(4), P(5), I(6), P(7))
ENTRY(moe_combine_backward, "ppiplllppp", P(0), P(1), I(2), P(3), L(4), L(5), L(6), P(7), P(8), P(9))

#define ROW(name) {#name, (PyCFunction)(void (*)(void))call_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {ROW(mxfp4_quantize),       ROW(mxfp4_dequantize),
                                ROW(mxfp4_linear),         ROW(mxfp4_linear_backward),
                                ROW(moe_route),            ROW(moe_route_backward),
                                ROW(moe_layout),           ROW(mxfp4_experts_linear),
                                ROW(mxfp4_experts_weight_grad), ROW(moe_combine),
                                ROW(moe_combine_f32),
                                ROW(moe_combine_backward), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
