/* tokens_py.c -- CPython entry points of the token operators.
 *
 * The package's other functions go through ctypes, which converts the twenty arguments of a
 * call in about 2 us; at decode sizes that is as long as the launch itself.  These wrappers take
 * the same arguments as plain integers (addresses, or None), call the C entry point with the
 * interpreter's lock released, and return its status.  They are private: tokens.py checks the
 * tensors and calls them. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/moe.h"

static int bad_count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return 1;
}
static void *ptr(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }
static long num(PyObject *o) { return PyLong_AsLong(o); }
/* an int argument: out of range raises OverflowError */
static int num32(PyObject *o) {
  long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v > 2147483647L || v < -2147483647L - 1)
    PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
  return (int)v;
}

#define P(i) ptr(a[i])
#define L(i) num(a[i])
#define I(i) num32(a[i])
#define RUN(call)                        \
  do {                                   \
    int returned;                        \
    if (PyErr_Occurred()) return NULL;   \
    Py_BEGIN_ALLOW_THREADS               \
    returned = (call);                   \
    Py_END_ALLOW_THREADS                 \
    return PyLong_FromLong(returned);    \
  } while (0)

static PyObject *rmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 17)) return NULL;
  int T = I(0), H = I(1), dt = I(4), norm = I(9), group = I(10);
  void *x = P(2), *add = P(5), *w = P(7), *resid = P(11), *q = P(13), *scale = P(15), *st = P(16);
  long ldx = L(3), lda = L(6), ldr = L(12), ldq = L(14);
  float eps = (float)PyFloat_AsDouble(a[8]);
  RUN(moe_rmsnorm_e4m3(T, H, x, ldx, (moe_dtype)dt, add, lda, w, eps, norm, group, resid, ldr,
                       (uint8_t *)q, ldq, (float *)scale, st));
}

static PyObject *sort(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 8)) return NULL;
  int T = I(0), k = I(1), E = I(2);
  void *ids = P(3), *off = P(4), *perm = P(5), *pos = P(6), *st = P(7);
  RUN(moe_sort_tokens(T, k, E, (const int32_t *)ids, (int32_t *)off, (int32_t *)perm,
                      (int32_t *)pos, st));
}

static PyObject *dispatch(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 15)) return NULL;
  int T = I(0), k = I(1), E = I(2), H = I(3), dt = I(4), S = I(10);
  void *x = P(5), *pos = P(7), *off = P(8), *xs = P(9), *sc = P(11), *scs = P(13), *st = P(14);
  long ldx = L(6), ldsc = L(12);
  RUN(moe_dispatch_rows(T, k, E, H, (moe_dtype)dt, x, ldx, (const int32_t *)pos,
                        (const int32_t *)off, xs, S, (const float *)sc, ldsc, (float *)scs, st));
}

static PyObject *combine(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 13)) return NULL;
  int T = I(0), k = I(1), H = I(2), yt = I(4), ot = I(11);
  void *y = P(3), *pos = P(5), *w = P(6), *add = P(7), *out = P(9), *st = P(12);
  long lda = L(8), ldo = L(10);
  RUN(moe_combine_rows(T, k, H, y, (moe_dtype)yt, (const int32_t *)pos, (const float *)w, add, lda,
                       out, ldo, (moe_dtype)ot, st));
}

static PyObject *combine_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 14)) return NULL;
  int T = I(0), k = I(1), E = I(2), H = I(3), dt = I(4);
  void *dout = P(5), *y = P(7), *pos = P(8), *off = P(9), *w = P(10), *dy = P(11), *dw = P(12),
       *st = P(13);
  long ldd = L(6);
  RUN(moe_combine_rows_grad(T, k, E, H, (moe_dtype)dt, dout, ldd, y, (const int32_t *)pos,
                            (const int32_t *)off, (const float *)w, dy, (float *)dw, st));
}

static PyObject *dispatch_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 10)) return NULL;
  int T = I(0), k = I(1), H = I(2), dt = I(3), xt = I(8);
  void *dxs = P(4), *pos = P(5), *dx = P(6), *st = P(9);
  long ldx = L(7);
  RUN(moe_dispatch_rows_grad(T, k, H, (moe_dtype)dt, dxs, (const int32_t *)pos, dx, ldx,
                             (moe_dtype)xt, st));
}

static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (bad_count(n, 20)) return NULL;
  int R = I(0), N = I(1), K = I(2), E = I(3), dt = I(6), act = I(11), ot = I(17);
  void *x = P(4), *xs = P(7), *w = P(8), *ws = P(9), *bias = P(10), *res = P(12), *off = P(14),
       *out = P(15), *status = P(18), *st = P(19);
  long ldx = L(5), ldr = L(13), ldo = L(16);
  RUN(moe_linear(R, N, K, E, x, ldx, (moe_dtype)dt, (const float *)xs, w, (const float *)ws,
                 (const float *)bias, (moe_act)act, res, ldr, (const int32_t *)off, out, ldo,
                 (moe_dtype)ot, (int32_t *)status, st));
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(rmsnorm),      METHOD(sort),          METHOD(dispatch),
                                METHOD(combine),      METHOD(combine_grad),  METHOD(dispatch_grad),
                                METHOD(linear),       {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens_native", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tokens_native(void) { return PyModule_Create(&module); }
