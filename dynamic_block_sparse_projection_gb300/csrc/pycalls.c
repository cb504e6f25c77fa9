// pycalls.c — Python entries to the calls of dsv.h that take structures.
//
// ctypes passes a structure by value through a copy object and libffi, about
// 1 us each on a Grace core: more than a small launch takes.  These functions
// take the same arguments in the same order (structures as objects that export
// their bytes, such as binding.py's ctypes structures; addresses as ints or
// None), so binding.py puts them in the ctypes functions' place.  Measured, host
// time of a call: see binding.py.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "dsv.h"

static int bytes_of(PyObject* o, void* dst, size_t n) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return 0;
  const int fits = (size_t)b.len == n;
  if (fits) memcpy(dst, b.buf, n);
  PyBuffer_Release(&b);
  if (!fits) PyErr_Format(PyExc_TypeError, "expected a structure of %zu bytes", n);
  return fits;
}
static int address_of(PyObject* o, void** p) {
  *p = NULL;
  if (o == Py_None) return 1;
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
  *p = (void*)(uintptr_t)v;
  return 1;
}
static int i64_of(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}
static int i32_of(PyObject* o, int32_t* v) {
  int64_t w;
  if (!i64_of(o, &w)) return 0;
  if (w < INT32_MIN || w > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "the value does not fit in 32 bits");
    return 0;
  }
  *v = (int32_t)w;
  return 1;
}
static int size_of(PyObject* o, size_t* v) {
  const unsigned long long w = PyLong_AsUnsignedLongLong(o);
  if (w == (unsigned long long)-1 && PyErr_Occurred()) return 0;
  *v = (size_t)w;
  return 1;
}
static int f32_of(PyObject* o, float* v) {
  const double w = PyFloat_AsDouble(o);
  *v = (float)w;
  return !(w == -1.0 && PyErr_Occurred());
}
static int count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return 0;
}

static PyObject* rope_axes_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_view x, y;
  dsv_rope r;
  void *pos, *weight, *stream;
  int64_t pos_b;
  float eps;
  if (!count_is(n, 8) || !bytes_of(a[0], &x, sizeof x) || !address_of(a[1], &pos) || !i64_of(a[2], &pos_b) ||
      !bytes_of(a[3], &r, sizeof r) || !address_of(a[4], &weight) || !f32_of(a[5], &eps) ||
      !bytes_of(a[6], &y, sizeof y) || !address_of(a[7], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_rope_axes_fwd(x, pos, pos_b, r, weight, eps, y, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* rope_axes_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_view dy, x, dx;
  dsv_rope r;
  void *pos, *weight, *dweight, *ws, *stream;
  int64_t pos_b;
  size_t bytes;
  float eps;
  if (!count_is(n, 12) || !bytes_of(a[0], &dy, sizeof dy) || !bytes_of(a[1], &x, sizeof x) ||
      !address_of(a[2], &pos) || !i64_of(a[3], &pos_b) || !bytes_of(a[4], &r, sizeof r) ||
      !address_of(a[5], &weight) || !f32_of(a[6], &eps) || !bytes_of(a[7], &dx, sizeof dx) ||
      !address_of(a[8], &dweight) || !address_of(a[9], &ws) || !size_of(a[10], &bytes) || !address_of(a[11], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_rope_axes_bwd(dy, x, pos, pos_b, r, weight, eps, dx, dweight, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* packed_attn_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_view Q, K, V, O;
  dsv_packed p;
  void *q_ptr, *k_ptr, *lse, *ws, *stream;
  int32_t causal;
  size_t bytes;
  float scale;
  if (!count_is(n, 13) || !bytes_of(a[0], &Q, sizeof Q) || !bytes_of(a[1], &K, sizeof K) ||
      !bytes_of(a[2], &V, sizeof V) || !bytes_of(a[3], &p, sizeof p) || !address_of(a[4], &q_ptr) ||
      !address_of(a[5], &k_ptr) || !i32_of(a[6], &causal) || !f32_of(a[7], &scale) || !bytes_of(a[8], &O, sizeof O) ||
      !address_of(a[9], &lse) || !address_of(a[10], &ws) || !size_of(a[11], &bytes) || !address_of(a[12], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_packed_attn_fwd(Q, K, V, p, q_ptr, k_ptr, causal, scale, O, lse, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* packed_attn_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_view Q, K, V, O, dO, dQ, dK, dV;
  dsv_packed p;
  void *lse, *q_ptr, *k_ptr, *ws, *stream;
  int32_t causal;
  size_t bytes;
  float scale;
  if (!count_is(n, 17) || !bytes_of(a[0], &Q, sizeof Q) || !bytes_of(a[1], &K, sizeof K) ||
      !bytes_of(a[2], &V, sizeof V) || !bytes_of(a[3], &O, sizeof O) || !bytes_of(a[4], &dO, sizeof dO) ||
      !address_of(a[5], &lse) || !bytes_of(a[6], &p, sizeof p) || !address_of(a[7], &q_ptr) ||
      !address_of(a[8], &k_ptr) || !i32_of(a[9], &causal) || !f32_of(a[10], &scale) ||
      !bytes_of(a[11], &dQ, sizeof dQ) || !bytes_of(a[12], &dK, sizeof dK) || !bytes_of(a[13], &dV, sizeof dV) ||
      !address_of(a[14], &ws) || !size_of(a[15], &bytes) || !address_of(a[16], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_packed_attn_bwd(Q, K, V, O, dO, lse, p, q_ptr, k_ptr, causal, scale, dQ, dK, dV, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

#define ENTRY(name) {"dsv_" #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, "dsv_" #name " of dsv.h"}
static PyMethodDef methods[] = {ENTRY(rope_axes_fwd), ENTRY(rope_axes_bwd), ENTRY(packed_attn_fwd),
                                ENTRY(packed_attn_bwd), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "dsv_calls", "calls of dsv.h that take structures", -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_dsv_calls(void) { return PyModule_Create(&module); }
