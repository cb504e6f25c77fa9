// pycalls.c — Python entries to the calls of dsv.h that take structures, and the
// views they take.
//
// Host time is what the smallest calls cost.  ctypes passes a structure by value
// through a copy object and libffi, about 1 us each on a Grace core, and a view
// built in Python takes another 1 us with its tensor's checks; a small kernel's
// launch takes 3.  The functions have the same arguments in the same order as
// dsv.h's (views as View objects, other structures as objects that export their
// bytes, addresses as ints or None), so binding.py puts them in the ctypes
// functions' place.  Measured, host time of a call: packed forward of a few
// short clips 26 -> 22 us, its gradient 47 -> 39, a rotation 15.5 -> 14.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <string.h>
#include <structmember.h>

#include "dsv.h"

// ---------------------------------------------------------------------------
// dsv_view
// ---------------------------------------------------------------------------
typedef struct {
  PyObject_HEAD
  dsv_view v;
} View;
static PyTypeObject ViewType;

static int address_of(PyObject* o, void** p) {
  *p = NULL;
  if (o == Py_None) return 1;
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
  *p = (void*)(uintptr_t)v;
  return 1;
}
static PyObject* view_make(void* ptr, int64_t b, int64_t h, int64_t t) {
  View* o = PyObject_New(View, &ViewType);
  if (o == NULL) return NULL;
  o->v.ptr = ptr;
  o->v.batch_stride = b;
  o->v.head_stride = h;
  o->v.token_stride = t;
  return (PyObject*)o;
}
static PyObject* view_new(PyTypeObject* type, PyObject* args, PyObject* kw) {
  PyObject* address;
  long long b, h, t;
  void* ptr;
  if (kw != NULL && PyDict_GET_SIZE(kw) != 0) {
    PyErr_SetString(PyExc_TypeError, "View(ptr, batch_stride, head_stride, token_stride)");
    return NULL;
  }
  if (!PyArg_ParseTuple(args, "OLLL", &address, &b, &h, &t) || !address_of(address, &ptr)) return NULL;
  return view_make(ptr, b, h, t);
}
static void view_free(PyObject* o) { PyObject_Free(o); }
static PyObject* view_ptr(PyObject* o, void* unused) {
  void* p = ((View*)o)->v.ptr;
  if (p == NULL) Py_RETURN_NONE;
  return PyLong_FromUnsignedLongLong((unsigned long long)(uintptr_t)p);
}
static PyMemberDef view_members[] = {
    {"batch_stride", T_LONGLONG, offsetof(View, v.batch_stride), READONLY, NULL},
    {"head_stride", T_LONGLONG, offsetof(View, v.head_stride), READONLY, NULL},
    {"token_stride", T_LONGLONG, offsetof(View, v.token_stride), READONLY, NULL},
    {NULL, 0, 0, 0, NULL}};
static PyGetSetDef view_getset[] = {{"ptr", view_ptr, NULL, NULL, NULL}, {NULL, NULL, NULL, NULL, NULL}};
static PyTypeObject ViewType = {
    PyVarObject_HEAD_INIT(NULL, 0).tp_name = "dsv_calls.View",
    .tp_basicsize = sizeof(View),
    .tp_flags = Py_TPFLAGS_DEFAULT,
    .tp_doc = "dsv_view: the address and element strides of a [batch, heads, tokens, d] tensor",
    .tp_new = view_new,
    .tp_dealloc = view_free,
    .tp_members = view_members,
    .tp_getset = view_getset,
};

static PyObject *s_dtype, *s_get_device, *s_stride, *s_data_ptr;

// The view of a [.., heads, tokens, d] tensor, NULL without an error set where
// its type, device or last stride is another than asked for.
static PyObject* view_of_tensor(PyObject* t, PyObject* dtype, long index) {
  PyObject* got = PyObject_GetAttr(t, s_dtype);
  if (got == NULL) return NULL;
  const int same = got == dtype;
  Py_DECREF(got);
  if (!same) return NULL;
  if ((got = PyObject_CallMethodNoArgs(t, s_get_device)) == NULL) return NULL;
  const long at = PyLong_AsLong(got);
  Py_DECREF(got);
  if (at != index || PyErr_Occurred()) return NULL;
  PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
  if (st == NULL) return NULL;
  PyObject* made = NULL;
  const Py_ssize_t n = PyTuple_Check(st) ? PyTuple_GET_SIZE(st) : 0;
  if (n == 3 || n == 4) {
    long long v[4] = {0, 0, 0, 0};
    for (Py_ssize_t i = 0; i < n; ++i) v[i + 4 - n] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    if (!PyErr_Occurred() && v[3] == 1 && (got = PyObject_CallMethodNoArgs(t, s_data_ptr)) != NULL) {
      void* ptr;
      if (address_of(got, &ptr)) made = view_make(ptr, v[0], v[1], v[2]);
      Py_DECREF(got);
    }
  }
  Py_DECREF(st);
  return made;
}
// row_views(dtype, index, *tensors): a tuple of their views (None: the null
// view), or None where one of them is not `dtype` on device `index` with a
// contiguous last dimension.
static PyObject* row_views(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n < 2) {
    PyErr_SetString(PyExc_TypeError, "row_views(dtype, index, *tensors)");
    return NULL;
  }
  const long index = PyLong_AsLong(a[1]);
  if (index == -1 && PyErr_Occurred()) return NULL;
  PyObject* all = PyTuple_New(n - 2);
  for (Py_ssize_t i = 2; all != NULL && i < n; ++i) {
    PyObject* v = a[i] == Py_None ? view_make(NULL, 0, 0, 0) : view_of_tensor(a[i], a[0], index);
    if (v == NULL) {
      Py_DECREF(all);
      if (PyErr_Occurred()) return NULL;
      Py_RETURN_NONE;
    }
    PyTuple_SET_ITEM(all, i - 2, v);
  }
  return all;
}

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
static int view_of(PyObject* o, dsv_view* v) {
  if (Py_TYPE(o) != &ViewType) {
    PyErr_Format(PyExc_TypeError, "expected a View, got %.80s", Py_TYPE(o)->tp_name);
    return 0;
  }
  *v = ((View*)o)->v;
  return 1;
}
static int bytes_of(PyObject* o, void* dst, size_t n) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return 0;
  const int fits = (size_t)b.len == n;
  if (fits) memcpy(dst, b.buf, n);
  PyBuffer_Release(&b);
  if (!fits) PyErr_Format(PyExc_TypeError, "expected a structure of %zu bytes", n);
  return fits;
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
  if (!count_is(n, 8) || !view_of(a[0], &x) || !address_of(a[1], &pos) || !i64_of(a[2], &pos_b) ||
      !bytes_of(a[3], &r, sizeof r) || !address_of(a[4], &weight) || !f32_of(a[5], &eps) ||
      !view_of(a[6], &y) || !address_of(a[7], &stream))
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
  if (!count_is(n, 12) || !view_of(a[0], &dy) || !view_of(a[1], &x) ||
      !address_of(a[2], &pos) || !i64_of(a[3], &pos_b) || !bytes_of(a[4], &r, sizeof r) ||
      !address_of(a[5], &weight) || !f32_of(a[6], &eps) || !view_of(a[7], &dx) ||
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
  if (!count_is(n, 13) || !view_of(a[0], &Q) || !view_of(a[1], &K) ||
      !view_of(a[2], &V) || !bytes_of(a[3], &p, sizeof p) || !address_of(a[4], &q_ptr) ||
      !address_of(a[5], &k_ptr) || !i32_of(a[6], &causal) || !f32_of(a[7], &scale) || !view_of(a[8], &O) ||
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
  if (!count_is(n, 17) || !view_of(a[0], &Q) || !view_of(a[1], &K) ||
      !view_of(a[2], &V) || !view_of(a[3], &O) || !view_of(a[4], &dO) ||
      !address_of(a[5], &lse) || !bytes_of(a[6], &p, sizeof p) || !address_of(a[7], &q_ptr) ||
      !address_of(a[8], &k_ptr) || !i32_of(a[9], &causal) || !f32_of(a[10], &scale) ||
      !view_of(a[11], &dQ) || !view_of(a[12], &dK) || !view_of(a[13], &dV) ||
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
                                ENTRY(packed_attn_bwd),
                                {"row_views", (PyCFunction)(void (*)(void))row_views, METH_FASTCALL,
                                 "views of rows of one type on one device, or None"},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "dsv_calls", "calls of dsv.h that take structures", -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_dsv_calls(void) {
  if (PyType_Ready(&ViewType) != 0) return NULL;
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (s_dtype == NULL || s_get_device == NULL || s_stride == NULL || s_data_ptr == NULL) return NULL;
  PyObject* m = PyModule_Create(&module);
  if (m == NULL) return NULL;
  Py_INCREF(&ViewType);
  if (PyModule_AddObject(m, "View", (PyObject*)&ViewType) != 0) {
    Py_DECREF(&ViewType);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
