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

static PyObject *s_dtype, *s_get_device, *s_stride, *s_data_ptr, *s_shape, *s_is_contiguous;

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
// dsv_rows
// ---------------------------------------------------------------------------
typedef struct {
  PyObject_HEAD
  dsv_rows v;
} Rows;
static PyTypeObject RowsType;
static PyObject* types[4];               // the dtypes of dsv_type, in its order (set_types)
static PyObject* dtype_i32;              // and int32

static PyObject* rows_make(void* ptr, int64_t stride, int32_t type) {
  Rows* o = PyObject_New(Rows, &RowsType);
  if (o == NULL) return NULL;
  o->v.ptr = ptr;
  o->v.stride = stride;
  o->v.type = type;
  return (PyObject*)o;
}
static PyObject* rows_new(PyTypeObject* type, PyObject* args, PyObject* kw) {
  PyObject* address;
  long long stride;
  int of;
  void* ptr;
  if (kw != NULL && PyDict_GET_SIZE(kw) != 0) {
    PyErr_SetString(PyExc_TypeError, "Rows(ptr, stride, type)");
    return NULL;
  }
  if (!PyArg_ParseTuple(args, "OLi", &address, &stride, &of) || !address_of(address, &ptr)) return NULL;
  return rows_make(ptr, stride, of);
}
static PyObject* rows_ptr(PyObject* o, void* unused) {
  void* p = ((Rows*)o)->v.ptr;
  if (p == NULL) Py_RETURN_NONE;
  return PyLong_FromUnsignedLongLong((unsigned long long)(uintptr_t)p);
}
static PyMemberDef rows_members[] = {{"stride", T_LONGLONG, offsetof(Rows, v.stride), READONLY, NULL},
                                     {"type", T_INT, offsetof(Rows, v.type), READONLY, NULL},
                                     {NULL, 0, 0, 0, NULL}};
static PyGetSetDef rows_getset[] = {{"ptr", rows_ptr, NULL, NULL, NULL}, {NULL, NULL, NULL, NULL, NULL}};
static PyTypeObject RowsType = {
    PyVarObject_HEAD_INIT(NULL, 0).tp_name = "dsv_calls.Rows",
    .tp_basicsize = sizeof(Rows),
    .tp_flags = Py_TPFLAGS_DEFAULT,
    .tp_doc = "dsv_rows: the address, row stride and type of a matrix",
    .tp_new = rows_new,
    .tp_dealloc = view_free,
    .tp_members = rows_members,
    .tp_getset = rows_getset,
};
static PyObject* set_types(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "set_types(bf16, f32, e4m3, e5m2, int32)");
    return NULL;
  }
  for (int i = 0; i < 5; ++i) {
    PyObject** to = i < 4 ? &types[i] : &dtype_i32;
    Py_INCREF(a[i]);
    Py_XDECREF(*to);
    *to = a[i];
  }
  Py_RETURN_NONE;
}
// The rows of a 2D tensor, NULL without an error set where its type, device or
// last stride is another than a matrix has.
static PyObject* rows_of_tensor(PyObject* t, long index) {
  PyObject* got = PyObject_GetAttr(t, s_dtype);
  if (got == NULL) return NULL;
  int type = 0;
  while (type < 4 && got != types[type]) ++type;
  Py_DECREF(got);
  if (type == 4) return NULL;
  if ((got = PyObject_CallMethodNoArgs(t, s_get_device)) == NULL) return NULL;
  const long at = PyLong_AsLong(got);
  Py_DECREF(got);
  if (at != index || PyErr_Occurred()) return NULL;
  PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
  if (st == NULL) return NULL;
  PyObject* made = NULL;
  if (PyTuple_Check(st) && PyTuple_GET_SIZE(st) == 2) {
    const long long r = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 0)), c = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 1));
    if (!PyErr_Occurred() && c == 1 && (got = PyObject_CallMethodNoArgs(t, s_data_ptr)) != NULL) {
      void* ptr;
      if (address_of(got, &ptr)) made = rows_make(ptr, r, type);
      Py_DECREF(got);
    }
  }
  Py_DECREF(st);
  return made;
}
// matrices(index, *tensors): a tuple of their rows (None: null), or None where
// one of them is not a matrix of a known type on device `index` with
// contiguous rows.
static PyObject* matrices(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n < 1) {
    PyErr_SetString(PyExc_TypeError, "matrices(index, *tensors)");
    return NULL;
  }
  const long index = PyLong_AsLong(a[0]);
  if (index == -1 && PyErr_Occurred()) return NULL;
  PyObject* all = PyTuple_New(n - 1);
  for (Py_ssize_t i = 1; all != NULL && i < n; ++i) {
    PyObject* v = a[i] == Py_None ? rows_make(NULL, 0, 0) : rows_of_tensor(a[i], index);
    if (v == NULL) {
      Py_DECREF(all);
      if (PyErr_Occurred()) return NULL;
      Py_RETURN_NONE;
    }
    PyTuple_SET_ITEM(all, i - 1, v);
  }
  return all;
}

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
static int rows_of(PyObject* o, dsv_rows* v) {
  if (Py_TYPE(o) != &RowsType) {
    PyErr_Format(PyExc_TypeError, "expected Rows, got %.80s", Py_TYPE(o)->tp_name);
    return 0;
  }
  *v = ((Rows*)o)->v;
  return 1;
}
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

static PyObject* layer_norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, y;
  dsv_norm p;
  void *ptr, *weight, *bias, *stats, *stream;
  if (!count_is(n, 8) || !rows_of(a[0], &x) || !bytes_of(a[1], &p, sizeof p) || !address_of(a[2], &ptr) ||
      !address_of(a[3], &weight) || !address_of(a[4], &bias) || !rows_of(a[5], &y) || !address_of(a[6], &stats) ||
      !address_of(a[7], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_layer_norm_fwd(x, p, ptr, weight, bias, y, stats, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* layer_norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows dy, x, dx;
  dsv_norm p;
  void *stats, *ptr, *weight, *dweight, *dbias, *ws, *stream;
  size_t bytes;
  if (!count_is(n, 12) || !rows_of(a[0], &dy) || !rows_of(a[1], &x) || !address_of(a[2], &stats) ||
      !bytes_of(a[3], &p, sizeof p) || !address_of(a[4], &ptr) || !address_of(a[5], &weight) || !rows_of(a[6], &dx) ||
      !address_of(a[7], &dweight) || !address_of(a[8], &dbias) || !address_of(a[9], &ws) || !size_of(a[10], &bytes) ||
      !address_of(a[11], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_layer_norm_bwd(dy, x, stats, p, ptr, weight, dx, dweight, dbias, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* quantize_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, q, qt;
  int32_t R, C, rows;
  void *scale, *scale_t, *stream;
  if (!count_is(n, 9) || !rows_of(a[0], &x) || !i32_of(a[1], &R) || !i32_of(a[2], &C) || !i32_of(a[3], &rows) ||
      !rows_of(a[4], &q) || !address_of(a[5], &scale) || !rows_of(a[6], &qt) || !address_of(a[7], &scale_t) ||
      !address_of(a[8], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_quantize_fp8(x, R, C, rows, q, scale, qt, scale_t, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* matmul_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, y, c;
  dsv_matmul p;
  void *sx, *sy, *stream;
  if (!count_is(n, 7) || !rows_of(a[0], &x) || !address_of(a[1], &sx) || !rows_of(a[2], &y) || !address_of(a[3], &sy) ||
      !bytes_of(a[4], &p, sizeof p) || !rows_of(a[5], &c) || !address_of(a[6], &stream))
    return NULL;
  dsv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = dsv_matmul_fp8(x, sx, y, sy, p, c, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// ---------------------------------------------------------------------------
// The calls on matrices from the tensors themselves
// ---------------------------------------------------------------------------
// What binding.py's checks cost is most of a small call's host time, so the common
// call is checked here: None where anything is not as it has to be (or a size does
// not fit), and binding.py then finds out what and says so.  Measured, host time of
// a call on a Grace core: norm 17.0 -> 9.8 us, its
// gradient 26.5 -> 18.4, quantiser 13.9 -> 9.2, product 15.6 -> 9.2.
static int fits(long long v) { return v >= INT32_MIN && v <= INT32_MAX; }
// sizes of an n-dimensional tensor
static int sizes_of(PyObject* t, int n, long long* v) {
  PyObject* st = PyObject_GetAttr(t, s_shape);
  if (st == NULL) return 0;
  int ok = PyTuple_Check(st) && PyTuple_GET_SIZE(st) == n;
  for (int i = 0; ok && i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    ok = !(v[i] == -1 && PyErr_Occurred());
  }
  Py_DECREF(st);
  return ok;
}
// A contiguous tensor of `dtype` on device `index` (None: null) with these sizes.
static int array_of(PyObject* t, PyObject* dtype, long index, int n, const long long* want, void** ptr) {
  *ptr = NULL;
  if (t == Py_None) return 1;
  PyObject* got = PyObject_GetAttr(t, s_dtype);
  if (got == NULL) return 0;
  Py_DECREF(got);
  if (got != dtype) return 0;
  if ((got = PyObject_CallMethodNoArgs(t, s_get_device)) == NULL) return 0;
  const long at = PyLong_AsLong(got);
  Py_DECREF(got);
  if (at != index) return 0;
  if ((got = PyObject_CallMethodNoArgs(t, s_is_contiguous)) == NULL) return 0;
  const int whole = got == Py_True;
  Py_DECREF(got);
  long long have[2];
  if (!whole || !sizes_of(t, n, have)) return 0;
  for (int i = 0; i < n; ++i)
    if (have[i] != want[i]) return 0;
  if ((got = PyObject_CallMethodNoArgs(t, s_data_ptr)) == NULL) return 0;
  const int ok = address_of(got, ptr);
  Py_DECREF(got);
  return ok;
}
// A matrix on device `index`, and its sizes (want: those it must have).
static int matrix_of(PyObject* t, long index, dsv_rows* v, long long* size, const long long* want) {
  PyObject* r = rows_of_tensor(t, index);
  if (r == NULL) return 0;
  *v = ((Rows*)r)->v;
  Py_DECREF(r);
  if (!sizes_of(t, 2, size) || !fits(size[0]) || !fits(size[1])) return 0;
  return want == NULL || (size[0] == want[0] && size[1] == want[1]);
}
static PyObject* not_so(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}
// The rows of weights that x's rows divide into; 0: not a valid combination.
static int weights_of(PyObject* weight, PyObject* ptr, long index, const long long* size, long long* S, int* dims,
                      void** w, void** p) {
  long long want[2] = {1, size[1]};
  *S = 1;
  *dims = 1;
  *p = NULL;
  if (ptr != Py_None) {
    long long n;
    if (!sizes_of(ptr, 1, &n) || n < 1 || !array_of(ptr, dtype_i32, index, 1, &n, p)) return 0;
    *S = n - 1;
    *dims = 2;
  } else if (weight != Py_None) {
    long long have[2];
    if (sizes_of(weight, 2, have)) {
      *S = have[0];
      *dims = 2;
      if (*S < 1 || size[0] % *S != 0) return 0;
    } else {
      PyErr_Clear();
    }
  }
  want[0] = *S;
  return fits(*S) && array_of(weight, types[1], index, *dims, *dims == 2 ? want : &size[1], w);
}

// norm_fwd(x, weight, bias, seq_ptr, eps, y, stats, index, stream): status or None
static PyObject* norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, y;
  dsv_norm p;
  void *ptr, *w, *b, *st, *stream;
  long long size[2], ysize[2], S;
  int dims;
  if (!count_is(n, 9)) return NULL;
  const long index = PyLong_AsLong(a[7]);
  if (index < 0 || !f32_of(a[4], &p.eps) || !matrix_of(a[0], index, &x, size, NULL) ||
      !weights_of(a[1], a[3], index, size, &S, &dims, &w, &ptr))
    return not_so();
  const long long vec[2] = {S, size[1]}, two[2] = {2, size[0]};
  if ((a[2] != Py_None && a[1] == Py_None) || !array_of(a[2], types[1], index, dims, dims == 2 ? vec : &size[1], &b) ||
      !matrix_of(a[5], index, &y, ysize, size) || y.type != DSV_BF16 || x.type > DSV_F32 ||
      !array_of(a[6], types[1], index, 2, two, &st) || !address_of(a[8], &stream))
    return not_so();
  p.T = (int32_t)size[0], p.C = (int32_t)size[1], p.S = (int32_t)S;
  dsv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = dsv_layer_norm_fwd(x, p, ptr, w, b, y, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

// norm_bwd_bytes(x, weight, seq_ptr, index): the gradient's workspace, or None
static PyObject* norm_bwd_bytes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_norm p;
  void *w, *ptr;
  long long size[2], S;
  int dims;
  if (!count_is(n, 4)) return NULL;
  const long index = PyLong_AsLong(a[3]);
  if (index < 0 || !sizes_of(a[0], 2, size) || !fits(size[0]) || !fits(size[1]) ||
      !weights_of(a[1], a[2], index, size, &S, &dims, &w, &ptr))
    return not_so();
  p.T = (int32_t)size[0], p.C = (int32_t)size[1], p.S = (int32_t)S, p.eps = 1e-6f;
  return PyLong_FromSize_t(dsv_layer_norm_bwd_workspace_bytes(p));
}
// norm_bwd(dy, x, stats, weight, seq_ptr, dx, dweight, dbias, workspace, bytes, index, stream): status or None
static PyObject* norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows dy, x, dx;
  dsv_norm p;
  void *ptr, *w, *dw, *db, *st, *ws, *stream;
  long long size[2], other[2], S;
  size_t bytes;
  int dims;
  if (!count_is(n, 12)) return NULL;
  const long index = PyLong_AsLong(a[10]);
  if (index < 0 || !matrix_of(a[1], index, &x, size, NULL) || !matrix_of(a[0], index, &dy, other, size) ||
      !matrix_of(a[5], index, &dx, other, size) || dy.type != DSV_BF16 || x.type > DSV_F32 || dx.type != x.type ||
      !weights_of(a[3], a[4], index, size, &S, &dims, &w, &ptr))
    return not_so();
  const long long vec[2] = {S, size[1]}, two[2] = {2, size[0]};
  const long long* want = dims == 2 ? vec : &size[1];
  if (!array_of(a[2], types[1], index, 2, two, &st) || !array_of(a[6], types[1], index, dims, want, &dw) ||
      !array_of(a[7], types[1], index, dims, want, &db) || !address_of(a[8], &ws) || !size_of(a[9], &bytes) ||
      !address_of(a[11], &stream))
    return not_so();
  p.T = (int32_t)size[0], p.C = (int32_t)size[1], p.S = (int32_t)S, p.eps = 1e-6f;
  dsv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = dsv_layer_norm_bwd(dy, x, st, p, ptr, w, dx, dw, db, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

// quantize(x, rows, q, scale, qt, scale_t, index, stream): status or None
static PyObject* quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, q, qt = {NULL, 0, 0};
  int32_t rows;
  void *scale, *scale_t = NULL, *stream;
  long long size[2], other[2];
  if (!count_is(n, 8)) return NULL;
  const long index = PyLong_AsLong(a[6]);
  if (index < 0 || !i32_of(a[1], &rows) || (rows != 1 && rows != 128) || !matrix_of(a[0], index, &x, size, NULL) ||
      !matrix_of(a[2], index, &q, other, size) || x.type > DSV_F32 || q.type < DSV_E4M3)
    return not_so();
  const long long cb = (size[1] + 127) / 128, rb = (size[0] + 127) / 128;
  const long long turned[2] = {size[1], size[0]}, sc[2] = {cb, rows == 1 ? size[0] : rb}, sct[2] = {rb, rows == 1 ? size[1] : cb};
  if (!array_of(a[3], types[1], index, 2, sc, &scale)) return not_so();
  if (a[4] != Py_None && (!matrix_of(a[4], index, &qt, other, turned) || qt.type != q.type ||
                          !array_of(a[5], types[1], index, 2, sct, &scale_t)))
    return not_so();
  if (!address_of(a[7], &stream)) return not_so();
  dsv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = dsv_quantize_fp8(x, (int32_t)size[0], (int32_t)size[1], rows, q, scale, qt, scale_t, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

static int scale_of(PyObject* t, long index, long long R, long long K, int32_t* rows, void** ptr) {
  long long have[2];
  const long long kb = (K + 127) / 128;
  if (t == Py_None || !sizes_of(t, 2, have) || have[0] != kb) return 0;
  *rows = have[1] == R ? 1 : 128;
  if (*rows == 128 && have[1] != (R + 127) / 128) return 0;
  return array_of(t, types[1], index, 2, have, ptr);
}
// matmul(a, a_scale, b, b_scale, c, accumulate, index, stream): status or None
static PyObject* matmul(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  dsv_rows x, y, c;
  dsv_matmul p;
  void *sx, *sy, *stream;
  long long xs[2], ys[2], cs[2];
  if (!count_is(n, 8)) return NULL;
  const long index = PyLong_AsLong(a[6]);
  if (index < 0 || !i32_of(a[5], &p.accumulate) || !matrix_of(a[0], index, &x, xs, NULL) ||
      !matrix_of(a[2], index, &y, ys, NULL) || xs[1] != ys[1] || x.type < DSV_E4M3 || y.type < DSV_E4M3)
    return not_so();
  const long long want[2] = {xs[0], ys[0]};
  if (!matrix_of(a[4], index, &c, cs, want) || c.type > DSV_F32 || (p.accumulate && c.type != DSV_F32) ||
      !scale_of(a[1], index, xs[0], xs[1], &p.a_rows, &sx) || !scale_of(a[3], index, ys[0], ys[1], &p.b_rows, &sy) ||
      !address_of(a[7], &stream))
    return not_so();
  p.M = (int32_t)xs[0], p.N = (int32_t)ys[0], p.K = (int32_t)xs[1];
  dsv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = dsv_matmul_fp8(x, sx, y, sy, p, c, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, "checked and called from tensors, or None"}
#define ENTRY(name) {"dsv_" #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, "dsv_" #name " of dsv.h"}
static PyMethodDef methods[] = {ENTRY(rope_axes_fwd), ENTRY(rope_axes_bwd), ENTRY(packed_attn_fwd),
                                ENTRY(packed_attn_bwd), ENTRY(layer_norm_fwd), ENTRY(layer_norm_bwd),
                                ENTRY(quantize_fp8), ENTRY(matmul_fp8),
                                FAST(norm_fwd), FAST(norm_bwd), FAST(norm_bwd_bytes), FAST(quantize), FAST(matmul),
                                {"set_types", (PyCFunction)(void (*)(void))set_types, METH_FASTCALL,
                                 "the dtypes of dsv_type"},
                                {"matrices", (PyCFunction)(void (*)(void))matrices, METH_FASTCALL,
                                 "rows of matrices on one device, or None"},
                                {"row_views", (PyCFunction)(void (*)(void))row_views, METH_FASTCALL,
                                 "views of rows of one type on one device, or None"},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "dsv_calls", "calls of dsv.h that take structures", -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_dsv_calls(void) {
  if (PyType_Ready(&ViewType) != 0 || PyType_Ready(&RowsType) != 0) return NULL;
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  if (s_dtype == NULL || s_get_device == NULL || s_stride == NULL || s_data_ptr == NULL || s_shape == NULL ||
      s_is_contiguous == NULL)
    return NULL;
  PyObject* m = PyModule_Create(&module);
  if (m == NULL) return NULL;
  Py_INCREF(&ViewType);
  if (PyModule_AddObject(m, "View", (PyObject*)&ViewType) != 0) {
    Py_DECREF(&ViewType);
    Py_DECREF(m);
    return NULL;
  }
  Py_INCREF(&RowsType);
  if (PyModule_AddObject(m, "Rows", (PyObject*)&RowsType) != 0) {
    Py_DECREF(&RowsType);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
