/*
 * Marshalling of the serving step's calls for Python.  A step makes several of them, each a
 * few microseconds of GPU work, and converting their twenty arguments through ctypes takes
 * as long as the work; here it takes about one microsecond.  A pointer argument is None, an
 * int or an object with data_ptr(); a stream None, an int or an object with cuda_stream; a
 * host array anything with a buffer; a shape None or a PagedShape, whose type is handed over
 * by set_shape_type.  The functions return the call's status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tpk.h"

static PyObject *s_data_ptr, *s_cuda_stream;
static PyTypeObject* shape_type;

/* The argument list of one call, read in order; `bad` once one did not convert. */
typedef struct {
  PyObject* const* args;
  Py_ssize_t n, at;
  int bad;
} reader;

/* The next argument; NULL after one that did not convert (its exception is set) or past the
 * last one. */
static PyObject* take(reader* r) {
  if (r->at >= r->n) r->bad = 1;
  return r->bad ? NULL : r->args[r->at++];
}

static void* as_pointer(PyObject* o, int* bad) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) *bad = 1;
  return p;
}

static void* pointer(reader* r) {
  PyObject* o = take(r);
  if (!o || o == Py_None) return NULL;
  if (PyLong_Check(o)) return as_pointer(o, &r->bad);
  PyObject* v = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!v) {
    if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
      PyErr_Clear();
      PyErr_Format(PyExc_TypeError, "cannot take a device pointer from %R", (PyObject*)Py_TYPE(o));
    }
    r->bad = 1;
    return NULL;
  }
  void* p = as_pointer(v, &r->bad);
  Py_DECREF(v);
  return p;
}

static tpk_stream_t stream(reader* r) {
  PyObject* o = take(r);
  if (!o || o == Py_None) return NULL;
  if (PyLong_Check(o)) return (tpk_stream_t)as_pointer(o, &r->bad);
  PyObject* v = PyObject_GetAttr(o, s_cuda_stream);
  if (!v) {
    r->bad = 1;
    return NULL;
  }
  void* p = as_pointer(v, &r->bad);
  Py_DECREF(v);
  return (tpk_stream_t)p;
}

static int64_t wide(reader* r) {
  PyObject* o = take(r);
  const long long v = o ? PyLong_AsLongLong(o) : 0;
  if (v == -1 && PyErr_Occurred()) r->bad = 1;
  return v;
}

static int narrow(reader* r) {
  const int64_t v = wide(r);
  if (!r->bad && (v < INT32_MIN || v > INT32_MAX)) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
    r->bad = 1;
  }
  return (int)v;
}

/* A buffer of at least `bytes` bytes, or NULL for None; released by the caller. */
static const void* buffer(reader* r, Py_buffer* b, Py_ssize_t bytes) {
  PyObject* o = take(r);
  b->obj = NULL;
  if (!o || o == Py_None) return NULL;
  if (PyObject_GetBuffer(o, b, PyBUF_SIMPLE) != 0) {
    r->bad = 1;
    return NULL;
  }
  if (b->len < bytes) {
    PyErr_Format(PyExc_ValueError, "a buffer of %zd bytes, not %zd", b->len, bytes);
    r->bad = 1;
  }
  return b->buf;
}

static const tpk_paged_shape* shape_of(reader* r, Py_buffer* b) {
  PyObject* o = r->at < r->n ? r->args[r->at] : NULL;
  const tpk_paged_shape* s = buffer(r, b, sizeof(tpk_paged_shape));
  if (s && !r->bad && !(shape_type && PyObject_TypeCheck(o, shape_type))) {
    PyErr_Format(PyExc_TypeError, "a PagedShape, not %R", (PyObject*)Py_TYPE(o));
    r->bad = 1;
  }
  return s;
}

static PyObject* done(reader* r, tpk_status st) {
  if (r->bad || r->at != r->n) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return NULL;
  }
  return PyLong_FromLong((long)st);
}

/* Calls with the lock released: a launch may wait for room in the queue. */
#define RUN(r, call)                \
  tpk_status st = TPK_ERR_INVALID;  \
  if (!(r).bad && (r).at == (r).n) { \
    Py_BEGIN_ALLOW_THREADS st = call; \
    Py_END_ALLOW_THREADS            \
  }

static PyObject* kv_tables_update(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  reader r = {args, n, 0, 0};
  const int n_req = narrow(&r), max_pages = narrow(&r);
  const int32_t *len_old = pointer(&r), *len_new = pointer(&r);
  int32_t *table = pointer(&r), *free_slots = pointer(&r);
  const int free_cap = narrow(&r);
  const int32_t* n_free_in = pointer(&r);
  int32_t *n_free_out = pointer(&r), *len_out = pointer(&r), *granted = pointer(&r), *tok_off = pointer(&r);
  int64_t* slot_map = pointer(&r);
  int32_t *positions = pointer(&r), *token_req = pointer(&r);
  const int max_tokens = narrow(&r);
  const tpk_stream_t s = stream(&r);
  RUN(r, tpk_kv_tables_update(n_req, max_pages, len_old, len_new, table, free_slots, free_cap, n_free_in, n_free_out,
                              len_out, granted, tok_off, slot_map, positions, token_req, max_tokens, s));
  return done(&r, st);
}

static PyObject* kv_rope_append(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  reader r = {args, n, 0, 0};
  Py_buffer sb, ab;
  const tpk_paged_shape* shape = shape_of(&r, &sb);
  const int n_tokens = narrow(&r);
  const void* q = pointer(&r);
  const int64_t q_stride = wide(&r);
  const void* k = pointer(&r);
  const int64_t k_stride = wide(&r);
  const void* v = pointer(&r);
  const int64_t v_stride = wide(&r);
  const int32_t* positions = pointer(&r);
  const int n_axes = narrow(&r);
  const uint8_t* axis_of = buffer(&r, &ab, 0);
  const float* inv_freq = pointer(&r);
  const int rot_dim = narrow(&r), interleaved = narrow(&r);
  const int64_t* slot_map = pointer(&r);
  void* q_out = pointer(&r);
  const int64_t q_out_stride = wide(&r);
  void *k_pool = pointer(&r), *v_pool = pointer(&r);
  const tpk_stream_t s = stream(&r);
  if (!r.bad && axis_of && ab.len != rot_dim / 2) {
    PyErr_Format(PyExc_ValueError, "axis_of has %zd bytes, not %d", ab.len, rot_dim / 2);
    r.bad = 1;
  }
  RUN(r, tpk_kv_rope_append(shape, n_tokens, q, q_stride, k, k_stride, v, v_stride, positions, n_axes, axis_of,
                            inv_freq, rot_dim, interleaved, slot_map, q_out, q_out_stride, k_pool, v_pool, s));
  if (sb.obj) PyBuffer_Release(&sb);
  if (ab.obj) PyBuffer_Release(&ab);
  return done(&r, st);
}

static PyObject* decode_attn_paged(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  reader r = {args, n, 0, 0};
  Py_buffer sb;
  const tpk_paged_shape* shape = shape_of(&r, &sb);
  const int n_req = narrow(&r);
  const void* q = pointer(&r);
  const int64_t q_stride = wide(&r);
  const void *k_pool = pointer(&r), *v_pool = pointer(&r);
  const int32_t *table = pointer(&r), *n_tokens = pointer(&r), *tok_begin = pointer(&r);
  void* o = pointer(&r);
  const int64_t o_stride = wide(&r);
  const int o_f32 = narrow(&r);
  float* lse = pointer(&r);
  void* ws = pointer(&r);
  const int64_t ws_bytes = wide(&r);
  const tpk_stream_t s = stream(&r);
  RUN(r, tpk_decode_attn_paged(shape, n_req, q, q_stride, k_pool, v_pool, table, n_tokens, tok_begin, o, o_stride,
                               o_f32, lse, ws, ws_bytes < 0 ? 0 : (size_t)ws_bytes, s));
  if (sb.obj) PyBuffer_Release(&sb);
  return done(&r, st);
}

static PyObject* cross_attn_paged(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  reader r = {args, n, 0, 0};
  Py_buffer sb;
  const tpk_paged_shape* shape = shape_of(&r, &sb);
  const int n_req = narrow(&r), n_q = narrow(&r);
  const void* q = pointer(&r);
  const int64_t q_stride = wide(&r);
  const int32_t* q_off = pointer(&r);
  const void *k_pool = pointer(&r), *v_pool = pointer(&r);
  const int32_t *table = pointer(&r), *n_tokens = pointer(&r), *kv_range = pointer(&r);
  void* o = pointer(&r);
  const int64_t o_stride = wide(&r);
  float* lse = pointer(&r);
  void* ws = pointer(&r);
  const int64_t ws_bytes = wide(&r);
  const tpk_stream_t s = stream(&r);
  RUN(r, tpk_cross_attn_paged(shape, n_req, n_q, q, q_stride, q_off, k_pool, v_pool, table, n_tokens, kv_range, o,
                              o_stride, lse, ws, ws_bytes < 0 ? 0 : (size_t)ws_bytes, s));
  if (sb.obj) PyBuffer_Release(&sb);
  return done(&r, st);
}

static PyObject* set_shape_type(PyObject* self, PyObject* type) {
  (void)self;
  if (!PyType_Check(type)) return PyErr_Format(PyExc_TypeError, "a type, not %R", type);
  Py_INCREF(type);
  Py_XSETREF(shape_type, (PyTypeObject*)type);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(kv_tables_update), METHOD(kv_rope_append), METHOD(decode_attn_paged),
                                METHOD(cross_attn_paged), {"set_shape_type", set_shape_type, METH_O, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tpk_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tpk_call(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_data_ptr || !s_cuda_stream) return NULL;
  return PyModule_Create(&module);
}
