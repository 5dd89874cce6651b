/*
 * Argument marshalling of the per-step calls for runtime.py (CPython C API): a
 * decode step's kernels take a few microseconds, less than building their
 * argument structs in Python does.  Reads the tensors' type, device, shape,
 * strides and address through their Python methods (no torch headers), checks
 * them, fills the structs of include/kvq.h and calls the library's functions,
 * whose addresses bind() takes from the loaded library.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "kvq.h"

typedef kvq_status (*norm_rope_fn)(const kvq_rotary*, int, int, const int32_t*, const kvq_heads*,
                                   const kvq_heads*, int, float, const float*, const kvq_heads*,
                                   const kvq_heads*, int32_t*, void*);
typedef kvq_status (*rope_append_fn)(const kvq_cache*, const kvq_rotary*, int, int, const int32_t*,
                                     const int32_t*, const kvq_heads*, const kvq_heads*,
                                     const kvq_heads*, const kvq_heads*, const kvq_heads*, int,
                                     float, const float*, int32_t*, void*);
typedef kvq_status (*decode_shared_fn)(const kvq_cache*, const kvq_decode_params*, int,
                                       const int32_t*, int, const void*, float*, float*, uint32_t*,
                                       void*, void*);

static norm_rope_fn p_norm_rope;
static rope_append_fn p_rope_append;
static decode_shared_fn p_decode_shared;

static PyObject *s_dtype, *s_get_device, *s_shape, *s_stride, *s_data_ptr, *s_numel,
    *s_is_contiguous;
static PyObject *t_bf16, *t_u8, *t_i32, *t_f32;   /* torch dtypes (singletons) */

/* ------------------------------------------------------------------ helpers */
static int refuse(const char* what, const char* why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", what, why);
  return -1;
}

static int method_long(PyObject* t, PyObject* name, long long* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int address(PyObject* t, void** out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return -1;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* A CUDA tensor of the given device and type. */
static int here(PyObject* t, PyObject* dtype, long dev, const char* what) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  const int same = d == dtype;
  if (!same) PyErr_Format(PyExc_ValueError, "%s: expected %R, got %R", what, dtype, d);
  Py_DECREF(d);
  if (!same) return -1;
  long long at;
  if (method_long(t, s_get_device, &at)) return -1;
  if (at != dev) {
    PyErr_Format(PyExc_ValueError, "%s: expected a tensor on cuda:%ld (the current device)", what,
                 dev);
    return -1;
  }
  return 0;
}

/* Sizes and strides; returns the number of dimensions (at most 4) or -1. */
static int layout(PyObject* t, long long* size, long long* stride, const char* what) {
  PyObject* sh = PyObject_GetAttr(t, s_shape);
  if (!sh) return -1;
  PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
  if (!st) {
    Py_DECREF(sh);
    return -1;
  }
  int n = -1;
  if (PyTuple_Check(sh) && PyTuple_Check(st) && PyTuple_GET_SIZE(sh) == PyTuple_GET_SIZE(st)) {
    n = (int)PyTuple_GET_SIZE(sh);
    for (int i = 0; i < n && i < 4; ++i) {
      size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(sh, i));
      stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    }
  }
  Py_DECREF(sh);
  Py_DECREF(st);
  if (PyErr_Occurred()) return -1;
  return n < 0 || n > 4 ? refuse(what, "expected a tensor of at most four dimensions") : n;
}

/* Rows of heads [tokens][heads][dim] or [batch][tokens][heads][dim] whose
 * tokens lie at one stride; their tokens and dim. */
typedef struct {
  kvq_heads h;
  int n;
  long long size[4], tokens, dim;
} rows_t;

static int rows(PyObject* t, PyObject* dtype, long dev, const char* what, rows_t* r) {
  long long st[4];
  if (here(t, dtype, dev, what)) return -1;
  if ((r->n = layout(t, r->size, st, what)) < 0) return -1;
  const int n = r->n;
  long long tok = 0;
  int one = 0;
  if (n == 3) {
    tok = st[0];
    one = 1;
    r->tokens = r->size[0];
  } else if (n == 4) {   /* one token per request: the requests are the tokens */
    tok = r->size[1] == 1 ? st[0] : st[1];
    one = r->size[0] <= 1 || r->size[1] <= 1 || st[0] == r->size[1] * tok;
    r->tokens = r->size[0] * r->size[1];
  }
  if (!one || st[n - 1] != 1)
    return refuse(what, "expected [(batch,) tokens][heads][dim] rows, dim dense, the tokens at one "
                        "stride");
  r->dim = r->size[n - 1];
  if (r->size[n - 2] > INT32_MAX) return refuse(what, "too many heads");
  r->h.num_heads = (int32_t)r->size[n - 2];
  /* the stride of a single token or head is never used, and torch's may be any */
  r->h.token_stride = r->tokens > 1 ? tok : 0;
  r->h.head_stride = r->h.num_heads > 1 ? st[n - 2] : r->dim;
  return address(t, &r->h.data);
}

/* A dense int32 array of n entries. */
static int index_array(PyObject* t, long long n, long dev, const char* what, const int32_t** out) {
  long long numel;
  void* p;
  if (here(t, t_i32, dev, what) || method_long(t, s_numel, &numel)) return -1;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!c) return -1;
  const int dense = c == Py_True;
  Py_DECREF(c);
  if (numel != n || !dense) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous entries", what, n);
    return -1;
  }
  if (address(t, &p)) return -1;
  *out = (const int32_t*)p;
  return 0;
}

static int optional_address(PyObject* t, void** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  if (PyLong_Check(t)) {
    *out = PyLong_AsVoidPtr(t);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
  }
  return address(t, out);
}

/* The error flag: int32 on the device (kernels write it), or its address. */
static int flag_address(PyObject* t, long dev, void** out) {
  long long numel;
  if (t != Py_None && !PyLong_Check(t)) {
    if (here(t, t_i32, dev, "error_flag") || method_long(t, s_numel, &numel)) return -1;
    if (numel < 1) return refuse("error_flag", "expected one entry");
  }
  return optional_address(t, out);
}

/* One float per head, dense. */
static int head_scales(PyObject* t, long long n, long dev, const float** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  long long numel;
  void* p;
  if (here(t, t_f32, dev, "q_head_scale") || method_long(t, s_numel, &numel)) return -1;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!c) return -1;
  const int dense = c == Py_True;
  Py_DECREF(c);
  if (numel != n || !dense) return refuse("q_head_scale", "expected one scale per query head");
  if (address(t, &p)) return -1;
  *out = (const float*)p;
  return 0;
}

static int as_int(PyObject* o, int32_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "an argument does not fit 32 bits");
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

static int as_float(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

/* Calls with the interpreter released hold no Python object. */
#define CALL(status, expr)      \
  do {                          \
    Py_BEGIN_ALLOW_THREADS      \
    status = (expr);            \
    Py_END_ALLOW_THREADS        \
  } while (0)

/* ------------------------------------------------------------------- calls */
/* bind(norm_rope, rope_append, decode_shared, bfloat16, uint8, int32, float32) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind: seven arguments");
    return NULL;
  }
  p_norm_rope = (norm_rope_fn)PyLong_AsVoidPtr(a[0]);
  p_rope_append = (rope_append_fn)PyLong_AsVoidPtr(a[1]);
  p_decode_shared = (decode_shared_fn)PyLong_AsVoidPtr(a[2]);
  if (PyErr_Occurred()) return NULL;
  PyObject** const types[4] = {&t_bf16, &t_u8, &t_i32, &t_f32};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[3 + i]);
    Py_XSETREF(*types[i], a[3 + i]);
  }
  Py_RETURN_NONE;
}

/* norm_rope(device, stream, rotary, q_norm len, k_norm len, q, k, positions,
 *           q_out, k_out, q_fp8, q_scale, q_head_scale, error_flag) -> status;
 * rotary is the struct's address, a norm's length -1 where it has none. */
static PyObject* norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 14 || !p_norm_rope) {
    PyErr_SetString(PyExc_TypeError, "norm_rope: fourteen arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  void *stream, *flag;
  const kvq_rotary* rot = (const kvq_rotary*)PyLong_AsVoidPtr(a[2]);
  const long nq = PyLong_AsLong(a[3]), nk = PyLong_AsLong(a[4]);
  const int fp8 = PyObject_IsTrue(a[10]);
  float scale;
  if (PyErr_Occurred() || optional_address(a[1], &stream) || as_float(a[11], &scale) ||
      flag_address(a[13], dev, &flag))
    return NULL;
  PyObject *q = a[5], *k = a[6];
  rows_t qr, qo, kr, ko;
  const float* hs = NULL;
  const int32_t* pos = NULL;
  long long T = -1, D = -1;
  if (q != Py_None) {
    if (rows(q, t_bf16, dev, "q", &qr) || rows(a[8], fp8 ? t_u8 : t_bf16, dev, "q_out", &qo) ||
        head_scales(a[12], qr.h.num_heads, dev, &hs))
      return NULL;
    T = qr.tokens;
    D = qr.dim;
    if (qr.n != 3) return refuse("q", "expected [tokens][heads][dim]"), NULL;
    if (qo.tokens != T || qo.dim != D || qo.h.num_heads != qr.h.num_heads)
      return refuse("q_out", "expected q's shape"), NULL;
    if (nq >= 0 && nq != D) return refuse("q_norm", "expected one weight per element"), NULL;
  }
  if (k != Py_None) {
    if (rows(k, t_bf16, dev, "k", &kr) || rows(a[9], t_bf16, dev, "k_out", &ko)) return NULL;
    if (kr.n != 3) return refuse("k", "expected [tokens][heads][dim]"), NULL;
    if (q != Py_None && (kr.tokens != T || kr.dim != D))
      return refuse("k", "expected q's tokens and dim"), NULL;
    T = kr.tokens;
    D = kr.dim;
    if (ko.tokens != T || ko.dim != D || ko.h.num_heads != kr.h.num_heads)
      return refuse("k_out", "expected k's shape"), NULL;
    if (nk >= 0 && nk != D) return refuse("k_norm", "expected one weight per element"), NULL;
  }
  if (T < 0) return refuse("norm_rope", "q or k is needed"), NULL;
  if (a[7] != Py_None && index_array(a[7], T, dev, "positions", &pos)) return NULL;
  if (T > INT32_MAX || D > INT32_MAX) return refuse("norm_rope", "too many tokens"), NULL;
  kvq_status st = KVQ_OK;
  if (T > 0)
    CALL(st, p_norm_rope(rot, (int)D, (int)T, pos, q != Py_None ? &qr.h : NULL,
                         q != Py_None ? &qo.h : NULL, fp8, scale, hs, k != Py_None ? &kr.h : NULL,
                         k != Py_None ? &ko.h : NULL, (int32_t*)flag, stream));
  return PyLong_FromLong(st);
}

/* rope_append(device, stream, cache, requests, rotary, q_norm len, k_norm len,
 *             k, v, kpe, start_pos, new_lens, q, q_out, q_fp8, q_scale,
 *             q_head_scale, error_flag) -> status;
 * cache and rotary are the structs' addresses, requests the block table's. */
static PyObject* rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 18 || !p_rope_append) {
    PyErr_SetString(PyExc_TypeError, "rope_append: eighteen arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  void *stream, *flag;
  const kvq_cache* c = (const kvq_cache*)PyLong_AsVoidPtr(a[2]);
  const long long requests = PyLong_AsLongLong(a[3]);
  const kvq_rotary* rot = (const kvq_rotary*)PyLong_AsVoidPtr(a[4]);
  const long nq = PyLong_AsLong(a[5]), nk = PyLong_AsLong(a[6]);
  const int fp8 = PyObject_IsTrue(a[14]);
  float scale;
  if (PyErr_Occurred() || !c || optional_address(a[1], &stream) || as_float(a[15], &scale) ||
      flag_address(a[17], dev, &flag)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "rope_append: no cache");
    return NULL;
  }
  const int mla = c->rope_dim > 0;
  rows_t kr, vr, er, qr, qo;
  const int32_t *start = NULL, *lens = NULL;
  const float* hs = NULL;
  if (rows(a[7], t_bf16, dev, "k_new", &kr)) return NULL;
  if (kr.n != 4 || kr.h.num_heads != c->num_kv_heads || kr.dim != c->head_dim)
    return refuse("k_new", "expected [batch][tokens][kv heads][dim] of the cache's"), NULL;
  const long long B = kr.size[0], T = kr.size[1];
  if (B > requests) return refuse("k_new", "more requests than the block table has"), NULL;
  if (B > INT32_MAX || T > INT32_MAX) return refuse("k_new", "too many tokens"), NULL;
  if (nk >= 0 && nk != c->head_dim)
    return refuse("k_norm", "expected one weight per element"), NULL;
  if (mla != (a[8] == Py_None) || mla != (a[9] != Py_None))
    return refuse("v_new", "expected v_new, or for MLA kpe_new"), NULL;
  if (!mla) {
    if (rows(a[8], t_bf16, dev, "v_new", &vr)) return NULL;
    if (vr.n != 4 || vr.size[0] != B || vr.size[1] != T || vr.h.num_heads != kr.h.num_heads ||
        vr.dim != kr.dim)
      return refuse("v_new", "expected k_new's shape"), NULL;
  } else {
    if (rows(a[9], t_bf16, dev, "kpe_new", &er)) return NULL;
    if (er.n != 4 || er.size[0] != B || er.size[1] != T || er.h.num_heads != 1 ||
        er.dim != c->rope_dim)
      return refuse("kpe_new", "expected [batch][tokens][1][rope]"), NULL;
  }
  PyObject* q = a[12];
  if (q != Py_None) {
    if (rows(q, t_bf16, dev, "q", &qr) || rows(a[13], fp8 ? t_u8 : t_bf16, dev, "q_out", &qo) ||
        head_scales(a[16], qr.h.num_heads, dev, &hs))
      return NULL;
    if (qr.n != 4 || qr.size[0] != B || qr.size[1] != T || qr.dim != c->head_dim)
      return refuse("q", "expected [batch][tokens][heads][dim]"), NULL;
    if (qo.tokens != B * T || qo.dim != qr.dim || qo.h.num_heads != qr.h.num_heads)
      return refuse("q_out", "expected q's shape"), NULL;
    if (nq >= 0 && nq != qr.dim) return refuse("q_norm", "expected one weight per element"), NULL;
  }
  kvq_status st = KVQ_OK;
  if (B > 0 && T > 0) {
    if (index_array(a[10], B, dev, "start_pos", &start)) return NULL;
    if (a[11] != Py_None && index_array(a[11], B, dev, "new_lens", &lens)) return NULL;
    CALL(st, p_rope_append(c, rot, (int)B, (int)T, start, lens, &kr.h, mla ? NULL : &vr.h,
                           mla ? &er.h : NULL, q != Py_None ? &qr.h : NULL,
                           q != Py_None ? &qo.h : NULL, fp8, scale, hs, (int32_t*)flag, stream));
  }
  return PyLong_FromLong(st);
}

/* decode_shared(device, stream, cache, params, prefix_len, prefix_table,
 *               prefix_splits, q, seq_lens, part_o, part_lse, counters, out,
 *               error_flag) -> status;
 * params' seq_lens and error_flag are filled in here. */
static PyObject* decode_shared(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 14 || !p_decode_shared) {
    PyErr_SetString(PyExc_TypeError, "decode_shared: fourteen arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  const kvq_cache* c = (const kvq_cache*)PyLong_AsVoidPtr(a[2]);
  const kvq_decode_params* given = (const kvq_decode_params*)PyLong_AsVoidPtr(a[3]);
  void *stream, *flag, *table, *po, *pl, *cn, *out;
  int32_t len, splits;
  if (PyErr_Occurred() || !c || !given) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "decode_shared: no cache or parameters");
    return NULL;
  }
  if (optional_address(a[1], &stream) || as_int(a[4], &len) || optional_address(a[5], &table) ||
      as_int(a[6], &splits) || optional_address(a[9], &po) || optional_address(a[10], &pl) ||
      optional_address(a[11], &cn) || optional_address(a[12], &out) ||
      flag_address(a[13], dev, &flag))
    return NULL;
  kvq_decode_params p = *given;
  rows_t qr;
  if (rows(a[7], p.q_fp8 ? t_u8 : t_bf16, dev, "q", &qr)) return NULL;
  if (qr.n != 3 || qr.tokens != p.batch || qr.h.num_heads != p.num_q_heads || qr.dim != p.qk_dim ||
      qr.h.head_stride != qr.dim || (p.batch > 1 && qr.h.token_stride != qr.dim * qr.h.num_heads))
    return refuse("q", "expected a contiguous [batch][heads][dim]"), NULL;
  if (index_array(a[8], p.batch, dev, "seq_lens", &p.seq_lens)) return NULL;
  p.error_flag = (int32_t*)flag;
  kvq_status st = KVQ_OK;
  if (p.batch > 0)
    CALL(st, p_decode_shared(c, &p, len, (const int32_t*)table, splits, qr.h.data, (float*)po,
                             (float*)pl, (uint32_t*)cn, out, stream));
  return PyLong_FromLong(st);
}

/* block_table(device, table, requests): refuses a table that is not a dense int32
 * [at least requests][pages] there. */
static PyObject* block_table(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "block_table: three arguments");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  const long long requests = PyLong_AsLongLong(a[2]);
  long long size[4], stride[4];
  if (PyErr_Occurred() || here(a[1], t_i32, dev, "block_table")) return NULL;
  const int d = layout(a[1], size, stride, "block_table");
  if (d < 0) return NULL;
  if (d != 2 || (size[1] > 1 && stride[1] != 1) || (size[0] > 1 && stride[0] != size[1]))
    return refuse("block_table", "expected a contiguous [batch][pages]"), NULL;
  if (size[0] < requests) return refuse("block_table", "fewer rows than requests"), NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "The library's functions."},
    {"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, "kvq_norm_rope"},
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, "kvq_rope_append"},
    {"decode_shared", (PyCFunction)(void (*)(void))decode_shared, METH_FASTCALL,
     "kvq_decode_shared"},
    {"block_table", (PyCFunction)(void (*)(void))block_table, METH_FASTCALL,
     "The check of a call's block table."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_call",
                                    "Marshalling of the per-step calls (see runtime.py).", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kvq_call(void) {
  struct {
    PyObject** to;
    const char* name;
  } const names[] = {{&s_dtype, "dtype"},     {&s_get_device, "get_device"},
                     {&s_shape, "shape"},     {&s_stride, "stride"},
                     {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
                     {&s_is_contiguous, "is_contiguous"}};
  for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
