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

typedef kvq_status (*plan_step_fn)(const kvq_page_plan*, void*);
typedef kvq_status (*append_slots_fn)(const kvq_cache*, const kvq_rotary*, int, const int32_t*,
                                      const int64_t*, const kvq_heads*, const kvq_heads*,
                                      const kvq_heads*, const kvq_heads*, const kvq_heads*, int,
                                      float, const float*, int32_t*, void*);
typedef kvq_status (*decode_diff_fn)(const kvq_cache*, const kvq_decode_params*, const kvq_diff*,
                                     const void*, float*, float*, uint32_t*, void*, void*);
typedef kvq_status (*chunk_fn)(const kvq_cache*, const kvq_decode_params*, const kvq_diff*, int,
                               const int32_t*, const void*, void*, size_t, void*, void*);

static norm_rope_fn p_norm_rope;
static rope_append_fn p_rope_append;
static decode_shared_fn p_decode_shared;
static plan_step_fn p_plan_step;
static append_slots_fn p_append_slots;
static decode_diff_fn p_decode_diff;
static chunk_fn p_chunk;

static PyObject *s_dtype, *s_get_device, *s_shape, *s_stride, *s_data_ptr, *s_numel,
    *s_is_contiguous;
static PyObject *t_bf16, *t_u8, *t_i32, *t_f32, *t_i64;   /* torch dtypes (singletons) */

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

/* A dense array of n entries of the type. */
static int dense_array(PyObject* t, PyObject* dtype, long long n, long dev, const char* what,
                       void** out) {
  long long numel;
  if (here(t, dtype, dev, what) || method_long(t, s_numel, &numel)) return -1;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!c) return -1;
  const int dense = c == Py_True;
  Py_DECREF(c);
  if (numel != n || !dense) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous entries", what, n);
    return -1;
  }
  return address(t, out);
}

static int index_array(PyObject* t, long long n, long dev, const char* what, const int32_t** out) {
  void* p;
  if (dense_array(t, t_i32, n, dev, what, &p)) return -1;
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
/* bind(norm_rope, rope_append, decode_shared, plan_step, rope_append_slots,
 *      decode_diff, chunk_attention, bfloat16, uint8, int32, float32, int64) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 12) {
    PyErr_SetString(PyExc_TypeError, "bind: twelve arguments");
    return NULL;
  }
  p_norm_rope = (norm_rope_fn)PyLong_AsVoidPtr(a[0]);
  p_rope_append = (rope_append_fn)PyLong_AsVoidPtr(a[1]);
  p_decode_shared = (decode_shared_fn)PyLong_AsVoidPtr(a[2]);
  p_plan_step = (plan_step_fn)PyLong_AsVoidPtr(a[3]);
  p_append_slots = (append_slots_fn)PyLong_AsVoidPtr(a[4]);
  p_decode_diff = (decode_diff_fn)PyLong_AsVoidPtr(a[5]);
  p_chunk = (chunk_fn)PyLong_AsVoidPtr(a[6]);
  if (PyErr_Occurred()) return NULL;
  PyObject** const types[5] = {&t_bf16, &t_u8, &t_i32, &t_f32, &t_i64};
  for (int i = 0; i < 5; ++i) {
    Py_INCREF(a[7 + i]);
    Py_XSETREF(*types[i], a[7 + i]);
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

/* plan_step(device, stream, plan, seq_lens, add_lens, seq_lens_out, free_count_out,
 *           error_flag) -> status;
 * plan is the struct's address; None leaves the lengths or the count updated in place. */
static PyObject* plan_step(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 8 || !p_plan_step) {
    PyErr_SetString(PyExc_TypeError, "plan_step: eight arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  const kvq_page_plan* given = (const kvq_page_plan*)PyLong_AsVoidPtr(a[2]);
  void *stream, *flag;
  if (PyErr_Occurred() || !given) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "plan_step: no plan");
    return NULL;
  }
  if (optional_address(a[1], &stream) || flag_address(a[7], dev, &flag)) return NULL;
  kvq_page_plan p = *given;
  const int32_t *lens_out = NULL, *count_out = NULL;
  if (index_array(a[3], p.batch, dev, "seq_lens", &p.seq_lens) ||
      index_array(a[4], p.batch, dev, "add_lens", &p.add_lens) ||
      (a[5] != Py_None && index_array(a[5], p.batch, dev, "seq_lens_out", &lens_out)) ||
      (a[6] != Py_None && index_array(a[6], 1, dev, "count_out", &count_out)))
    return NULL;
  p.seq_lens_out = (int32_t*)(a[5] != Py_None ? lens_out : p.seq_lens);
  p.free_count_out = (int32_t*)(a[6] != Py_None ? count_out : p.free_count);
  p.error_flag = (int32_t*)flag;
  kvq_status st;
  CALL(st, p_plan_step(&p, stream));
  return PyLong_FromLong(st);
}

/* append_slots(device, stream, cache, rotary, q_norm len, k_norm len, k, v, kpe, slots,
 *              positions, q, q_out, q_fp8, q_scale, q_head_scale, error_flag) -> status */
static PyObject* append_slots(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 17 || !p_append_slots) {
    PyErr_SetString(PyExc_TypeError, "append_slots: seventeen arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  void *stream, *flag;
  const kvq_cache* c = (const kvq_cache*)PyLong_AsVoidPtr(a[2]);
  const kvq_rotary* rot = (const kvq_rotary*)PyLong_AsVoidPtr(a[3]);
  const long nq = PyLong_AsLong(a[4]), nk = PyLong_AsLong(a[5]);
  const int fp8 = PyObject_IsTrue(a[13]);
  float scale;
  if (PyErr_Occurred() || !c || !rot || optional_address(a[1], &stream) ||
      as_float(a[14], &scale) || flag_address(a[16], dev, &flag)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "append_slots: no cache or rotation");
    return NULL;
  }
  const int mla = c->rope_dim > 0;
  rows_t kr, vr, er, qr, qo;
  void *slots = NULL, *pos = NULL;
  const float* hs = NULL;
  if (rows(a[6], t_bf16, dev, "k", &kr)) return NULL;
  if (kr.n != 3 || kr.h.num_heads != c->num_kv_heads || kr.dim != c->head_dim)
    return refuse("k", "expected [tokens][kv heads][dim] of the cache's"), NULL;
  const long long T = kr.tokens;
  if (T > INT32_MAX) return refuse("k", "too many tokens"), NULL;
  if (nk >= 0 && nk != c->head_dim)
    return refuse("k_norm", "expected one weight per element"), NULL;
  if (mla != (a[7] == Py_None) || mla != (a[8] != Py_None))
    return refuse("v", "expected v, or for MLA kpe"), NULL;
  if (!mla) {
    if (rows(a[7], t_bf16, dev, "v", &vr)) return NULL;
    if (vr.n != 3 || vr.tokens != T || vr.h.num_heads != kr.h.num_heads || vr.dim != kr.dim)
      return refuse("v", "expected k's shape"), NULL;
  } else {
    if (rows(a[8], t_bf16, dev, "kpe", &er)) return NULL;
    if (er.n != 3 || er.tokens != T || er.h.num_heads != 1 || er.dim != c->rope_dim)
      return refuse("kpe", "expected [tokens][1][rope]"), NULL;
  }
  PyObject* q = a[11];
  if (q != Py_None) {
    if (rows(q, t_bf16, dev, "q", &qr) || rows(a[12], fp8 ? t_u8 : t_bf16, dev, "q_out", &qo) ||
        head_scales(a[15], qr.h.num_heads, dev, &hs))
      return NULL;
    if (qr.n != 3 || qr.tokens != T || qr.dim != c->head_dim)
      return refuse("q", "expected [tokens][heads][dim]"), NULL;
    if (qo.tokens != T || qo.dim != qr.dim || qo.h.num_heads != qr.h.num_heads)
      return refuse("q_out", "expected q's shape"), NULL;
    if (nq >= 0 && nq != qr.dim) return refuse("q_norm", "expected one weight per element"), NULL;
  }
  if (dense_array(a[9], t_i64, T, dev, "slots", &slots)) return NULL;
  if (a[10] != Py_None && dense_array(a[10], t_i32, T, dev, "positions", &pos)) return NULL;
  kvq_status st = KVQ_OK;
  if (T > 0)
    CALL(st, p_append_slots(c, rot, (int)T, (const int32_t*)pos, (const int64_t*)slots, &kr.h,
                            mla ? NULL : &vr.h, mla ? &er.h : NULL, q != Py_None ? &qr.h : NULL,
                            q != Py_None ? &qo.h : NULL, fp8, scale, hs, (int32_t*)flag, stream));
  return PyLong_FromLong(st);
}

/* A dense [tokens][heads][dim] of queries that the parameters describe; its tokens. */
static int query_rows(PyObject* t, const kvq_decode_params* p, long dev, rows_t* r) {
  if (rows(t, p->q_fp8 ? t_u8 : t_bf16, dev, "q", r)) return -1;
  if (r->n != 3 || r->h.num_heads != p->num_q_heads || r->dim != p->qk_dim ||
      r->h.head_stride != r->dim ||
      (r->tokens > 1 && r->h.token_stride != r->dim * r->h.num_heads))
    return refuse("q", "expected a contiguous [tokens][heads][dim]");
  return 0;
}

/* decode_diff(device, stream, cache, params, diff, q, seq_lens, part_o, part_lse,
 *             counters, out, error_flag) -> status;
 * cache, params and diff are the structs' addresses. */
static PyObject* decode_diff(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 12 || !p_decode_diff) {
    PyErr_SetString(PyExc_TypeError, "decode_diff: twelve arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  const kvq_cache* c = (const kvq_cache*)PyLong_AsVoidPtr(a[2]);
  const kvq_decode_params* given = (const kvq_decode_params*)PyLong_AsVoidPtr(a[3]);
  const kvq_diff* d = (const kvq_diff*)PyLong_AsVoidPtr(a[4]);
  void *stream, *flag, *po, *pl, *cn, *out;
  if (PyErr_Occurred() || !c || !given || !d) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "decode_diff: no cache or parameters");
    return NULL;
  }
  if (optional_address(a[1], &stream) || optional_address(a[7], &po) ||
      optional_address(a[8], &pl) || optional_address(a[9], &cn) ||
      optional_address(a[10], &out) || flag_address(a[11], dev, &flag))
    return NULL;
  kvq_decode_params p = *given;
  rows_t qr;
  if (query_rows(a[5], &p, dev, &qr)) return NULL;
  if (qr.tokens != p.batch) return refuse("q", "expected one token per request"), NULL;
  if (index_array(a[6], p.batch, dev, "seq_lens", &p.seq_lens)) return NULL;
  p.error_flag = (int32_t*)flag;
  kvq_status st = KVQ_OK;
  if (p.batch > 0)
    CALL(st, p_decode_diff(c, &p, d, qr.h.data, (float*)po, (float*)pl, (uint32_t*)cn, out, stream));
  return PyLong_FromLong(st);
}

/* chunk_attention(device, stream, cache, params, diff, q, q_offsets, seq_lens,
 *                 workspace, bytes, out, out type, error_flag) -> status;
 * diff may be 0, out is a tensor of q's shape. */
static PyObject* chunk_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 13 || !p_chunk) {
    PyErr_SetString(PyExc_TypeError, "chunk_attention: thirteen arguments, after bind");
    return NULL;
  }
  const long dev = PyLong_AsLong(a[0]);
  const kvq_cache* c = (const kvq_cache*)PyLong_AsVoidPtr(a[2]);
  const kvq_decode_params* given = (const kvq_decode_params*)PyLong_AsVoidPtr(a[3]);
  const kvq_diff* d = (const kvq_diff*)PyLong_AsVoidPtr(a[4]);
  const long long bytes = PyLong_AsLongLong(a[9]);
  void *stream, *flag, *ws;
  if (PyErr_Occurred() || !c || !given) {
    if (!PyErr_Occurred())
      PyErr_SetString(PyExc_ValueError, "chunk_attention: no cache or parameters");
    return NULL;
  }
  if (optional_address(a[1], &stream) || optional_address(a[8], &ws) ||
      flag_address(a[12], dev, &flag))
    return NULL;
  kvq_decode_params p = *given;
  rows_t qr, o;
  const int32_t* offsets;
  if (query_rows(a[5], &p, dev, &qr)) return NULL;
  if (index_array(a[6], (long long)p.batch + 1, dev, "q_offsets", &offsets) ||
      index_array(a[7], p.batch, dev, "seq_lens", &p.seq_lens))
    return NULL;
  if (rows(a[10], a[11], dev, "out", &o)) return NULL;
  if (o.n != 3 || o.tokens != qr.tokens || o.h.num_heads != p.num_q_heads || o.dim != p.v_dim ||
      o.h.head_stride != o.dim || (o.tokens > 1 && o.h.token_stride != o.dim * o.h.num_heads))
    return refuse("out", "expected a contiguous [tokens][heads][dim]"), NULL;
  if (qr.tokens > INT32_MAX) return refuse("q", "too many tokens"), NULL;
  p.error_flag = (int32_t*)flag;
  kvq_status st = KVQ_OK;
  if (p.batch > 0 && qr.tokens > 0)
    CALL(st, p_chunk(c, &p, d, (int)qr.tokens, offsets, qr.h.data, ws, (size_t)bytes, o.h.data,
                     stream));
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
    {"plan_step", (PyCFunction)(void (*)(void))plan_step, METH_FASTCALL, "kvq_plan_step"},
    {"append_slots", (PyCFunction)(void (*)(void))append_slots, METH_FASTCALL,
     "kvq_rope_append_slots"},
    {"decode_diff", (PyCFunction)(void (*)(void))decode_diff, METH_FASTCALL, "kvq_decode_diff"},
    {"chunk_attention", (PyCFunction)(void (*)(void))chunk_attention, METH_FASTCALL,
     "kvq_chunk_attention"},
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
