/* Argument marshalling of the rotating appends and the 8-bit-cache decode for
 * Python: reads the tensors' pointers, shapes and strides, refuses what the
 * library could not see (types, shapes, strided tables, short plans, tensors on
 * the host or another device), and calls the C ABI.
 * Plain CPython C API; the functions' addresses come from libmla.py, which has
 * loaded the library.  An 8-bit append takes 5.5 us of a Grace host, its launch
 * 2.1 among them, against 9.3 with fewer checks in Python and the call through
 * ctypes (whose conversions alone take 2.2); with a small batch that is the
 * call's time (1 token, 16 heads: 10.9 -> 5.9 us). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "mla.h"

static __typeof__(&mla_rope_append) f_append;
static __typeof__(&mla_rope_append_fp8) f_append_fp8;
static __typeof__(&mla_decode_fp8) f_decode;
static __typeof__(&mla_decode_fp8_f32) f_decode_f32;
static __typeof__(&mla_decode_fp8_plan) f_plan;
static __typeof__(&mla_decode_fp8_plan_size) f_plan_size;
static int (*f_device)(int*);          /* cudaGetDevice */
static PyObject* f_stream;             /* torch's current stream of a device */

static PyObject *s_shape, *s_stride, *s_data_ptr, *s_dtype, *s_contiguous, *s_nbytes,
    *s_get_device, *s_cuda_stream;

/* torch's types, an object each; e4m3 codes may also come as bytes. */
static PyObject *t_bf16[2], *t_f32[2], *t_i32[2], *t_e4m3[2];

/* NULL, with a ValueError unless an exception is on its way already. */
static PyObject* refuse(const char* why) {
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, why);
  return NULL;
}
#define NEED(cond, why) \
  do {                  \
    if (!(cond)) return refuse(why); \
  } while (0)

/* The n numbers of a tuple; 0 when it is something else or an error came. */
static int numbers(PyObject* tuple, int n, int64_t* out) {
  int ok = tuple && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n;
  for (int i = 0; ok && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) ok = 0;
  }
  Py_XDECREF(tuple);
  return ok;
}
static int shape_of(PyObject* t, int n, int64_t* out) {
  return numbers(PyObject_GetAttr(t, s_shape), n, out);
}
static int strides_of(PyObject* t, int n, int64_t* out) {
  return numbers(PyObject_CallMethodNoArgs(t, s_stride), n, out);
}
static int64_t number(PyObject* x) {   /* -1 on an error */
  if (!x) return -1;
  const int64_t v = PyLong_AsLongLong(x);
  Py_DECREF(x);
  return v;
}
static int has_type(PyObject* t, PyObject* const* type) {
  PyObject* x = PyObject_GetAttr(t, s_dtype);
  const int ok = x && (x == type[0] || x == type[1]);
  Py_XDECREF(x);
  return ok;
}
static int contiguous(PyObject* t) {
  PyObject* x = PyObject_CallMethodNoArgs(t, s_contiguous);
  const int ok = x && PyObject_IsTrue(x) == 1;
  Py_XDECREF(x);
  return ok;
}
static void* pointer(PyObject* t) {    /* NULL is refused by the library */
  PyObject* x = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!x) return NULL;
  void* p = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return p;
}
/* The current device's number if each of n tensors (NULL and None pass) lies on
 * it, else -1: the kernels would fault on host memory or another device's. */
static int on_device(PyObject* const* t, int n) {
  int64_t at = -1;
  for (int i = 0; i < n; ++i) {
    if (!t[i] || t[i] == Py_None) continue;
    const int64_t d = number(PyObject_CallMethodNoArgs(t[i], s_get_device));
    if (d < 0 || (at >= 0 && d != at)) return -1;
    at = d;
  }
  int now = -1;
  return at >= 0 && f_device(&now) == 0 && now == at ? now : -1;
}
/* The handle of a stream (a number or torch's object); for None that of torch's
 * current one, without the object around it (0.1 against 2.9 us a call). */
static void* stream_of(PyObject* stream, int device) {
  if (PyLong_Check(stream)) return PyLong_AsVoidPtr(stream);
  PyObject* x;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLong(device);
    if (!d) return NULL;
    x = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
  } else {
    x = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!x) return NULL;
  void* p = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return p;
}
static int dim(int64_t v) { return v >= 0 && v <= INT32_MAX; }

/* A cache of pages [pages, 64, 1, 576]. */
static int cache_ok(PyObject* t, PyObject* const* type, int64_t* pages) {
  int64_t s[4];
  *pages = 0;
  if (!shape_of(t, 4, s) || s[1] != 64 || s[2] != 1 || s[3] != 576 || !dim(s[0]) ||
      !has_type(t, type) || !contiguous(t))
    return 0;
  *pages = s[0];
  return 1;
}
/* scales [pages, 64 / scale_tokens]. */
static int scales_ok(PyObject* t, int64_t pages, int* scale_tokens) {
  int64_t s[2];
  if (!shape_of(t, 2, s) || s[0] != pages || s[1] < 1 || s[1] > 64 || 64 % s[1] != 0 ||
      !has_type(t, t_f32) || !contiguous(t))
    return 0;
  *scale_tokens = (int)(64 / s[1]);
  return 1;
}
static int table_ok(PyObject* t, int64_t batch, int64_t* max_pages) {
  int64_t s[2];
  if (!shape_of(t, 2, s) || s[0] < batch || !dim(s[1]) || !has_type(t, t_i32) || !contiguous(t))
    return 0;
  *max_pages = s[1];
  return 1;
}
static int lengths_ok(PyObject* t, int64_t batch) {
  int64_t n;
  return shape_of(t, 1, &n) && n >= batch && has_type(t, t_i32) && contiguous(t);
}

static const char kKvNew[] = "kv_new must be bf16 [B, s_new, 576], its last dim contiguous";
static const char kQueries[] =
    "q_rope and q_out come together, bf16 [B, s_new, h_q, 64], their last dim contiguous";
static const char kCosSin[] = "cos_sin must be fp32 [max_positions, 64], contiguous";
static const char kTable[] = "block_table must be int32 [B, max_pages], contiguous";
static const char kLengths[] = "cache_seqlens and new_lens must be int32 [B], contiguous";
static const char kCache16[] = "kv_cache must be bf16 [pages, 64, 1, 576], contiguous";
static const char kCache8[] = "kv_cache must be float8_e4m3fn or uint8 [pages, 64, 1, 576], contiguous";
static const char kDevice[] = "every tensor must be on the current CUDA device";
static const char kPlan[] = "tile_meta must be contiguous, of mla_decode_fp8_plan_size bytes";
static const char kScales[] = "scales must be fp32 [pages, 64 / scale_tokens], contiguous";

/* append(kv_new, kv_cache, scales or None, block_table, cache_seqlens, cos_sin,
 *        q_rope, q_out, new_lens, interleaved, stream) -> status */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  NEED(n == 11, "append takes 11 arguments");
  PyObject *kv = a[0], *cache = a[1], *scales = a[2], *table = a[3], *lens = a[4], *cs = a[5],
           *q = a[6], *qo = a[7], *news = a[8];
  const int interleaved = PyObject_IsTrue(a[9]);
  if (PyErr_Occurred()) return NULL;
  const int fp8 = scales != Py_None;
  int64_t ks[3], kt[3], qs[4], qt[4] = {0, 0, 0, 1}, os[4], ot[4] = {0, 0, 0, 1}, cd[2], pages,
          max_pages;
  int g = 0;
  NEED(shape_of(kv, 3, ks) && ks[2] == 576 && dim(ks[0]) && dim(ks[1]) && strides_of(kv, 3, kt) &&
           kt[2] == 1 && has_type(kv, t_bf16),
       kKvNew);
  const int queries = q != Py_None;
  NEED(queries == (qo != Py_None), kQueries);
  if (queries) {
    NEED(shape_of(q, 4, qs) && qs[0] == ks[0] && qs[1] == ks[1] && dim(qs[2]) && qs[3] == 64 &&
             shape_of(qo, 4, os) && os[0] == qs[0] && os[1] == qs[1] && os[2] == qs[2] &&
             os[3] == 64 && strides_of(q, 4, qt) && strides_of(qo, 4, ot) && qt[3] == 1 &&
             ot[3] == 1 && has_type(q, t_bf16) && has_type(qo, t_bf16),
         kQueries);
  }
  NEED(cache_ok(cache, fp8 ? t_e4m3 : t_bf16, &pages), fp8 ? kCache8 : kCache16);
  if (fp8) NEED(scales_ok(scales, pages, &g), kScales);
  NEED(table_ok(table, ks[0], &max_pages), kTable);
  NEED(lengths_ok(lens, ks[0]) && (news == Py_None || lengths_ok(news, ks[0])), kLengths);
  NEED(shape_of(cs, 2, cd) && cd[1] == 64 && dim(cd[0]) && has_type(cs, t_f32) && contiguous(cs),
       kCosSin);
  PyObject* const all[] = {kv, cache, scales, table, lens, cs, q, qo, news};
  const int device = on_device(all, 9);
  NEED(device >= 0, kDevice);
  void* stream = stream_of(a[10], device);
  const void *p_kv = pointer(kv), *p_q = queries ? pointer(q) : NULL;
  void *p_qo = queries ? pointer(qo) : NULL, *p_cache = pointer(cache);
  float* p_sc = fp8 ? (float*)pointer(scales) : NULL;
  const int32_t *p_table = (const int32_t*)pointer(table), *p_lens = (const int32_t*)pointer(lens),
                *p_new = news == Py_None ? NULL : (const int32_t*)pointer(news);
  const float* p_cs = (const float*)pointer(cs);
  if (PyErr_Occurred()) return NULL;
  const int h = queries ? (int)qs[2] : 0;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fp8 ? f_append_fp8(p_kv, kt[0], kt[1], p_q, qt[0], qt[1], qt[2], p_qo, ot[0], ot[1], ot[2],
                          p_cache, p_sc, g, (int)pages, p_table, (int)max_pages, p_lens, p_new,
                          p_cs, (int)cd[0], interleaved, (int)ks[0], (int)ks[1], h, stream)
           : f_append(p_kv, kt[0], kt[1], p_q, qt[0], qt[1], qt[2], p_qo, ot[0], ot[1], ot[2],
                      p_cache, (int)pages, p_table, (int)max_pages, p_lens, p_new, p_cs,
                      (int)cd[0], interleaved, (int)ks[0], (int)ks[1], h, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* decode(f32, q, kv_cache, scales, block_table, cache_seqlens, tile_meta, out,
 *        lse, softmax_scale, workspace, stream) -> status */
static PyObject* py_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  NEED(n == 12, "decode takes 12 arguments");
  const int f32 = PyObject_IsTrue(a[0]);
  PyObject *q = a[1], *cache = a[2], *scales = a[3], *table = a[4], *lens = a[5], *meta = a[6],
           *out = a[7], *lse = a[8], *ws = a[10];
  const double scale = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred()) return NULL;
  int64_t qs[4], os[4], ls[3], pages, max_pages;
  int g = 0;
  NEED(shape_of(q, 4, qs) && dim(qs[0]) && dim(qs[1]) && dim(qs[2]) && qs[3] == 576 &&
           has_type(q, t_bf16) && contiguous(q),
       "q must be bf16 [B, s_q, h_q, 576], contiguous");
  NEED(shape_of(out, 4, os) && os[0] == qs[0] && os[1] == qs[1] && os[2] == qs[2] && os[3] == 512 &&
           has_type(out, f32 ? t_f32 : t_bf16) && contiguous(out),
       "out must be [B, s_q, h_q, 512] of the call's type, contiguous");
  NEED(shape_of(lse, 3, ls) && ls[0] == qs[0] && ls[1] == qs[2] && ls[2] == qs[1] &&
           has_type(lse, t_f32) && contiguous(lse),
       "lse must be fp32 [B, h_q, s_q], contiguous");
  NEED(cache_ok(cache, t_e4m3, &pages), kCache8);
  NEED(scales_ok(scales, pages, &g), kScales);
  NEED(table_ok(table, qs[0], &max_pages), kTable);
  NEED(lengths_ok(lens, qs[0]), kLengths);
  PyObject* const all[] = {q, cache, scales, table, lens, meta, out, lse, ws};
  const int device = on_device(all, 9);
  NEED(device >= 0, kDevice);
  NEED(contiguous(meta) && number(PyObject_GetAttr(meta, s_nbytes)) >=
                               (int64_t)f_plan_size((int)qs[0], (int)qs[1], (int)qs[2], device),
       kPlan);
  NEED(contiguous(ws), "workspace must be contiguous");
  void* stream = stream_of(a[11], device);
  const void *p_q = pointer(q), *p_cache = pointer(cache), *p_meta = pointer(meta);
  const float* p_sc = (const float*)pointer(scales);
  const int32_t *p_table = (const int32_t*)pointer(table), *p_lens = (const int32_t*)pointer(lens);
  void *p_out = pointer(out), *p_ws = pointer(ws);
  float* p_lse = (float*)pointer(lse);
  const int64_t ws_bytes = number(PyObject_GetAttr(ws, s_nbytes));
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f32 ? f_decode_f32(p_q, p_cache, p_sc, g, (int)pages, p_table, (int)max_pages, p_lens,
                          (int)qs[0], (int)qs[1], (int)qs[2], p_meta, (float*)p_out, p_lse,
                          (float)scale, p_ws, (size_t)ws_bytes, stream)
           : f_decode(p_q, p_cache, p_sc, g, (int)pages, p_table, (int)max_pages, p_lens,
                      (int)qs[0], (int)qs[1], (int)qs[2], p_meta, p_out, p_lse, (float)scale, p_ws,
                      (size_t)ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* plan(cache_seqlens, s_q, h_q, tile_meta, stream) -> status */
static PyObject* py_plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  NEED(n == 5, "plan takes 5 arguments");
  const long s_q = PyLong_AsLong(a[1]), h_q = PyLong_AsLong(a[2]);
  if (PyErr_Occurred()) return NULL;
  int64_t batch;
  NEED(shape_of(a[0], 1, &batch) && dim(batch) && has_type(a[0], t_i32) && contiguous(a[0]),
       "cache_seqlens must be int32 [B], contiguous");
  NEED(dim(s_q) && dim(h_q), "s_q and h_q out of range");
  PyObject* const all[] = {a[0], a[3]};
  const int device = on_device(all, 2);
  NEED(device >= 0, kDevice);
  NEED(contiguous(a[3]), kPlan);
  void* stream = stream_of(a[4], device);
  const int32_t* p_lens = (const int32_t*)pointer(a[0]);
  void* p_meta = pointer(a[3]);
  const int64_t bytes = number(PyObject_GetAttr(a[3], s_nbytes));
  if (PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_plan(p_lens, (int)batch, (int)s_q, (int)h_q, p_meta, (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* bind(seven addresses, current_stream, five types): append, append_fp8, decode,
 * decode_f32, plan, plan_size, cudaGetDevice; bfloat16, float32, int32,
 * float8_e4m3fn, uint8 */
static PyObject* py_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  NEED(n == 13, "bind takes 7 addresses, a function and 5 types");
  void* p[7];
  for (int i = 0; i < 7; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return NULL;
  f_append = (__typeof__(f_append))p[0];
  f_append_fp8 = (__typeof__(f_append_fp8))p[1];
  f_decode = (__typeof__(f_decode))p[2];
  f_decode_f32 = (__typeof__(f_decode_f32))p[3];
  f_plan = (__typeof__(f_plan))p[4];
  f_plan_size = (__typeof__(f_plan_size))p[5];
  f_device = (__typeof__(f_device))p[6];
  Py_INCREF(a[7]);
  Py_XSETREF(f_stream, a[7]);
  PyObject** const to[] = {t_bf16, t_f32, t_i32, t_e4m3};
  for (int i = 0; i < 4; ++i) {
    for (int k = 0; k < 2; ++k) {
      PyObject* type = a[i == 3 && k ? 12 : 8 + i];
      Py_INCREF(type);
      Py_XSETREF(to[i][k], type);
    }
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, NULL},
    {"plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, NULL},
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_shape, "shape"},       {&s_stride, "stride"},
               {&s_data_ptr, "data_ptr"}, {&s_dtype, "dtype"},
               {&s_contiguous, "is_contiguous"}, {&s_nbytes, "nbytes"},
               {&s_get_device, "get_device"}, {&s_cuda_stream, "cuda_stream"}};
  for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i) {
    *names[i].to = PyUnicode_InternFromString(names[i].name);
    if (!*names[i].to) return NULL;
  }
  return PyModule_Create(&module);
}
