/*
 * CPython side of the grouped-query entry points: checks the tensors of one call and makes it.
 *
 * A decode step's calls take 3 to 10 us on the GPU, and the same checks and marshalling written
 * in Python with ctypes took 8 us of a call's 13 (13 tensors, four attributes each, 30 converted
 * arguments). Here they take about 3. Only the stable CPython API is used: tensors are looked at
 * through their Python attributes, the library is called through the addresses that ctypes
 * resolved (bind), and streams and devices come from torch's own functions.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/tts.h"

typedef tts_status (*append_fn)(const void*, int64_t, int32_t, const void*, int64_t, const void*,
                                int64_t, int64_t, const int32_t*, const int32_t*, int32_t, int32_t,
                                int32_t, int32_t, const float*, int32_t, const int32_t*, int32_t,
                                void*, void*, float*, float*, tts_dtype, int32_t, int32_t, void*,
                                void*, uint32_t*, void*);
typedef tts_status (*decode_fn)(const void*, int64_t, const int32_t*, int32_t, int32_t, int32_t,
                                int32_t, int32_t, const void*, const void*, const float*,
                                const float*, tts_dtype, int32_t, int32_t, const int32_t*, int32_t,
                                const int32_t*, int32_t, int32_t, float, void*, tts_dtype, float*,
                                void*, size_t, uint32_t*, void*);
typedef tts_status (*window_fn)(const void*, const void*, const void*, tts_dtype, int64_t, int64_t,
                                const int32_t*, const int32_t*, int32_t, int32_t, int32_t, int32_t,
                                int32_t, int32_t, int32_t, int32_t, float, void*, tts_dtype, float*,
                                void*, size_t, uint32_t*, void*);

static append_fn f_append;
static decode_fn f_decode;
static window_fn f_window;
static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride, *s_nbytes;
static PyObject *d_bf16, *d_f32, *d_u8, *d_e4m3, *d_i32;
static PyObject *raw_stream, *get_device, *set_device;

typedef struct {
  void* ptr;
  PyObject* dtype; /* one of torch's dtype objects, which live as long as the process */
  int nd;
  int64_t shape[4];
} Tensor;

static int refuse(const char* what, const char* why) {
  if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s %s", what, why);
  return -1;
}

static int64_t call_int(PyObject* t, PyObject* method) {
  PyObject* r = PyObject_CallMethodNoArgs(t, method);
  if (r == NULL) return -1;
  const int64_t v = (int64_t)PyLong_AsUnsignedLongLongMask(r);
  Py_DECREF(r);
  return v;
}

static int sizes(PyObject* tuple, int64_t* out, int most) {
  if (tuple == NULL || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > most) return -1;
  const int n = (int)PyTuple_GET_SIZE(tuple);
  for (int i = 0; i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  return n;
}

/* dtype, shape and address of a tensor on device `dev`; not yet whether it is contiguous. */
static int look(PyObject* t, const char* name, long dev, Tensor* o) {
  o->dtype = PyObject_GetAttr(t, s_dtype);
  if (o->dtype == NULL) {
    PyErr_Clear();
    return refuse(name, "must be a CUDA tensor");
  }
  Py_DECREF(o->dtype);
  const int64_t at = call_int(t, s_get_device);
  if (at < 0) {
    PyErr_Clear();
    return refuse(name, "must be a CUDA tensor");
  }
  if (at != dev) return refuse(name, "must be on the device of the call's other tensors");
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  o->nd = sizes(shape, o->shape, 4);
  Py_XDECREF(shape);
  if (o->nd < 0) return refuse(name, "has too many dimensions");
  o->ptr = (void*)(uintptr_t)call_int(t, s_data_ptr);
  return PyErr_Occurred() ? -1 : 0;
}

static int contiguous(PyObject* t, const char* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (r == NULL) return -1;
  const int ok = r == Py_True;
  Py_DECREF(r);
  return ok ? 0 : refuse(name, "must be contiguous");
}

/* A contiguous tensor of one type with nd dimensions (nd < 0: any). */
static int plain(PyObject* t, const char* name, long dev, PyObject* dtype, int nd, Tensor* o) {
  if (look(t, name, dev, o) < 0) return -1;
  if (dtype != NULL && o->dtype != dtype) {
    PyErr_Format(PyExc_ValueError, "%s must be %S, got %S", name, dtype, o->dtype);
    return -1;
  }
  if (nd >= 0 && o->nd != nd) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", name, nd);
    return -1;
  }
  return contiguous(t, name);
}
/* The same, or None: a null address. */
static int optional(PyObject* t, const char* name, long dev, PyObject* dtype, int nd, Tensor* o) {
  if (t != Py_None) return plain(t, name, dev, dtype, nd, o);
  o->ptr = NULL;
  o->dtype = NULL;
  o->nd = 0;
  return 0;
}
static int64_t count(const Tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->nd; ++i) n *= t->shape[i];
  return n;
}

/* [tokens, heads, d] bf16 whose heads are contiguous: a view of a packed projection passes. */
static int rows(PyObject* t, const char* name, long dev, Tensor* o, int64_t* stride) {
  if (look(t, name, dev, o) < 0) return -1;
  if (o->dtype != d_bf16 || o->nd != 3) return refuse(name, "must be bf16 [tokens, heads, head_dim]");
  int64_t s[4];
  PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
  const int n = sizes(st, s, 4);
  Py_XDECREF(st);
  if (n != 3) return refuse(name, "has no strides");
  if (s[2] != 1 || (s[1] != o->shape[2] && o->shape[1] != 1))
    return refuse(name, "must have the heads of a token contiguous");
  *stride = o->shape[0] > 1 ? s[0] : o->shape[1] * o->shape[2];
  return 0;
}

typedef struct {
  Tensor k, v, ks, vs;
  tts_dtype code;
} Cache;
static int cache(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, long dev, Cache* c) {
  if (plain(k, "k_cache", dev, NULL, 4, &c->k) < 0) return -1;
  const int f8 = c->k.dtype == d_u8 || c->k.dtype == d_e4m3;
  if (!f8 && c->k.dtype != d_bf16)
    return refuse("k_cache", "must be bf16, or uint8 / float8_e4m3fn codes");
  if (plain(v, "v_cache", dev, c->k.dtype, 4, &c->v) < 0) return -1;
  for (int i = 0; i < 4; ++i)
    if (c->k.shape[i] != c->v.shape[i])
      return refuse("k_cache and v_cache", "must have the same shape");
  if ((ks != Py_None) != f8 || (vs != Py_None) != f8)
    return refuse("k_scale and v_scale", "go with an e4m3 cache");
  c->code = f8 ? TTS_E4M3 : TTS_BF16;
  if (optional(ks, "k_scale", dev, d_f32, 2, &c->ks) < 0) return -1;
  if (optional(vs, "v_scale", dev, d_f32, 2, &c->vs) < 0) return -1;
  if (f8 && (c->ks.shape[0] != c->k.shape[0] || c->ks.shape[1] != c->k.shape[1] ||
             c->vs.shape[0] != c->k.shape[0] || c->vs.shape[1] != c->k.shape[1]))
    return refuse("k_scale and v_scale", "must be [pages, heads_kv]");
  return 0;
}

static int fits32(int64_t x, const char* name) {
  return x >= INT32_MIN && x <= INT32_MAX ? 0 : refuse(name, "is out of range");
}
static int int32_arg(PyObject* o, const char* name, int32_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = (int32_t)v;
  return fits32(v, name);
}

static int make_current(long dev) {
  PyObject* d = PyLong_FromLong(dev);
  PyObject* r = d == NULL ? NULL : PyObject_CallOneArg(set_device, d);
  Py_XDECREF(d);
  Py_XDECREF(r);
  return r == NULL ? -1 : 0;
}
/* The current stream of `dev`, that device made current (*back: the one to restore, or -1). Where
 * that fails, the device that was current is so again. */
static int enter(long dev, void** stream, long* back) {
  *back = -1;
  PyObject* now = PyObject_CallNoArgs(get_device);
  if (now == NULL) return -1;
  const long cur = PyLong_AsLong(now);
  Py_DECREF(now);
  if (cur == -1 && PyErr_Occurred()) return -1;
  if (cur != dev) {
    if (make_current(dev) < 0) return -1;
    *back = cur;
  }
  PyObject* d = PyLong_FromLong(dev);
  PyObject* s = d == NULL ? NULL : PyObject_CallOneArg(raw_stream, d);
  Py_XDECREF(d);
  if (s == NULL) {
    if (*back >= 0) {
      PyObject *type, *value, *trace;
      PyErr_Fetch(&type, &value, &trace);
      if (make_current(*back) < 0) PyErr_Clear();
      PyErr_Restore(type, value, trace);
    }
    return -1;
  }
  *stream = (void*)(uintptr_t)PyLong_AsUnsignedLongLongMask(s);
  Py_DECREF(s);
  return 0;
}
static PyObject* leave(long back, int status) {
  if (back >= 0 && make_current(back) < 0) return NULL;
  return PyLong_FromLong(status);
}

static long device_of(PyObject* t, const char* name) {
  const int64_t dev = call_int(t, s_get_device);
  if (PyErr_Occurred()) PyErr_Clear();
  if (dev < 0) refuse(name, "must be a CUDA tensor");
  return (long)dev;
}

static int nargs_are(Py_ssize_t n, Py_ssize_t want) {
  if (f_append == NULL) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return -1;
  }
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, n);
  return -1;
}

static PyObject* rope_kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (nargs_are(n, 15) < 0) return NULL;
  PyObject *k = a[0], *v = a[1], *q = a[11];
  const long dev = device_of(k, "k");
  if (dev < 0) return NULL;
  Cache c;
  if (cache(a[2], a[3], a[8], a[9], dev, &c) < 0) return NULL;
  const int64_t hkv = c.k.shape[1], d = c.k.shape[3];
  Tensor tk, tv, tq, qo, ko, pt, past, cu, cs, st;
  int64_t k_stride, v_stride, q_stride = 0, hq = 0, max_pos = 0;
  if (rows(k, "k", dev, &tk, &k_stride) < 0 || rows(v, "v", dev, &tv, &v_stride) < 0) return NULL;
  const int64_t total = tk.shape[0];
  if (tk.shape[1] != hkv || tk.shape[2] != d || tv.shape[0] != total || tv.shape[1] != hkv ||
      tv.shape[2] != d) {
    refuse("k and v", "must be [tokens, heads_kv, head_dim] with the cache's heads");
    return NULL;
  }
  if (plain(a[4], "page_tables", dev, d_i32, 2, &pt) < 0 ||
      plain(a[5], "past_lens", dev, d_i32, -1, &past) < 0 ||
      plain(a[6], "cu_new", dev, d_i32, -1, &cu) < 0)
    return NULL;
  const int64_t batch = count(&past);
  if (pt.shape[0] != batch || count(&cu) != batch + 1) {
    refuse("page_tables, past_lens, cu_new", "must be [batch, max_pages], [batch], [batch + 1]");
    return NULL;
  }
  int32_t max_new;
  if (int32_arg(a[7], "max_new", &max_new) < 0) return NULL;
  if (optional(a[10], "cos_sin", dev, d_f32, 3, &cs) < 0) return NULL;
  if (a[10] != Py_None) {  /* a table of no positions has a null address: not `no rotation` */
    if (cs.shape[0] < 1 || cs.shape[1] != d / 2 || cs.shape[2] != 2) {
      refuse("cos_sin", "must be [max_pos, head_dim/2, 2] with a position at least");
      return NULL;
    }
    max_pos = cs.shape[0];
  }
  tq.ptr = qo.ptr = NULL;
  if (q != Py_None) {
    if (rows(q, "q", dev, &tq, &q_stride) < 0) return NULL;
    hq = tq.shape[1];
    if (tq.shape[0] != total || tq.shape[2] != d) {
      refuse("q", "must be [tokens, heads, head_dim]");
      return NULL;
    }
    if (plain(a[12], "q_out", dev, d_bf16, 3, &qo) < 0) return NULL;
    if (qo.shape[0] != total || qo.shape[1] != hq || qo.shape[2] != d) {
      refuse("q_out", "must have q's shape");
      return NULL;
    }
  } else if (a[12] != Py_None) {
    refuse("q_out", "goes with q");
    return NULL;
  }
  if (optional(a[13], "k_out", dev, d_bf16, 3, &ko) < 0) return NULL;
  if (a[13] != Py_None && (ko.shape[0] != total || ko.shape[1] != hkv || ko.shape[2] != d)) {
    refuse("k_out", "must have k's shape");
    return NULL;
  }
  if (optional(a[14], "status", dev, d_i32, -1, &st) < 0) return NULL;
  if (fits32(batch, "batch") < 0 || fits32(c.k.shape[0], "pages") < 0 ||
      fits32(pt.shape[1], "max_pages") < 0 || fits32(max_pos, "max_pos") < 0)
    return NULL;
  void* stream;
  long back;
  if (enter(dev, &stream, &back) < 0) return NULL;
  tts_status status;
  Py_BEGIN_ALLOW_THREADS  /* a launch may block */
  status = f_append(tq.ptr, q_stride, (int32_t)hq, tk.ptr, k_stride, tv.ptr, v_stride, total,
                    cu.ptr, past.ptr, (int32_t)batch, max_new, (int32_t)hkv, (int32_t)d, cs.ptr,
                    (int32_t)max_pos, pt.ptr, (int32_t)pt.shape[1], c.k.ptr, c.v.ptr, c.ks.ptr,
                    c.vs.ptr, c.code, (int32_t)c.k.shape[0], (int32_t)c.k.shape[2], qo.ptr, ko.ptr,
                    st.ptr, stream);
  Py_END_ALLOW_THREADS
  return leave(back, status);
}

/* out and lse of an attention call on q [tokens, heads, d]. */
static int results(PyObject* out, PyObject* lse, long dev, const Tensor* q, Tensor* to, Tensor* tl) {
  if (plain(out, "out", dev, NULL, 3, to) < 0) return -1;
  if ((to->dtype != d_f32 && to->dtype != d_bf16) || to->shape[0] != q->shape[0] ||
      to->shape[1] != q->shape[1] || to->shape[2] != q->shape[2])
    return refuse("out", "must be fp32 or bf16 of q's shape");
  if (optional(lse, "lse", dev, d_f32, 2, tl) < 0) return -1;
  if (lse != Py_None && (tl->shape[0] != q->shape[0] || tl->shape[1] != q->shape[1]))
    return refuse("lse", "must be [tokens, heads]");
  return 0;
}
static int scratch(PyObject* ws, long dev, Tensor* t, size_t* bytes) {
  if (optional(ws, "workspace", dev, NULL, -1, t) < 0) return -1;
  *bytes = 0;
  if (ws == Py_None) return 0;
  PyObject* n = PyObject_GetAttr(ws, s_nbytes);
  if (n == NULL) return -1;
  *bytes = (size_t)PyLong_AsUnsignedLongLongMask(n);
  Py_DECREF(n);
  return 0;
}

static PyObject* attn_decode_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (nargs_are(n, 16) < 0) return NULL;
  const long dev = device_of(a[0], "q");
  if (dev < 0) return NULL;
  Cache c;
  if (cache(a[1], a[2], a[3], a[4], dev, &c) < 0) return NULL;
  Tensor q, pt, lens, cu, out, lse, ws, st;
  if (plain(a[0], "q", dev, d_bf16, 3, &q) < 0 ||
      plain(a[5], "page_tables", dev, d_i32, 2, &pt) < 0 ||
      plain(a[6], "kv_lens", dev, d_i32, -1, &lens) < 0 ||
      optional(a[7], "cu_seqlens_q", dev, d_i32, -1, &cu) < 0 ||
      results(a[12], a[13], dev, &q, &out, &lse) < 0)
    return NULL;
  const int64_t batch = count(&lens), d = c.k.shape[3];
  if (q.shape[2] != d) {
    refuse("q", "must be [tokens, heads, head_dim]");
    return NULL;
  }
  if (pt.shape[0] != batch) {
    refuse("page_tables, kv_lens", "must be [batch, max_pages], [batch]");
    return NULL;
  }
  if (a[7] != Py_None ? count(&cu) != batch + 1 : q.shape[0] != batch) {
    refuse("cu_seqlens_q", "must be [batch + 1]; without it q has one token per request");
    return NULL;
  }
  int32_t max_q, window, sinks;
  if (int32_arg(a[8], "max_seqlen_q", &max_q) < 0 || int32_arg(a[9], "window", &window) < 0 ||
      int32_arg(a[10], "sinks", &sinks) < 0)
    return NULL;
  const double scale = PyFloat_AsDouble(a[11]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  size_t bytes;
  if (scratch(a[14], dev, &ws, &bytes) < 0 || optional(a[15], "status", dev, d_i32, -1, &st) < 0)
    return NULL;
  if (fits32(batch, "batch") < 0 || fits32(c.k.shape[0], "pages") < 0 ||
      fits32(pt.shape[1], "max_pages") < 0)
    return NULL;
  void* stream;
  long back;
  if (enter(dev, &stream, &back) < 0) return NULL;
  tts_status status;
  Py_BEGIN_ALLOW_THREADS  /* a launch may block */
  status = f_decode(q.ptr, q.shape[0], cu.ptr, (int32_t)batch, max_q, (int32_t)q.shape[1],
                    (int32_t)c.k.shape[1], (int32_t)d, c.k.ptr, c.v.ptr, c.ks.ptr, c.vs.ptr, c.code,
                    (int32_t)c.k.shape[0], (int32_t)c.k.shape[2], pt.ptr, (int32_t)pt.shape[1],
                    lens.ptr, window, sinks, (float)scale, out.ptr,
                    out.dtype == d_bf16 ? TTS_BF16 : TTS_F32, lse.ptr, ws.ptr, bytes, st.ptr,
                    stream);
  Py_END_ALLOW_THREADS
  return leave(back, status);
}

static PyObject* attn_fwd_varlen_window(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (nargs_are(n, 14) < 0) return NULL;
  const long dev = device_of(a[0], "q");
  if (dev < 0) return NULL;
  Tensor q, k, v, cq, ck, out, lse, ws, st;
  if (plain(a[0], "q", dev, NULL, 3, &q) < 0) return NULL;
  if (q.dtype != d_bf16 && q.dtype != d_f32) {
    refuse("q, k, v", "must share dtype bf16 or fp32");
    return NULL;
  }
  if (plain(a[1], "k", dev, q.dtype, 3, &k) < 0 || plain(a[2], "v", dev, q.dtype, 3, &v) < 0)
    return NULL;
  if (k.shape[0] != v.shape[0] || k.shape[1] != v.shape[1] || k.shape[2] != v.shape[2] ||
      q.shape[2] != k.shape[2]) {
    refuse("k and v", "must have the same shape and q's head_dim");
    return NULL;
  }
  if (plain(a[3], "cu_seqlens_q", dev, d_i32, -1, &cq) < 0 ||
      plain(a[4], "cu_seqlens_k", dev, d_i32, -1, &ck) < 0 ||
      results(a[10], a[11], dev, &q, &out, &lse) < 0)
    return NULL;
  const int64_t batch = count(&cq) - 1;
  if (batch < 1 || count(&ck) != batch + 1) {
    refuse("cu_seqlens_q and cu_seqlens_k", "must be [batch + 1]");
    return NULL;
  }
  int32_t max_q, max_k, window, sinks;
  if (int32_arg(a[5], "max_seqlen_q", &max_q) < 0 || int32_arg(a[6], "max_seqlen_k", &max_k) < 0 ||
      int32_arg(a[7], "window", &window) < 0 || int32_arg(a[8], "sinks", &sinks) < 0)
    return NULL;
  const double scale = PyFloat_AsDouble(a[9]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  size_t bytes;
  if (scratch(a[12], dev, &ws, &bytes) < 0 || optional(a[13], "status", dev, d_i32, -1, &st) < 0)
    return NULL;
  if (fits32(batch, "batch") < 0) return NULL;
  void* stream;
  long back;
  if (enter(dev, &stream, &back) < 0) return NULL;
  tts_status status;
  Py_BEGIN_ALLOW_THREADS  /* a launch may block */
  status = f_window(q.ptr, k.ptr, v.ptr, q.dtype == d_f32 ? TTS_F32 : TTS_BF16, q.shape[0],
                    k.shape[0], cq.ptr, ck.ptr, (int32_t)batch, max_q, max_k, (int32_t)q.shape[1],
                    (int32_t)k.shape[1], (int32_t)q.shape[2], window, sinks, (float)scale, out.ptr,
                    out.dtype == d_bf16 ? TTS_BF16 : TTS_F32, lse.ptr, ws.ptr, bytes, st.ptr,
                    stream);
  Py_END_ALLOW_THREADS
  return leave(back, status);
}

/* bind((append, decode, window addresses), (bf16, fp32, uint8, e4m3, int32),
 *      (raw_stream, get_device, set_device)) */
static PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long f[3];
  PyObject* d[5];
  PyObject* t[3];
  if (!PyArg_ParseTuple(args, "(KKK)(OOOOO)(OOO)", &f[0], &f[1], &f[2], &d[0], &d[1], &d[2], &d[3],
                        &d[4], &t[0], &t[1], &t[2]))
    return NULL;
  f_append = (append_fn)(uintptr_t)f[0];
  f_decode = (decode_fn)(uintptr_t)f[1];
  f_window = (window_fn)(uintptr_t)f[2];
  PyObject** keep[8] = {&d_bf16, &d_f32, &d_u8, &d_e4m3, &d_i32, &raw_stream, &get_device, &set_device};
  for (int i = 0; i < 8; ++i) {
    PyObject* o = i < 5 ? d[i] : t[i - 5];
    Py_INCREF(o);
    Py_XSETREF(*keep[i], o);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(addresses, dtypes, torch functions)"},
    {"rope_kv_append", (PyCFunction)(void (*)(void))rope_kv_append, METH_FASTCALL, NULL},
    {"attn_decode_paged", (PyCFunction)(void (*)(void))attn_decode_paged, METH_FASTCALL, NULL},
    {"attn_fwd_varlen_window", (PyCFunction)(void (*)(void))attn_fwd_varlen_window, METH_FASTCALL,
     NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", NULL, -1, methods, NULL, NULL,
                                    NULL, NULL};

PyMODINIT_FUNC PyInit__native(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  if (!s_dtype || !s_shape || !s_get_device || !s_is_contiguous || !s_data_ptr || !s_stride ||
      !s_nbytes)
    return NULL;
  return PyModule_Create(&module);
}
