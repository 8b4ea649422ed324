/*
 * The argument marshalling of the attention calls and of those for several continuations, for torch tensors
 * and calls whose sizes and strides have been seen before: a decode step's kernels take 4 to 7 us, and checking and unpacking its
 * tensors in Python took as long.  Everything else (the first call of a combination, errors) is
 * attention.py's and branching.py's: a function here returns None for "not seen, or not to my liking",
 * and they then check again and say what is wrong.  Tensors are seen through their Python
 * attributes only.
 *
 * The interpreter lock is let go around the library's call: a launch blocks while the stream's queue is full.
 *
 * Results: None, an int (a libgdn status that is not GDN_OK), or what the call returns.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "gdn.h"

static PyObject *n_shape, *n_stride, *n_dtype, *n_device, *n_get_device, *n_data_ptr, *n_is_contiguous, *n_nbytes;
/* set by bind() */
static PyObject *t_bf16, *t_f32, *t_f64, *t_i32, *f_empty, *f_empty_like, *f_stream, *dense_format, *f_current;
static PyObject *kw_format, *kw_dtype, *kw_dtype_device;
static gdn_status (*c_paged)(const gdn_attn_shape *, const void *, const void *, const void *, const void *,
                             const int32_t *, const int32_t *, const int32_t *, void *, float *, void *, size_t, void *);
static gdn_status (*c_prefix)(const gdn_attn_shape *, const void *, const void *, const void *, const void *,
                              const int32_t *, const int32_t *, const int32_t *, const int32_t *, void *, float *,
                              void *, size_t, void *);
static gdn_status (*c_append)(const gdn_attn_shape *, const void *, const void *, const void *, const float *,
                              const float *, float, const double *, const int32_t *, const int32_t *, const int32_t *,
                              const int32_t *, const int32_t *, void *, void *, void *, void *);
static gdn_status (*c_tree)(const gdn_attn_shape *, const void *, const void *, const void *, const void *,
                            const int32_t *, const int32_t *, const int32_t *, const int32_t *, const int32_t *, void *,
                            float *, void *, size_t, void *);
static gdn_status (*c_verify)(const gdn_shape *, const void *, const void *, const void *, const float *, const float *,
                              const float *, const int32_t *, const int32_t *, void *, float *, void *);
static gdn_status (*c_select)(const gdn_beam_shape *, const void *, const float *, const uint8_t *, float *, int32_t *,
                              int32_t *, void *, size_t, void *);
static gdn_status (*c_reorder)(int32_t, int32_t, int32_t, int64_t, const int32_t *, void *, void *);
static gdn_status (*c_norm)(int64_t, int32_t, gdn_dtype, const void *, const void *, const float *, float, void *,
                            void *, float *, int32_t, void *);

/* The helpers return 1 (yes), 0 (no) or -1 (a Python error is set). */

static int has_type(PyObject *t, PyObject *type) {
  PyObject *d = PyObject_GetAttr(t, n_dtype);
  if (!d) return -1;
  const int same = d == type;
  Py_DECREF(d);
  return same;
}
static int on_device(PyObject *t, long device) {
  PyObject *d = PyObject_CallMethodNoArgs(t, n_get_device);
  if (!d) return -1;
  const long v = PyLong_AsLong(d);
  Py_DECREF(d);
  if (v == -1 && PyErr_Occurred()) return -1;
  return v == device;
}
static int is_dense(PyObject *t) {
  PyObject *d = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  if (!d) return -1;
  const int yes = d == Py_True;
  Py_DECREF(d);
  return yes;
}
/* A tensor (None passes with `maybe`) of this type on this device, contiguous where asked. */
static int good(PyObject *t, PyObject *type, long device, int dense, int maybe) {
  int r;
  if (t == Py_None) return maybe;
  if ((r = has_type(t, type)) != 1 || (r = on_device(t, device)) != 1) return r;
  return dense ? is_dense(t) : 1;
}
/* Address of a tensor, 0 for None; the error is told apart by PyErr_Occurred(). */
static uintptr_t address(PyObject *t) {
  if (t == Py_None) return 0;
  PyObject *p = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!p) return 0;
  const unsigned long long v = PyLong_AsUnsignedLongLong(p);
  Py_DECREF(p);
  return (uintptr_t)v;
}
/* The tensor's device, which has to be the current one: the library launches there. */
static int device_of(PyObject *t, long *device) {
  PyObject *d = PyObject_CallMethodNoArgs(t, n_get_device);
  if (!d) return -1;
  *device = PyLong_AsLong(d);
  Py_DECREF(d);
  if (PyErr_Occurred()) return -1;
  if (*device < 0) return 0;
  if (!(d = PyObject_CallNoArgs(f_current))) return -1;
  const long current = PyLong_AsLong(d);
  Py_DECREF(d);
  return PyErr_Occurred() ? -1 : current == *device;
}
static int stream_of(long device, void **stream) {
  PyObject *n = PyLong_FromLong(device), *s = n ? PyObject_CallOneArg(f_stream, n) : NULL;
  Py_XDECREF(n);
  if (!s) return -1;
  *stream = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(s);
  Py_DECREF(s);
  return PyErr_Occurred() ? -1 : 1;
}
/* Key under construction: steals each item; a NULL item spoils it. */
static void put(PyObject *key, Py_ssize_t *at, PyObject *item, int *bad) {
  if (!item) *bad = 1;
  PyTuple_SET_ITEM(key, (*at)++, item);
}
static PyObject *shape_of(PyObject *t) {
  if (t == Py_None) return Py_NewRef(Py_None);
  return PyObject_GetAttr(t, n_shape);
}
static PyObject *strides_of(PyObject *t) { return PyObject_CallMethodNoArgs(t, n_stride); }

/* What attention.py keeps for the key (a borrowed reference), NULL if nothing; takes the key. */
static PyObject *look_up(PyObject *made, PyObject *key, int bad) {
  PyObject *v = bad ? NULL : PyDict_GetItemWithError(made, key);
  Py_DECREF(key);
  return v;
}
/* The gdn_attn_shape of such an entry (struct, pointer, address); a copy, since the entry may go
 * while torch is called. */
static gdn_attn_shape struct_of(PyObject *entry) {
  return *(const gdn_attn_shape *)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(entry, 2));
}
static PyObject *like(PyObject *t) {
  PyObject *args[2] = {t, dense_format};
  return PyObject_Vectorcall(f_empty_like, args, 1, kw_format);
}
/* An output that was given: bf16, contiguous, of q's shape. */
static int output(PyObject *o, PyObject *q, long device) {
  int r = good(o, t_bf16, device, 1, 0);
  if (r != 1) return r;
  PyObject *a = shape_of(o), *b = shape_of(q);
  r = a && b ? PyObject_RichCompareBool(a, b, Py_EQ) : -1;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}
static PyObject *no(int r) {
  if (r < 0) return NULL;
  Py_RETURN_NONE;
}
#define NEED(x)                \
  do {                         \
    const int r_ = (x);        \
    if (r_ != 1) return no(r_); \
  } while (0)

/* A contiguous int32 vector of as many entries as `like` has rows. */
static int one_a_row(PyObject *t, PyObject *like, long device) {
  const int r = good(t, t_i32, device, 1, 0);
  if (r != 1) return r;
  PyObject *a = shape_of(t), *b = shape_of(like);
  int same = a && b && PyTuple_GET_SIZE(a) == 1 && PyTuple_GET_SIZE(b) > 0
                 ? PyObject_RichCompareBool(PyTuple_GET_ITEM(a, 0), PyTuple_GET_ITEM(b, 0), Py_EQ)
                 : a && b ? 0 : -1;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return same;
}

/* attend(made, q, k_cache, v_cache, prefix_table, prefix_len, page_table, kv_lens, cu_seqlens, gate,
 *        scale, o, workspace[, parents]): with parents (not None) gdn_tree_attention */
static PyObject *attend(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 13 && count != 14) return PyErr_Format(PyExc_TypeError, "attend takes 13 or 14 arguments");
  PyObject *up = count == 14 ? a[13] : Py_None;
  PyObject *made = a[0], *q = a[1], *k = a[2], *v = a[3], *prefix = a[4], *prefix_len = a[5], *table = a[6],
           *lens = a[7], *cu = a[8], *gate = a[9], *scale = a[10], *o = a[11], *ws = a[12];
  long device;
  if (ws == Py_None) Py_RETURN_NONE;
  NEED(device_of(q, &device));
  NEED(has_type(q, t_bf16));
  NEED(good(k, t_bf16, device, 0, 0));
  NEED(good(v, t_bf16, device, 0, 0));
  NEED(good(gate, t_bf16, device, 0, 1));
  NEED(good(table, t_i32, device, 1, 0));
  NEED(good(lens, t_i32, device, 1, 0));
  NEED(good(cu, t_i32, device, 1, 1));
  NEED(good(prefix, t_i32, device, 1, 1));
  NEED(on_device(ws, device));
  NEED(is_dense(ws));
  if (up != Py_None) {
    if (cu == Py_None) Py_RETURN_NONE;
    NEED(one_a_row(up, q, device));
  }
  PyObject *key = PyTuple_New(13);
  if (!key) return NULL;
  Py_ssize_t at = 0;
  int bad = 0;
  put(key, &at, shape_of(q), &bad);
  put(key, &at, strides_of(q), &bad);
  put(key, &at, shape_of(k), &bad);
  put(key, &at, strides_of(k), &bad);
  put(key, &at, shape_of(v), &bad);
  put(key, &at, strides_of(v), &bad);
  put(key, &at, shape_of(table), &bad);
  put(key, &at, shape_of(lens), &bad);
  put(key, &at, shape_of(cu), &bad);
  if (gate == Py_None) {
    put(key, &at, Py_NewRef(Py_None), &bad);
  } else {
    PyObject *s = shape_of(gate), *t = s ? strides_of(gate) : NULL, *pair = t ? PyTuple_Pack(2, s, t) : NULL;
    Py_XDECREF(s);
    Py_XDECREF(t);
    put(key, &at, pair, &bad);
  }
  put(key, &at, Py_NewRef(scale), &bad);
  put(key, &at, shape_of(prefix), &bad);
  put(key, &at, Py_NewRef(prefix_len), &bad);
  PyObject *entry = look_up(made, key, bad);
  if (!entry) return no(PyErr_Occurred() ? -1 : 0);
  const gdn_attn_shape s = struct_of(entry);
  if (o != Py_None) NEED(output(o, q, device));
  void *stream;
  NEED(stream_of(device, &stream));
  PyObject *bytes = PyObject_GetAttr(ws, n_nbytes);
  if (!bytes) return NULL;
  const size_t ws_bytes = PyLong_AsSize_t(bytes);
  Py_DECREF(bytes);
  PyObject *out = o == Py_None ? like(q) : Py_NewRef(o);
  if (!out) return NULL;
  const void *pq = (void *)address(q), *pg = (void *)address(gate), *pk = (void *)address(k),
             *pv = (void *)address(v);
  const int32_t *pt = (int32_t *)address(table), *pl = (int32_t *)address(lens), *pc = (int32_t *)address(cu),
                *pp = (int32_t *)address(prefix), *pu = (int32_t *)address(up);
  void *po = (void *)address(out), *pw = (void *)address(ws);
  if (PyErr_Occurred()) {
    Py_DECREF(out);
    return NULL;
  }
  gdn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = up != Py_None     ? c_tree(&s, pq, pg, pk, pv, pp, pt, pl, pc, pu, po, NULL, pw, ws_bytes, stream)
       : prefix == Py_None ? c_paged(&s, pq, pg, pk, pv, pt, pl, pc, po, NULL, pw, ws_bytes, stream)
                           : c_prefix(&s, pq, pg, pk, pv, pp, pt, pl, pc, po, NULL, pw, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  if (st == GDN_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(st);
}

/* A weight vector of `n` float32, or None. */
static int vector(PyObject *t, Py_ssize_t n, long device, int maybe) {
  if (t == Py_None) return maybe;
  const int r = good(t, t_f32, device, 1, 0);
  if (r != 1) return r;
  PyObject *s = shape_of(t);
  if (!s) return -1;
  const int same = PyTuple_GET_SIZE(s) == 1 && PyLong_AsSsize_t(PyTuple_GET_ITEM(s, 0)) == n;
  Py_DECREF(s);
  return same;
}

/* append(made, q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens, positions,
 *        rope_axis, q_norm, k_norm, eps, q_out, prefix_len) */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 17) return PyErr_Format(PyExc_TypeError, "append takes 17 arguments");
  PyObject *made = a[0], *q = a[1], *k = a[2], *v = a[3], *kc = a[4], *vc = a[5], *table = a[6], *lens = a[7],
           *freq = a[8], *cu = a[9], *pos = a[10], *axis = a[11], *qn = a[12], *kn = a[13], *q_out = a[15],
           *prefix_len = a[16];
  const double eps = PyFloat_AsDouble(a[14]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  long device;
  NEED(device_of(q, &device));
  NEED(has_type(q, t_bf16));
  NEED(good(k, t_bf16, device, 0, 0));
  NEED(good(v, t_bf16, device, 0, 0));
  NEED(good(kc, t_bf16, device, 0, 0));
  NEED(good(vc, t_bf16, device, 0, 0));
  NEED(good(table, t_i32, device, 1, 0));
  NEED(good(lens, t_i32, device, 1, 0));
  NEED(good(cu, t_i32, device, 1, 1));
  NEED(good(pos, t_i32, device, 1, 1));
  NEED(good(axis, t_i32, device, 1, 1));
  NEED(good(freq, t_f64, device, 1, 1));
  PyObject *key = PyTuple_New(17);
  if (!key) return NULL;
  Py_ssize_t at = 0;
  int bad = 0;
  PyObject *strided[5] = {q, k, v, kc, vc};
  for (int i = 0; i < 5; ++i) {
    put(key, &at, shape_of(strided[i]), &bad);
    put(key, &at, strides_of(strided[i]), &bad);
  }
  PyObject *plain[6] = {table, lens, freq, cu, pos, axis};
  for (int i = 0; i < 6; ++i) put(key, &at, shape_of(plain[i]), &bad);
  put(key, &at, Py_NewRef(prefix_len), &bad);
  PyObject *entry = look_up(made, key, bad);
  if (!entry) return no(PyErr_Occurred() ? -1 : 0);
  const gdn_attn_shape s = struct_of(entry);
  NEED(vector(qn, s.head_dim, device, 1));
  NEED(vector(kn, s.head_dim, device, 1));
  if (q_out != Py_None) NEED(output(q_out, q, device));
  void *stream;
  NEED(stream_of(device, &stream));
  PyObject *out = q_out == Py_None ? like(q) : Py_NewRef(q_out);
  if (!out) return NULL;
  const void *pq = (void *)address(q), *pk = (void *)address(k), *pv = (void *)address(v);
  const float *pqn = (float *)address(qn), *pkn = (float *)address(kn);
  const double *pf = (double *)address(freq);
  const int32_t *pa = (int32_t *)address(axis), *pp = (int32_t *)address(pos), *pt = (int32_t *)address(table),
                *pl = (int32_t *)address(lens), *pc = (int32_t *)address(cu);
  void *po = (void *)address(out), *pkc = (void *)address(kc), *pvc = (void *)address(vc);
  if (PyErr_Occurred()) {
    Py_DECREF(out);
    return NULL;
  }
  gdn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = c_append(&s, pq, pk, pv, pqn, pkn, (float)eps, pf, pa, pp, pt, pl, pc, po, pkc, pvc, stream);
  Py_END_ALLOW_THREADS
  if (st == GDN_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(st);
}

/* norm(made, x, residual, weight, eps, out, group): all outputs new */
static PyObject *norm(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 7) return PyErr_Format(PyExc_TypeError, "norm takes 7 arguments");
  PyObject *made = a[0], *x = a[1], *residual = a[2], *weight = a[3];
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  long device;
  NEED(device_of(x, &device));
  NEED(is_dense(x));
  PyObject *type = PyObject_GetAttr(x, n_dtype), *shape = type ? shape_of(x) : NULL;
  if (!shape) {
    Py_XDECREF(type);
    return NULL;
  }
  int r = 1;
  if (residual != Py_None) {
    r = good(residual, type, device, 1, 0);
    if (r == 1) {
      PyObject *other = shape_of(residual);
      r = other ? PyObject_RichCompareBool(other, shape, Py_EQ) : -1;
      Py_XDECREF(other);
    }
  }
  PyObject *key = r == 1 ? PyTuple_New(5) : NULL, *entry = NULL;
  if (key) {
    static PyObject *tag;
    if (!tag) tag = PyUnicode_InternFromString("norm");
    Py_ssize_t at = 0;
    int bad = 0;
    put(key, &at, Py_XNewRef(tag), &bad);
    put(key, &at, Py_NewRef(shape), &bad);
    put(key, &at, Py_NewRef(type), &bad);
    put(key, &at, Py_NewRef(a[5]), &bad);
    put(key, &at, Py_NewRef(a[6]), &bad);
    entry = look_up(made, key, bad);  /* (rows, columns, code, output type, shape of the scales) */
  }
  const int same = entry && PyTuple_GET_ITEM(entry, 3) == type;
  Py_DECREF(type);
  Py_DECREF(shape);
  if (!entry) return no(r < 0 || PyErr_Occurred() ? -1 : 0);
  const int64_t rows = PyLong_AsLongLong(PyTuple_GET_ITEM(entry, 0));
  const int32_t cols = (int32_t)PyLong_AsLong(PyTuple_GET_ITEM(entry, 1));
  const gdn_dtype code = (gdn_dtype)PyLong_AsLong(PyTuple_GET_ITEM(entry, 2));
  const int32_t group = (int32_t)PyLong_AsLong(a[6]);
  PyObject *kind = Py_NewRef(PyTuple_GET_ITEM(entry, 3)), *scales = Py_NewRef(PyTuple_GET_ITEM(entry, 4));
  PyObject *h = NULL, *y = NULL, *scale = NULL, *result = NULL;
  void *stream;
  if ((r = vector(weight, cols, device, 0)) != 1 || (r = stream_of(device, &stream)) != 1) {
    result = no(r);
    goto end;
  }
  if (residual != Py_None && !(h = PyObject_CallOneArg(f_empty_like, x))) goto end;
  if (same) {
    y = PyObject_CallOneArg(f_empty_like, x);
  } else {
    PyObject *args[2] = {x, kind};
    y = PyObject_Vectorcall(f_empty_like, args, 1, kw_dtype);
  }
  if (!y) goto end;
  if (scales != Py_None) {
    PyObject *where = PyObject_GetAttr(x, n_device);
    if (!where) goto end;
    PyObject *args[3] = {scales, t_f32, where};
    scale = PyObject_Vectorcall(f_empty, args, 1, kw_dtype_device);
    Py_DECREF(where);
    if (!scale) goto end;
  }
  {
    const void *px = (void *)address(x), *pr = (void *)address(residual);
    const float *pw = (float *)address(weight);
    void *ph = h ? (void *)address(h) : NULL, *py = (void *)address(y);
    float *ps = scale ? (float *)address(scale) : NULL;
    if (PyErr_Occurred()) goto end;
    gdn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = c_norm(rows, cols, code, px, pr, pw, (float)eps, ph, py, ps, group, stream);
    Py_END_ALLOW_THREADS
    if (st != GDN_OK) result = PyLong_FromLong(st);
    else if (scale) result = PyTuple_Pack(3, y, scale, h ? h : x);
    else result = PyTuple_Pack(2, y, h ? h : x);
  }
end:
  Py_DECREF(kind);
  Py_DECREF(scales);
  Py_XDECREF(h);
  Py_XDECREF(y);
  Py_XDECREF(scale);
  return result;
}

/* Shape and type of a tensor, twice None for None. */
static void put_kind(PyObject *key, Py_ssize_t *at, PyObject *t, int *bad) {
  put(key, at, shape_of(t), bad);
  put(key, at, t == Py_None ? Py_NewRef(Py_None) : PyObject_GetAttr(t, n_dtype), bad);
}
/* A contiguous tensor on this device (None passes with `maybe`); its type is in the key. */
static int lies(PyObject *t, long device, int maybe) {
  if (t == Py_None) return maybe;
  const int r = on_device(t, device);
  return r == 1 ? is_dense(t) : r;
}
static PyObject *like_in(PyObject *t, PyObject *type) {
  PyObject *args[2] = {t, type};
  return PyObject_Vectorcall(f_empty_like, args, 1, kw_dtype);
}

/* verify(made, q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta, chunk) */
static PyObject *verify(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 12) return PyErr_Format(PyExc_TypeError, "verify takes 12 arguments");
  static PyObject *tag;
  if (!tag && !(tag = PyUnicode_InternFromString("verify"))) return NULL;
  long device;
  NEED(device_of(a[1], &device));
  for (int i = 1; i < 11; ++i) NEED(lies(a[i], device, i == 6 || i == 9 || i == 10));
  PyObject *key = PyTuple_New(22);
  if (!key) return NULL;
  Py_ssize_t at = 0;
  int bad = 0;
  put(key, &at, Py_NewRef(tag), &bad);
  for (int i = 1; i < 11; ++i) put_kind(key, &at, a[i], &bad);
  put(key, &at, Py_NewRef(a[11]), &bad);
  PyObject *entry = look_up(a[0], key, bad);
  if (!entry) return no(PyErr_Occurred() ? -1 : 0);
  const gdn_shape s = *(const gdn_shape *)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(entry, 2));
  void *stream;
  NEED(stream_of(device, &stream));
  PyObject *o = a[9] == Py_None ? PyObject_CallOneArg(f_empty_like, a[3]) : Py_NewRef(a[9]);
  PyObject *delta = !o ? NULL : a[10] == Py_None ? like_in(a[3], t_f32) : Py_NewRef(a[10]), *result = NULL;
  if (delta) {
    const void *p[8];
    for (int i = 0; i < 8; ++i) p[i] = (void *)address(a[1 + i]);
    void *po = (void *)address(o), *pd = (void *)address(delta);
    if (!PyErr_Occurred()) {
      gdn_status st;
      Py_BEGIN_ALLOW_THREADS
      st = c_verify(&s, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], po, pd, stream);
      Py_END_ALLOW_THREADS
      result = st == GDN_OK ? PyTuple_Pack(2, o, delta) : PyLong_FromLong(st);
    }
  }
  Py_XDECREF(o);
  Py_XDECREF(delta);
  return result;
}

/* select(made, logits, scores, top, finished, pad_token, workspace): all outputs new */
static PyObject *select_best(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 7) return PyErr_Format(PyExc_TypeError, "select takes 7 arguments");
  PyObject *made = a[0], *logits = a[1], *scores = a[2], *finished = a[4], *ws = a[6];
  static PyObject *tag;
  if (!tag && !(tag = PyUnicode_InternFromString("select"))) return NULL;
  long device;
  if (ws == Py_None) Py_RETURN_NONE;
  NEED(device_of(logits, &device));
  NEED(lies(scores, device, 0));
  NEED(lies(finished, device, 1));
  NEED(lies(ws, device, 0));
  PyObject *key = PyTuple_New(10);
  if (!key) return NULL;
  Py_ssize_t at = 0;
  int bad = 0;
  put(key, &at, Py_NewRef(tag), &bad);
  put(key, &at, shape_of(logits), &bad);
  put(key, &at, strides_of(logits), &bad);
  put(key, &at, PyObject_GetAttr(logits, n_dtype), &bad);
  put_kind(key, &at, scores, &bad);
  put_kind(key, &at, finished, &bad);
  put(key, &at, Py_NewRef(a[3]), &bad);
  put(key, &at, Py_NewRef(a[5]), &bad);
  PyObject *entry = look_up(made, key, bad);
  if (!entry) return no(PyErr_Occurred() ? -1 : 0);
  const gdn_beam_shape s = *(const gdn_beam_shape *)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(entry, 2));
  PyObject *shape = Py_NewRef(PyTuple_GET_ITEM(entry, 3));
  PyObject *out[3] = {NULL, NULL, NULL}, *result = NULL, *where = NULL, *bytes = NULL;
  void *stream;
  const int r = stream_of(device, &stream);
  if (r != 1) {
    result = no(r);
    goto end;
  }
  if (!(where = PyObject_GetAttr(logits, n_device)) || !(bytes = PyObject_GetAttr(ws, n_nbytes))) goto end;
  for (int i = 0; i < 3; ++i) {
    PyObject *args[3] = {shape, i ? t_i32 : t_f32, where};
    if (!(out[i] = PyObject_Vectorcall(f_empty, args, 1, kw_dtype_device))) goto end;
  }
  {
    const void *px = (void *)address(logits);
    const float *ps = (float *)address(scores);
    const uint8_t *pf = (uint8_t *)address(finished);
    void *po = (void *)address(out[0]), *pu = (void *)address(out[1]), *pt = (void *)address(out[2]),
         *pw = (void *)address(ws);
    const size_t ws_bytes = PyLong_AsSize_t(bytes);
    if (PyErr_Occurred()) goto end;
    gdn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = c_select(&s, px, ps, pf, (float *)po, (int32_t *)pu, (int32_t *)pt, pw, ws_bytes, stream);
    Py_END_ALLOW_THREADS
    result = st == GDN_OK ? PyTuple_Pack(3, out[0], out[1], out[2]) : PyLong_FromLong(st);
  }
end:
  for (int i = 0; i < 3; ++i) Py_XDECREF(out[i]);
  Py_DECREF(shape);
  Py_XDECREF(where);
  Py_XDECREF(bytes);
  return result;
}

/* reorder(made, rows, parents) */
static PyObject *reorder(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 3) return PyErr_Format(PyExc_TypeError, "reorder takes 3 arguments");
  PyObject *rows = a[1], *up = a[2];
  static PyObject *tag;
  if (!tag && !(tag = PyUnicode_InternFromString("reorder"))) return NULL;
  long device;
  NEED(device_of(rows, &device));
  NEED(is_dense(rows));
  NEED(lies(up, device, 0));
  PyObject *key = PyTuple_New(5);
  if (!key) return NULL;
  Py_ssize_t at = 0;
  int bad = 0;
  put(key, &at, Py_NewRef(tag), &bad);
  put_kind(key, &at, rows, &bad);
  put_kind(key, &at, up, &bad);
  PyObject *entry = look_up(a[0], key, bad); /* (layers, groups, beams, bytes of a row) */
  if (!entry) return no(PyErr_Occurred() ? -1 : 0);
  const int32_t layers = (int32_t)PyLong_AsLong(PyTuple_GET_ITEM(entry, 0)),
                groups = (int32_t)PyLong_AsLong(PyTuple_GET_ITEM(entry, 1)),
                beams = (int32_t)PyLong_AsLong(PyTuple_GET_ITEM(entry, 2));
  const int64_t row_bytes = PyLong_AsLongLong(PyTuple_GET_ITEM(entry, 3));
  void *stream;
  NEED(stream_of(device, &stream));
  void *pr = (void *)address(rows);
  const int32_t *pu = (int32_t *)address(up);
  if (PyErr_Occurred()) return NULL;
  gdn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = c_reorder(layers, groups, beams, row_bytes, pu, pr, stream);
  Py_END_ALLOW_THREADS
  return st == GDN_OK ? Py_NewRef(rows) : PyLong_FromLong(st);
}

/* bind(bfloat16, float32, float64, int32, empty, empty_like, raw_stream, contiguous_format,
 *      current_device, gdn_paged_attention, gdn_shared_prefix_attention, gdn_kv_append, gdn_add_rmsnorm,
 *      gdn_tree_attention, gdn_verify_tree, gdn_beam_select, gdn_beam_reorder) */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t count) {
  (void)self;
  if (count != 17) return PyErr_Format(PyExc_TypeError, "bind takes 17 arguments");
  PyObject **to[9] = {&t_bf16, &t_f32, &t_f64, &t_i32, &f_empty, &f_empty_like, &f_stream, &dense_format, &f_current};
  for (int i = 0; i < 9; ++i) Py_XSETREF(*to[i], Py_NewRef(a[i]));
  uintptr_t f[8];
  for (int i = 0; i < 8; ++i) f[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[9 + i]);
  if (PyErr_Occurred()) return NULL;
  *(uintptr_t *)&c_paged = f[0];
  *(uintptr_t *)&c_prefix = f[1];
  *(uintptr_t *)&c_append = f[2];
  *(uintptr_t *)&c_norm = f[3];
  *(uintptr_t *)&c_tree = f[4];
  *(uintptr_t *)&c_verify = f[5];
  *(uintptr_t *)&c_select = f[6];
  *(uintptr_t *)&c_reorder = f[7];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, NULL},
    {"verify", (PyCFunction)(void (*)(void))verify, METH_FASTCALL, NULL},
    {"select", (PyCFunction)(void (*)(void))select_best, METH_FASTCALL, NULL},
    {"reorder", (PyCFunction)(void (*)(void))reorder, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject **to[8] = {&n_shape, &n_stride, &n_dtype, &n_device, &n_get_device, &n_data_ptr, &n_is_contiguous, &n_nbytes};
  static const char *names[8] = {"shape", "stride", "dtype", "device", "get_device", "data_ptr", "is_contiguous", "nbytes"};
  for (int i = 0; i < 8; ++i)
    if (!(*to[i] = PyUnicode_InternFromString(names[i]))) return NULL;
  kw_format = Py_BuildValue("(s)", "memory_format");
  kw_dtype = Py_BuildValue("(s)", "dtype");
  kw_dtype_device = Py_BuildValue("(ss)", "dtype", "device");
  if (!kw_format || !kw_dtype || !kw_dtype_device) return NULL;
  return PyModule_Create(&module);
}
