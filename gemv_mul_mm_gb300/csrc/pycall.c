/*
 * pycall.c -- CPython bindings of the rotary, cache and attention operators
 * (include/qmm.h), used by qmm.py, and what those of pycall_layer.c share with them.
 *
 * A call on a decode step costs more on the host than on the GPU: through
 * ctypes and Python-level checks qrope took 7.6 us and qattn_decode 15 us, of
 * which the launches are 2 and 4. Here the tensors' attributes are read, checked
 * and passed on from C. Nothing of torch is compiled in: tensors are read
 * through their Python attributes, and what else is needed of torch (element
 * types, the current stream, an allocator) is handed over once by setup().
 */
#include "pycall.h"

/* ---- what setup() hands over */

static __typeof__(&qrope) f_qrope;
static __typeof__(&qkv_store) f_qkv_store;
static __typeof__(&qkv_load) f_qkv_load;
static __typeof__(&qattn_decode) f_qattn_decode;
static __typeof__(&qattn_decode_workspace_bytes) f_ws_bytes;
static __typeof__(&qattn_decode_splits) f_splits;

PyObject *dt_act[3], *dt_i32, *dt_i64, *dt_u8;
static PyObject *fn_stream;               /* device index -> raw stream */
static PyObject *fn_device;               /* () -> current device index */
static PyObject *fn_new;                  /* (shape, strides, dtype) -> tensor on the current device and stream */
static PyObject *fn_new_on;               /* (shape, strides, dtype, stream) -> tensor of that stream */
static PyObject *fn_check;                /* (status, name) -> raises */
static PyObject *s_data_ptr, *s_shape, *s_stride, *s_dtype, *s_get_device;

static int set_ref(PyObject **to, PyObject *o) {
    Py_INCREF(o);
    Py_XSETREF(*to, o);
    return 0;
}

static PyObject *setup(PyObject *self, PyObject *args) {
    unsigned long long a[8];
    PyObject *o[11];
    (void)self;
    if (!PyArg_ParseTuple(args, "(KKKKKKKK)(OOO)OOOOOOOO", &a[0], &a[1], &a[2], &a[3], &a[4], &a[5], &a[6], &a[7], &o[0], &o[1], &o[2], &o[3],
                          &o[4], &o[5], &o[6], &o[7], &o[8], &o[9], &o[10]))
        return NULL;
    f_qrope = (__typeof__(f_qrope))(uintptr_t)a[0];
    f_qkv_store = (__typeof__(f_qkv_store))(uintptr_t)a[1];
    f_qkv_load = (__typeof__(f_qkv_load))(uintptr_t)a[2];
    f_qattn_decode = (__typeof__(f_qattn_decode))(uintptr_t)a[3];
    f_ws_bytes = (__typeof__(f_ws_bytes))(uintptr_t)a[4];
    f_splits = (__typeof__(f_splits))(uintptr_t)a[5];
    f_qrmsnorm = (__typeof__(f_qrmsnorm))(uintptr_t)a[6];
    f_qmoe_route = (__typeof__(f_qmoe_route))(uintptr_t)a[7];
    for (int i = 0; i < 3; ++i) set_ref(&dt_act[i], o[i]);
    set_ref(&dt_i32, o[3]);
    set_ref(&dt_i64, o[4]);
    set_ref(&dt_u8, o[5]);
    set_ref(&fn_stream, o[6]);
    set_ref(&fn_device, o[7]);
    set_ref(&fn_new, o[8]);
    set_ref(&fn_new_on, o[9]);
    set_ref(&fn_check, o[10]);
    Py_RETURN_NONE;
}

/* ---- tensors */

/* A Python int from a call, or -1 with an exception. */
static int64_t as_i64(PyObject *o) {
    if (!o) return -1;
    const int64_t v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return v;
}

static int read_dims(PyObject *t, int64_t *to, const char *what) {
    int n = -1;
    if (t && PyTuple_Check(t) && PyTuple_GET_SIZE(t) <= 4) {
        n = (int)PyTuple_GET_SIZE(t);
        for (int i = 0; i < n; ++i) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    } else if (t) {
        PyErr_Format(PyExc_ValueError, "%s must be a tensor of at most four dimensions", what);
    }
    Py_XDECREF(t);
    return PyErr_Occurred() ? -1 : n;
}

int read_tensor(PyObject *o, Ten *t, const char *what) {
    PyObject *p = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!p) {
        if (PyErr_ExceptionMatches(PyExc_AttributeError)) PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return -1;
    }
    t->ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    t->nd = read_dims(PyObject_GetAttr(o, s_shape), t->shape, what);
    if (t->nd < 0 || read_dims(PyObject_CallMethodNoArgs(o, s_stride), t->stride, what) < 0) return -1;
    t->dtype = PyObject_GetAttr(o, s_dtype);
    if (!t->dtype) return -1;
    Py_DECREF(t->dtype);
    t->dev = (int)as_i64(PyObject_CallMethodNoArgs(o, s_get_device));
    return PyErr_Occurred() ? -1 : 0;
}

int act_of(PyObject *dtype, const char *what) {
    for (int i = 0; i < 3; ++i)
        if (dtype == dt_act[i]) return i;
    PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16, got %R", what, dtype);
    return -1;
}

int on_current(const Ten *t, const char *what) {
    if (t->dev < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", what);
        return -1;
    }
    const int64_t now = as_i64(PyObject_CallNoArgs(fn_device));
    if (PyErr_Occurred()) return -1;
    if (now != t->dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, which is not the current device", what, t->dev);
        return -1;
    }
    return 0;
}

int on(const Ten *t, int dev, const char *what) {
    if (t->dev == dev) return 0;
    PyErr_Format(PyExc_ValueError, "%s is on device %d, not on cuda:%d", what, t->dev, dev);
    return -1;
}

/* (tokens, heads, dim) with a contiguous last dimension; *n elements reachable */
static int rows_of(const Ten *t, const char *what, size_t *n) {
    if (t->nd != 3) {
        PyErr_Format(PyExc_ValueError, "%s must have three dimensions (tokens, heads, dim), got %d", what, t->nd);
        return -1;
    }
    if (t->shape[2] > 1 && t->stride[2] != 1) {
        PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", what);
        return -1;
    }
    *n = t->shape[0] && t->shape[1] && t->shape[2]
             ? (size_t)((t->shape[0] - 1) * t->stride[0] + (t->shape[1] - 1) * t->stride[1] + t->shape[2])
             : 0;
    return 0;
}

int same_shape(const Ten *a, const Ten *b) {
    if (a->nd != b->nd) return 0;
    for (int i = 0; i < a->nd; ++i)
        if (a->shape[i] != b->shape[i]) return 0;
    return 1;
}

int64_t numel(const Ten *t) {
    int64_t n = 1;
    for (int i = 0; i < t->nd; ++i) n *= t->shape[i];
    return n;
}

static int contiguous(const Ten *t) {
    int64_t want = 1;
    for (int i = t->nd - 1; i >= 0; --i) {
        if (t->shape[i] == 0) return 1;
        if (t->shape[i] != 1) {
            if (t->stride[i] != want) return 0;
            want *= t->shape[i];
        }
    }
    return 1;
}

int want(PyObject *o, Ten *t, PyObject *dtype, int64_t n, int dev, const char *what) {
    if (read_tensor(o, t, what)) return -1;
    if (t->dtype != dtype || !contiguous(t) || (n >= 0 && numel(t) != n)) {
        if (n >= 0) PyErr_Format(PyExc_ValueError, "%s must be a contiguous %R tensor of %lld elements", what, dtype, (long long)n);
        else PyErr_Format(PyExc_ValueError, "%s must be a contiguous %R tensor", what, dtype);
        return -1;
    }
    return on(t, dev, what);
}

/* A cache given as two (pages, bytes per page) uint8 tensors. */
typedef struct {
    void *k, *v;
    int64_t pages, stride;
    size_t bytes;
    int dev;
} Cache;

static int read_cache(PyObject *ko, PyObject *vo, Cache *c) {
    Ten k, v;
    if (read_tensor(ko, &k, "k_cache") || read_tensor(vo, &v, "v_cache")) return -1;
    if (k.nd != 2 || k.dtype != dt_u8 || (k.shape[1] > 1 && k.stride[1] != 1)) {
        PyErr_SetString(PyExc_ValueError, "k_cache must be a (pages, bytes per page) uint8 tensor with contiguous pages");
        return -1;
    }
    if (!same_shape(&k, &v) || v.dtype != dt_u8 || v.stride[0] != k.stride[0] || v.stride[1] != k.stride[1] || v.dev != k.dev) {
        PyErr_SetString(PyExc_ValueError, "v_cache must have k_cache's shape, strides, type and device");
        return -1;
    }
    c->k = k.ptr;
    c->v = v.ptr;
    c->dev = k.dev;
    c->pages = k.shape[0];
    c->stride = k.shape[0] > 1 ? k.stride[0] : k.shape[1];   /* one page alone has no stride to speak of */
    c->bytes = k.shape[0] ? (size_t)((k.shape[0] - 1) * c->stride + k.shape[1]) : 0;
    return 0;
}

int stream_of(PyObject *o, int dev, Stream *s) {
    PyObject *d = PyLong_FromLong(dev);
    if (!d) return -1;
    PyObject *r = PyObject_CallOneArg(fn_stream, d);
    Py_DECREF(d);
    if (!r) return -1;
    s->handle = PyLong_AsVoidPtr(r);
    s->other = 0;
    Py_DECREF(r);
    if (o != Py_None && !PyErr_Occurred()) {
        r = PyNumber_Long(o);
        if (!r) return -1;
        void *given = PyLong_AsVoidPtr(r);
        Py_DECREF(r);
        s->other = given != s->handle;
        s->handle = given;
    }
    return PyErr_Occurred() ? -1 : 0;
}

PyObject *new_tensor(int nd, const int64_t *shape, PyObject *dtype, const Stream *s, void **ptr) {
    PyObject *sh = PyTuple_New(nd), *st = PyTuple_New(nd), *t = NULL, *p;
    int64_t n = 1;
    if (!sh || !st) goto out;
    for (int i = nd - 1; i >= 0; --i) {
        PyObject *a = PyLong_FromLongLong(shape[i]), *b = PyLong_FromLongLong(n);
        if (!a || !b) {
            Py_XDECREF(a);
            Py_XDECREF(b);
            goto out;
        }
        PyTuple_SET_ITEM(sh, i, a);
        PyTuple_SET_ITEM(st, i, b);
        n *= shape[i] > 1 ? shape[i] : 1;
    }
    if (s->other) {
        t = PyObject_CallFunction(fn_new_on, "OOOK", sh, st, dtype, (unsigned long long)(uintptr_t)s->handle);
    } else {
        PyObject *args[3] = {sh, st, dtype};
        t = PyObject_Vectorcall(fn_new, args, 3, NULL);
    }
    if (t) {
        p = PyObject_CallMethodNoArgs(t, s_data_ptr);
        if (p) {
            *ptr = PyLong_AsVoidPtr(p);
            Py_DECREF(p);
        } else {
            Py_CLEAR(t);
        }
    }
out:
    Py_XDECREF(sh);
    Py_XDECREF(st);
    return t;
}

int failed(int rc, const char *name) {
    if (rc == QMM_OK) return 0;
    PyObject *r = PyObject_CallFunction(fn_check, "is", rc, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, rc);
    return 1;
}

int as_int(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
        return -1;
    }
    return (int)v;
}

int nargs_are(Py_ssize_t n, Py_ssize_t want_n, const char *name) {
    if (n == want_n && f_qrope) return 1;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, or setup() not called", name, n);
    return 0;
}

/* Reads a table of qrope_turns. */
static int want_turns(PyObject *o, Ten *t, int dev) {
    if (want(o, t, dt_i64, -1, dev, "turns")) return -1;
    if (numel(t) <= INT32_MAX / 2) return 0;
    PyErr_SetString(PyExc_ValueError, "turns has too many elements");
    return -1;
}

/* ---- the operators */

/* (X, positions, turns, layout, mscale, out or None, stream or None) */
static PyObject *py_qrope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten x, pos, turns, y;
    size_t xn, yn;
    Stream stream;
    (void)self;
    if (!nargs_are(n, 7, "qrope") || read_tensor(a[0], &x, "X")) return NULL;
    PyObject *out = a[5];
    const int dt = act_of(x.dtype, "X");
    if (dt < 0 || rows_of(&x, "X", &xn) || on_current(&x, "X") ||
        want(a[1], &pos, dt_i32, x.shape[0], x.dev, "positions") || want_turns(a[2], &turns, x.dev))
        return NULL;
    const int layout = as_int(a[3]);
    const float mscale = (float)PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred() || stream_of(a[6], x.dev, &stream)) return NULL;
    if (out == Py_None) {
        out = new_tensor(3, x.shape, x.dtype, &stream, &y.ptr);
        if (!out) return NULL;
        yn = (size_t)numel(&x);
        y.stride[0] = x.shape[1] * x.shape[2];
        y.stride[1] = x.shape[2];
    } else {
        if (read_tensor(out, &y, "out")) return NULL;
        if (!same_shape(&x, &y) || y.dtype != x.dtype) {
            PyErr_SetString(PyExc_ValueError, "out must have X's shape and type");
            return NULL;
        }
        if (on(&y, x.dev, "out") || rows_of(&y, "out", &yn)) return NULL;
        Py_INCREF(out);
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qrope(x.ptr, dt, xn, x.stride[0], x.stride[1], pos.ptr, turns.ptr, (int)(2 * numel(&turns)), layout, mscale, y.ptr, yn,
                 y.stride[0], y.stride[1], x.shape[0], x.shape[1], x.shape[2], stream.handle);
    Py_END_ALLOW_THREADS
    if (failed(rc, "qrope")) Py_CLEAR(out);
    return out;
}

/* (fmt, K, V, slots, k_cache, v_cache, page_size, positions or None, turns or None, layout, mscale, stream or None) */
static PyObject *py_qkv_store(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten k, v, slots, pos, turns;
    Cache c;
    size_t kn, vn;
    Stream stream;
    (void)self;
    if (!nargs_are(n, 12, "qkv_store") || read_tensor(a[1], &k, "K") || read_tensor(a[2], &v, "V")) return NULL;
    const int dt = act_of(k.dtype, "K");
    if (dt < 0) return NULL;
    if (v.dtype != k.dtype || !same_shape(&k, &v)) {
        PyErr_SetString(PyExc_ValueError, "V must have K's shape and type");
        return NULL;
    }
    if (rows_of(&k, "K", &kn) || rows_of(&v, "V", &vn) || on_current(&k, "K") || on(&v, k.dev, "V") ||
        want(a[3], &slots, dt_i64, k.shape[0], k.dev, "slots") || read_cache(a[4], a[5], &c))
        return NULL;
    if (c.dev != k.dev) {
        PyErr_SetString(PyExc_ValueError, "the cache is on another device than K");
        return NULL;
    }
    const int rope = a[7] != Py_None;
    if (rope != (a[8] != Py_None)) {
        PyErr_SetString(PyExc_ValueError, "positions and turns go together");
        return NULL;
    }
    if (rope && (want(a[7], &pos, dt_i32, k.shape[0], k.dev, "positions") || want_turns(a[8], &turns, k.dev)))
        return NULL;
    const int fmt = as_int(a[0]), page = as_int(a[6]), layout = as_int(a[9]);
    const float mscale = (float)PyFloat_AsDouble(a[10]);
    if (PyErr_Occurred() || stream_of(a[11], k.dev, &stream)) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qkv_store(fmt, k.ptr, kn, k.stride[0], k.stride[1], v.ptr, vn, v.stride[0], v.stride[1], dt, slots.ptr,
                     rope ? pos.ptr : NULL, rope ? turns.ptr : NULL, rope ? (int)(2 * numel(&turns)) : 0, layout, mscale, c.k, c.v,
                     c.bytes, c.pages, c.stride, page, k.shape[0], (int)k.shape[1], (int)k.shape[2], stream.handle);
    Py_END_ALLOW_THREADS
    if (failed(rc, "qkv_store")) return NULL;
    Py_RETURN_NONE;
}

/* (fmt, slots, k_cache, v_cache, page_size, n_kv_heads, head_dim, element type or None, stream or None) */
static PyObject *py_qkv_load(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten slots;
    Cache c;
    Stream stream;
    void *kp, *vp;
    (void)self;
    if (!nargs_are(n, 9, "qkv_load") || read_cache(a[2], a[3], &c)) return NULL;
    PyObject *dtype = a[7] == Py_None ? dt_act[0] : a[7];
    const int dt = act_of(dtype, "dtype");
    Ten here = {.dev = c.dev};
    if (dt < 0 || on_current(&here, "k_cache") || want(a[1], &slots, dt_i64, -1, c.dev, "slots")) return NULL;
    const int fmt = as_int(a[0]), page = as_int(a[4]);
    const int64_t shape[3] = {numel(&slots), PyLong_AsLongLong(a[5]), PyLong_AsLongLong(a[6])};
    if (PyErr_Occurred() || stream_of(a[8], c.dev, &stream)) return NULL;
    if (shape[1] < 0 || shape[2] < 0 || shape[1] > (1 << 20) || shape[2] > (1 << 20)) {
        PyErr_SetString(PyExc_ValueError, "n_kv_heads or head_dim out of range");
        return NULL;
    }
    PyObject *k = new_tensor(3, shape, dtype, &stream, &kp), *v = k ? new_tensor(3, shape, dtype, &stream, &vp) : NULL;
    if (!v) {
        Py_XDECREF(k);
        return NULL;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qkv_load(fmt, slots.ptr, c.k, c.v, c.bytes, c.pages, c.stride, page, kp, vp, dt, (size_t)(shape[0] * shape[1] * shape[2]),
                    shape[0], (int)shape[1], (int)shape[2], stream.handle);
    Py_END_ALLOW_THREADS
    PyObject *r = failed(rc, "qkv_load") ? NULL : PyTuple_Pack(2, k, v);
    Py_DECREF(k);
    Py_DECREF(v);
    return r;
}

/* (fmt, q, k_cache, v_cache, block_table, seq_lens, page_size, n_kv_heads, scale or None, window, softcap, max_len or None,
   out or None, return_lse, workspace or None, stream or None) */
static PyObject *py_qattn_decode(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten q, table, lens, t;
    Cache c;
    size_t qn;
    Stream stream;
    void *optr, *lptr = NULL, *wptr = NULL;
    PyObject *out = NULL, *lse = NULL, *ws = NULL, *r = NULL;
    (void)self;
    if (!nargs_are(n, 16, "qattn_decode") || read_tensor(a[1], &q, "q")) return NULL;
    const int dt = act_of(q.dtype, "q");
    if (dt < 0 || rows_of(&q, "q", &qn) || on_current(&q, "q") || read_cache(a[2], a[3], &c) ||
        read_tensor(a[4], &table, "block_table"))
        return NULL;
    const int64_t B = q.shape[0], H = q.shape[1], D = q.shape[2];
    if (c.dev != q.dev) {
        PyErr_SetString(PyExc_ValueError, "the cache is on another device than q");
        return NULL;
    }
    if (table.dtype != dt_i32 || table.nd != 2 || table.shape[0] != B || (table.shape[1] > 1 && table.stride[1] != 1)) {
        PyErr_SetString(PyExc_ValueError, "block_table must be an int32 tensor (sequences, pages) with contiguous rows");
        return NULL;
    }
    if (on(&table, q.dev, "block_table") || want(a[5], &lens, dt_i32, B, q.dev, "seq_lens")) return NULL;
    const int fmt = as_int(a[0]), page = as_int(a[6]), kv = as_int(a[7]);
    const int window = as_int(a[9]);
    const double scale = a[8] == Py_None ? 0.0 : PyFloat_AsDouble(a[8]);
    const float softcap = (float)PyFloat_AsDouble(a[10]);
    const int64_t width = table.shape[1];
    int64_t max_len = a[11] == Py_None ? width * page : PyLong_AsLongLong(a[11]);
    const int with_lse = PyObject_IsTrue(a[13]);
    if (PyErr_Occurred() || stream_of(a[15], q.dev, &stream)) return NULL;
    if (max_len > (1 << 30)) max_len = a[11] == Py_None ? 1 << 30 : INT32_MAX;   /* refused below where the caller asked for it */
    if (max_len < -1) max_len = -1;
    if (H > INT32_MAX || D > INT32_MAX || width > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "q or block_table too large");
        return NULL;
    }
    if (a[12] == Py_None) {
        out = new_tensor(3, q.shape, q.dtype, &stream, &optr);
        if (!out) return NULL;
    } else {
        if (want(a[12], &t, q.dtype, B * H * D, q.dev, "out")) return NULL;
        out = a[12];
        optr = t.ptr;
        Py_INCREF(out);
    }
    if (with_lse && !(lse = new_tensor(2, q.shape, dt_act[0], &stream, &lptr))) goto done;
    int64_t wn = 0;
    if (a[14] == Py_None) {
        if (f_splits(fmt, dt, B, (int)H, kv, (int)D, (int)max_len, window) > 1)
            wn = (int64_t)f_ws_bytes(fmt, dt, B, (int)H, kv, (int)D, (int)max_len, window);
        if (wn && !(ws = new_tensor(1, &wn, dt_u8, &stream, &wptr))) goto done;
    } else {
        if (read_tensor(a[14], &t, "workspace") || on(&t, q.dev, "workspace")) goto done;
        if (t.dtype != dt_u8 || !contiguous(&t)) {
            PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
            goto done;
        }
        wptr = t.ptr;
        wn = numel(&t);
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qattn_decode(fmt, q.ptr, dt, qn, q.stride[0], q.stride[1], c.k, c.v, c.bytes, c.pages, c.stride, page, table.ptr,
                        B ? (size_t)((B - 1) * table.stride[0] + width) : 0, table.stride[0], (int)width, lens.ptr, (int)max_len, B,
                        (int)H, kv, (int)D, a[8] == Py_None ? (float)(1.0 / __builtin_sqrt(D > 0 ? (double)D : 1.0)) : (float)scale,
                        window, softcap, optr, (size_t)(B * H * D), lptr, wptr, (size_t)wn, stream.handle);
    Py_END_ALLOW_THREADS
    if (!failed(rc, "qattn_decode")) {
        if (with_lse) {
            r = PyTuple_Pack(2, out, lse);
        } else {
            Py_INCREF(out);
            r = out;
        }
    }
done:
    Py_XDECREF(out);
    Py_XDECREF(lse);
    Py_XDECREF(ws);
    return r;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Entry points and what is used of torch."},
    {"qrope", (PyCFunction)(void (*)(void))py_qrope, METH_FASTCALL, NULL},
    {"qkv_store", (PyCFunction)(void (*)(void))py_qkv_store, METH_FASTCALL, NULL},
    {"qkv_load", (PyCFunction)(void (*)(void))py_qkv_load, METH_FASTCALL, NULL},
    {"qattn_decode", (PyCFunction)(void (*)(void))py_qattn_decode, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    if (!s_data_ptr || !s_shape || !s_stride || !s_dtype || !s_get_device) return NULL;
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, layer_methods)) Py_CLEAR(m);
    return m;
}
