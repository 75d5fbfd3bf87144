/*
 * pycall_layer.c -- CPython bindings of the norm and the router (include/qmm.h).
 */
#include "pycall.h"

__typeof__(&qrmsnorm) f_qrmsnorm;
__typeof__(&qmoe_route) f_qmoe_route;

/* (tokens, dim) or (tokens, heads, dim) with a contiguous last dimension as
 * tokens, heads and dim; *n elements reachable */
typedef struct {
    int64_t T, H, D, ts, hs;
    size_t n;
} Dims;

static int dims_of(const Ten *t, Dims *d, const char *what) {
    if (t->nd != 2 && t->nd != 3) {
        PyErr_Format(PyExc_ValueError, "%s must have two or three dimensions (tokens, heads, dim), got %d", what, t->nd);
        return -1;
    }
    const int last = t->nd - 1;
    d->T = t->shape[0];
    d->ts = t->stride[0];
    d->H = last == 2 ? t->shape[1] : 1;
    d->hs = last == 2 ? t->stride[1] : 0;
    d->D = t->shape[last];
    if (d->D > 1 && t->stride[last] != 1) {
        PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", what);
        return -1;
    }
    d->n = d->T && d->H && d->D ? (size_t)((d->T - 1) * d->ts + (d->H - 1) * d->hs + d->D) : 0;
    return 0;
}

static int read_rows(PyObject *o, Ten *t, Dims *d, int dev, const char *what) {
    return read_tensor(o, t, what) || on(t, dev, what) || dims_of(t, d, what) ? -1 : 0;
}

/* (X, weight or None, eps, residual or None, residual_out or None, out or None, element type, or True for Q8_0 rows,
   weight_offset, stream or None) */
static PyObject *py_qrmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten x, w, r, ro, y;
    Dims xd, rd = {0}, od = {0}, yd;
    Stream stream;
    (void)self;
    if (!nargs_are(n, 9, "qrmsnorm") || read_tensor(a[0], &x, "X")) return NULL;
    const int xt = act_of(x.dtype, "X");
    if (xt < 0 || dims_of(&x, &xd, "X") || on_current(&x, "X")) return NULL;
    const int weighted = a[1] != Py_None, res = a[3] != Py_None, given = a[5] != Py_None, q8 = a[6] == Py_True;
    if (weighted && want(a[1], &w, dt_act[0], xd.D, x.dev, "weight")) return NULL;
    const float eps = (float)PyFloat_AsDouble(a[2]), offset = (float)PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return NULL;
    int rt = 0;
    if (res) {
        if (read_rows(a[3], &r, &rd, x.dev, "residual") || (rt = act_of(r.dtype, "residual")) < 0) return NULL;
        if (!same_shape(&r, &x)) {
            PyErr_SetString(PyExc_ValueError, "residual must have X's shape");
            return NULL;
        }
        ro = r;                           /* in place unless there is another */
        od = rd;
        if (a[4] != Py_None) {
            if (read_rows(a[4], &ro, &od, x.dev, "residual_out")) return NULL;
            if (!same_shape(&ro, &x) || ro.dtype != r.dtype) {
                PyErr_SetString(PyExc_ValueError, "residual_out must have residual's shape and type");
                return NULL;
            }
        }
    } else if (a[4] != Py_None) {
        PyErr_SetString(PyExc_ValueError, "residual_out goes with residual");
        return NULL;
    }
    PyObject *type = q8 ? dt_u8 : a[6];
    int yt = QMM_NORM_Q8_0;
    if (!q8 && (yt = act_of(type, "out_dtype")) < 0) return NULL;
    if (stream_of(a[8], x.dev, &stream)) return NULL;
    int64_t shape[3] = {x.shape[0], x.nd == 3 ? x.shape[1] : 0, 0};
    shape[x.nd - 1] = q8 ? xd.D / 32 * 34 : xd.D;
    PyObject *out = a[5];
    if (given) {
        if (read_rows(out, &y, &yd, x.dev, "out")) return NULL;
        int same = y.dtype == type && y.nd == x.nd;
        for (int i = 0; same && i < x.nd; ++i) same = y.shape[i] == shape[i];
        if (!same) {
            PyErr_SetString(PyExc_ValueError, q8 ? "out must be a uint8 tensor of X's rows, 34 bytes for each 32 elements"
                                                 : "out must have X's shape and the output type");
            return NULL;
        }
        Py_INCREF(out);
    } else {
        out = new_tensor(x.nd, shape, type, &stream, &y.ptr);
        if (!out) return NULL;
        yd = xd;
        yd.D = shape[x.nd - 1];
        yd.hs = yd.D;
        yd.ts = yd.H * yd.D;
        yd.n = (size_t)(yd.T * yd.ts);
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qrmsnorm(x.ptr, xt, xd.n, xd.ts, xd.hs, res ? r.ptr : NULL, rt, rd.n, rd.ts, rd.hs, res ? ro.ptr : NULL, od.n, od.ts, od.hs,
                    weighted ? w.ptr : NULL, weighted ? (size_t)xd.D : 0, offset, eps, y.ptr, yt, yd.n, yd.ts, yd.hs, xd.T, xd.H,
                    xd.D, stream.handle);
    Py_END_ALLOW_THREADS
    if (failed(rc, "qrmsnorm")) Py_CLEAR(out);
    return out;
}

/* (logits, top_k, score, bias or None, groups, top_groups, group_top, renorm, scale, ids or None, weights or None, stream or None) */
static PyObject *py_qmoe_route(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Ten x, b, it, wt;
    Dims d;
    Stream stream;
    (void)self;
    if (!nargs_are(n, 12, "qmoe_route") || read_tensor(a[0], &x, "logits")) return NULL;
    const int dt = act_of(x.dtype, "logits");
    if (dt < 0 || dims_of(&x, &d, "logits") || on_current(&x, "logits")) return NULL;
    if (x.nd != 2 || d.D > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "logits must be (tokens, experts)");
        return NULL;
    }
    const int biased = a[3] != Py_None;
    if (biased && want(a[3], &b, dt_act[0], d.D, x.dev, "bias")) return NULL;
    const int k = as_int(a[1]), score = as_int(a[2]), groups = as_int(a[4]), top_groups = as_int(a[5]), group_top = as_int(a[6]);
    const int renorm = PyObject_IsTrue(a[7]);
    const float scale = (float)PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred() || stream_of(a[11], x.dev, &stream)) return NULL;
    if (k < 0 || k > (1 << 20)) {
        PyErr_SetString(PyExc_ValueError, "top_k out of range");
        return NULL;
    }
    const int64_t shape[2] = {d.T, k};
    PyObject *ids = NULL, *weights = NULL, *r = NULL;
    if (a[9] == Py_None) {
        if (!(ids = new_tensor(2, shape, dt_i32, &stream, &it.ptr))) goto done;
    } else {
        if (want(a[9], &it, dt_i32, d.T * k, x.dev, "ids")) goto done;
        ids = a[9];
        Py_INCREF(ids);
    }
    if (a[10] == Py_None) {
        if (!(weights = new_tensor(2, shape, dt_act[0], &stream, &wt.ptr))) goto done;
    } else {
        if (want(a[10], &wt, dt_act[0], d.T * k, x.dev, "weights")) goto done;
        weights = a[10];
        Py_INCREF(weights);
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f_qmoe_route(x.ptr, dt, d.n, d.ts, biased ? b.ptr : NULL, score, groups, top_groups, group_top, k, renorm, scale, it.ptr,
                      wt.ptr, (size_t)(d.T * k), d.T, (int)d.D, stream.handle);
    Py_END_ALLOW_THREADS
    if (!failed(rc, "qmoe_route")) r = PyTuple_Pack(2, ids, weights);
done:
    Py_XDECREF(ids);
    Py_XDECREF(weights);
    return r;
}

PyMethodDef layer_methods[] = {
    {"qrmsnorm", (PyCFunction)(void (*)(void))py_qrmsnorm, METH_FASTCALL, NULL},
    {"qmoe_route", (PyCFunction)(void (*)(void))py_qmoe_route, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
