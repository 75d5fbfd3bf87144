/*
 * pycall.h -- what the CPython bindings of the serving operators share: torch's
 * objects handed over by setup(), tensors read through their Python attributes,
 * argument checks, new tensors. (Defined in pycall.c.)
 */
#ifndef QMM_PYCALL_H
#define QMM_PYCALL_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "qmm.h"

extern PyObject *dt_act[3];               /* torch.float32, float16, bfloat16: qmm_dtype order */
extern PyObject *dt_i32, *dt_i64, *dt_u8;

typedef struct {
    void *ptr;
    PyObject *dtype;                      /* borrowed: element types live as long as torch */
    int nd, dev;
    int64_t shape[4], stride[4];
} Ten;

/* The stream of a call: the caller's handle, or the current one of `dev`. New
 * tensors come from the pool of the stream that uses them: one of the current
 * stream's could still be in use there, and a workspace would be handed out
 * again there while the kernels of the other stream run. */
typedef struct {
    void *handle;
    int other;                            /* not the current stream */
} Stream;

int read_tensor(PyObject *o, Ten *t, const char *what);
/* The qmm_dtype of an f32 / f16 / bf16 element type, or -1 with an exception. */
int act_of(PyObject *dtype, const char *what);
/* Kernels launch on the current device: the first tensor has to be there. */
int on_current(const Ten *t, const char *what);
int on(const Ten *t, int dev, const char *what);
int same_shape(const Ten *a, const Ten *b);
int64_t numel(const Ten *t);
/* Reads a contiguous tensor of `dtype` and `n` elements (-1: any) on `dev`. */
int want(PyObject *o, Ten *t, PyObject *dtype, int64_t n, int dev, const char *what);
int stream_of(PyObject *o, int dev, Stream *s);
/* A new contiguous tensor; *ptr its address. */
PyObject *new_tensor(int nd, const int64_t *shape, PyObject *dtype, const Stream *s, void **ptr);
/* Raises for a status other than QMM_OK. */
int failed(int rc, const char *name);
/* A C int, or -1 with an exception. */
int as_int(PyObject *o);
/* Whether a call has its arguments, and setup() was called. */
int nargs_are(Py_ssize_t n, Py_ssize_t want_n, const char *name);

/* pycall_layer.c: the norm and the router */
extern __typeof__(&qrmsnorm) f_qrmsnorm;
extern __typeof__(&qmoe_route) f_qmoe_route;
extern PyMethodDef layer_methods[];

#endif
