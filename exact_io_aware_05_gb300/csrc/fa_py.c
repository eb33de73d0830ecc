/*
 * fa_py.c -- CPython module _fa_py: the checks and the calls of the rotary and paged-cache
 * entry points (include/fa.h) without ctypes.
 *
 * These calls take 3 to 15 us on the device, and a serving step makes several: marshalling them in
 * Python and ctypes took 7 to 9 us each on the host, here it takes 3 to 5.  Every function checks its tensors
 * (types, shapes, device, contiguity) and calls the C entry point; it returns the status, or None where a
 * check does not pass or the tensors' device is not current: exact_io_aware_05_gb300/fa.py then goes
 * through its own checks, which say what is wrong, and through ctypes.  No torch headers: tensors
 * are read through their Python attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/fa.h"

typedef int (*rope_fn)(const fa_heads *, const fa_heads *, int, const int *, const fa_rope_spec *, int, int, int, int,
                       fa_stream_t);
typedef int (*append_fn)(const fa_kv_cache *, const fa_heads *, const fa_heads *, const fa_heads *, const fa_heads *,
                         const int *, const fa_rope_spec *, const int *, int, fa_stream_t);
typedef int (*decode_fn)(const fa_kv_cache *, const void *, void *, float *, int, int, int, float, int, void *, size_t,
                         fa_stream_t);
typedef int (*evict_fn)(const fa_kv_cache *, int, int, int, float *, int *, int *, int *, fa_stream_t);

static rope_fn call_rope;
static append_fn call_append;
static decode_fn call_decode;
static evict_fn call_evict;

/* torch's dtypes and two of its functions, and the names of attributes */
static PyObject *t_bf16, *t_f32, *t_i32, *f_stream, *f_device;
static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_stride, *n_nbytes, *n_cuda_stream;

/* A Python integer that is handed over (its reference is taken): 0 and *ok = 0 on any error. */
static long long taken_int(PyObject *x, int *ok)
{
    long long v = 0;
    if (!x || !PyLong_Check(x)) {
        *ok = 0;
    } else {
        v = PyLong_AsLongLong(x);
        if (v == -1 && PyErr_Occurred())
            *ok = 0;
    }
    Py_XDECREF(x);
    return v;
}

static int has_dtype(PyObject *t, PyObject *dtype)
{
    PyObject *x = PyObject_GetAttr(t, n_dtype);
    if (!x)
        PyErr_Clear();
    Py_XDECREF(x);
    return x && x == dtype;
}

static int on_device(PyObject *t, long long index)
{
    int ok = 1;
    const long long d = taken_int(PyObject_CallMethodNoArgs(t, n_get_device), &ok);
    return ok && d == index;
}

static int is_contiguous(PyObject *t)
{
    PyObject *x = PyObject_CallMethodNoArgs(t, n_is_contiguous);
    Py_XDECREF(x);
    return x == Py_True;
}

static int data_of(PyObject *t, void **p)
{
    int ok = 1;
    PyObject *x = PyObject_CallMethodNoArgs(t, n_data_ptr);
    if (!x || !PyLong_Check(x))
        ok = 0;
    else
        *p = PyLong_AsVoidPtr(x);
    Py_XDECREF(x);
    return ok && !PyErr_Occurred();
}

/* n sizes or strides of a tensor (attr: the name of its tuple; call: a method's name) */
static int tuple_of(PyObject *t, PyObject *name, int call, int n, long long *out)
{
    PyObject *x = call ? PyObject_CallMethodNoArgs(t, name) : PyObject_GetAttr(t, name);
    int ok = x && PyTuple_Check(x) && PyTuple_GET_SIZE(x) == n;
    for (int i = 0; ok && i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(x, i));
        ok = !(out[i] == -1 && PyErr_Occurred());
    }
    Py_XDECREF(x);
    return ok;
}

/* A contiguous tensor of the given type and shape on device `index`; its address in *p. */
static int plain(PyObject *t, PyObject *dtype, int n, const long long *shape, long long index, void **p)
{
    long long s[4];
    if (!has_dtype(t, dtype) || !tuple_of(t, n_shape, 0, n, s) || !on_device(t, index) || !is_contiguous(t))
        return 0;
    for (int i = 0; i < n; ++i)
        if (s[i] != shape[i])
            return 0;
    return data_of(t, p);
}

/* The strides and the address of a tensor of shape s. */
static int strided(PyObject *t, const long long *s, fa_heads *out)
{
    long long st[4];
    if (!tuple_of(t, n_stride, 1, 4, st) || st[3] != 1 || s[1] > INT_MAX)
        return 0;
    /* the stride of a dimension of one entry is never used: torch leaves any value there */
    out->stride_b = s[0] > 1 ? st[0] : 0;
    out->stride_h = s[1] > 1 ? st[1] : 0;
    out->stride_t = s[2] > 1 ? st[2] : 0;
    out->H = (int)s[1];
    return data_of(t, &out->data);
}

/* A [B, H, T, d] tensor by strides; H < 0: any number of heads. */
static int heads(PyObject *t, PyObject *dtype, long long B, long long H, long long T, long long d, long long index,
                 fa_heads *out)
{
    long long s[4];
    if (!has_dtype(t, dtype) || !tuple_of(t, n_shape, 0, 4, s) || !on_device(t, index))
        return 0;
    if (s[0] != B || (H >= 0 && s[1] != H) || s[2] != T || s[3] != d)
        return 0;
    return strided(t, s, out);
}

/* The stream to launch on, if `index` is the current device. */
static int stream_of(PyObject *stream, PyObject *index, long long dev, fa_stream_t *out)
{
    int ok = 1;
    long long v;
    if (!f_device || dev < 0 || taken_int(PyObject_CallNoArgs(f_device), &ok) != dev || !ok)
        return 0;   /* not set up, or another device */
    if (stream == Py_None) {
        v = taken_int(PyObject_CallOneArg(f_stream, index), &ok);
    } else if (PyLong_Check(stream)) {
        Py_INCREF(stream);
        v = taken_int(stream, &ok);
    } else {
        v = taken_int(PyObject_GetAttr(stream, n_cuda_stream), &ok);
    }
    *out = (fa_stream_t)(intptr_t)v;
    return ok;
}

static PyObject *slow(void)
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

static int int_arg(PyObject *x, int *out)
{
    int over;
    const long v = PyLong_Check(x) ? PyLong_AsLongAndOverflow(x, &over) : (over = 1, 0);
    if (over || v < INT_MIN || v > INT_MAX)
        return 0;
    *out = (int)v;
    return 1;
}

/* rope(spec, q, q_out, k, k_out, positions, inverse, stream) */
static PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 8)
        return PyErr_Format(PyExc_TypeError, "rope: 8 arguments");
    const fa_rope_spec *spec = (const fa_rope_spec *)PyLong_AsVoidPtr(a[0]);
    if (!spec)
        return slow();
    fa_heads x[2], y[2];
    void *pos;
    fa_stream_t s;
    long long shape[4];
    int ok = 1, inverse;
    PyObject *dtype = has_dtype(a[1], t_bf16) ? t_bf16 : has_dtype(a[1], t_f32) ? t_f32 : NULL;
    PyObject *index = PyObject_CallMethodNoArgs(a[1], n_get_device);
    Py_XINCREF(index);
    const long long dev = taken_int(index, &ok);
    if (!dtype || !ok || !tuple_of(a[1], n_shape, 0, 4, shape))
        goto no;
    const long long B = shape[0], T = shape[2], d = shape[3], at[3] = {spec->n_axes, B, T};
    const int two = a[3] != Py_None;
    if (d != spec->d || two != (a[4] != Py_None) || B > INT_MAX || T > INT_MAX || !int_arg(a[6], &inverse) ||
        !plain(a[5], t_i32, 3, at, dev, &pos) || !strided(a[1], shape, &x[0]) ||
        !heads(a[2], dtype, B, x[0].H, T, d, dev, &y[0]))
        goto no;
    if (two && (!heads(a[3], dtype, B, -1, T, d, dev, &x[1]) || !heads(a[4], dtype, B, x[1].H, T, d, dev, &y[1])))
        goto no;
    if (!stream_of(a[7], index, dev, &s))
        goto no;
    Py_DECREF(index);
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call_rope(x, y, two ? 2 : 1, (const int *)pos, spec, (int)B, (int)T, dtype == t_bf16 ? FA_BF16 : FA_F32, inverse, s);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
no:
    Py_XDECREF(index);
    return slow();
}

/* append(cache, index, k, v, positions, spec, q, q_out, new_lens, stream); spec None or an address */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 10)
        return PyErr_Format(PyExc_TypeError, "append: 10 arguments");
    const fa_kv_cache *c = (const fa_kv_cache *)PyLong_AsVoidPtr(a[0]);
    if (!c)
        return slow();
    int ok = 1;
    Py_INCREF(a[1]);
    const long long dev = taken_int(a[1], &ok);
    const fa_rope_spec *spec = a[5] == Py_None ? NULL : (const fa_rope_spec *)PyLong_AsVoidPtr(a[5]);
    fa_heads k, v, q, qo;
    void *pos = NULL, *new_lens = NULL;
    fa_stream_t s;
    long long shape[4];
    if (!ok || PyErr_Occurred() || !tuple_of(a[2], n_shape, 0, 4, shape) || shape[2] > INT_MAX)
        return slow();
    const long long B = c->B, T = shape[2], d = c->d, lens[1] = {B};
    const int rotate = spec != NULL, with_q = a[6] != Py_None;
    if (rotate != (a[4] != Py_None) || with_q != (a[7] != Py_None) || (with_q && !rotate) ||
        shape[0] != B || shape[1] != c->Hkv || shape[3] != d || !has_dtype(a[2], t_bf16) || !on_device(a[2], dev) ||
        !strided(a[2], shape, &k) || !heads(a[3], t_bf16, B, c->Hkv, T, d, dev, &v))
        return slow();
    if (rotate) {
        const long long at[3] = {spec->n_axes, B, T};
        if (!plain(a[4], t_i32, 3, at, dev, &pos))
            return slow();
    }
    if (with_q && (!heads(a[6], t_bf16, B, -1, T, d, dev, &q) || !heads(a[7], t_bf16, B, q.H, T, d, dev, &qo)))
        return slow();
    if (a[8] != Py_None && !plain(a[8], t_i32, 1, lens, dev, &new_lens))
        return slow();
    if (!stream_of(a[9], a[1], dev, &s))
        return slow();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call_append(c, &k, &v, with_q ? &q : NULL, with_q ? &qo : NULL, (const int *)pos, spec, (const int *)new_lens,
                     (int)T, s);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
}

/* decode(cache, index, q, o, lse, scale, workspace, causal, accumulate, stream) */
static PyObject *py_decode(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 10)
        return PyErr_Format(PyExc_TypeError, "decode: 10 arguments");
    const fa_kv_cache *c = (const fa_kv_cache *)PyLong_AsVoidPtr(a[0]);
    if (!c)
        return slow();
    int ok = 1;
    Py_INCREF(a[1]);
    const long long dev = taken_int(a[1], &ok);
    void *q, *o, *lse, *ws;
    fa_stream_t s;
    long long shape[4];
    if (!ok || !tuple_of(a[2], n_shape, 0, 4, shape) || shape[0] != c->B || shape[1] > INT_MAX || shape[2] > INT_MAX ||
        shape[3] != c->d || !has_dtype(a[2], t_bf16) || !on_device(a[2], dev) || !is_contiguous(a[2]) || !data_of(a[2], &q))
        return slow();
    const double scale = PyFloat_AsDouble(a[5]);
    const int causal = PyObject_IsTrue(a[7]), accumulate = PyObject_IsTrue(a[8]);
    if (PyErr_Occurred() || !plain(a[3], t_bf16, 4, shape, dev, &o) ||
        !plain(a[4], t_f32, 3, shape, dev, &lse) || !on_device(a[6], dev) || !is_contiguous(a[6]) || !data_of(a[6], &ws))
        return slow();
    const long long bytes = taken_int(PyObject_GetAttr(a[6], n_nbytes), &ok);
    if (!ok || !stream_of(a[9], a[1], dev, &s))
        return slow();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call_decode(c, q, o, (float *)lse, (int)shape[1], (int)shape[2], causal, (float)scale, accumulate, ws,
                     (size_t)bytes, s);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
}

/* evict(cache, index, budget, weight_out, order_out, lens_out, kept, n_first, n_recent, stream) */
static PyObject *py_evict(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 10)
        return PyErr_Format(PyExc_TypeError, "evict: 10 arguments");
    const fa_kv_cache *c = (const fa_kv_cache *)PyLong_AsVoidPtr(a[0]);
    if (!c)
        return slow();
    int ok = 1, budget, n_first, n_recent;
    Py_INCREF(a[1]);
    const long long dev = taken_int(a[1], &ok);
    void *weight, *order = NULL, *lens, *kept;
    fa_stream_t s;
    if (!ok || !int_arg(a[2], &budget) || !int_arg(a[7], &n_first) || !int_arg(a[8], &n_recent))
        return slow();
    const long long slots[3] = {c->B, c->Hkv, (long long)c->max_pages * c->page_size}, seqs[1] = {c->B},
                    keep[3] = {c->B, c->Hkv, budget};
    if ((a[4] != Py_None) != (c->order != NULL) || !plain(a[3], t_f32, 3, slots, dev, &weight) ||
        (a[4] != Py_None && !plain(a[4], t_i32, 3, slots, dev, &order)) || !plain(a[5], t_i32, 1, seqs, dev, &lens) ||
        !plain(a[6], t_i32, 3, keep, dev, &kept) || !stream_of(a[9], a[1], dev, &s))
        return slow();
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call_evict(c, budget, n_first, n_recent, (float *)weight, (int *)order, (int *)lens, (int *)kept, s);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
}

/* setup(bfloat16, float32, int32, stream function, device function, addresses of the four entry points) */
static PyObject *py_setup(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 9)
        return PyErr_Format(PyExc_TypeError, "setup: 9 arguments");
    PyObject **keep[5] = {&t_bf16, &t_f32, &t_i32, &f_stream, &f_device};
    void *fn[4];
    for (int i = 0; i < 4; ++i) {
        fn[i] = PyLong_AsVoidPtr(a[5 + i]);
        if (!fn[i])
            return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "setup: a null entry point");
    }
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*keep[i], a[i]);
    }
    call_rope = (rope_fn)fn[0];
    call_append = (append_fn)fn[1];
    call_decode = (decode_fn)fn[2];
    call_evict = (evict_fn)fn[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, NULL},
    {"evict", (PyCFunction)(void (*)(void))py_evict, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_py", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fa_py(void)
{
    PyObject **names[8] = {&n_dtype, &n_shape, &n_get_device, &n_is_contiguous, &n_data_ptr, &n_stride, &n_nbytes, &n_cuda_stream};
    const char *text[8] = {"dtype", "shape", "get_device", "is_contiguous", "data_ptr", "stride", "nbytes", "cuda_stream"};
    for (int i = 0; i < 8; ++i)
        if (!(*names[i] = PyUnicode_InternFromString(text[i])))
            return NULL;
    return PyModule_Create(&module);
}
