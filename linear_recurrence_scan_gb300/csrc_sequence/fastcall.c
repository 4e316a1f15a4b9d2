/* fastcall.c -- the state-space layer's latency-bound calls without the
 * interpreter between the tensors and the C entry points.
 *
 * A single token's kernel takes a few microseconds; asking ten tensors for
 * their type, shape, strides and address from Python takes longer.  Each
 * function here does what its namesake in state_space.py does for arguments
 * in the usual form (plain CUDA tensors of the right type and shape, element
 * stride 1, no gradient wanted, outside forward-mode differentiation, on the
 * current device) and returns None for any others, which then take the
 * Python way and its error messages.  It needs Python.h alone; the
 * entry points' addresses come from the loaded library.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "rlscan.h"

typedef struct Tensor {
    PyObject *object;
    const void *data;
    int dims;
    int64_t size[3], stride[3];
} Tensor;

static PyObject *g_tensor, *g_parameter, *g_f32, *g_bf16, *g_i32, *g_u8, *g_bool, *g_fp8, *g_empty,
    *g_raw_stream, *g_grad_enabled, *g_norm_result, *g_current_device, *g_forward_ad,
    *g_changed;
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_requires_grad, *s_device, *s_level, *kw_empty;

static size_t (*f_scan_ws)(const rlscan_selective_scan_args *);
static rlscan_status (*f_scan)(const rlscan_selective_scan_args *, void *, float *, float *, void *, size_t,
                               rlscan_stream_t);
static rlscan_status (*f_scan_step)(const rlscan_selective_scan_args *, float *, int64_t, const int32_t *, void *,
                                    rlscan_stream_t);
static rlscan_status (*f_conv)(const rlscan_causal_conv_args *, void *, void *, rlscan_stream_t);
static rlscan_status (*f_conv_step)(const rlscan_causal_conv_args *, void *, int64_t, const int32_t *, void *,
                                    rlscan_stream_t);
static rlscan_status (*f_norm)(const void *, int64_t, const void *, int64_t, const float *, int64_t, int64_t, float,
                               rlscan_dtype, rlscan_dtype, void *, float *, void *, rlscan_stream_t);

/* 1 and the numbers of a tuple of 1 to 3 integers, else 0 */
static int numbers(PyObject *tuple, int64_t *to, int *count)
{
    if (tuple == NULL || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) < 1 || PyTuple_GET_SIZE(tuple) > 3) return 0;
    *count = (int)PyTuple_GET_SIZE(tuple);
    for (int i = 0; i < *count; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (to[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

static int call_number(PyObject *t, PyObject *method, int64_t *to)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, method);
    if (r == NULL) return 0;
    *to = (int64_t)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

/* A plain tensor of type `dtype` (NULL: any) on `device` (-1: any CUDA
 * device, which it becomes) that wants no gradient. */
static int look(PyObject *t, Tensor *o, PyObject *dtype, int64_t *device)
{
    if ((PyObject *)Py_TYPE(t) != g_tensor && (PyObject *)Py_TYPE(t) != g_parameter) return 0;
    o->object = t;
    PyObject *v = PyObject_GetAttr(t, s_dtype);
    if (v == NULL) return 0;
    const int fits = dtype == NULL || v == dtype;
    Py_DECREF(v);
    if (!fits) return 0;
    int64_t at;
    if (!call_number(t, s_get_device, &at) || at < 0 || (*device >= 0 && at != *device)) return 0;
    *device = at;
    v = PyObject_GetAttr(t, s_requires_grad);
    if (v == NULL) return 0;
    const int wants = v != Py_False;
    Py_DECREF(v);
    if (wants) {
        v = PyObject_CallNoArgs(g_grad_enabled);
        if (v == NULL) return 0;
        const int on = v != Py_False;
        Py_DECREF(v);
        if (on) return 0;
    }
    int n = 0;
    v = PyObject_GetAttr(t, s_shape);
    int ok = numbers(v, o->size, &o->dims);
    Py_XDECREF(v);
    if (!ok) return 0;
    v = PyObject_CallMethodNoArgs(t, s_stride);
    ok = numbers(v, o->stride, &n) && n == o->dims;
    Py_XDECREF(v);
    if (!ok) return 0;
    int64_t p;
    if (!call_number(t, s_data_ptr, &p)) return 0;
    o->data = (const void *)(intptr_t)p;
    return 1;
}

static int sized(const Tensor *t, int dims, int64_t a, int64_t b, int64_t c)
{
    return t->dims == dims && t->size[0] == a && (dims < 2 || t->size[1] == b) && (dims < 3 || t->size[2] == c);
}

static int dense(const Tensor *t)
{
    int64_t each = 1;
    for (int i = t->dims - 1; i >= 0; --i) {
        if (t->size[i] != 1 && t->stride[i] != each) return 0;
        each *= t->size[i];
    }
    return 1;
}

/* an activation of the given sizes: element stride 1 */
static int act(PyObject *t, rlscan_array3 *o, PyObject *dtype, int64_t *device, int dims, int64_t a, int64_t b, int64_t c)
{
    Tensor v;
    if (!look(t, &v, dtype, device) || !sized(&v, dims, a, b, c) || v.stride[dims - 1] != 1) return 0;
    o->data = v.data;
    o->row_stride = v.stride[0];
    o->token_stride = dims == 3 ? v.stride[1] : 0;
    return 1;
}

/* a dense array, or None where that is allowed */
static int array(PyObject *t, const void **o, PyObject *dtype, int64_t *device, int needed, int dims, int64_t a, int64_t b,
                 int64_t c)
{
    *o = NULL;
    if (t == Py_None) return !needed;
    Tensor v;
    if (!look(t, &v, dtype, device) || !sized(&v, dims, a, b, c) || !dense(&v)) return 0;
    *o = v.data;
    return 1;
}

static int flags(PyObject *t, const void **o, int64_t *device, int64_t N, int64_t T)
{
    if (array(t, o, g_u8, device, 0, 2, N, T, 0)) return 1;
    return !PyErr_Occurred() && array(t, o, g_bool, device, 0, 2, N, T, 0);
}

static PyObject *new_tensor(PyObject *like, int dims, int64_t a, int64_t b, int64_t c, PyObject *dtype, void **data)
{
    PyObject *device = PyObject_GetAttr(like, s_device);
    if (device == NULL) return NULL;
    PyObject *shape = dims == 1 ? Py_BuildValue("(L)", (long long)a)
                      : dims == 2 ? Py_BuildValue("(LL)", (long long)a, (long long)b)
                                  : Py_BuildValue("(LLL)", (long long)a, (long long)b, (long long)c);
    PyObject *r = NULL;
    if (shape != NULL) {
        PyObject *args[3] = {shape, dtype, device};
        r = PyObject_Vectorcall(g_empty, args, 1, kw_empty);
        Py_DECREF(shape);
    }
    Py_DECREF(device);
    int64_t p;
    if (r != NULL && !call_number(r, s_data_ptr, &p)) Py_CLEAR(r);
    if (r != NULL) *data = (void *)(intptr_t)p;
    return r;
}

/* the current stream of `device`, which has to be the current device */
static int stream_of(int64_t device, rlscan_stream_t *s)
{
    PyObject *d = PyObject_CallNoArgs(g_current_device);
    if (d == NULL) return 0;
    if (PyLong_AsLongLong(d) != device) {
        Py_DECREF(d);
        return 0;
    }
    PyObject *r = PyObject_CallOneArg(g_raw_stream, d);
    Py_DECREF(d);
    if (r == NULL) return 0;
    *s = (rlscan_stream_t)(intptr_t)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

/* whether tensors may carry tangents: inside a dual level (-1: none) */
static int dual_level(void)
{
    PyObject *v = PyObject_GetAttr(g_forward_ad, s_level);
    if (v == NULL) return 1;
    const long level = PyLong_AsLong(v);
    Py_DECREF(v);
    return level >= 0 || PyErr_Occurred() != NULL;
}

/* "not in the usual form": the Python way takes over, and says what is wrong */
static PyObject *other_way(void)
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

static int io_type(PyObject *x, PyObject **dtype, int64_t *code)
{
    PyObject *v = PyObject_GetAttr(x, s_dtype);
    if (v == NULL) return 0;
    Py_DECREF(v);  /* types are immortal module attributes */
    *dtype = v;
    *code = v == g_bf16 ? RLSCAN_BF16 : RLSCAN_F32;
    return v == g_bf16 || v == g_f32;
}

/* x, delta, A, B, C, D, z, delta_bias, delta_softplus at args[0..8] */
static int scan_args(PyObject *const *args, rlscan_selective_scan_args *a, PyObject **dtype, int64_t *device, int step)
{
    Tensor x, A;
    const void *p;
    const int dims = step ? 2 : 3;
    if (!io_type(args[0], dtype, &a->dtype) || !look(args[0], &x, *dtype, device) || x.dims != dims ||
        x.stride[dims - 1] != 1)
        return 0;
    a->N = x.size[0];
    a->T = step ? 1 : x.size[1];
    a->D = x.size[dims - 1];
    a->x.data = x.data;
    a->x.row_stride = x.stride[0];
    a->x.token_stride = step ? 0 : x.stride[1];
    if (!look(args[2], &A, g_f32, device) || A.dims != 2 || A.size[0] != a->D || !dense(&A)) return 0;
    a->A = (const float *)A.data;
    a->S = A.size[1];
    if (args[8] != Py_True && args[8] != Py_False) return 0;
    a->delta_softplus = args[8] == Py_True;
    const int64_t second = step ? a->D : a->T, states = step ? a->S : a->T;
    if (!act(args[1], &a->delta, *dtype, device, dims, a->N, second, a->D) ||
        !act(args[3], &a->B, *dtype, device, dims, a->N, states, a->S) ||
        !act(args[4], &a->C, *dtype, device, dims, a->N, states, a->S))
        return 0;
    a->z.data = NULL;
    a->z.row_stride = a->z.token_stride = 0;
    if (args[6] != Py_None && !act(args[6], &a->z, *dtype, device, dims, a->N, second, a->D)) return 0;
    if (!array(args[5], &p, g_f32, device, 0, 1, a->D, 0, 0)) return 0;
    a->skip = (const float *)p;
    if (!array(args[7], &p, g_f32, device, 0, 1, a->D, 0, 0)) return 0;
    a->delta_bias = (const float *)p;
    a->initial_state = NULL;
    a->resets = NULL;
    a->lengths = NULL;
    return 1;
}

/* selective_scan(x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, resets, lengths) */
static PyObject *selective_scan(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_selective_scan_args a;
    PyObject *dtype;
    int64_t device = -1;
    const void *init, *resets, *lengths;
    rlscan_stream_t s;
    if (n != 12 || dual_level() || !scan_args(args, &a, &dtype, &device, 0) ||
        !array(args[9], &init, g_f32, &device, 0, 3, a.N, a.D, a.S) || !flags(args[10], &resets, &device, a.N, a.T) ||
        !array(args[11], &lengths, g_i32, &device, 0, 1, a.N, 0, 0) || !stream_of(device, &s))
        return other_way();
    a.initial_state = (const float *)init;
    a.resets = (const uint8_t *)resets;
    a.lengths = (const int32_t *)lengths;
    void *yp, *fp, *wp = NULL;
    const size_t bytes = f_scan_ws(&a);
    PyObject *y = new_tensor(args[0], 3, a.N, a.T, a.D, dtype, &yp);
    PyObject *final = y != NULL ? new_tensor(args[0], 3, a.N, a.D, a.S, g_f32, &fp) : NULL;
    PyObject *ws = final != NULL && bytes > 0 ? new_tensor(args[0], 1, (int64_t)bytes, 0, 0, g_u8, &wp) : NULL;
    PyObject *r = NULL;
    if (final != NULL && (bytes == 0 || ws != NULL) &&
        f_scan(&a, yp, (float *)fp, NULL, wp, bytes, s) == RLSCAN_OK)
        r = PyTuple_Pack(2, y, final);
    Py_XDECREF(y);
    Py_XDECREF(final);
    Py_XDECREF(ws);
    return r != NULL ? r : other_way();
}

/* y of a call that has updated its state, which autograd is told */
static PyObject *updated(PyObject *state, PyObject *y)
{
    PyObject *r = PyObject_CallOneArg(g_changed, state);
    if (r == NULL) Py_CLEAR(y);
    Py_XDECREF(r);
    return y;
}

/* selective_scan_step(state, x, delta, A, B, C, D, z, delta_bias, delta_softplus, slots) */
static PyObject *selective_scan_step(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_selective_scan_args a;
    PyObject *dtype;
    int64_t device = -1;
    Tensor state;
    const void *slots;
    rlscan_stream_t s;
    if (n != 11 || dual_level() || !scan_args(args + 1, &a, &dtype, &device, 1) || !look(args[0], &state, g_f32, &device) ||
        !sized(&state, 3, state.size[0], a.D, a.S) || !dense(&state) ||
        !array(args[10], &slots, g_i32, &device, 0, 1, a.N, 0, 0) || !stream_of(device, &s))
        return other_way();
    void *yp;
    PyObject *y = new_tensor(args[1], 2, a.N, a.D, 0, dtype, &yp);
    if (y != NULL &&
        f_scan_step(&a, (float *)state.data, state.size[0], (const int32_t *)slots, yp, s) == RLSCAN_OK)
        return updated(args[0], y);
    Py_XDECREF(y);
    return other_way();
}

/* x, weight, bias, activation at args[0..3] */
static int conv_args(PyObject *const *args, rlscan_causal_conv_args *a, PyObject **dtype, int64_t *device, int step)
{
    Tensor x, w;
    const void *p;
    const int dims = step ? 2 : 3;
    if (!io_type(args[0], dtype, &a->dtype) || !look(args[0], &x, *dtype, device) || x.dims != dims ||
        x.stride[dims - 1] != 1)
        return 0;
    a->N = x.size[0];
    a->T = step ? 1 : x.size[1];
    a->D = x.size[dims - 1];
    a->x.data = x.data;
    a->x.row_stride = x.stride[0];
    a->x.token_stride = step ? 0 : x.stride[1];
    if (!look(args[1], &w, g_f32, device) || w.dims != 2 || w.size[0] != a->D || !dense(&w)) return 0;
    a->weight = (const float *)w.data;
    a->K = w.size[1];
    if (!array(args[2], &p, g_f32, device, 0, 1, a->D, 0, 0)) return 0;
    a->bias = (const float *)p;
    a->silu = args[3] != Py_None;
    if (a->silu && (!PyUnicode_Check(args[3]) || PyUnicode_CompareWithASCIIString(args[3], "silu") != 0)) return 0;
    a->initial_state = NULL;
    a->resets = NULL;
    a->lengths = NULL;
    return 1;
}

/* causal_conv(x, weight, bias, activation, initial_state, resets, lengths) */
static PyObject *causal_conv(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_causal_conv_args a;
    PyObject *dtype;
    int64_t device = -1;
    const void *resets, *lengths;
    rlscan_stream_t s;
    if (n != 7 || dual_level() || !conv_args(args, &a, &dtype, &device, 0) || a.K < 2 ||
        !array(args[4], &a.initial_state, dtype, &device, 0, 3, a.N, a.K - 1, a.D) ||
        !flags(args[5], &resets, &device, a.N, a.T) || !array(args[6], &lengths, g_i32, &device, 0, 1, a.N, 0, 0) ||
        !stream_of(device, &s))
        return other_way();
    a.resets = (const uint8_t *)resets;
    a.lengths = (const int32_t *)lengths;
    void *yp, *fp;
    PyObject *y = new_tensor(args[0], 3, a.N, a.T, a.D, dtype, &yp);
    PyObject *final = y != NULL ? new_tensor(args[0], 3, a.N, a.K - 1, a.D, dtype, &fp) : NULL;
    PyObject *r = NULL;
    if (final != NULL && f_conv(&a, yp, fp, s) == RLSCAN_OK) r = PyTuple_Pack(2, y, final);
    Py_XDECREF(y);
    Py_XDECREF(final);
    return r != NULL ? r : other_way();
}

/* causal_conv_step(state, x, weight, bias, activation, slots) */
static PyObject *causal_conv_step(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_causal_conv_args a;
    PyObject *dtype;
    int64_t device = -1;
    Tensor state;
    const void *slots;
    rlscan_stream_t s;
    if (n != 6 || dual_level() || !conv_args(args + 1, &a, &dtype, &device, 1) || a.K < 2 ||
        !look(args[0], &state, dtype, &device) ||
        !sized(&state, 3, state.size[0], a.K - 1, a.D) || !dense(&state) ||
        !array(args[5], &slots, g_i32, &device, 0, 1, a.N, 0, 0) || !stream_of(device, &s))
        return other_way();
    void *yp;
    PyObject *y = new_tensor(args[1], 2, a.N, a.D, 0, dtype, &yp);
    if (y != NULL && f_conv_step(&a, (void *)state.data, state.size[0], (const int32_t *)slots, yp, s) == RLSCAN_OK)
        return updated(args[0], y);
    Py_XDECREF(y);
    return other_way();
}

/* add_rms_norm(x, weight, residual, eps, out_dtype), x of two dimensions */
static PyObject *add_rms_norm(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    Tensor x, r;
    PyObject *dtype, *rtype = NULL;
    int64_t device = -1, code, rcode = RLSCAN_F32;
    const void *w;
    rlscan_stream_t s;
    if (n != 5 || dual_level() || !io_type(args[0], &dtype, &code) || !look(args[0], &x, dtype, &device) || x.dims != 2 ||
        x.stride[1] != 1 || !array(args[1], &w, g_f32, &device, 1, 1, x.size[1], 0, 0) || !PyFloat_Check(args[3]))
        return other_way();
    const int eight = args[4] == g_fp8, summed = args[2] != Py_None;
    if (!eight && args[4] != Py_None && args[4] != dtype) return other_way();
    r.data = NULL;
    r.stride[0] = 0;
    if (summed && (!io_type(args[2], &rtype, &rcode) || (rtype != dtype && rtype != g_f32) ||
                   !look(args[2], &r, rtype, &device) || !sized(&r, 2, x.size[0], x.size[1], 0) || r.stride[1] != 1))
        return other_way();
    if (!stream_of(device, &s)) return other_way();
    const int64_t M = x.size[0], D = x.size[1];
    void *yp, *hp = NULL, *sp = NULL;
    PyObject *y = new_tensor(args[0], 2, M, D, 0, eight ? g_fp8 : dtype, &yp), *h = NULL, *sc = NULL, *result = NULL;
    if (y != NULL && summed) h = new_tensor(args[0], 2, M, D, 0, rtype, &hp);
    if (y != NULL && eight) sc = new_tensor(args[0], 2, M, (D + 127) / 128, 0, g_f32, &sp);
    if (y != NULL && (!summed || h != NULL) && (!eight || sc != NULL) &&
        f_norm(x.data, x.stride[0], r.data, r.stride[0], (const float *)w, M, D, (float)PyFloat_AS_DOUBLE(args[3]),
               (rlscan_dtype)code, (rlscan_dtype)rcode, yp, (float *)sp, hp, s) == RLSCAN_OK) {
        PyObject *out[3] = {y, summed ? h : Py_None, eight ? sc : Py_None};
        result = PyObject_Vectorcall(g_norm_result, out, 3, NULL);
    }
    Py_XDECREF(y);
    Py_XDECREF(h);
    Py_XDECREF(sc);
    return result != NULL ? result : other_way();
}

/* setup(torch, RmsNorm, raw stream function, current device function, torch.autograd.forward_ad, increment_version,
 * addresses of the six entry points) */
static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *torch, *result, *stream, *device, *forward_ad, *changed;
    unsigned long long f[6];
    if (!PyArg_ParseTuple(args, "OOOOOOKKKKKK", &torch, &result, &stream, &device, &forward_ad, &changed, &f[0], &f[1],
                          &f[2], &f[3], &f[4], &f[5]))
        return NULL;
    const struct {
        PyObject **to;
        const char *name;
    } names[] = {{&g_tensor, "Tensor"}, {&g_f32, "float32"}, {&g_bf16, "bfloat16"}, {&g_i32, "int32"}, {&g_u8, "uint8"},
                 {&g_bool, "bool"}, {&g_fp8, "float8_e4m3fn"}, {&g_empty, "empty"}, {&g_grad_enabled, "is_grad_enabled"}};
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if ((*names[i].to = PyObject_GetAttrString(torch, names[i].name)) == NULL) return NULL;
    PyObject *nn = PyObject_GetAttrString(torch, "nn");
    if (nn == NULL) return NULL;
    g_parameter = PyObject_GetAttrString(nn, "Parameter");
    Py_DECREF(nn);
    if (g_parameter == NULL) return NULL;
    Py_INCREF(result);
    g_norm_result = result;
    Py_INCREF(stream);
    g_raw_stream = stream;
    Py_INCREF(device);
    g_current_device = device;
    Py_INCREF(forward_ad);
    g_forward_ad = forward_ad;
    Py_INCREF(changed);
    g_changed = changed;
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_requires_grad = PyUnicode_InternFromString("requires_grad");
    s_device = PyUnicode_InternFromString("device");
    s_level = PyUnicode_InternFromString("_current_level");
    kw_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device || !s_requires_grad || !s_device || !s_level ||
        !kw_empty)
        return NULL;
    f_scan_ws = (size_t (*)(const rlscan_selective_scan_args *))(uintptr_t)f[0];
    f_scan = (rlscan_status (*)(const rlscan_selective_scan_args *, void *, float *, float *, void *, size_t,
                                rlscan_stream_t))(uintptr_t)f[1];
    f_scan_step = (rlscan_status (*)(const rlscan_selective_scan_args *, float *, int64_t, const int32_t *, void *,
                                     rlscan_stream_t))(uintptr_t)f[2];
    f_conv = (rlscan_status (*)(const rlscan_causal_conv_args *, void *, void *, rlscan_stream_t))(uintptr_t)f[3];
    f_conv_step = (rlscan_status (*)(const rlscan_causal_conv_args *, void *, int64_t, const int32_t *, void *,
                                     rlscan_stream_t))(uintptr_t)f[4];
    f_norm = (rlscan_status (*)(const void *, int64_t, const void *, int64_t, const float *, int64_t, int64_t, float,
                                rlscan_dtype, rlscan_dtype, void *, float *, void *, rlscan_stream_t))(uintptr_t)f[5];
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, NULL}, FAST(selective_scan), FAST(selective_scan_step),
                                FAST(causal_conv), FAST(causal_conv_step), FAST(add_rms_norm), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
