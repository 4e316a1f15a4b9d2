/* fastcall.c -- the latency-bound calls of the state-space layer and of the
 * token policy's other operators without the interpreter between the tensors
 * and the C entry points.
 *
 * A single token's kernel takes a few microseconds; asking ten tensors for
 * their type, shape, strides and address from Python takes longer.  Each
 * function here does what its namesake in state_space.py or token_policy.py
 * does for arguments
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
    *g_changed, *g_i64, *g_gated_grads, *g_projection_grads;
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

/* ---- the token policy's other operators ------------------------------------- */

static rlscan_status (*f_gated)(const rlscan_gated_scan_args *, void *, float *, float *, rlscan_stream_t);
static size_t (*f_gated_back_ws)(const rlscan_gated_scan_args *);
static rlscan_status (*f_gated_back)(const rlscan_gated_scan_args *, const rlscan_array3 *, const float *, const float *,
                                     const rlscan_gated_scan_grads *, void *, size_t, rlscan_stream_t);
static rlscan_status (*f_gated_step)(const rlscan_gated_scan_args *, float *, int64_t, const int32_t *, void *, rlscan_stream_t);
static size_t (*f_projection_ws)(const rlscan_gated_projection_args *);
static rlscan_status (*f_projection)(const rlscan_gated_projection_args *, void *, void *, size_t, rlscan_stream_t);
static size_t (*f_projection_back_ws)(const rlscan_gated_projection_args *);
static rlscan_status (*f_projection_back)(const rlscan_gated_projection_args *, const void *, int64_t, void *, void *, void *,
                                          void *, size_t, rlscan_stream_t);
static rlscan_status (*f_distill)(const rlscan_distill_args *, float *, float *, rlscan_stream_t);
static rlscan_status (*f_distill_both)(const rlscan_distill_args *, const float *, float *, float *, void *, rlscan_stream_t);

static int is_empty(const int64_t *sizes, int n)
{
    for (int i = 0; i < n; ++i)
        if (sizes[i] == 0) return 1;
    return 0;
}

/* x, gate, input_gate, log_decay at args[0..3] */
static int gated_args(PyObject *const *args, rlscan_gated_scan_args *a, PyObject **dtype, int64_t *device, int step)
{
    Tensor x;
    const void *p;
    const int dims = step ? 2 : 3;
    if (!io_type(args[0], dtype, &a->dtype) || !look(args[0], &x, *dtype, device) || x.dims != dims || x.stride[dims - 1] != 1 ||
        is_empty(x.size, dims))
        return 0;
    a->N = x.size[0];
    a->T = step ? 1 : x.size[1];
    a->D = x.size[dims - 1];
    a->x.data = x.data;
    a->x.row_stride = x.stride[0];
    a->x.token_stride = step ? 0 : x.stride[1];
    const int64_t second = step ? a->D : a->T;
    if (!act(args[1], &a->gate, *dtype, device, dims, a->N, second, a->D) ||
        !act(args[2], &a->input_gate, *dtype, device, dims, a->N, second, a->D) || !array(args[3], &p, g_f32, device, 1, 1, a->D, 0, 0))
        return 0;
    a->log_decay = (const float *)p;
    a->initial_state = NULL;
    a->resets = NULL;
    a->lengths = NULL;
    return 1;
}

/* gated_scan(x, gate, input_gate, log_decay, initial_state, resets, lengths, return_checkpoints) */
static PyObject *gated_scan(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_gated_scan_args a;
    PyObject *dtype;
    int64_t device = -1;
    const void *init, *resets, *lengths;
    rlscan_stream_t s;
    if (n != 8 || dual_level() || !gated_args(args, &a, &dtype, &device, 0) || (args[7] != Py_True && args[7] != Py_False) ||
        !array(args[4], &init, g_f32, &device, 0, 2, a.N, a.D, 0) || !flags(args[5], &resets, &device, a.N, a.T) ||
        !array(args[6], &lengths, g_i32, &device, 0, 1, a.N, 0, 0) || !stream_of(device, &s))
        return other_way();
    a.initial_state = (const float *)init;
    a.resets = (const uint8_t *)resets;
    a.lengths = (const int32_t *)lengths;
    const int marks = args[7] == Py_True;
    void *yp, *fp, *mp = NULL;
    PyObject *y = new_tensor(args[0], 3, a.N, a.T, a.D, dtype, &yp);
    PyObject *final = y != NULL ? new_tensor(args[0], 2, a.N, a.D, 0, g_f32, &fp) : NULL;
    const int64_t count = (a.T + RLSCAN_GATED_SCAN_CHECKPOINT - 1) / RLSCAN_GATED_SCAN_CHECKPOINT;
    PyObject *kept = final != NULL && marks ? new_tensor(args[0], 3, a.N, count, a.D, g_f32, &mp) : NULL;
    PyObject *r = NULL;
    if (final != NULL && (!marks || kept != NULL) && f_gated(&a, yp, (float *)fp, (float *)mp, s) == RLSCAN_OK)
        r = marks ? PyTuple_Pack(3, y, final, kept) : PyTuple_Pack(2, y, final);
    Py_XDECREF(y);
    Py_XDECREF(final);
    Py_XDECREF(kept);
    return r != NULL ? r : other_way();
}

/* gated_scan_backward(grad_y, x, gate, input_gate, log_decay, checkpoints, resets, lengths, grad_final_state) */
static PyObject *gated_scan_backward(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_gated_scan_args a;
    rlscan_array3 gy;
    PyObject *dtype;
    int64_t device = -1;
    const void *marks, *final, *resets, *lengths;
    rlscan_stream_t s;
    if (n != 9 || dual_level() || !gated_args(args + 1, &a, &dtype, &device, 0)) return other_way();
    const int64_t count = (a.T + RLSCAN_GATED_SCAN_CHECKPOINT - 1) / RLSCAN_GATED_SCAN_CHECKPOINT;
    if (!act(args[0], &gy, dtype, &device, 3, a.N, a.T, a.D) || !array(args[5], &marks, g_f32, &device, 1, 3, a.N, count, a.D) ||
        !flags(args[6], &resets, &device, a.N, a.T) || !array(args[7], &lengths, g_i32, &device, 0, 1, a.N, 0, 0) ||
        !array(args[8], &final, g_f32, &device, 0, 2, a.N, a.D, 0) || !stream_of(device, &s))
        return other_way();
    a.resets = (const uint8_t *)resets;
    a.lengths = (const int32_t *)lengths;
    const size_t bytes = f_gated_back_ws(&a);
    void *p[5], *wp = NULL;
    PyObject *out[5] = {NULL, NULL, NULL, NULL, NULL}, *ws = NULL, *r = NULL;
    int ok = 1;
    for (int i = 0; i < 3 && ok; ++i) ok = (out[i] = new_tensor(args[1], 3, a.N, a.T, a.D, dtype, &p[i])) != NULL;
    ok = ok && (out[3] = new_tensor(args[1], 1, a.D, 0, 0, g_f32, &p[3])) != NULL;
    ok = ok && (out[4] = new_tensor(args[1], 2, a.N, a.D, 0, g_f32, &p[4])) != NULL;
    if (ok && bytes > 0) ok = (ws = new_tensor(args[1], 1, (int64_t)bytes, 0, 0, g_u8, &wp)) != NULL;
    if (ok) {
        const rlscan_gated_scan_grads g = {p[0], p[1], p[2], (float *)p[3], (float *)p[4]};
        if (f_gated_back(&a, &gy, (const float *)final, (const float *)marks, &g, wp, bytes, s) == RLSCAN_OK)
            r = PyObject_Vectorcall(g_gated_grads, out, 5, NULL);
    }
    for (int i = 0; i < 5; ++i) Py_XDECREF(out[i]);
    Py_XDECREF(ws);
    return r != NULL ? r : other_way();
}

/* gated_scan_step(state, x, gate, input_gate, log_decay, slots) */
static PyObject *gated_scan_step(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_gated_scan_args a;
    PyObject *dtype;
    int64_t device = -1;
    Tensor state;
    const void *slots;
    rlscan_stream_t s;
    if (n != 6 || dual_level() || !gated_args(args + 1, &a, &dtype, &device, 1) || !look(args[0], &state, g_f32, &device) ||
        !sized(&state, 2, state.size[0], a.D, 0) || !dense(&state) || !array(args[5], &slots, g_i32, &device, 0, 1, a.N, 0, 0) ||
        !stream_of(device, &s))
        return other_way();
    void *yp;
    PyObject *y = new_tensor(args[1], 2, a.N, a.D, 0, dtype, &yp);
    if (y != NULL && f_gated_step(&a, (float *)state.data, state.size[0], (const int32_t *)slots, yp, s) == RLSCAN_OK)
        return updated(args[0], y);
    Py_XDECREF(y);
    return other_way();
}

/* x, gate_weight, up_weight, activation at args[0..3], x of two dimensions */
static int projection_args(PyObject *const *args, rlscan_gated_projection_args *a, int64_t *device)
{
    Tensor x, g, u;
    if (!look(args[0], &x, g_bf16, device) || x.dims != 2 || x.stride[1] != 1 || !look(args[1], &g, g_bf16, device) || g.dims != 2 ||
        g.stride[1] != 1 || !look(args[2], &u, g_bf16, device) || !sized(&u, 2, g.size[0], g.size[1], 0) || u.stride[1] != 1 ||
        g.size[1] != x.size[1] || is_empty(x.size, 2) || is_empty(g.size, 2) || !PyUnicode_Check(args[3]))
        return 0;
    if (PyUnicode_CompareWithASCIIString(args[3], "silu") == 0)
        a->activation = RLSCAN_SILU;
    else if (PyUnicode_CompareWithASCIIString(args[3], "gelu") == 0)
        a->activation = RLSCAN_GELU;
    else
        return 0;
    a->M = x.size[0];
    a->D = x.size[1];
    a->F = g.size[0];
    a->x = x.data;
    a->x_stride = x.stride[0];
    a->gate_weight = g.data;
    a->gate_stride = g.stride[0];
    a->up_weight = u.data;
    a->up_stride = u.stride[0];
    return 1;
}

/* gated_projection(x, gate_weight, up_weight, activation) */
static PyObject *gated_projection(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_gated_projection_args a;
    int64_t device = -1;
    rlscan_stream_t s;
    if (n != 4 || dual_level() || !projection_args(args, &a, &device) || !stream_of(device, &s)) return other_way();
    const size_t bytes = f_projection_ws(&a);
    void *hp, *wp = NULL;
    PyObject *h = new_tensor(args[0], 2, a.M, a.F, 0, g_bf16, &hp);
    PyObject *ws = h != NULL && bytes > 0 ? new_tensor(args[0], 1, (int64_t)bytes, 0, 0, g_u8, &wp) : NULL;
    const int ok = h != NULL && (bytes == 0 || ws != NULL) && f_projection(&a, hp, wp, bytes, s) == RLSCAN_OK;
    Py_XDECREF(ws);
    if (ok) return h;
    Py_XDECREF(h);
    return other_way();
}

/* gated_projection_backward(grad_h, x, gate_weight, up_weight, activation) */
static PyObject *gated_projection_backward(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_gated_projection_args a;
    Tensor gh;
    int64_t device = -1;
    rlscan_stream_t s;
    if (n != 5 || dual_level() || !projection_args(args + 1, &a, &device) || !look(args[0], &gh, g_bf16, &device) ||
        !sized(&gh, 2, a.M, a.F, 0) || gh.stride[1] != 1 || !stream_of(device, &s))
        return other_way();
    const size_t bytes = f_projection_back_ws(&a);
    void *p[3], *wp = NULL;
    PyObject *out[3] = {NULL, NULL, NULL}, *ws = NULL, *r = NULL;
    int ok = (out[0] = new_tensor(args[1], 2, a.M, a.D, 0, g_bf16, &p[0])) != NULL;
    for (int i = 1; i < 3 && ok; ++i) ok = (out[i] = new_tensor(args[1], 2, a.F, a.D, 0, g_bf16, &p[i])) != NULL;
    if (ok && bytes > 0) ok = (ws = new_tensor(args[1], 1, (int64_t)bytes, 0, 0, g_u8, &wp)) != NULL;
    if (ok && f_projection_back(&a, gh.data, gh.stride[0], p[0], p[1], p[2], wp, bytes, s) == RLSCAN_OK)
        r = PyObject_Vectorcall(g_projection_grads, out, 3, NULL);
    for (int i = 0; i < 3; ++i) Py_XDECREF(out[i]);
    Py_XDECREF(ws);
    return r != NULL ? r : other_way();
}

/* logits, teacher_logits, teacher_tokens, temperature, mask at args[0..4] */
static int distill_args(PyObject *const *args, rlscan_distill_args *a, PyObject **dtype, int64_t *device)
{
    Tensor z, t, k;
    PyObject *ttype;
    const void *mask;
    if (!io_type(args[0], dtype, &a->dtype) || !look(args[0], &z, *dtype, device) || z.dims != 3 || z.stride[2] != 1 ||
        is_empty(z.size, 3) || !io_type(args[1], &ttype, &a->teacher_dtype) || !look(args[1], &t, ttype, device) || t.dims != 3 ||
        !sized(&t, 3, z.size[0], z.size[1], t.size[2]) || !dense(&t) || !look(args[2], &k, NULL, device) ||
        !sized(&k, 3, t.size[0], t.size[1], t.size[2]) || !dense(&k) || !PyFloat_Check(args[3]) ||
        !flags(args[4], &mask, device, z.size[0], z.size[1]))
        return 0;
    PyObject *v = PyObject_GetAttr(args[2], s_dtype);
    if (v == NULL) return 0;
    Py_DECREF(v);
    if (v != g_i32 && v != g_i64) return 0;
    a->token_bytes = v == g_i64 ? 8 : 4;
    a->N = z.size[0];
    a->T = z.size[1];
    a->V = z.size[2];
    a->K = t.size[2];
    a->logits.data = z.data;
    a->logits.row_stride = z.stride[0];
    a->logits.token_stride = z.stride[1];
    a->teacher_logits = t.data;
    a->teacher_tokens = k.data;
    a->mask = (const uint8_t *)mask;
    a->temperature = PyFloat_AS_DOUBLE(args[3]);
    return 1;
}

/* distill_loss(logits, teacher_logits, teacher_tokens, temperature, mask) */
static PyObject *distill_loss(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_distill_args a;
    PyObject *dtype;
    int64_t device = -1;
    rlscan_stream_t s;
    if (n != 5 || dual_level() || !distill_args(args, &a, &dtype, &device) || !stream_of(device, &s)) return other_way();
    void *lp;
    PyObject *loss = new_tensor(args[0], 2, a.N, a.T, 0, g_f32, &lp);
    if (loss != NULL && f_distill(&a, (float *)lp, NULL, s) == RLSCAN_OK) return loss;
    Py_XDECREF(loss);
    return other_way();
}

/* distill_loss_and_grad(grad_loss, logits, teacher_logits, teacher_tokens, temperature, mask) */
static PyObject *distill_loss_and_grad(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    rlscan_distill_args a;
    PyObject *dtype;
    int64_t device = -1;
    const void *weight;
    rlscan_stream_t s;
    if (n != 6 || dual_level() || !distill_args(args + 1, &a, &dtype, &device) ||
        !array(args[0], &weight, g_f32, &device, 1, 2, a.N, a.T, 0) || !stream_of(device, &s))
        return other_way();
    void *lp, *np, *gp;
    PyObject *loss = new_tensor(args[1], 2, a.N, a.T, 0, g_f32, &lp), *r = NULL;
    PyObject *norm = loss != NULL ? new_tensor(args[1], 3, a.N, a.T, 2, g_f32, &np) : NULL;
    PyObject *grad = norm != NULL ? new_tensor(args[1], 3, a.N, a.T, a.V, dtype, &gp) : NULL;
    if (grad != NULL && f_distill_both(&a, (const float *)weight, (float *)lp, (float *)np, gp, s) == RLSCAN_OK)
        r = PyTuple_Pack(2, loss, grad);
    Py_XDECREF(loss);
    Py_XDECREF(norm);
    Py_XDECREF(grad);
    return r != NULL ? r : other_way();
}

/* setup_token_policy(torch, GatedScanGrads, GatedProjectionGrads, addresses of the ten entry points), behind setup */
static PyObject *setup_token_policy(PyObject *self, PyObject *args)
{
    PyObject *torch, *gated, *projection;
    unsigned long long f[10];
    if (!PyArg_ParseTuple(args, "OOOKKKKKKKKKK", &torch, &gated, &projection, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6],
                          &f[7], &f[8], &f[9]))
        return NULL;
    if ((g_i64 = PyObject_GetAttrString(torch, "int64")) == NULL) return NULL;
    Py_INCREF(gated);
    g_gated_grads = gated;
    Py_INCREF(projection);
    g_projection_grads = projection;
    f_gated = (rlscan_status (*)(const rlscan_gated_scan_args *, void *, float *, float *, rlscan_stream_t))(uintptr_t)f[0];
    f_gated_back_ws = (size_t (*)(const rlscan_gated_scan_args *))(uintptr_t)f[1];
    f_gated_back = (rlscan_status (*)(const rlscan_gated_scan_args *, const rlscan_array3 *, const float *, const float *,
                                      const rlscan_gated_scan_grads *, void *, size_t, rlscan_stream_t))(uintptr_t)f[2];
    f_gated_step = (rlscan_status (*)(const rlscan_gated_scan_args *, float *, int64_t, const int32_t *, void *,
                                      rlscan_stream_t))(uintptr_t)f[3];
    f_projection_ws = (size_t (*)(const rlscan_gated_projection_args *))(uintptr_t)f[4];
    f_projection = (rlscan_status (*)(const rlscan_gated_projection_args *, void *, void *, size_t, rlscan_stream_t))(uintptr_t)f[5];
    f_projection_back_ws = (size_t (*)(const rlscan_gated_projection_args *))(uintptr_t)f[6];
    f_projection_back = (rlscan_status (*)(const rlscan_gated_projection_args *, const void *, int64_t, void *, void *, void *,
                                           void *, size_t, rlscan_stream_t))(uintptr_t)f[7];
    f_distill = (rlscan_status (*)(const rlscan_distill_args *, float *, float *, rlscan_stream_t))(uintptr_t)f[8];
    f_distill_both = (rlscan_status (*)(const rlscan_distill_args *, const float *, float *, float *, void *,
                                        rlscan_stream_t))(uintptr_t)f[9];
    Py_RETURN_NONE;
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
                                FAST(causal_conv), FAST(causal_conv_step), FAST(add_rms_norm),
                                {"setup_token_policy", setup_token_policy, METH_VARARGS, NULL}, FAST(gated_scan),
                                FAST(gated_scan_backward), FAST(gated_scan_step), FAST(gated_projection),
                                FAST(gated_projection_backward), FAST(distill_loss), FAST(distill_loss_and_grad), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
