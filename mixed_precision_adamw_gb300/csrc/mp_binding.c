/*
 * mp_binding.c — CPython extension `_binding`: the calls of mp_block.h from
 * Python without ctypes, for the ordinary case. A kernel of a few microseconds is
 * otherwise behind its own arguments' checks: RMS norm of one row took 8.8 us a
 * call through ctypes (1.7 of them its conversion of 24 arguments, 5 the checks in
 * Python), of which the launch is 2.
 *
 * Every function takes the arguments of its namesake in block.py by position and
 * either makes the call and returns the status, or, wherever an argument is not
 * plainly right, touches nothing and returns None; block.py then goes through its
 * own checks, which name what is wrong (or know how to pass it on). Only Python's
 * C API is used: tensors are asked for their attributes, so the extension
 * belongs to no version of PyTorch.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "mp_block.h"

static struct {
    PyTypeObject* tensor;            /* torch.Tensor, torch.nn.Parameter */
    PyTypeObject* parameter;
    PyObject* dtype[3];              /* of MP_BF16, MP_FP16, MP_FP32 */
    PyObject *uint8, *e4m3, *int32, *int64;
    PyObject *device, *raw_stream;   /* the current device; a device's current stream */
    PyObject *s_get_device, *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_cuda_stream;
} G;

typedef int (*rms_forward_fn)(void*, void*, float*, void*, void*, void*, void*, const void*, const void*, const void*,
                              int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int32_t,
                              int32_t, int32_t, void*);
typedef int (*rms_backward_fn)(void*, void*, const void*, const void*, const void*, const void*, const void*,
                               const float*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int32_t, int32_t,
                               void*, size_t, void*);
typedef int (*rope_fn)(void*, const void*, void*, const void*, const uint64_t*, const void*, int64_t, int64_t, int32_t,
                       int32_t, int32_t, int32_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                       int64_t, float, int32_t, int32_t, int32_t, int32_t, void*);
typedef int (*gated_forward_fn)(void*, void*, void*, void*, void*, const void*, const void*, int64_t, int64_t, int64_t,
                                int64_t, int64_t, int64_t, int64_t, int32_t, int32_t, void*);
typedef int (*gated_backward_fn)(void*, void*, void*, const void*, const void*, const void*, const void*, const void*,
                                 int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int32_t,
                                 int32_t, void*);
typedef int (*pack_fn)(void*, void*, const void*, int64_t, int64_t, int64_t, int64_t, int32_t, int32_t, void*);
typedef int (*unpack_fn)(void*, const void*, const void*, int64_t, int64_t, int64_t, int64_t, int32_t, int32_t, void*);

static struct {
    rms_forward_fn rms_forward;
    rms_backward_fn rms_backward;
    rope_fn rope;
    gated_forward_fn gated_forward;
    gated_backward_fn gated_backward;
    pack_fn pack;
    unpack_fn unpack;
} F;

/* ---- arguments -------------------------------------------------------------- */

typedef struct {
    long device;
    void* stream;
} Call;

typedef struct { /* a tensor of at most three dimensions */
    void* p;
    PyObject* dtype; /* borrowed: dtypes live as long as PyTorch does */
    int dims;
    int64_t size[3], stride[3];
} Tensor;

static int numbers(PyObject* t, int64_t* to, int dims) {
    for (int i = 0; i < dims; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (to[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* What a CUDA tensor on the call's device is; 0 if `t` is none or has other than `dims` dimensions. */
static int tensor(PyObject* t, const Call* call, int dims, Tensor* to) {
    PyObject* v;
    if (Py_TYPE(t) != G.tensor && Py_TYPE(t) != G.parameter) return 0;
    if (!(v = PyObject_CallMethodNoArgs(t, G.s_get_device))) return 0;
    const long device = PyLong_AsLong(v);
    Py_DECREF(v);
    if (device != call->device) return 0;
    if (!(to->dtype = PyObject_GetAttr(t, G.s_dtype))) return 0;
    Py_DECREF(to->dtype);
    if (!(v = PyObject_GetAttr(t, G.s_shape))) return 0;
    int ok = PyTuple_Check(v) && PyTuple_GET_SIZE(v) == dims && numbers(v, to->size, dims);
    Py_DECREF(v);
    if (!ok || !(v = PyObject_CallMethodNoArgs(t, G.s_stride))) return 0;
    ok = PyTuple_Check(v) && PyTuple_GET_SIZE(v) == dims && numbers(v, to->stride, dims);
    Py_DECREF(v);
    if (!ok || !(v = PyObject_CallMethodNoArgs(t, G.s_data_ptr))) return 0;
    to->p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    to->dims = dims;
    return !PyErr_Occurred();
}

static int type_code(PyObject* dtype) {
    for (int i = 0; i < 3; ++i)
        if (dtype == G.dtype[i]) return i;
    return -1;
}

/* The first matrix of a call, of any element type, with contiguous rows. */
static int matrix(PyObject* t, const Call* call, Tensor* to, int* code) {
    return tensor(t, call, 2, to) && (*code = type_code(to->dtype)) >= 0 && to->stride[1] == 1 &&
           to->stride[0] >= to->size[1];
}

/* A further one, of its shape and type; None if that is allowed. */
static int like(PyObject* t, const Call* call, const Tensor* x, int optional, Tensor* to) {
    if (t == Py_None) {
        to->p = NULL;
        to->stride[0] = 0;
        return optional;
    }
    return tensor(t, call, 2, to) && to->dtype == x->dtype && to->size[0] == x->size[0] &&
           to->size[1] == x->size[1] && to->stride[1] == 1 && to->stride[0] >= to->size[1];
}

/* A contiguous vector of n elements; the caller looks at its dtype. */
static int vector(PyObject* t, const Call* call, int64_t n, Tensor* to) {
    if (t == Py_None) {
        to->p = NULL;
        to->dtype = NULL;
        return 1;
    }
    return tensor(t, call, 1, to) && to->size[0] == n && (n <= 1 || to->stride[0] == 1);
}

/* Rows in 8 bits and their scales; kind 0 for None. */
static int rows8(PyObject* t, PyObject* scale, const Call* call, int64_t rows, int64_t d, Tensor* to, Tensor* s,
                 int* kind) {
    *kind = 0;
    to->p = s->p = NULL;
    to->stride[0] = 0;
    if (t == Py_None && scale == Py_None) return 1;
    if (!tensor(t, call, 2, to) || (to->dtype != G.e4m3 && to->dtype != G.uint8) || to->size[0] != rows ||
        to->size[1] != d || to->stride[1] != 1 || to->stride[0] < d)
        return 0;
    PyObject* dtype = PyObject_GetAttr(scale, G.s_dtype);
    if (!dtype) return 0;
    Py_DECREF(dtype);
    if (dtype == G.dtype[MP_FP32]) {
        *kind = MP_SCALE_ROW;
        return vector(scale, call, rows, s);
    }
    const int64_t blocks = (d + 31) / 32;
    *kind = MP_SCALE_BLOCK;
    return dtype == G.uint8 && tensor(scale, call, 2, s) && s->size[0] == rows && s->size[1] == blocks &&
           (blocks == 1 || s->stride[1] == 1) && (rows <= 1 || s->stride[0] == blocks);
}

static int begin(Call* call, PyObject* stream) {
    PyObject* v = PyObject_CallNoArgs(G.device);
    if (!v) return 0;
    call->device = PyLong_AsLong(v);
    if (stream == Py_None) {
        PyObject* s = PyObject_CallOneArg(G.raw_stream, v);
        Py_DECREF(v);
        if (!(v = s)) return 0;
    } else if (PyLong_Check(stream)) {
        Py_DECREF(v);
        v = Py_NewRef(stream);
    } else {
        Py_DECREF(v);
        if (!(v = PyObject_GetAttr(stream, G.s_cuda_stream))) return 0;
    }
    call->stream = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

static PyObject* not_plain(void) {
    PyErr_Clear(); /* block.py's own checks find it again */
    Py_RETURN_NONE;
}

#define MADE(call_)                 \
    int status_;                    \
    Py_BEGIN_ALLOW_THREADS;         \
    status_ = (call_);              \
    Py_END_ALLOW_THREADS;           \
    return PyLong_FromLong(status_)

/* ---- the calls ---------------------------------------------------------------- */

/* y, x, weight, eps, residual, h, rstd, y8, y8_scale, h8, h8_scale, stream */
static PyObject* rmsnorm_forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor y, x, w, res, h, rstd, y8, y8s, h8, h8s;
    int code, kind, hkind, wcode = MP_FP32;
    (void)self;
    if (n != 12 || !F.rms_forward || !begin(&call, a[11]) || !matrix(a[1], &call, &x, &code) ||
        !like(a[0], &call, &x, 1, &y) || !vector(a[2], &call, x.size[1], &w) || !like(a[4], &call, &x, 1, &res) ||
        !like(a[5], &call, &x, 1, &h) || !vector(a[6], &call, x.size[0], &rstd) ||
        !rows8(a[7], a[8], &call, x.size[0], x.size[1], &y8, &y8s, &kind) ||
        !rows8(a[9], a[10], &call, x.size[0], x.size[1], &h8, &h8s, &hkind) || hkind == MP_SCALE_ROW ||
        (rstd.dtype && rstd.dtype != G.dtype[MP_FP32]) || (w.dtype && (wcode = type_code(w.dtype)) < 0))
        return not_plain();
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return not_plain();
    MADE(F.rms_forward(y.p, h.p, rstd.p, y8.p, y8s.p, h8.p, h8s.p, x.p, res.p, w.p, x.size[0], x.size[1], y.stride[0],
                       h.stride[0], y8.stride[0], h8.stride[0], x.stride[0], res.stride[0], (float)eps, code, wcode,
                       kind, call.stream));
}

/* dx, dweight, dy, h, weight, rstd, dh, h_scale, workspace, stream */
static PyObject* rmsnorm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor dx, dw, dy, h, hs, w, rstd, dh, ws;
    int code, kind, wcode = MP_FP32;
    (void)self;
    if (n != 10 || !F.rms_backward || !begin(&call, a[9]) || !matrix(a[2], &call, &dy, &code) ||
        !like(a[0], &call, &dy, 1, &dx) || !vector(a[1], &call, dy.size[1], &dw) ||
        !vector(a[4], &call, dy.size[1], &w) || !vector(a[5], &call, dy.size[0], &rstd) || !rstd.p ||
        !like(a[6], &call, &dy, 1, &dh) || rstd.dtype != G.dtype[MP_FP32])
        return not_plain();
    if (a[7] == Py_None) {
        hs.p = NULL;
        if (!like(a[3], &call, &dy, 0, &h)) return not_plain();
    } else if (!rows8(a[3], a[7], &call, dy.size[0], dy.size[1], &h, &hs, &kind) || kind != MP_SCALE_BLOCK) {
        return not_plain();
    }
    if ((w.dtype && (wcode = type_code(w.dtype)) < 0) || (dw.dtype && w.dtype && dw.dtype != w.dtype) ||
        (dw.dtype && (wcode = type_code(dw.dtype)) < 0))
        return not_plain();
    ws.p = NULL;
    ws.size[0] = 0;
    if (a[8] != Py_None &&
        (!tensor(a[8], &call, 1, &ws) || ws.dtype != G.uint8 || (ws.size[0] > 1 && ws.stride[0] != 1)))
        return not_plain();
    MADE(F.rms_backward(dx.p, dw.p, dy.p, dh.p, h.p, hs.p, w.p, rstd.p, dy.size[0], dy.size[1], dx.stride[0],
                        dy.stride[0], dh.stride[0], h.stride[0], code, wcode, ws.p, (size_t)ws.size[0], call.stream));
}

/* [tokens, heads, head_dim], the token's distance the larger (block.py passes other orders on). */
static int heads_of(PyObject* t, const Call* call, const Tensor* x, Tensor* to) {
    return tensor(t, call, 3, to) && to->stride[2] == 1 && to->stride[1] >= to->size[2] && to->size[1] <= 1024 &&
           to->stride[1] < ((int64_t)1 << 40) &&
           to->stride[0] >= (to->size[1] - 1) * to->stride[1] + to->size[2] &&
           (!x || (to->dtype == x->dtype && to->size[0] == x->size[0] && to->size[2] == x->size[2]));
}

/* q_out, q, k_out, k, turns, positions, first_position, interleaved, inverse, factor, stream */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor qo, q, ko, k, turns, pos;
    int code, icode = MP_INT64;
    (void)self;
    if (n != 11 || !F.rope || !begin(&call, a[10]) || !heads_of(a[1], &call, NULL, &q) ||
        (code = type_code(q.dtype)) < 0 || !heads_of(a[0], &call, &q, &qo) || qo.size[1] != q.size[1])
        return not_plain();
    k.p = ko.p = NULL;
    k.size[1] = k.stride[0] = k.stride[1] = ko.stride[0] = ko.stride[1] = 0;
    if (a[3] != Py_None && (!heads_of(a[3], &call, &q, &k) || !heads_of(a[2], &call, &q, &ko) || ko.size[1] != k.size[1]))
        return not_plain();
    if ((a[3] == Py_None && a[2] != Py_None) || !tensor(a[4], &call, 1, &turns) || turns.dtype != G.int64 ||
        turns.size[0] > 512 || (turns.size[0] > 1 && turns.stride[0] != 1) || !vector(a[5], &call, q.size[0], &pos))
        return not_plain();
    if (pos.dtype == G.int32)
        icode = MP_INT32;
    else if (pos.dtype && pos.dtype != G.int64)
        return not_plain();
    const int64_t first = PyLong_AsLongLong(a[6]);
    const int interleaved = PyObject_IsTrue(a[7]), inverse = PyObject_IsTrue(a[8]);
    const double factor = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred() || q.size[2] > 1024) return not_plain();
    MADE(F.rope(qo.p, q.p, ko.p, k.p, turns.p, pos.p, first, q.size[0], (int32_t)q.size[1], (int32_t)k.size[1],
                (int32_t)q.size[2], 2 * (int32_t)turns.size[0], qo.stride[0], qo.stride[1], q.stride[0], q.stride[1],
                ko.stride[0], ko.stride[1], k.stride[0], k.stride[1], (float)factor, interleaved, inverse, code, icode,
                call.stream));
}

/* y, gate, up, activation, gate8, gate8_scale, up8, up8_scale, stream */
static PyObject* gated_forward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor y, g, u, g8, g8s, u8, u8s;
    int code, gkind, ukind;
    (void)self;
    if (n != 9 || !F.gated_forward || !begin(&call, a[8]) || !matrix(a[1], &call, &g, &code) ||
        !like(a[0], &call, &g, 0, &y) || !like(a[2], &call, &g, 1, &u) ||
        !rows8(a[4], a[5], &call, g.size[0], g.size[1], &g8, &g8s, &gkind) || gkind == MP_SCALE_ROW ||
        !rows8(a[6], a[7], &call, g.size[0], g.size[1], &u8, &u8s, &ukind) || ukind == MP_SCALE_ROW)
        return not_plain();
    const long act = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) return not_plain();
    MADE(F.gated_forward(y.p, g8.p, g8s.p, u8.p, u8s.p, g.p, u.p, g.size[0], g.size[1], y.stride[0], g8.stride[0],
                         u8.stride[0], g.stride[0], u.stride[0], (int32_t)act, code, call.stream));
}

/* dgate, dup, dy, gate, up, activation, gate_scale, up_scale, y, stream */
static PyObject* gated_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor dg, du, dy, g, gs, u, us, y;
    int code, kind;
    (void)self;
    if (n != 10 || !F.gated_backward || !begin(&call, a[9]) || !matrix(a[2], &call, &dy, &code) ||
        !like(a[0], &call, &dy, 0, &dg) || !like(a[1], &call, &dy, 1, &du) || !like(a[8], &call, &dy, 1, &y) ||
        (a[1] == Py_None) != (a[4] == Py_None))
        return not_plain();
    if (a[6] == Py_None) {
        gs.p = us.p = NULL;
        if (a[7] != Py_None || !like(a[3], &call, &dy, 0, &g) || !like(a[4], &call, &dy, 1, &u)) return not_plain();
    } else if (!rows8(a[3], a[6], &call, dy.size[0], dy.size[1], &g, &gs, &kind) || kind != MP_SCALE_BLOCK ||
               !rows8(a[4], a[7], &call, dy.size[0], dy.size[1], &u, &us, &kind) || kind == MP_SCALE_ROW) {
        return not_plain();
    }
    const long act = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return not_plain();
    MADE(F.gated_backward(dg.p, du.p, y.p, dy.p, g.p, gs.p, u.p, us.p, dy.size[0], dy.size[1], dg.stride[0],
                          du.stride[0], y.stride[0], dy.stride[0], g.stride[0], u.stride[0], (int32_t)act, code,
                          call.stream));
}

/* q, scale, x, stream */
static PyObject* pack8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor q, s, x;
    int code, kind;
    (void)self;
    if (n != 4 || !F.pack || !begin(&call, a[3]) || !matrix(a[2], &call, &x, &code) ||
        !rows8(a[0], a[1], &call, x.size[0], x.size[1], &q, &s, &kind) || !kind)
        return not_plain();
    MADE(F.pack(q.p, s.p, x.p, x.size[0], x.size[1], q.stride[0], x.stride[0], code, kind, call.stream));
}

/* x, q, scale, stream */
static PyObject* unpack8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Call call;
    Tensor q, s, x;
    int code, kind;
    (void)self;
    if (n != 4 || !F.unpack || !begin(&call, a[3]) || !matrix(a[0], &call, &x, &code) ||
        !rows8(a[1], a[2], &call, x.size[0], x.size[1], &q, &s, &kind) || !kind)
        return not_plain();
    MADE(F.unpack(x.p, q.p, s.p, x.size[0], x.size[1], x.stride[0], q.stride[0], code, kind, call.stream));
}

/* tensor, parameter, (bf16, fp16, fp32, uint8, e4m3, int32, int64), device, raw_stream, (addresses of the library's
 * functions in the order of F) */
static PyObject* bind(PyObject* self, PyObject* args) {
    PyObject *tensor_type, *parameter_type, *dt[7], *device, *raw_stream, *v[7];
    (void)self;
    if (!PyArg_ParseTuple(args, "OO(OOOOOOO)OO(OOOOOOO)", &tensor_type, &parameter_type, &dt[0], &dt[1], &dt[2], &dt[3],
                          &dt[4], &dt[5], &dt[6], &device, &raw_stream, &v[0], &v[1], &v[2], &v[3], &v[4], &v[5],
                          &v[6]))
        return NULL;
    void* at[7];
    for (int i = 0; i < 7; ++i) {
        at[i] = PyLong_AsVoidPtr(v[i]);
        if (PyErr_Occurred()) return NULL;
    }
    /* kept for the life of the process */
    G.tensor = (PyTypeObject*)Py_NewRef(tensor_type);
    G.parameter = (PyTypeObject*)Py_NewRef(parameter_type);
    for (int i = 0; i < 3; ++i) G.dtype[i] = Py_NewRef(dt[i]);
    G.uint8 = Py_NewRef(dt[3]);
    G.e4m3 = Py_NewRef(dt[4]);
    G.int32 = Py_NewRef(dt[5]);
    G.int64 = Py_NewRef(dt[6]);
    G.device = Py_NewRef(device);
    G.raw_stream = Py_NewRef(raw_stream);
    F.rms_forward = (rms_forward_fn)at[0];
    F.rms_backward = (rms_backward_fn)at[1];
    F.rope = (rope_fn)at[2];
    F.gated_forward = (gated_forward_fn)at[3];
    F.gated_backward = (gated_backward_fn)at[4];
    F.pack = (pack_fn)at[5];
    F.unpack = (unpack_fn)at[6];
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL}, FAST(rmsnorm_forward), FAST(rmsnorm_backward), FAST(rope),
    FAST(gated_forward), FAST(gated_backward), FAST(pack8), FAST(unpack8), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    G.s_get_device = PyUnicode_InternFromString("get_device");
    G.s_dtype = PyUnicode_InternFromString("dtype");
    G.s_shape = PyUnicode_InternFromString("shape");
    G.s_stride = PyUnicode_InternFromString("stride");
    G.s_data_ptr = PyUnicode_InternFromString("data_ptr");
    G.s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!G.s_get_device || !G.s_dtype || !G.s_shape || !G.s_stride || !G.s_data_ptr || !G.s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
