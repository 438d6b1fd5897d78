/*
 * _fastcall: a minimal CPython extension that calls moe_finalize_ex of the
 * loaded libmoe_finalize.so.  ctypes converts each of the call's twenty
 * arguments through its generic machinery on every call, which costs more
 * host time than the decode-size kernel takes on the GPU.  Here call_now
 * converts them directly, and pack/call go further for repeated calls: the
 * arguments are packed once into a C struct (a capsule) and each call passes
 * only the stream.  checked_call does the Python binding's argument checks
 * on DLPack descriptions of the tensors before calling; checked_linear and
 * checked_gated, checked_backward, checked_expert and checked_permute do so for
 * the calls of moe_ffn.h, and call_backward, call_expert and call_permute
 * convert those calls' arguments.  Nothing here computes anything.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <stdlib.h>

typedef int (*finalize_ex_fn)(const void *permuted_out, int64_t P, const int32_t *idx_map,
                              const void *weights, int wkind, float routed_scale,
                              const void *shared_out, const void *residual, const void *gamma,
                              float eps, void *out, void *residual_out, void *norm_out, int T,
                              int K, int H, int splits_hint, int threads_hint, unsigned flags,
                              void *stream);

typedef struct {
    finalize_ex_fn fn;
    const void *permuted_out;
    int64_t P;
    const int32_t *idx_map;
    const void *weights;
    int wkind;
    float routed_scale;
    const void *shared_out, *residual, *gamma;
    float eps;
    void *out, *residual_out, *norm_out;
    int T, K, H, splits, threads;
    unsigned flags;
} bound_call;

static const char *kCapsule = "moe_finalize_bound_call";

static void free_bound(PyObject *cap) {
    free(PyCapsule_GetPointer(cap, kCapsule));
}

static void *as_ptr(PyObject *o) {
    return o == Py_None ? NULL : PyLong_AsVoidPtr(o);
}

/* Converts the twenty positional arguments (fn_address, permuted_out, P,
 * idx_map, weights, wkind, routed_scale, shared_out, residual, gamma, eps,
 * out, residual_out, norm_out, T, K, H, splits, threads, flags) into `b`.
 * Pointers are ints (or None), as tensor.data_ptr() gives them.  Returns 0,
 * or -1 with a Python error set. */
static int parse_call(PyObject *const *a, bound_call *b) {
    b->fn = (finalize_ex_fn)as_ptr(a[0]);
    b->permuted_out = as_ptr(a[1]);
    b->P = (int64_t)PyLong_AsLongLong(a[2]);
    b->idx_map = (const int32_t *)as_ptr(a[3]);
    b->weights = as_ptr(a[4]);
    b->wkind = (int)PyLong_AsLong(a[5]);
    b->routed_scale = (float)PyFloat_AsDouble(a[6]);
    b->shared_out = as_ptr(a[7]);
    b->residual = as_ptr(a[8]);
    b->gamma = as_ptr(a[9]);
    b->eps = (float)PyFloat_AsDouble(a[10]);
    b->out = as_ptr(a[11]);
    b->residual_out = as_ptr(a[12]);
    b->norm_out = as_ptr(a[13]);
    b->T = (int)PyLong_AsLong(a[14]);
    b->K = (int)PyLong_AsLong(a[15]);
    b->H = (int)PyLong_AsLong(a[16]);
    b->splits = (int)PyLong_AsLong(a[17]);
    b->threads = (int)PyLong_AsLong(a[18]);
    b->flags = (unsigned)PyLong_AsUnsignedLong(a[19]);
    if (PyErr_Occurred()) return -1;
    if (!b->fn) {
        PyErr_SetString(PyExc_ValueError, "null function pointer");
        return -1;
    }
    return 0;
}

static int enqueue(const bound_call *b, void *stream) {
    return b->fn(b->permuted_out, b->P, b->idx_map, b->weights, b->wkind, b->routed_scale,
                 b->shared_out, b->residual, b->gamma, b->eps, b->out, b->residual_out,
                 b->norm_out, b->T, b->K, b->H, b->splits, b->threads, b->flags, stream);
}

/* pack(<the twenty arguments>) -> capsule holding them */
static PyObject *pack(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 20) {
        PyErr_SetString(PyExc_TypeError, "pack takes 20 arguments");
        return NULL;
    }
    bound_call *b = (bound_call *)calloc(1, sizeof(bound_call));
    if (!b) return PyErr_NoMemory();
    if (parse_call(args, b) != 0) {
        free(b);
        return NULL;
    }
    return PyCapsule_New(b, kCapsule, free_bound);
}

/* call_now(<the twenty arguments>, stream_handle) -> status of one
 * moe_finalize_ex call, with nothing kept */
static PyObject *call_now(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 21) {
        PyErr_SetString(PyExc_TypeError, "call_now takes 21 arguments");
        return NULL;
    }
    bound_call b;
    if (parse_call(args, &b) != 0) return NULL;
    void *stream = as_ptr(args[20]);
    if (PyErr_Occurred()) return NULL;
    return PyLong_FromLong(enqueue(&b, stream));
}

/* ---------------------------------------------------------------------------
 * checked_call: the checks of the Python binding, done here on DLPack
 * descriptions of the tensors (one capsule per tensor, as torch's
 * to_dlpack() makes them), then one moe_finalize_ex call.  Reading a
 * tensor's device, dtype, shape, strides and address costs one DLPack
 * export instead of six attribute lookups.
 *
 * The structures below are the DLPack interchange format (DLTensor inside a
 * DLManagedTensor, capsule name "dltensor"): a public interface that any
 * consumer has to lay out the same way.  The capsules are only read; each
 * one's own destructor releases its tensor.
 */
typedef struct {
    int32_t device_type;
    int32_t device_id;
} dl_device;

typedef struct {
    uint8_t code;
    uint8_t bits;
    uint16_t lanes;
} dl_dtype;

typedef struct {
    void *data;
    dl_device device;
    int32_t ndim;
    dl_dtype dtype;
    int64_t *shape;
    int64_t *strides;
    uint64_t byte_offset;
} dl_tensor;

typedef struct {
    dl_tensor t;
    void *manager_ctx;
    void (*deleter)(void *self);
} dl_managed;

enum { DL_INT = 0, DL_FLOAT = 2, DL_BFLOAT = 4 };
enum { DL_CUDA = 2 };

/* a tensor description; NULL for None (or on error, with a Python error) */
static const dl_tensor *described(PyObject *cap) {
    if (cap == Py_None) return NULL;
    dl_managed *m = (dl_managed *)PyCapsule_GetPointer(cap, "dltensor");
    return m ? &m->t : NULL;
}

/* 1 when t is a dense row-major array on CUDA device `dev` of element type
 * (code, bits), with ndim dimensions; its sizes go to dims */
static int dense(const dl_tensor *t, int dev, uint8_t code, uint8_t bits, int ndim,
                 int64_t *dims) {
    if (!t || t->device.device_type != DL_CUDA || t->device.device_id != dev) return 0;
    if (t->dtype.code != code || t->dtype.bits != bits || t->dtype.lanes != 1) return 0;
    if (t->ndim != ndim) return 0;
    int64_t stride = 1;
    for (int d = ndim - 1; d >= 0; --d) {
        dims[d] = t->shape[d];
        if (t->strides && t->shape[d] != 1 && t->strides[d] != stride) return 0;
        stride *= t->shape[d];
    }
    return 1;
}

static void *address(const dl_tensor *t) {
    return t ? (void *)((char *)t->data + t->byte_offset) : NULL;
}

/* checked_call(fn_address, wkind, weight_code, weight_bits, routed_scale,
 *              eps, device, splits, threads, flags, stream, permuted_out,
 *              idx_map, weights, shared_out, residual, gamma, out,
 *              residual_out, norm_out) -> status
 * The last nine are DLPack capsules or None.  Returns moe_finalize_ex's
 * status, or -1 when a tensor fails the binding's checks (wrong device,
 * dtype, rank, shape or layout, or a missing or extra tensor): the caller
 * then runs its own checks to report which. */
static PyObject *checked_call(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 20) {
        PyErr_SetString(PyExc_TypeError, "checked_call takes 20 arguments");
        return NULL;
    }
    finalize_ex_fn fn = (finalize_ex_fn)as_ptr(a[0]);
    const int wkind = (int)PyLong_AsLong(a[1]);
    const uint8_t wcode = (uint8_t)PyLong_AsLong(a[2]);
    const uint8_t wbits = (uint8_t)PyLong_AsLong(a[3]);
    const float scale = (float)PyFloat_AsDouble(a[4]);
    const float eps = (float)PyFloat_AsDouble(a[5]);
    const int dev = (int)PyLong_AsLong(a[6]);
    const int splits = (int)PyLong_AsLong(a[7]);
    const int threads = (int)PyLong_AsLong(a[8]);
    const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[9]);
    void *stream = as_ptr(a[10]);
    if (PyErr_Occurred()) return NULL;
    if (!fn) {
        PyErr_SetString(PyExc_ValueError, "null function pointer");
        return NULL;
    }
    const dl_tensor *t[9];
    for (int i = 0; i < 9; ++i) {
        t[i] = described(a[11 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    const dl_tensor *x = t[0], *idx = t[1], *w = t[2], *sh = t[3], *res = t[4], *gam = t[5],
                    *out = t[6], *rout = t[7], *nout = t[8];
    int64_t xd[2], id[2], d2[2], d1[1];
    int ok = dense(x, dev, DL_BFLOAT, 16, 2, xd) && dense(idx, dev, DL_INT, 32, 2, id) &&
             dense(w, dev, wcode, wbits, 2, d2) && d2[0] == id[0] && d2[1] == id[1] &&
             dense(sh, dev, DL_BFLOAT, 16, 2, d2) && d2[0] == id[0] && d2[1] == xd[1];
    const int norm = res != NULL;
    if (ok && (norm != (gam != NULL) || norm != (rout != NULL) || norm != (nout != NULL) ||
               (!norm && !out)))
        ok = 0;
    const dl_tensor *rows[4] = {res, out, rout, nout};
    for (int i = 0; ok && i < 4; ++i)
        if (rows[i])
            ok = dense(rows[i], dev, DL_BFLOAT, 16, 2, d2) && d2[0] == id[0] && d2[1] == xd[1];
    if (ok && gam) ok = dense(gam, dev, DL_BFLOAT, 16, 1, d1) && d1[0] == xd[1];
    if (ok && (xd[1] > 0x7FFFFFFF || id[0] > 0x7FFFFFFF || id[1] > 0x7FFFFFFF)) ok = 0;
    if (!ok) return PyLong_FromLong(-1);
    return PyLong_FromLong(fn(address(x), xd[0], (const int32_t *)address(idx), address(w),
                              wkind, scale, address(sh), address(res), address(gam), eps,
                              address(out), address(rout), address(nout), (int)id[0],
                              (int)id[1], (int)xd[1], splits, threads, flags, stream));
}

/* ---------------------------------------------------------------------------
 * checked_linear / checked_gated: the same for moe_linear and moe_gated_ffn.
 *
 * checked_linear(fn_address, activation, out_fp32, device, stream, x, weight,
 *                bias, residual, out, preact) -> status
 * checked_gated(fn_address, activation, device, stream, x, weight, bias, out,
 *               preact) -> status
 * The tensors are DLPack capsules or None; -1 when one fails the checks.  out
 * and preact may be addresses (ints): the caller made them for this call, of
 * the right type and shape. */
typedef int (*linear_fn)(const void *x, const void *weight, const void *bias,
                         const void *residual, int act, void *out, int out_type, void *preact,
                         int T, int N, int K, void *stream);
typedef int (*gated_fn)(const void *x, const void *weight, const void *bias, int act, void *out,
                        void *preact, int T, int I, int H, void *stream);

/* an output: its description in *t, or its address in *at when it is an int */
static int output(PyObject *o, const dl_tensor **t, void **at) {
    *t = NULL;
    *at = NULL;
    if (PyLong_Check(o)) *at = PyLong_AsVoidPtr(o);
    else *t = described(o);
    if (*t) *at = address(*t);
    return !PyErr_Occurred();
}

/* 1 when the optional bf16 operand t is absent, or dense [a, b] (b < 0: [a]) */
static int optional_bf16(const dl_tensor *t, int dev, int64_t a, int64_t b) {
    int64_t d[2];
    if (!t) return 1;
    if (b < 0) return dense(t, dev, DL_BFLOAT, 16, 1, d) && d[0] == a;
    return dense(t, dev, DL_BFLOAT, 16, 2, d) && d[0] == a && d[1] == b;
}

static PyObject *checked_linear(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 11) {
        PyErr_SetString(PyExc_TypeError, "checked_linear takes 11 arguments");
        return NULL;
    }
    linear_fn fn = (linear_fn)as_ptr(a[0]);
    const int act = (int)PyLong_AsLong(a[1]);
    const int fp32 = (int)PyLong_AsLong(a[2]);
    const int dev = (int)PyLong_AsLong(a[3]);
    void *stream = as_ptr(a[4]);
    if (PyErr_Occurred()) return NULL;
    const dl_tensor *t[6];
    for (int i = 0; i < 4; ++i) {
        t[i] = described(a[5 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    void *out, *preact;
    if (!output(a[9], &t[4], &out) || !output(a[10], &t[5], &preact)) return NULL;
    int64_t x[2], w[2], o[2];
    const int ok = fn && dense(t[0], dev, DL_BFLOAT, 16, 2, x) &&
                   dense(t[1], dev, DL_BFLOAT, 16, 2, w) && w[1] == x[1] &&
                   (t[4] ? dense(t[4], dev, fp32 ? DL_FLOAT : DL_BFLOAT, fp32 ? 32 : 16, 2, o) &&
                               o[0] == x[0] && o[1] == w[0]
                         : out || !x[0]) &&
                   optional_bf16(t[2], dev, w[0], -1) &&
                   optional_bf16(t[3], dev, x[0], w[0]) && optional_bf16(t[5], dev, x[0], w[0]) &&
                   x[0] <= 0x7FFFFFFF && x[1] <= 0x7FFFFFFF && w[0] <= 0x7FFFFFFF;
    if (!ok) return PyLong_FromLong(-1);
    return PyLong_FromLong(fn(address(t[0]), address(t[1]), address(t[2]), address(t[3]), act,
                              out, fp32, preact, (int)x[0], (int)w[0],
                              (int)x[1], stream));
}

static PyObject *checked_gated(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 9) {
        PyErr_SetString(PyExc_TypeError, "checked_gated takes 9 arguments");
        return NULL;
    }
    gated_fn fn = (gated_fn)as_ptr(a[0]);
    const int act = (int)PyLong_AsLong(a[1]);
    const int dev = (int)PyLong_AsLong(a[2]);
    void *stream = as_ptr(a[3]);
    if (PyErr_Occurred()) return NULL;
    const dl_tensor *t[5];
    for (int i = 0; i < 3; ++i) {
        t[i] = described(a[4 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    void *out, *preact;
    if (!output(a[7], &t[3], &out) || !output(a[8], &t[4], &preact)) return NULL;
    int64_t x[2], w[2], o[2];
    const int ok = fn && dense(t[0], dev, DL_BFLOAT, 16, 2, x) &&
                   dense(t[1], dev, DL_BFLOAT, 16, 2, w) && w[1] == x[1] && w[0] % 2 == 0 &&
                   (t[3] ? dense(t[3], dev, DL_BFLOAT, 16, 2, o) && o[0] == x[0] &&
                               2 * o[1] == w[0]
                         : out || !x[0]) &&
                   optional_bf16(t[2], dev, w[0], -1) && optional_bf16(t[4], dev, x[0], w[0]) &&
                   x[0] <= 0x7FFFFFFF && x[1] <= 0x7FFFFFFF && w[0] <= 0x7FFFFFFF;
    if (!ok) return PyLong_FromLong(-1);
    return PyLong_FromLong(fn(address(t[0]), address(t[1]), address(t[2]), act, out,
                              preact, (int)x[0], (int)(w[0] / 2), (int)x[1], stream));
}

/* ---------------------------------------------------------------------------
 * call_backward, call_expert, call_permute: the entry points of moe_ffn.h with
 * many arguments, converted directly.  The first argument is the function's
 * address, the others are its own in order, pointers as ints or None; the
 * tensors were checked by the binding. */
typedef int (*backward_fn)(const void *dout, const void *x, const void *weight, int act,
                           const void *preact, void *dx, void *dweight, void *dbias, int T,
                           int n, int K, void *workspace, size_t workspace_bytes, void *stream);
typedef int (*expert_fn)(const void *x, int64_t T, const int32_t *row_token,
                         const int32_t *offsets, const int32_t *counts, const void *weight,
                         const void *bias, int act, void *out, int64_t P, int E, int M, int K,
                         void *stream);
typedef int (*permute_fn)(const int32_t *ids, int T, int K, int E, int tile, int32_t *idx_map,
                          int32_t *row_token, int64_t P, int32_t *offsets, int32_t *counts,
                          void *workspace, size_t workspace_bytes, void *stream);

enum { MOST_ARGS = 15 };

/* n ints (or None, as 0) into v; 0, or -1 with a Python error */
static int parse_ints(PyObject *const *a, Py_ssize_t nargs, int n, const char *name,
                      long long *v) {
    if (nargs != n) {
        PyErr_Format(PyExc_TypeError, "%s takes %d arguments", name, n);
        return -1;
    }
    for (int i = 0; i < n; ++i) v[i] = a[i] == Py_None ? 0 : PyLong_AsLongLong(a[i]);
    if (PyErr_Occurred()) return -1;
    if (!v[0]) {
        PyErr_SetString(PyExc_ValueError, "null function pointer");
        return -1;
    }
    return 0;
}

/* PTR(i): argument i as a pointer; INT(i): as an int, out of range as -1 */
#define PTR(i) ((void *)(intptr_t)v[i])
#define INT(i) (v[i] < -1 || v[i] > 0x7FFFFFFF ? -1 : (int)v[i])

static PyObject *call_backward(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    long long v[MOST_ARGS];
    if (parse_ints(a, nargs, 15, "call_backward", v) != 0) return NULL;
    return PyLong_FromLong(((backward_fn)PTR(0))(PTR(1), PTR(2), PTR(3), INT(4), PTR(5), PTR(6),
                                                 PTR(7), PTR(8), INT(9), INT(10), INT(11),
                                                 PTR(12), (size_t)v[13], PTR(14)));
}

static PyObject *call_expert(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    long long v[MOST_ARGS];
    if (parse_ints(a, nargs, 15, "call_expert", v) != 0) return NULL;
    return PyLong_FromLong(((expert_fn)PTR(0))(PTR(1), v[2], PTR(3), PTR(4), PTR(5), PTR(6),
                                               PTR(7), INT(8), PTR(9), v[10], INT(11), INT(12),
                                               INT(13), PTR(14)));
}

static PyObject *call_permute(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    long long v[MOST_ARGS];
    if (parse_ints(a, nargs, 14, "call_permute", v) != 0) return NULL;
    return PyLong_FromLong(((permute_fn)PTR(0))(PTR(1), INT(2), INT(3), INT(4), INT(5), PTR(6),
                                                PTR(7), v[8], PTR(9), PTR(10), PTR(11),
                                                (size_t)v[12], PTR(13)));
}

/* checked_backward(fn_address, gated, activation, device, stream, dout, x,
 *                  weight, preact, dx, dweight, dbias, workspace,
 *                  workspace_bytes) -> status
 * The checks of the binding's backward calls, then the call.  dout to preact
 * are DLPack capsules (preact or None), the gradients capsules, addresses of
 * outputs made for this call, or None; workspace is an address or None.  -1
 * when a tensor fails the checks. */
static PyObject *checked_backward(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 14) {
        PyErr_SetString(PyExc_TypeError, "checked_backward takes 14 arguments");
        return NULL;
    }
    backward_fn fn = (backward_fn)as_ptr(a[0]);
    const int gated = (int)PyLong_AsLong(a[1]);
    const int act = (int)PyLong_AsLong(a[2]);
    const int dev = (int)PyLong_AsLong(a[3]);
    void *stream = as_ptr(a[4]);
    void *workspace = as_ptr(a[12]);
    const size_t bytes = (size_t)PyLong_AsUnsignedLongLong(a[13]);
    if (PyErr_Occurred()) return NULL;
    const dl_tensor *t[4], *o[3];
    void *grad[3];
    for (int i = 0; i < 4; ++i) {
        t[i] = described(a[5 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    for (int i = 0; i < 3; ++i) {
        o[i] = NULL;
        grad[i] = NULL;
        if (a[9 + i] != Py_None && !output(a[9 + i], &o[i], &grad[i])) return NULL;
    }
    int64_t d[3], x[3], w[3];
    int ok = fn && dense(t[0], dev, DL_BFLOAT, 16, 2, d) && dense(t[1], dev, DL_BFLOAT, 16, 2, x) &&
             dense(t[2], dev, DL_BFLOAT, 16, 2, w) && x[0] == d[0] && w[1] == x[1] &&
             w[0] == (gated ? 2 * d[1] : d[1]);
    ok = ok && (gated || act ? t[3] != NULL : 1) && optional_bf16(t[3], dev, d[0], w[0]);
    ok = ok && optional_bf16(o[0], dev, x[0], x[1]) && optional_bf16(o[1], dev, w[0], w[1]) &&
         optional_bf16(o[2], dev, w[0], -1) && d[0] <= 0x7FFFFFFF && d[1] <= 0x7FFFFFFF &&
         x[1] <= 0x7FFFFFFF;
    if (!ok) return PyLong_FromLong(-1);
    /* the preactivations of the identity are not read */
    return PyLong_FromLong(fn(address(t[0]), address(t[1]), address(t[2]), act,
                              gated || act ? address(t[3]) : NULL, grad[0], grad[1], grad[2],
                              (int)d[0], (int)d[1], (int)x[1], workspace, bytes, stream));
}

/* checked_expert(fn_address, gated, activation, device, stream, x, row_token,
 *                offsets, counts, weight, bias, out) -> status
 * Likewise for the expert products: capsules; row_token and bias may be None,
 * out an address. */
static PyObject *checked_expert(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 12) {
        PyErr_SetString(PyExc_TypeError, "checked_expert takes 12 arguments");
        return NULL;
    }
    expert_fn fn = (expert_fn)as_ptr(a[0]);
    const int gated = (int)PyLong_AsLong(a[1]);
    const int act = (int)PyLong_AsLong(a[2]);
    const int dev = (int)PyLong_AsLong(a[3]);
    void *stream = as_ptr(a[4]);
    if (PyErr_Occurred()) return NULL;
    const dl_tensor *t[6], *o;
    void *out;
    for (int i = 0; i < 6; ++i) {
        t[i] = described(a[5 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    if (!output(a[11], &o, &out)) return NULL;
    int64_t x[3], r[3], f[3], c[3], w[3], b[3];
    int ok = fn && dense(t[0], dev, DL_BFLOAT, 16, 2, x) && dense(t[4], dev, DL_BFLOAT, 16, 3, w) &&
             w[2] == x[1] && dense(t[2], dev, DL_INT, 32, 1, f) && f[0] == w[0] + 1 &&
             dense(t[3], dev, DL_INT, 32, 1, c) && c[0] == w[0] && (!gated || w[1] % 2 == 0);
    ok = ok && (!t[1] || dense(t[1], dev, DL_INT, 32, 1, r)) &&
         (!t[5] || (dense(t[5], dev, DL_BFLOAT, 16, 2, b) && b[0] == w[0] && b[1] == w[1]));
    if (!ok) return PyLong_FromLong(-1);
    const int64_t P = t[1] ? r[0] : x[0], M = gated ? w[1] / 2 : w[1];
    ok = (o ? optional_bf16(o, dev, P, M) : out || !P) && w[0] <= 0x7FFFFFFF && M <= 0x7FFFFFFF &&
         x[1] <= 0x7FFFFFFF;
    if (!ok) return PyLong_FromLong(-1);
    return PyLong_FromLong(fn(address(t[0]), x[0], (const int32_t *)address(t[1]),
                              (const int32_t *)address(t[2]), (const int32_t *)address(t[3]),
                              address(t[4]), address(t[5]), act, out, P, (int)w[0], (int)M,
                              (int)x[1], stream));
}

/* 1 when the output t is dense int32 [a, b] (b < 0: [a]), or was given by its
 * address (null only when it is empty) */
static int int32_output(const dl_tensor *t, const void *at, int dev, int64_t a, int64_t b) {
    int64_t d[2];
    if (!t) return at || a * b == 0;
    if (b < 0) return dense(t, dev, DL_INT, 32, 1, d) && d[0] == a;
    return dense(t, dev, DL_INT, 32, 2, d) && d[0] == a && d[1] == b;
}

/* checked_permute(fn_address, device, stream, E, tile, P, expert_ids, idx_map,
 *                 row_token, offsets, counts, workspace, workspace_bytes) ->
 * status.  Likewise for moe_permute: expert_ids is a capsule, the outputs
 * capsules or addresses, workspace an address or None; P is the size of a
 * row_token given by its address. */
static PyObject *checked_permute(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 13) {
        PyErr_SetString(PyExc_TypeError, "checked_permute takes 13 arguments");
        return NULL;
    }
    permute_fn fn = (permute_fn)as_ptr(a[0]);
    const int dev = (int)PyLong_AsLong(a[1]);
    void *stream = as_ptr(a[2]);
    const int64_t E = PyLong_AsLongLong(a[3]), tile = PyLong_AsLongLong(a[4]);
    int64_t P = PyLong_AsLongLong(a[5]);
    void *workspace = as_ptr(a[11]);
    const size_t bytes = (size_t)PyLong_AsUnsignedLongLong(a[12]);
    if (PyErr_Occurred()) return NULL;
    const dl_tensor *ids = described(a[6]), *o[4];
    void *at[4];
    if (PyErr_Occurred()) return NULL;
    for (int i = 0; i < 4; ++i)
        if (!output(a[7 + i], &o[i], &at[i])) return NULL;
    int64_t d[2], r[1];
    int ok = fn && dense(ids, dev, DL_INT, 32, 2, d) && d[0] <= 0x7FFFFFFF && d[1] <= 0x7FFFFFFF &&
             E >= 0 && E < 0x7FFFFFFF && tile >= 0 && tile <= 0x7FFFFFFF;
    if (ok && o[1]) {
        ok = dense(o[1], dev, DL_INT, 32, 1, r);
        P = r[0];
    }
    ok = ok && int32_output(o[0], at[0], dev, d[0], d[1]) && int32_output(o[1], at[1], dev, P, -1) &&
         int32_output(o[2], at[2], dev, E + 1, -1) && int32_output(o[3], at[3], dev, E, -1);
    if (!ok) return PyLong_FromLong(-1);
    return PyLong_FromLong(fn((const int32_t *)address(ids), (int)d[0], (int)d[1], (int)E,
                              (int)tile, (int32_t *)at[0], (int32_t *)at[1], P, (int32_t *)at[2],
                              (int32_t *)at[3], workspace, bytes, stream));
}

/* call_size(fn_address, a, b) -> a size_t function of two ints */
static PyObject *call_size(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    long long v[MOST_ARGS];
    if (parse_ints(a, nargs, 3, "call_size", v) != 0) return NULL;
    return PyLong_FromSize_t(((size_t(*)(int, int))PTR(0))(INT(1), INT(2)));
}

/* permute_sizes(moe_permute_rows, moe_permute_workspace_bytes, T, K, E, tile)
 * -> (rows, workspace bytes); the first two are the functions' addresses */
static PyObject *permute_sizes(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    (void)self;
    long long v[MOST_ARGS];
    if (parse_ints(a, nargs, 6, "permute_sizes", v) != 0) return NULL;
    if (!v[1]) {
        PyErr_SetString(PyExc_ValueError, "null function pointer");
        return NULL;
    }
    const int64_t rows = ((int64_t(*)(int, int, int, int))PTR(0))(INT(2), INT(3), INT(4), INT(5));
    const size_t bytes = ((size_t(*)(int, int, int))PTR(1))(INT(2), INT(3), INT(4));
    return Py_BuildValue("Ln", (long long)rows, (Py_ssize_t)bytes);
}

#undef PTR
#undef INT

/* call(capsule, stream_handle) -> status of moe_finalize_ex */
static PyObject *call(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "call(capsule, stream)");
        return NULL;
    }
    bound_call *b = (bound_call *)PyCapsule_GetPointer(args[0], kCapsule);
    if (!b) return NULL;
    void *stream = as_ptr(args[1]);
    if (PyErr_Occurred()) return NULL;
    return PyLong_FromLong(enqueue(b, stream));
}

static PyMethodDef methods[] = {
    {"pack", (PyCFunction)(void (*)(void))pack, METH_FASTCALL,
     "Pack a moe_finalize_ex call into a capsule."},
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL,
     "Enqueue a packed call on a stream; returns the status."},
    {"call_now", (PyCFunction)(void (*)(void))call_now, METH_FASTCALL,
     "Enqueue one moe_finalize_ex call from its arguments; returns the status."},
    {"checked_call", (PyCFunction)(void (*)(void))checked_call, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one moe_finalize_ex call."},
    {"checked_linear", (PyCFunction)(void (*)(void))checked_linear, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one moe_linear call."},
    {"checked_gated", (PyCFunction)(void (*)(void))checked_gated, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one moe_gated_ffn call."},
    {"call_backward", (PyCFunction)(void (*)(void))call_backward, METH_FASTCALL,
     "Call moe_linear_backward or moe_gated_ffn_backward."},
    {"call_expert", (PyCFunction)(void (*)(void))call_expert, METH_FASTCALL,
     "Call moe_expert_gated_ffn or moe_expert_linear."},
    {"call_permute", (PyCFunction)(void (*)(void))call_permute, METH_FASTCALL,
     "Call moe_permute."},
    {"checked_backward", (PyCFunction)(void (*)(void))checked_backward, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one backward call."},
    {"checked_expert", (PyCFunction)(void (*)(void))checked_expert, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one expert product."},
    {"checked_permute", (PyCFunction)(void (*)(void))checked_permute, METH_FASTCALL,
     "Check DLPack-described tensors and enqueue one moe_permute call."},
    {"call_size", (PyCFunction)(void (*)(void))call_size, METH_FASTCALL,
     "Call a size function of two ints."},
    {"permute_sizes", (PyCFunction)(void (*)(void))permute_sizes, METH_FASTCALL,
     "Call moe_permute_rows and moe_permute_workspace_bytes."},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
