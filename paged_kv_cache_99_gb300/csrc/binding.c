/*
 * Python calls of the operators that a server makes many times per step outside a CUDA
 * graph: they check a dozen tensors each and launch kernels of a few microseconds, so the
 * checks are made here rather than in Python and the arguments passed without ctypes (host
 * time of a call on the Grace cores: the rotation 11.0 -> 5.2 us, the decode with attention
 * weights, three launches, 13.5 -> 8, the eviction 10 -> 4.5, the table 6 -> 3; where tensors
 * are read directly, by tensor_info.cpp, a call of twelve tensors 6.3 -> 3.0, a commit of 28
 * layers' caches 29.7 -> 10.3).  Same rules
 * as the package's other calls: TypeError for what is no CUDA tensor or of another type, ValueError
 * for a wrong shape, layout or device; the tensors' device is current for the call, the
 * default stream is that device's current one.  Each returns the library's status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "pa.h"
#include "tensor_info.h"

/* absent where tensor_info.cpp could not be built */
#pragma weak pa_tensor_info

enum { BF16 = 1, FP16 = 2, U8 = 4, E4M3 = 8, F32 = 16, I32 = 32, I64 = 64 };
enum { HALVES = BF16 | FP16, CACHES = BF16 | FP16 | U8 | E4M3 };
#define NUM_TYPES 7

static const char* const type_names[NUM_TYPES] = {"bfloat16", "float16", "uint8", "float8_e4m3fn",
                                                  "float32",  "int32",   "int64"};
static PyObject* types[NUM_TYPES];
static PyTypeObject* tensor_type;
static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr, *s_is_contiguous;
static PyObject *torch_c, *s_raw_stream, *s_current_device, *s_set_device;   /* torch._C and its functions */

typedef struct {
    void* ptr;
    long long shape[4], numel, step;   /* step: elements from one token to the next (rows only) */
    int ndim, type;                    /* type: one of the bits above */
} Tensor;

/* Takes over a reference to an int object (NULL: an error is set). */
static int as_int(PyObject* o, long long* out) {
    if (!o) return -1;
    *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int info_of(PyObject* t, TensorInfo* info) { return pa_tensor_info && pa_tensor_info(t, info) == 0; }

static int device_of(PyObject* t, const char* name, long long* device) {
    TensorInfo info;
    if (info_of(t, &info)) *device = info.device;
    else if (!PyObject_TypeCheck(t, tensor_type)) *device = -1;
    else if (as_int(PyObject_CallMethodNoArgs(t, s_get_device), device)) return -1;
    if (*device >= 0) return 0;
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return -1;
}

/* Reads a tensor of one of `allowed` types on `device` with ndim dimensions (0: any).  rows: each
 * token's heads are contiguous, with any stride between tokens; otherwise it is contiguous. */
static int take(PyObject* t, const char* name, int allowed, int ndim, long long device, int rows, Tensor* out) {
    long long dev, ptr = 0, strides[3];
    TensorInfo info;
    const int known = info_of(t, &info);
    if (known) {
        dev = info.device;
        if (dev < 0) {
            PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
            return -1;
        }
        out->type = info.type < 0 ? 0 : 1 << info.type;
    } else if (device_of(t, name, &dev)) {
        return -1;
    }
    if (!known || !(out->type & allowed)) {
        PyObject* dtype = PyObject_GetAttr(t, s_dtype);
        if (!dtype) return -1;
        out->type = 0;
        for (int i = 0; i < NUM_TYPES; ++i)
            if (dtype == types[i]) out->type = 1 << i;
        if (!(out->type & allowed)) {
            PyErr_Format(PyExc_TypeError, "%s: dtype %S is not one it can have", name, dtype);
            Py_DECREF(dtype);
            return -1;
        }
        Py_DECREF(dtype);
    }
    if (dev != device) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%lld, not on cuda:%lld", name, dev, device);
        return -1;
    }
    Py_ssize_t n;
    out->numel = 1;
    if (known) {
        n = info.ndim;
        for (Py_ssize_t i = 0; i < n; ++i) {
            out->numel *= info.shape[i];
            if (i < 4) out->shape[i] = info.shape[i];
        }
    } else {
        PyObject* shape = PyObject_GetAttr(t, s_shape);
        if (!shape) return -1;
        n = PyTuple_Check(shape) ? PyTuple_GET_SIZE(shape) : -1;
        for (Py_ssize_t i = 0; i < n; ++i) {
            const long long d = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
            out->numel *= d;
            if (i < 4) out->shape[i] = d;
        }
        Py_DECREF(shape);
        if (PyErr_Occurred()) return -1;
    }
    out->ndim = (int)n;
    if (ndim && n != ndim) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, not %zd", name, ndim, n);
        return -1;
    }
    for (int i = 0; i < ndim; ++i) {           /* the library takes them as ints */
        if (out->shape[i] > INT_MAX) {
            PyErr_Format(PyExc_ValueError, "%s: dimension %d is too large", name, i);
            return -1;
        }
    }
    if (rows) {
        const long long heads = out->shape[1], d = out->shape[2];
        if (known) {
            for (int i = 0; i < 3; ++i) strides[i] = info.stride[i];
        } else {
            PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
            if (!st) return -1;
            for (int i = 0; i < 3; ++i) strides[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
            Py_DECREF(st);
        }
        if (out->shape[0] && ((strides[2] != 1 && d > 1) || (strides[1] != d && heads > 1))) {
            PyErr_Format(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
            return -1;
        }
        out->step = out->shape[0] > 1 ? strides[0] : heads * d;     /* a single token's stride means nothing */
    } else {
        int contiguous;
        if (known) {
            contiguous = info.contiguous;
        } else {
            PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
            if (!c) return -1;
            contiguous = c == Py_True;
            Py_DECREF(c);
        }
        if (!contiguous) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            return -1;
        }
    }
    if (known) {
        out->ptr = info.ptr;
    } else {
        if (as_int(PyObject_CallMethodNoArgs(t, s_data_ptr), &ptr)) return -1;
        out->ptr = (void*)ptr;
    }
    return 0;
}

/* An argument that may be None (a null pointer then). */
static int take_or_none(PyObject* t, const char* name, int allowed, int ndim, long long device, Tensor* out) {
    if (t != Py_None) return take(t, name, allowed, ndim, device, 0, out);
    memset(out, 0, sizeof *out);
    return 0;
}

static int same_shape(const Tensor* a, const Tensor* b) {
    if (a->ndim != b->ndim) return 0;
    for (int i = 0; i < a->ndim; ++i)
        if (a->shape[i] != b->shape[i]) return 0;
    return 1;
}

static int is(const Tensor* a, long long d0, long long d1, long long d2) {    /* -1: no such dimension */
    return a->shape[0] == d0 && (d1 < 0 || a->shape[1] == d1) && (d2 < 0 || a->shape[2] == d2);
}

static int mismatch(void) {
    PyErr_SetString(PyExc_ValueError, "shape mismatch");
    return -1;
}

/* pa_dtype of a 16-bit tensor, and of a cache with its scales (checked: both or none, one value or
 * one per KV head); -1 with an error set. */
static int half_code(const Tensor* t) { return t->type == BF16 ? PA_BF16 : PA_FP16; }

static int cache_code(const Tensor* cache, const Tensor* ks, const Tensor* vs, long long heads) {
    if (cache->type & HALVES) return half_code(cache);
    if (!ks->ptr || !vs->ptr) {
        PyErr_SetString(PyExc_TypeError, "an FP8 cache needs k_scale and v_scale");
        return -1;
    }
    if (ks->numel != vs->numel || (ks->numel != 1 && ks->numel != heads)) {
        PyErr_SetString(PyExc_ValueError, "FP8 scales must hold one value or one per KV head, K and V alike");
        return -1;
    }
    return ks->numel == 1 ? PA_FP8_E4M3 : PA_FP8_E4M3_PER_HEAD;
}

static int check_workspace(const Tensor* ws) {
    if (!ws->ptr || ws->numel >= 256) return 0;
    PyErr_SetString(PyExc_ValueError, "workspace: at least 256 bytes");
    return -1;
}

/* The call's stream (None: the device's current one), and the device made current; *back: the device
 * to go back to, or -1. */
static int enter(long long device, PyObject* stream, void** raw, long long* back) {
    long long s, current;
    PyObject* dev = PyLong_FromLongLong(device);
    if (!dev) return -1;
    if (as_int(stream == Py_None ? PyObject_CallMethodOneArg(torch_c, s_raw_stream, dev) : Py_NewRef(stream), &s) ||
        as_int(PyObject_CallMethodNoArgs(torch_c, s_current_device), &current)) {
        Py_DECREF(dev);
        return -1;
    }
    *raw = (void*)s;
    *back = -1;
    if (current != device) {
        PyObject* r = PyObject_CallMethodOneArg(torch_c, s_set_device, dev);
        if (!r) {
            Py_DECREF(dev);
            return -1;
        }
        Py_DECREF(r);
        *back = current;
    }
    Py_DECREF(dev);
    return 0;
}

static PyObject* leave(long long back, pa_status status) {
    if (back >= 0) {
        PyObject* dev = PyLong_FromLongLong(back);
        PyObject* r = dev ? PyObject_CallMethodOneArg(torch_c, s_set_device, dev) : NULL;
        Py_XDECREF(dev);
        if (!r) return NULL;
        Py_DECREF(r);
    }
    return PyLong_FromLong(status);
}

static int want_args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return -1;
}

/* cos_sin, freqs (a buffer of float64), attention, stream */
static PyObject* rope_table(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor t;
    long long dev, back;
    void* stream;
    if (want_args(n, 4) || device_of(a[0], "cos_sin", &dev) || take(a[0], "cos_sin", F32, 2, dev, 0, &t)) return NULL;
    const double attention = PyFloat_AsDouble(a[2]);
    if (attention == -1.0 && PyErr_Occurred()) return NULL;
    Py_buffer f;
    if (PyObject_GetBuffer(a[1], &f, PyBUF_SIMPLE)) return NULL;
    PyObject* res = NULL;
    if (f.len % sizeof(double) || t.shape[1] != 2 * (long long)(f.len / sizeof(double))) {
        PyErr_SetString(PyExc_ValueError, "cos_sin must be [max_positions, 2 * len(freqs)]");
    } else if (!enter(dev, a[3], &stream, &back)) {
        res = leave(back, pa_rope_table(t.ptr, (int)t.shape[0], (int)t.shape[1], f.buf, (float)attention,
                                        (pa_stream_t)stream));
    }
    PyBuffer_Release(&f);
    return res;
}

/* q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, interleaved, k_scale, v_scale,
 * workspace, stream */
static PyObject* rope_and_cache(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor qo, q, k, v, kc, vc, slots, pos, table, ks, vs, ws;
    long long dev, back;
    void* stream;
    if (want_args(n, 14) || device_of(a[1], "q", &dev) || take(a[1], "q", HALVES, 3, dev, 1, &q) ||
        take(a[0], "q_out", q.type, 3, dev, 1, &qo) || take(a[2], "k", q.type, 3, dev, 1, &k) ||
        take(a[3], "v", q.type, 3, dev, 1, &v) || take(a[4], "k_cache", CACHES, 4, dev, 0, &kc) ||
        take(a[5], "v_cache", kc.type, 4, dev, 0, &vc) || take(a[6], "slot_mapping", I64, 1, dev, 0, &slots) ||
        take(a[7], "positions", I64, 1, dev, 0, &pos) || take(a[8], "cos_sin", F32, 2, dev, 0, &table) ||
        take_or_none(a[10], "k_scale", F32, 0, dev, &ks) || take_or_none(a[11], "v_scale", F32, 0, dev, &vs) ||
        take_or_none(a[12], "workspace", U8, 0, dev, &ws) || check_workspace(&ws))
        return NULL;
    const long long T = q.shape[0], H = k.shape[1], d = q.shape[2];
    if (!same_shape(&qo, &q) || !is(&k, T, H, d) || !same_shape(&v, &k) || !same_shape(&vc, &kc) ||
        kc.shape[1] != H || kc.shape[3] != d || !is(&slots, T, -1, -1) || !is(&pos, T, -1, -1))
        return mismatch(), NULL;
    const int code = cache_code(&kc, &ks, &vs, H);
    const int interleaved = PyObject_IsTrue(a[9]);
    if (code < 0 || interleaved < 0 || enter(dev, a[13], &stream, &back)) return NULL;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_rope_and_cache(qo.ptr, qo.step, q.ptr, q.step, k.ptr, k.step, v.ptr, v.step, kc.ptr, vc.ptr, slots.ptr,
                           pos.ptr, table.ptr, (int)table.shape[0], (int)table.shape[1],
                           interleaved ? PA_ROPE_INTERLEAVED : PA_ROPE_HALF, (int)T, (int)q.shape[1], (int)H, (int)d,
                           (int)kc.shape[2], (int)kc.shape[0], (pa_dtype)half_code(&q), (pa_dtype)code, ks.ptr, vs.ptr,
                           ws.ptr, (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

/* out, weights_out, q, k_cache, v_cache, block_tables, seq_lens, scale, workspace, weights_in, k_scale,
 * v_scale, stream */
static PyObject* decode_weights(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor out, wo, q, kc, vc, bt, sl, ws, wi, ks, vs;
    long long dev, back;
    void* stream;
    if (want_args(n, 13) || device_of(a[2], "q", &dev) || take(a[2], "q", HALVES, 3, dev, 0, &q) ||
        take(a[0], "out", q.type, 3, dev, 0, &out) || take(a[1], "weights_out", F32, 3, dev, 0, &wo) ||
        take(a[3], "k_cache", CACHES, 4, dev, 0, &kc) || take(a[4], "v_cache", kc.type, 4, dev, 0, &vc) ||
        take(a[5], "block_tables", I32, 2, dev, 0, &bt) || take(a[6], "seq_lens", I32, 1, dev, 0, &sl) ||
        take(a[8], "workspace", U8, 0, dev, 0, &ws) || take_or_none(a[9], "weights_in", F32, 3, dev, &wi) ||
        take_or_none(a[10], "k_scale", F32, 0, dev, &ks) || take_or_none(a[11], "v_scale", F32, 0, dev, &vs))
        return NULL;
    const long long B = q.shape[0], H = kc.shape[1];
    if (!same_shape(&out, &q) || !same_shape(&vc, &kc) || kc.shape[3] != q.shape[2] || bt.shape[0] != B ||
        !is(&sl, B, -1, -1) || !is(&wo, B, H, -1) || (a[9] != Py_None && !same_shape(&wi, &wo)))
        return mismatch(), NULL;
    const int code = cache_code(&kc, &ks, &vs, H);
    const double scale = PyFloat_AsDouble(a[7]);
    if (code < 0 || (scale == -1.0 && PyErr_Occurred()) || enter(dev, a[12], &stream, &back)) return NULL;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_decode_weights(out.ptr, wo.ptr, wi.ptr, wo.shape[2], q.ptr, kc.ptr, vc.ptr, bt.ptr, (int)bt.shape[1], sl.ptr,
                           (int)B, (int)q.shape[1], (int)H, (int)q.shape[2], (int)kc.shape[2], (int)kc.shape[0],
                           (float)scale, (pa_dtype)half_code(&q), (pa_dtype)code, ks.ptr, vs.ptr, ws.ptr,
                           (size_t)ws.numel, (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

/* kept, seq_lens_out, weights_out, weights, k_cache, v_cache, block_tables, seq_lens, new_tables, budget,
 * sinks, recent, workspace, stream */
static PyObject* evict(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor kept, lo, wo, w, kc, vc, bt, sl, nt, ws;
    long long dev, back, budget, sinks, recent;
    void* stream;
    if (want_args(n, 14) || device_of(a[4], "k_cache", &dev) || take(a[4], "k_cache", CACHES, 4, dev, 0, &kc) ||
        take(a[5], "v_cache", kc.type, 4, dev, 0, &vc) || take(a[3], "weights", F32, 3, dev, 0, &w) ||
        take(a[2], "weights_out", F32, 3, dev, 0, &wo) || take(a[0], "kept", I32, 3, dev, 0, &kept) ||
        take(a[1], "seq_lens_out", I32, 1, dev, 0, &lo) || take(a[6], "block_tables", I32, 2, dev, 0, &bt) ||
        take(a[7], "seq_lens", I32, 1, dev, 0, &sl) || take(a[8], "new_tables", I32, 2, dev, 0, &nt) ||
        take_or_none(a[12], "workspace", U8, 0, dev, &ws) || check_workspace(&ws) ||
        as_int(PyNumber_Index(a[9]), &budget) || as_int(PyNumber_Index(a[10]), &sinks) ||
        as_int(PyNumber_Index(a[11]), &recent))
        return NULL;
    const long long B = w.shape[0], H = kc.shape[1];
    if (!same_shape(&vc, &kc) || w.shape[1] != H || !same_shape(&wo, &w) || !is(&kept, B, H, -1) || kept.shape[2] != budget ||
        !is(&sl, B, -1, -1) || !is(&lo, B, -1, -1) || bt.shape[0] != B || nt.shape[0] != B)
        return mismatch(), NULL;
    if (budget > INT_MAX || sinks > INT_MAX || recent > INT_MAX || sinks < 0 || recent < 0)
        return PyLong_FromLong(PA_ERR_INVALID_ARG);
    const int code = kc.type & HALVES ? half_code(&kc) : PA_FP8_E4M3;
    if (enter(dev, a[13], &stream, &back)) return NULL;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_evict(kept.ptr, lo.ptr, wo.ptr, w.ptr, w.shape[2], kc.ptr, vc.ptr, bt.ptr, (int)bt.shape[1], sl.ptr, nt.ptr,
                  (int)nt.shape[1], (int)B, (int)budget, (int)sinks, (int)recent, (int)H, (int)kc.shape[3],
                  (int)kc.shape[2], (int)kc.shape[0], (pa_dtype)code, ws.ptr, (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

/* q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight, k_weight, eps,
 * weight_offset, axes (None or a buffer of bytes), interleaved, k_scale, v_scale, workspace, stream */
static PyObject* norm_rope_and_cache(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor qo, q, k, v, kc, vc, slots, pos, table, qw, kw, ks, vs, ws;
    long long dev, back;
    void* stream;
    if (want_args(n, 19) || device_of(a[1], "q", &dev) || take(a[1], "q", HALVES, 3, dev, 1, &q) ||
        take(a[0], "q_out", q.type, 3, dev, 1, &qo) || take(a[2], "k", q.type, 3, dev, 1, &k) ||
        take(a[3], "v", q.type, 3, dev, 1, &v) || take(a[4], "k_cache", CACHES, 4, dev, 0, &kc) ||
        take(a[5], "v_cache", kc.type, 4, dev, 0, &vc) || take(a[6], "slot_mapping", I64, 1, dev, 0, &slots) ||
        take(a[7], "positions", I64, 0, dev, 0, &pos) || take(a[8], "cos_sin", F32, 2, dev, 0, &table) ||
        take_or_none(a[9], "q_weight", q.type, 1, dev, &qw) || take_or_none(a[10], "k_weight", q.type, 1, dev, &kw) ||
        take_or_none(a[15], "k_scale", F32, 0, dev, &ks) || take_or_none(a[16], "v_scale", F32, 0, dev, &vs) ||
        take_or_none(a[17], "workspace", U8, 0, dev, &ws) || check_workspace(&ws))
        return NULL;
    const long long T = q.shape[0], H = k.shape[1], d = q.shape[2];
    if (pos.ndim == 1) {                            /* one axis */
        pos.shape[1] = pos.shape[0];
        pos.shape[0] = 1;
    } else if (pos.ndim != 2) {
        PyErr_SetString(PyExc_ValueError, "positions must be [tokens] or [axes, tokens]");
        return NULL;
    }
    if (!same_shape(&qo, &q) || !is(&k, T, H, d) || !same_shape(&v, &k) || !same_shape(&vc, &kc) ||
        kc.shape[1] != H || kc.shape[3] != d || !is(&slots, T, -1, -1) || pos.shape[1] != T ||
        (a[9] != Py_None && !is(&qw, d, -1, -1)) || (a[10] != Py_None && !is(&kw, d, -1, -1)))
        return mismatch(), NULL;
    if (pos.shape[0] > INT_MAX) return PyLong_FromLong(PA_ERR_UNSUPPORTED);
    const int code = cache_code(&kc, &ks, &vs, H);
    const int interleaved = PyObject_IsTrue(a[14]);
    const double eps = PyFloat_AsDouble(a[11]);
    const double offset = eps == -1.0 && PyErr_Occurred() ? 0.0 : PyFloat_AsDouble(a[12]);
    if (code < 0 || interleaved < 0 || PyErr_Occurred()) return NULL;
    Py_buffer axes = {0};
    if (a[13] != Py_None) {
        if (PyObject_GetBuffer(a[13], &axes, PyBUF_SIMPLE)) return NULL;
        if (axes.itemsize != 1 || 2 * (long long)axes.len != table.shape[1]) {
            PyErr_SetString(PyExc_ValueError, "axes must hold one byte for every pair of cos_sin's columns");
            PyBuffer_Release(&axes);
            return NULL;
        }
    }
    PyObject* res = NULL;
    if (!enter(dev, a[18], &stream, &back)) {
        pa_status st;
        Py_BEGIN_ALLOW_THREADS
        st = pa_norm_rope_and_cache(qo.ptr, qo.step, q.ptr, q.step, k.ptr, k.step, v.ptr, v.step, qw.ptr, kw.ptr, (float)eps,
                                    (float)offset, kc.ptr, vc.ptr, slots.ptr, pos.ptr, (int)pos.shape[0], axes.buf,
                                    table.ptr, (int)table.shape[0], (int)table.shape[1],
                                    interleaved ? PA_ROPE_INTERLEAVED : PA_ROPE_HALF, (int)T, (int)q.shape[1], (int)H,
                                    (int)d, (int)kc.shape[2], (int)kc.shape[0], (pa_dtype)half_code(&q), (pa_dtype)code,
                                    ks.ptr, vs.ptr, ws.ptr, (pa_stream_t)stream);
        Py_END_ALLOW_THREADS
        res = leave(back, st);
    }
    if (a[13] != Py_None) PyBuffer_Release(&axes);
    return res;
}

/* What the two calls with scores or masks that are not plain have alike: out, q, query_start_loc,
 * k_cache, v_cache, block_tables, seq_lens first, workspace, cap, window, k_scale, v_scale. */
typedef struct {
    Tensor out, q, qsl, kc, vc, bt, sl, ws, ks, vs;
    long long dev, window;
    double scale, cap;
    int code;
} Scored;

static int take_scored(PyObject* const* a, PyObject* scale, PyObject* ws, PyObject* cap, PyObject* window, PyObject* ks,
                       PyObject* vs, Scored* c) {
    if (device_of(a[1], "q", &c->dev) || take(a[1], "q", HALVES, 3, c->dev, 0, &c->q) ||
        take(a[0], "out", c->q.type, 3, c->dev, 0, &c->out) || take(a[2], "query_start_loc", I32, 1, c->dev, 0, &c->qsl) ||
        take(a[3], "k_cache", CACHES, 4, c->dev, 0, &c->kc) || take(a[4], "v_cache", c->kc.type, 4, c->dev, 0, &c->vc) ||
        take(a[5], "block_tables", I32, 2, c->dev, 0, &c->bt) || take(a[6], "seq_lens", I32, 1, c->dev, 0, &c->sl) ||
        take(ws, "workspace", U8, 0, c->dev, 0, &c->ws) || take_or_none(ks, "k_scale", F32, 0, c->dev, &c->ks) ||
        take_or_none(vs, "v_scale", F32, 0, c->dev, &c->vs) || as_int(PyNumber_Index(window), &c->window))
        return -1;
    const long long B = c->sl.shape[0];
    if (!same_shape(&c->out, &c->q) || !same_shape(&c->vc, &c->kc) || c->kc.shape[3] != c->q.shape[2] ||
        c->bt.shape[0] != B || !is(&c->qsl, B + 1, -1, -1))
        return mismatch();
    c->code = cache_code(&c->kc, &c->ks, &c->vs, c->kc.shape[1]);
    if (c->code < 0) return -1;
    c->scale = PyFloat_AsDouble(scale);
    if (c->scale == -1.0 && PyErr_Occurred()) return -1;
    c->cap = PyFloat_AsDouble(cap);
    if (c->cap == -1.0 && PyErr_Occurred()) return -1;
    if (c->window > INT_MAX) c->window = INT_MAX;   /* wider than any sequence */
    if (c->window < 0) c->window = -1;              /* refused by the library */
    return 0;
}

/* out, q, query_start_loc, k_cache, v_cache, block_tables, seq_lens, scale, workspace, cap, slopes, window,
 * prefix_lens, k_scale, v_scale, stream */
static PyObject* mixed_scored(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Scored c;
    Tensor slopes, prefix;
    long long back;
    void* stream;
    if (want_args(n, 16) || take_scored(a, a[7], a[8], a[9], a[11], a[13], a[14], &c) ||
        take_or_none(a[10], "slopes", F32, 1, c.dev, &slopes) || take_or_none(a[12], "prefix_lens", I32, 1, c.dev, &prefix))
        return NULL;
    if ((a[10] != Py_None && !is(&slopes, c.q.shape[1], -1, -1)) || (a[12] != Py_None && !is(&prefix, c.sl.shape[0], -1, -1)))
        return mismatch(), NULL;
    if (enter(c.dev, a[15], &stream, &back)) return NULL;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_mixed_scored(c.out.ptr, c.q.ptr, c.qsl.ptr, c.kc.ptr, c.vc.ptr, c.bt.ptr, (int)c.bt.shape[1], c.sl.ptr, prefix.ptr,
                         slopes.ptr, (float)c.cap, (int)c.window, (int)c.sl.shape[0], (int)c.q.shape[0], (int)c.q.shape[1],
                         (int)c.kc.shape[1], (int)c.q.shape[2], (int)c.kc.shape[2], (int)c.kc.shape[0], (float)c.scale,
                         (pa_dtype)half_code(&c.q), (pa_dtype)c.code, c.ks.ptr, c.vs.ptr, c.ws.ptr, (size_t)c.ws.numel,
                         (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

/* out, q, query_start_loc, k_cache, v_cache, block_tables, seq_lens, masks, scale, workspace, cap, window, k_scale,
 * v_scale, stream */
static PyObject* tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Scored c;
    Tensor masks;
    long long back;
    void* stream;
    if (want_args(n, 15) || take_scored(a, a[8], a[9], a[10], a[11], a[12], a[13], &c) ||
        take(a[7], "masks", I64, 2, c.dev, 0, &masks))
        return NULL;
    if (masks.shape[0] != c.q.shape[0]) return mismatch(), NULL;
    if (enter(c.dev, a[14], &stream, &back)) return NULL;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_tree(c.out.ptr, c.q.ptr, c.qsl.ptr, c.kc.ptr, c.vc.ptr, c.bt.ptr, (int)c.bt.shape[1], c.sl.ptr, masks.ptr,
                 (int)masks.shape[1], (float)c.cap, (int)c.window, (int)c.sl.shape[0], (int)c.q.shape[0], (int)c.q.shape[1],
                 (int)c.kc.shape[1], (int)c.q.shape[2], (int)c.kc.shape[2], (int)c.kc.shape[0], (float)c.scale,
                 (pa_dtype)half_code(&c.q), (pa_dtype)c.code, c.ks.ptr, c.vs.ptr, c.ws.ptr, (size_t)c.ws.numel,
                 (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

#define MAX_LAYERS 1024

/* seq_lens_out, k_caches, v_caches (sequences of tensors), paths, path_lens, query_start_loc, block_tables,
 * seq_lens, workspace, stream */
static PyObject* tree_commit(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor lo, paths, pl, qsl, bt, sl, ws, first = {0}, c;
    long long dev, back;
    void *stream, *k[MAX_LAYERS], *v[MAX_LAYERS];
    if (want_args(n, 10) || device_of(a[7], "seq_lens", &dev) || take(a[7], "seq_lens", I32, 1, dev, 0, &sl) ||
        take(a[0], "seq_lens_out", I32, 1, dev, 0, &lo) || take(a[3], "paths", I32, 2, dev, 0, &paths) ||
        take(a[4], "path_lens", I32, 1, dev, 0, &pl) || take(a[5], "query_start_loc", I32, 1, dev, 0, &qsl) ||
        take(a[6], "block_tables", I32, 2, dev, 0, &bt) || take_or_none(a[8], "workspace", U8, 0, dev, &ws) ||
        check_workspace(&ws))
        return NULL;
    const long long B = sl.shape[0];
    if (!is(&lo, B, -1, -1) || paths.shape[0] != B || !is(&pl, B, -1, -1) || !is(&qsl, B + 1, -1, -1) || bt.shape[0] != B)
        return mismatch(), NULL;
    PyObject* ks = PySequence_Fast(a[1], "k_caches must be a sequence of tensors");
    PyObject* vs = ks ? PySequence_Fast(a[2], "v_caches must be a sequence of tensors") : NULL;
    if (!vs) {
        Py_XDECREF(ks);
        return NULL;
    }
    const Py_ssize_t layers = PySequence_Fast_GET_SIZE(ks);
    int bad = 0;
    if (layers < 1 || layers > MAX_LAYERS || PySequence_Fast_GET_SIZE(vs) != layers) {
        PyErr_Format(PyExc_ValueError, "k_caches and v_caches: 1 to %d layers, K and V alike", MAX_LAYERS);
        bad = 1;
    }
    for (Py_ssize_t i = 0; !bad && i < 2 * layers; ++i) {
        PyObject* t = PySequence_Fast_GET_ITEM(i & 1 ? vs : ks, i >> 1);
        bad = take(t, i & 1 ? "v_cache" : "k_cache", i ? first.type : CACHES, 4, dev, 0, &c);
        if (!bad && i && !same_shape(&c, &first)) bad = mismatch();
        if (bad) break;
        if (!i) first = c;
        (i & 1 ? v : k)[i >> 1] = c.ptr;
    }
    Py_DECREF(ks);
    Py_DECREF(vs);
    if (bad || enter(dev, a[9], &stream, &back)) return NULL;
    const int code = first.type & HALVES ? half_code(&first) : PA_FP8_E4M3;
    pa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = pa_tree_commit(lo.ptr, k, v, (int)layers, paths.ptr, pl.ptr, (int)paths.shape[1], qsl.ptr, bt.ptr, (int)bt.shape[1],
                        sl.ptr, (int)B, (int)first.shape[1], (int)first.shape[3], (int)first.shape[2], (int)first.shape[0],
                        (pa_dtype)code, ws.ptr, (pa_stream_t)stream);
    Py_END_ALLOW_THREADS
    return leave(back, st);
}

static PyMethodDef methods[] = {
    {"rope_table", (PyCFunction)(void (*)(void))rope_table, METH_FASTCALL, NULL},
    {"rope_and_cache", (PyCFunction)(void (*)(void))rope_and_cache, METH_FASTCALL, NULL},
    {"decode_weights", (PyCFunction)(void (*)(void))decode_weights, METH_FASTCALL, NULL},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, NULL},
    {"norm_rope_and_cache", (PyCFunction)(void (*)(void))norm_rope_and_cache, METH_FASTCALL, NULL},
    {"mixed_scored", (PyCFunction)(void (*)(void))mixed_scored, METH_FASTCALL, NULL},
    {"tree", (PyCFunction)(void (*)(void))tree, METH_FASTCALL, NULL},
    {"tree_commit", (PyCFunction)(void (*)(void))tree_commit, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* torch = PyImport_ImportModule("torch");
    if (!torch || !(torch_c = PyObject_GetAttrString(torch, "_C"))) return NULL;
    for (int i = 0; i < NUM_TYPES; ++i)
        if (!(types[i] = PyObject_GetAttrString(torch, type_names[i]))) return NULL;
    if (!(tensor_type = (PyTypeObject*)PyObject_GetAttrString(torch, "Tensor")) ||
        !(s_raw_stream = PyUnicode_InternFromString("_cuda_getCurrentRawStream")) ||
        !(s_current_device = PyUnicode_InternFromString("_cuda_getDevice")) ||
        !(s_set_device = PyUnicode_InternFromString("_cuda_setDevice")) ||
        !(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_shape = PyUnicode_InternFromString("shape")) ||
        !(s_stride = PyUnicode_InternFromString("stride")) ||
        !(s_get_device = PyUnicode_InternFromString("get_device")) ||
        !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) ||
        !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")))
        return NULL;
    Py_DECREF(torch);
    return PyModule_Create(&module);
}
