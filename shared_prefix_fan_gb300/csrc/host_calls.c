/* host_calls.c -- the host side of the calls of the 8-bit cache and of drafted trees, as a
 * CPython extension module.
 *
 * Most kernels behind these calls take 2 to 4 us in a drafting step, and a call through
 * ctypes with its checks in Python took 8 to 21 us of host time. Here the same checks, output
 * tensors and calls take 4 to 14, of which the launch is 2.5 and an output tensor made and
 * freed 1.9. The module holds no state of calls: it is handed torch's own functions and types
 * once (setup), and every call looks at its tensors again.
 *
 * Checks are binding.py's: every tensor contiguous, of its type and shape, on the CUDA device
 * of the call's first one; integers that do not fit 32 bits are refused. Results of a call on
 * a given stream come from that stream's memory (binding._empty_on).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "../../include/fanout.h"

/* What setup() is given; owned for the life of the process. */
enum { BF16, F8, U8, I32, I64, F32, N_TYPES };
static PyObject *g_type[N_TYPES];
static PyObject *g_empty, *g_raw_stream, *g_get_device, *g_device_guard, *g_empty_on, *g_handle_of,
    *g_raise;
static PyObject *s_dtype, *s_device, *s_shape, *s_is_contiguous, *s_data_ptr, *s_index, *s_is_cuda,
    *s_stride, *s_enter, *s_exit, *kw_empty;

/* One call: its device, where its results come from, and what it holds until it ends. */
#define MAX_HELD 8
typedef struct {
    PyObject *dev, *index, *stream, *empty;
    PyObject *held[MAX_HELD];
    int n_held;
} Call;

static void drop(Call *c) {
    for (int i = 0; i < c->n_held; ++i) Py_DECREF(c->held[i]);
    c->n_held = 0;
    Py_CLEAR(c->dev);
    Py_CLEAR(c->index);
    Py_CLEAR(c->empty);
}

/* The call's device is `first`'s, which has to be a CUDA tensor. */
static int begin(Call *c, PyObject *first, const char *name, PyObject *stream) {
    memset(c, 0, sizeof *c);
    c->stream = stream;
    PyObject *cuda = PyObject_GetAttr(first, s_is_cuda);
    if (!cuda) return -1;
    const int is_cuda = PyObject_IsTrue(cuda);
    Py_DECREF(cuda);
    c->dev = PyObject_GetAttr(first, s_device);
    if (!c->dev) return -1;
    if (is_cuda <= 0) {
        if (is_cuda == 0)
            PyErr_Format(PyExc_ValueError, "%s must be a tensor on a CUDA device, not %S", name, c->dev);
        goto bad;
    }
    c->index = PyObject_GetAttr(c->dev, s_index);
    if (!c->index) goto bad;
    if (stream == Py_None) {
        c->empty = Py_NewRef(g_empty);
    } else {
        PyObject *args[] = {c->dev, stream};
        c->empty = PyObject_Vectorcall(g_empty_on, args, 2, NULL);
    }
    if (c->empty) return 0;
bad:
    drop(c);
    return -1;
}

/* The sizes of t, at most `max` of them; their number, or -1. */
static int sizes(PyObject *t, Py_ssize_t *out, int max) {
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    if (!shape) return -1;
    int n = -1;
    if (PyTuple_Check(shape)) {
        n = (int)PyTuple_GET_SIZE(shape);
        for (int i = 0; i < n && i < max; ++i) {
            out[i] = PyLong_AsSsize_t(PyTuple_GET_ITEM(shape, i));
            if (out[i] == -1 && PyErr_Occurred()) n = -1;
        }
    } else {
        PyErr_SetString(PyExc_TypeError, "shape is no tuple");
    }
    Py_DECREF(shape);
    return n;
}

static int pointer(PyObject *t, void **p) {
    PyObject *v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return -1;
    *p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return *p == NULL && PyErr_Occurred() ? -1 : 0;
}

/* Type and device of t; 1 or 0, -1 with an exception. */
static int is_on(const Call *c, PyObject *t, int type) {
    PyObject *dtype = PyObject_GetAttr(t, s_dtype);
    if (!dtype) return -1;
    int ok = dtype == g_type[type];
    Py_DECREF(dtype);
    if (ok) {
        PyObject *dev = PyObject_GetAttr(t, s_device);
        if (!dev) return -1;
        ok = PyObject_RichCompareBool(dev, c->dev, Py_EQ);
        Py_DECREF(dev);
    }
    return ok;
}

/* A contiguous tensor of this type and shape (nd < 0: any; a size < 0: any) on the call's
 * device: its address. */
static int need(const Call *c, const char *name, PyObject *t, int type, int nd,
                const Py_ssize_t *shape, void **p) {
    int ok = is_on(c, t, type);
    if (ok < 0) return -1;
    if (ok) {
        PyObject *v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!v) return -1;
        ok = v == Py_True;
        Py_DECREF(v);
    }
    if (!ok) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous %S tensor on one CUDA device (%S)",
                     name, g_type[type], c->dev);
        return -1;
    }
    if (nd >= 0) {
        Py_ssize_t got[4] = {0};
        const int n = sizes(t, got, 4);
        if (n < 0 && PyErr_Occurred()) return -1;
        ok = n == nd;
        for (int i = 0; i < nd && ok; ++i) ok = shape[i] < 0 || shape[i] == got[i];
        if (!ok) {
            PyObject *have = PyObject_GetAttr(t, s_shape);
            PyErr_Format(PyExc_ValueError, "%s shape %S does not fit the other arguments", name,
                         have ? have : Py_None);
            Py_XDECREF(have);
            return -1;
        }
    }
    return pointer(t, p);
}

/* A new tensor, held by the call; its place in held, or -1. */
static int make(Call *c, int type, int nd, const Py_ssize_t *shape, void **p) {
    PyObject *size = PyTuple_New(nd);
    if (!size) return -1;
    for (int i = 0; i < nd; ++i) {
        PyObject *v = PyLong_FromSsize_t(shape[i]);
        if (!v) {
            Py_DECREF(size);
            return -1;
        }
        PyTuple_SET_ITEM(size, i, v);
    }
    PyObject *args[] = {size, g_type[type], c->dev};
    PyObject *t = PyObject_Vectorcall(c->empty, args, 1, kw_empty);
    Py_DECREF(size);
    if (!t) return -1;
    c->held[c->n_held++] = t;
    return pointer(t, p) < 0 ? -1 : c->n_held - 1;
}

/* Integers of the C calls: 32 bits. */
static int int32_of(PyObject *v, const char *name, int32_t *out) {
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(v, &overflow);
    if (x == -1 && PyErr_Occurred()) return -1;
    if (overflow || x < INT32_MIN || x > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: %S does not fit 32 bits", name, v);
        return -1;
    }
    *out = (int32_t)x;
    return 0;
}
static int size32(Py_ssize_t v, const char *name, int32_t *out) {
    if (v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: %zd does not fit 32 bits", name, v);
        return -1;
    }
    *out = (int32_t)v;
    return 0;
}
static int float_of(PyObject *v, float *out) {
    const double x = PyFloat_AsDouble(v);
    if (x == -1.0 && PyErr_Occurred()) return -1;
    *out = (float)x;
    return 0;
}

/* The stream's handle, and the call's device made current where another one is: a context
 * manager that has been entered (NULL: none), to be left by `leave`. */
static int enter(const Call *c, fanout_stream_t *handle, PyObject **guard) {
    *guard = NULL;
    PyObject *v = c->stream == Py_None ? PyObject_CallOneArg(g_raw_stream, c->index)
                                       : PyObject_CallOneArg(g_handle_of, c->stream);
    if (!v) return -1;
    *handle = (fanout_stream_t)PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!*handle && PyErr_Occurred()) return -1;
    PyObject *now = PyObject_CallNoArgs(g_get_device);
    if (!now) return -1;
    const int same = PyObject_RichCompareBool(now, c->index, Py_EQ);
    Py_DECREF(now);
    if (same < 0) return -1;
    if (!same) {
        PyObject *g = PyObject_CallOneArg(g_device_guard, c->index);
        if (!g) return -1;
        PyObject *r = PyObject_CallMethodNoArgs(g, s_enter);
        if (!r) {
            Py_DECREF(g);
            return -1;
        }
        Py_DECREF(r);
        *guard = g;
    }
    return 0;
}
static int leave(PyObject *guard, int rc, const char *name) {
    if (guard) {
        PyObject *r = PyObject_CallMethodObjArgs(guard, s_exit, Py_None, Py_None, Py_None, NULL);
        Py_DECREF(guard);
        if (!r) return -1;
        Py_DECREF(r);
    }
    if (rc != FANOUT_OK) {
        PyObject *r = PyObject_CallFunction(g_raise, "is", rc, name);
        Py_XDECREF(r);
        return -1;
    }
    return 0;
}
#define RUN(c, name, expr)                                        \
    do {                                                          \
        fanout_stream_t stream;                                   \
        PyObject *guard;                                          \
        int rc;                                                   \
        if (enter(&(c), &stream, &guard) < 0) goto done;          \
        Py_BEGIN_ALLOW_THREADS rc = (expr);                       \
        Py_END_ALLOW_THREADS if (leave(guard, rc, name) < 0) goto done; \
    } while (0)

static int arity(const char *name, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, want, n);
    return -1;
}

/* Rows [n, H_kv, d] of bf16 whose heads are packed: elements between rows, and the address. */
static int rows_of(const Call *c, const char *name, PyObject *t, Py_ssize_t n, Py_ssize_t h_kv,
                   Py_ssize_t d, int64_t *stride, void **p) {
    Py_ssize_t got[3] = {0}, step[3] = {0};
    const int ok = is_on(c, t, BF16);
    if (ok < 0) return -1;
    if (!ok) {
        PyErr_Format(PyExc_ValueError, "%s must be a bf16 tensor on %S", name, c->dev);
        return -1;
    }
    const int nd = sizes(t, got, 3);
    if (nd < 0 && PyErr_Occurred()) return -1;
    if (nd != 3 || got[0] != n || got[1] != h_kv || got[2] != d) {
        PyErr_Format(PyExc_ValueError, "%s must be [%zd, %zd, %zd]", name, n, h_kv, d);
        return -1;
    }
    *stride = h_kv * d;
    if (n > 0) {
        PyObject *s = PyObject_CallMethodNoArgs(t, s_stride);
        if (!s) return -1;
        for (int i = 0; i < 3; ++i) step[i] = PyLong_AsSsize_t(PyTuple_GET_ITEM(s, i));
        Py_DECREF(s);
        if (PyErr_Occurred()) return -1;
        if ((d > 1 && step[2] != 1) || (h_kv > 1 && step[1] != d)) {
            PyErr_Format(PyExc_ValueError, "%s: a row's heads must be packed", name);
            return -1;
        }
        if (n > 1) *stride = step[0];
    }
    return pointer(t, p);
}

/* A pair of 8-bit pools: their sizes [num_pages, H_kv, page_size, d] and addresses. */
static int pools_of(const Call *c, PyObject *k, PyObject *v, Py_ssize_t *shape, int32_t *size, void **kp,
                    void **vp) {
    static const Py_ssize_t any[4] = {-1, -1, -1, -1};
    if (need(c, "k_pages", k, F8, 4, any, kp) < 0 || sizes(k, shape, 4) < 0 ||
        need(c, "v_pages", v, F8, 4, shape, vp) < 0)
        return -1;
    for (int i = 0; i < 4; ++i)
        if (size32(shape[i], "pool size", size + i) < 0) return -1;
    return 0;
}

/* kv_append_q8(k_new, v_new, k_pages, v_pages, slots, k_scale, v_scale, stream) */
static PyObject *kv_append_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("kv_append_q8", n, 8) < 0) return NULL;
    Call c;
    if (begin(&c, a[2], "k_pages", a[7]) < 0) return NULL;
    PyObject *result = NULL;
    Py_ssize_t pool[4], rows[1];
    int32_t size[4], n_rows = 0;
    int64_t ks, vs;
    void *kn, *vn, *kp, *vp, *slots;
    float kg, vg;
    static const Py_ssize_t any[1] = {-1};
    if (pools_of(&c, a[2], a[3], pool, size, &kp, &vp) < 0 ||
        need(&c, "slots", a[4], I64, 1, any, &slots) < 0 || sizes(a[4], rows, 1) < 0 ||
        size32(rows[0], "slots", &n_rows) < 0 ||
        rows_of(&c, "k_new", a[0], rows[0], pool[1], pool[3], &ks, &kn) < 0 ||
        rows_of(&c, "v_new", a[1], rows[0], pool[1], pool[3], &vs, &vn) < 0 || float_of(a[5], &kg) < 0 ||
        float_of(a[6], &vg) < 0)
        goto done;
    RUN(c, "fanout_kv_append_q8",
        fanout_kv_append_q8(kn, vn, ks, vs, kp, vp, slots, n_rows, size[0], size[1], size[3], size[2], kg,
                            vg, stream));
    result = Py_NewRef(Py_None);
done:
    drop(&c);
    return result;
}

/* kv_read_q8(k_pages, v_pages, slots, k_scale, v_scale, k_out, v_out, stream) -> (k, v) */
static PyObject *kv_read_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("kv_read_q8", n, 8) < 0) return NULL;
    Call c;
    if (begin(&c, a[0], "k_pages", a[7]) < 0) return NULL;
    PyObject *result = NULL, *out[2] = {a[5], a[6]};
    Py_ssize_t pool[4], rows[1];
    int32_t size[4], n_rows = 0;
    int64_t stride[2];
    void *kp, *vp, *slots, *to[2];
    float kg, vg;
    static const Py_ssize_t any[1] = {-1};
    static const char *const names[2] = {"k_out", "v_out"};
    if (pools_of(&c, a[0], a[1], pool, size, &kp, &vp) < 0 ||
        need(&c, "slots", a[2], I64, 1, any, &slots) < 0 || sizes(a[2], rows, 1) < 0 ||
        size32(rows[0], "slots", &n_rows) < 0 || float_of(a[3], &kg) < 0 || float_of(a[4], &vg) < 0)
        goto done;
    const Py_ssize_t shape[3] = {rows[0], pool[1], pool[3]};
    for (int i = 0; i < 2; ++i) {
        if (out[i] == Py_None) {
            const int at = make(&c, BF16, 3, shape, &to[i]);
            if (at < 0) goto done;
            out[i] = c.held[at];
            stride[i] = shape[1] * shape[2];
        } else if (rows_of(&c, names[i], out[i], shape[0], shape[1], shape[2], &stride[i], &to[i]) < 0) {
            goto done;
        }
    }
    RUN(c, "fanout_kv_read_q8",
        fanout_kv_read_q8(kp, vp, slots, n_rows, size[0], size[1], size[3], size[2], kg, vg, to[0], to[1],
                          stride[0], stride[1], stream));
    result = PyTuple_Pack(2, out[0], out[1]);
done:
    drop(&c);
    return result;
}

/* tail: masks, positions, slots, stream */
static PyObject *tree_rows_of(PyObject *const *a, int32_t sinks, PyObject *const *tail) {
    int32_t prefix_len, page_size, words, window, B = 0, width = 0;
    if (int32_of(a[2], "prefix_len", &prefix_len) < 0 || int32_of(a[5], "page_size", &page_size) < 0 ||
        int32_of(a[6], "mask words", &words) < 0 || int32_of(a[7], "window", &window) < 0)
        return NULL;
    Call c;
    if (begin(&c, a[0], "parents", tail[3]) < 0) return NULL;
    PyObject *result = NULL, *out[3] = {tail[0], tail[1], tail[2]};
    static const Py_ssize_t any[2] = {-1, -1};
    static const char *const names[3] = {"masks", "positions", "slots"};
    static const int types[3] = {I32, I32, I64};
    Py_ssize_t rows[1], table[2];
    void *parents, *tp, *s, *l, *to[3];
    if (need(&c, "parents", a[0], I32, 1, any, &parents) < 0 || sizes(a[0], rows, 1) < 0 ||
        need(&c, "page_table", a[1], I32, 2, any, &tp) < 0 || sizes(a[1], table, 2) < 0 ||
        need(&c, "suffix_lens", a[3], I32, 1, table, &s) < 0 ||
        need(&c, "add_lens", a[4], I32, 1, table, &l) < 0 || size32(table[0], "page_table", &B) < 0 ||
        size32(table[1], "page_table", &width) < 0)
        goto done;
    for (int i = 0; i < 3; ++i) {
        const Py_ssize_t shape[2] = {rows[0], words};
        const int nd = i == 0 ? 2 : 1;
        if (out[i] == Py_None) {
            const int at = make(&c, types[i], nd, shape, &to[i]);
            if (at < 0) goto done;
            out[i] = c.held[at];
        } else if (need(&c, names[i], out[i], types[i], nd, shape, &to[i]) < 0) {
            goto done;
        }
    }
    RUN(c, "fanout_tree_rows",
        fanout_tree_rows_sinks(parents, tp, B, width, prefix_len, s, l, page_size, rows[0], words, window,
                               sinks, to[0], to[1], to[2], stream));
    result = PyTuple_Pack(3, out[0], out[1], out[2]);
done:
    drop(&c);
    return result;
}

/* tree_rows(parents, page_table, prefix_len, suffix_lens, add_lens, page_size, words, window,
 *           masks, positions, slots, stream) -> (masks, positions, slots) */
static PyObject *tree_rows(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return arity("tree_rows", n, 12) < 0 ? NULL : tree_rows_of(a, 0, a + 8);
}

/* the same with first keys: sinks behind window */
static PyObject *tree_rows_sinks(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int32_t sinks;
    if (arity("tree_rows_sinks", n, 13) < 0 || int32_of(a[8], "sinks", &sinks) < 0) return NULL;
    return tree_rows_of(a, sinks, a + 9);
}

/* tree_accept(parents, draft_tokens, target_tokens, first_tokens, add_lens, stream)
 *   -> (path, counts, next_tokens) */
static PyObject *tree_accept(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("tree_accept", n, 6) < 0) return NULL;
    Call c;
    if (begin(&c, a[0], "parents", a[5]) < 0) return NULL;
    PyObject *result = NULL;
    static const Py_ssize_t any[1] = {-1};
    Py_ssize_t rows[1], branches[1];
    int32_t B = 0;
    void *parents, *draft, *target, *first, *lens, *path, *counts, *after;
    if (need(&c, "parents", a[0], I32, 1, any, &parents) < 0 || sizes(a[0], rows, 1) < 0 ||
        need(&c, "draft_tokens", a[1], I64, 1, rows, &draft) < 0 ||
        need(&c, "target_tokens", a[2], I64, 1, rows, &target) < 0 ||
        need(&c, "add_lens", a[4], I32, 1, any, &lens) < 0 || sizes(a[4], branches, 1) < 0 ||
        need(&c, "first_tokens", a[3], I64, 1, branches, &first) < 0 ||
        size32(branches[0], "add_lens", &B) < 0 || make(&c, I32, 1, rows, &path) < 0 ||
        make(&c, I32, 1, branches, &counts) < 0 || make(&c, I64, 1, branches, &after) < 0)
        goto done;
    RUN(c, "fanout_tree_accept",
        fanout_tree_accept(parents, draft, target, first, lens, B, rows[0], path, counts, after, stream));
    result = PyTuple_Pack(3, c.held[0], c.held[1], c.held[2]);
done:
    drop(&c);
    return result;
}

/* A pair of pools of any kind, of pages of page_size tokens (*h_kv < 0: any number of heads). */
static int any_pools(const Call *c, PyObject *k, PyObject *v, int32_t page_size, int32_t *kind,
                     int32_t *pages, int32_t *h_kv, void **kp, void **vp) {
    PyObject *dtype = PyObject_GetAttr(k, s_dtype);
    if (!dtype) return -1;
    const int type = dtype == g_type[U8] ? U8 : dtype == g_type[F8] ? F8 : BF16;
    Py_DECREF(dtype);
    *kind = type == U8 ? FANOUT_KV_Q4 : type == F8 ? FANOUT_KV_Q8 : FANOUT_KV_BF16;
    const int nd = type == U8 ? 3 : 4;
    Py_ssize_t shape[4] = {-1, *h_kv, type == U8 ? (Py_ssize_t)page_size * FANOUT_Q4_ROW_BYTES : page_size, 128};
    if (need(c, "k_pages", k, type, nd, shape, kp) < 0 || sizes(k, shape, 4) < 0 ||
        need(c, "v_pages", v, type, nd, shape, vp) < 0)
        return -1;
    return size32(shape[0], "num_pages", pages) < 0 || size32(shape[1], "H_kv", h_kv) < 0 ? -1 : 0;
}

/* kv_keep(k_pages, v_pages, page_table, prefix_len, suffix_lens, add_lens, path, counts,
 *         page_size, stream) */
static PyObject *kv_keep(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("kv_keep", n, 10) < 0) return NULL;
    int32_t kind, pages, h_kv = -1, prefix_len, page_size, B = 0, width = 0;
    if (int32_of(a[3], "prefix_len", &prefix_len) < 0 || int32_of(a[8], "page_size", &page_size) < 0)
        return NULL;
    Call c;
    if (begin(&c, a[0], "k_pages", a[9]) < 0) return NULL;
    PyObject *result = NULL;
    static const Py_ssize_t any[2] = {-1, -1};
    Py_ssize_t table[2], rows[1];
    void *kp, *vp, *tp, *s, *l, *path, *counts;
    if (any_pools(&c, a[0], a[1], page_size, &kind, &pages, &h_kv, &kp, &vp) < 0 ||
        need(&c, "page_table", a[2], I32, 2, any, &tp) < 0 || sizes(a[2], table, 2) < 0 ||
        need(&c, "suffix_lens", a[4], I32, 1, table, &s) < 0 ||
        need(&c, "add_lens", a[5], I32, 1, table, &l) < 0 || need(&c, "path", a[6], I32, 1, any, &path) < 0 ||
        sizes(a[6], rows, 1) < 0 || need(&c, "counts", a[7], I32, 1, table, &counts) < 0 ||
        size32(table[0], "page_table", &B) < 0 || size32(table[1], "page_table", &width) < 0)
        goto done;
    RUN(c, "fanout_kv_keep",
        fanout_kv_keep(kp, vp, kind, tp, B, width, prefix_len, s, l, path, counts, rows[0], pages, h_kv, 128,
                       page_size, stream));
    result = Py_NewRef(Py_None);
done:
    drop(&c);
    return result;
}

/* What the two attention calls share. Host lengths: the address of int32 [2, B] (binding._lens). */
typedef struct {
    int32_t prefix_len, B, width, h_q, h_kv, d, page_size, window, sinks, code;
    const int32_t *lens;
    Py_ssize_t R;
    void *q, *table, *out, *lse;
    PyObject *out_t, *lse_t;
    float scale, k_scale, v_scale;
} Attn;

/* a: q .. scale as the calls below have them; tail: window, sinks, k_scale, v_scale, out, lse, bf16 out, want lse */
static int attn_of(Call *c, Attn *x, PyObject *const *a, PyObject *const *tail) {
    Py_ssize_t shape[3] = {0};
    int want, nd;
    if (int32_of(a[4], "prefix_len", &x->prefix_len) < 0 || int32_of(a[6], "branches", &x->B) < 0 ||
        int32_of(a[8], "h_q", &x->h_q) < 0 || int32_of(a[9], "h_kv", &x->h_kv) < 0 ||
        int32_of(a[10], "page_size", &x->page_size) < 0 || float_of(a[11], &x->scale) < 0 ||
        int32_of(tail[0], "window", &x->window) < 0 || int32_of(tail[1], "sinks", &x->sinks) < 0 ||
        float_of(tail[2], &x->k_scale) < 0 || float_of(tail[3], &x->v_scale) < 0)
        return -1;
    x->lens = PyLong_AsVoidPtr(a[5]);
    x->R = PyLong_AsSsize_t(a[7]);
    if (PyErr_Occurred() || (nd = sizes(a[0], shape, 3)) < 0) return -1;
    if (nd != 3) {
        PyErr_SetString(PyExc_ValueError, "q must be [R, H_q, d]");
        return -1;
    }
    if (x->R < 0 || x->h_q < 0 || x->h_kv < 0) {  // (a size below 0 would stand for any)
        PyErr_SetString(PyExc_ValueError, "rows and heads must not be negative");
        return -1;
    }
    Py_ssize_t rows[3] = {x->R, x->h_q, shape[2]}, table[2] = {x->B, -1};
    if (size32(shape[2], "d", &x->d) < 0 || need(c, "q", a[0], BF16, 3, rows, &x->q) < 0 ||
        need(c, "page_table", a[3], I32, 2, table, &x->table) < 0 || sizes(a[3], table, 2) < 0 ||
        size32(table[1], "page_table", &x->width) < 0 || (x->code = PyObject_IsTrue(tail[6])) < 0 ||
        (want = PyObject_IsTrue(tail[7])) < 0)
        return -1;
    const int type = x->code ? BF16 : F32;
    x->code = x->code ? FANOUT_OUT_BF16 : FANOUT_OUT_F32;
    x->out_t = tail[4];
    x->lse_t = tail[5];
    x->lse = NULL;
    if (x->out_t == Py_None) {
        const int at = make(c, type, 3, rows, &x->out);
        if (at < 0) return -1;
        x->out_t = c->held[at];
    } else if (need(c, "out", x->out_t, type, 3, rows, &x->out) < 0) {
        return -1;
    }
    if (x->lse_t != Py_None) return need(c, "lse", x->lse_t, F32, 2, rows, &x->lse);
    if (want) {
        const int at = make(c, F32, 2, rows, &x->lse);
        if (at < 0) return -1;
        x->lse_t = c->held[at];
    }
    return 0;
}

/* attn_q8(q, k_pages, v_pages, page_table, prefix_len, lens, B, R, h_q, h_kv, page_size, scale,
 *         causal, window, sinks, k_scale, v_scale, out, lse, bf16 out, want lse, stream)
 *   -> (out, lse) */
static PyObject *attn_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("attn_q8", n, 22) < 0) return NULL;
    Call c;
    if (begin(&c, a[0], "q", a[21]) < 0) return NULL;
    PyObject *result = NULL;
    Attn x;
    int32_t pages = 0;
    void *kp, *vp;
    const int causal = PyObject_IsTrue(a[12]);
    if (causal < 0 || attn_of(&c, &x, a, a + 13) < 0) goto done;
    Py_ssize_t pool[4] = {-1, x.h_kv, x.page_size < 0 ? 0 : x.page_size, x.d};
    if (need(&c, "k_pages", a[1], F8, 4, pool, &kp) < 0 || sizes(a[1], pool, 4) < 0 ||
        need(&c, "v_pages", a[2], F8, 4, pool, &vp) < 0 || size32(pool[0], "num_pages", &pages) < 0)
        goto done;
    RUN(c, "fanout_attn_q8",
        fanout_attn_q8(x.q, kp, vp, x.table, x.prefix_len, x.lens, x.lens + x.B, x.B, x.width, pages, x.h_q,
                       x.h_kv, x.d, x.page_size, x.scale, causal, x.k_scale, x.v_scale, x.window, x.sinks,
                       x.out, x.code, x.lse, stream));
    result = PyTuple_Pack(2, x.out_t, x.lse_t);
done:
    drop(&c);
    return result;
}

/* attn_tree(q, k_pages, v_pages, page_table, prefix_len, lens, B, R, h_q, h_kv, page_size, scale,
 *           masks, positions, window, sinks, k_scale, v_scale, out, lse, bf16 out, want lse, stream)
 *   -> (out, lse) */
static PyObject *attn_tree(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (arity("attn_tree", n, 23) < 0) return NULL;
    Call c;
    if (begin(&c, a[0], "q", a[22]) < 0) return NULL;
    PyObject *result = NULL;
    Attn x;
    int32_t kind, pages, words = 0;
    void *kp, *vp, *masks, *positions = NULL;
    if (attn_of(&c, &x, a, a + 14) < 0 ||
        any_pools(&c, a[1], a[2], x.page_size, &kind, &pages, &x.h_kv, &kp, &vp) < 0)
        goto done;
    Py_ssize_t mask[2] = {x.R, -1};
    if (need(&c, "masks", a[12], I32, 2, mask, &masks) < 0 || sizes(a[12], mask, 2) < 0 ||
        size32(mask[1], "masks", &words) < 0 ||
        (a[13] != Py_None && need(&c, "positions", a[13], I32, 1, mask, &positions) < 0))
        goto done;
    RUN(c, "fanout_attn_tree",
        fanout_attn_tree(x.q, kp, vp, kind, x.table, x.prefix_len, x.lens, x.lens + x.B, x.B, x.width,
                         pages, x.h_q, x.h_kv, x.d, x.page_size, x.scale, masks, words, positions, x.window,
                         x.sinks, x.k_scale, x.v_scale, x.out, x.code, x.lse, stream));
    result = PyTuple_Pack(2, x.out_t, x.lse_t);
done:
    drop(&c);
    return result;
}

/* setup(types, empty, raw_stream, get_device, device_guard, empty_on, handle_of, raise) */
static PyObject *setup(PyObject *self, PyObject *args) {
    PyObject *types, *f[7];
    if (!PyArg_ParseTuple(args, "O!OOOOOOO", &PyTuple_Type, &types, f, f + 1, f + 2, f + 3, f + 4, f + 5,
                          f + 6))
        return NULL;
    if (PyTuple_GET_SIZE(types) != N_TYPES) {
        PyErr_SetString(PyExc_ValueError, "setup: wrong number of types");
        return NULL;
    }
    for (int i = 0; i < N_TYPES; ++i) Py_XSETREF(g_type[i], Py_NewRef(PyTuple_GET_ITEM(types, i)));
    PyObject **const to[7] = {&g_empty, &g_raw_stream, &g_get_device, &g_device_guard, &g_empty_on,
                              &g_handle_of, &g_raise};
    for (int i = 0; i < 7; ++i) Py_XSETREF(*to[i], Py_NewRef(f[i]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"kv_append_q8", (PyCFunction)(void (*)(void))kv_append_q8, METH_FASTCALL, NULL},
    {"kv_read_q8", (PyCFunction)(void (*)(void))kv_read_q8, METH_FASTCALL, NULL},
    {"tree_rows", (PyCFunction)(void (*)(void))tree_rows, METH_FASTCALL, NULL},
    {"tree_rows_sinks", (PyCFunction)(void (*)(void))tree_rows_sinks, METH_FASTCALL, NULL},
    {"tree_accept", (PyCFunction)(void (*)(void))tree_accept, METH_FASTCALL, NULL},
    {"kv_keep", (PyCFunction)(void (*)(void))kv_keep, METH_FASTCALL, NULL},
    {"attn_q8", (PyCFunction)(void (*)(void))attn_q8, METH_FASTCALL, NULL},
    {"attn_tree", (PyCFunction)(void (*)(void))attn_tree, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_calls", NULL, -1, methods, NULL, NULL,
                                    NULL, NULL};

PyMODINIT_FUNC PyInit__host_calls(void) {
    static const struct {
        PyObject **to;
        const char *name;
    } names[] = {{&s_dtype, "dtype"},   {&s_device, "device"},     {&s_shape, "shape"},
                 {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"},
                 {&s_index, "index"},   {&s_is_cuda, "is_cuda"},   {&s_stride, "stride"},
                 {&s_enter, "__enter__"}, {&s_exit, "__exit__"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!*names[i].to && !(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    if (!kw_empty && !(kw_empty = Py_BuildValue("(OO)", s_dtype, s_device))) return NULL;
    return PyModule_Create(&module);
}
