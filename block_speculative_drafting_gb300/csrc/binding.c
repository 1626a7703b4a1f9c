/*
 * The hot half of target.py: what a call of the target's verification pass does
 * on the host, without ctypes.  These calls run once a layer and step, where
 * their 20 us of interpreted argument checks were longer than the kernels they
 * start; here a call's checks, descriptors and launch take about 8.
 *
 * Tensors are read through their Python attributes (shape, stride, data_ptr,
 * dtype, device), so that nothing here depends on how torch was built.  The
 * library's entry points come in as addresses (init).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdarg.h>
#include <stdint.h>

#include "../../include/dflash.h"

enum { F32 = DFLASH_F32, BF16 = DFLASH_BF16, F16 = DFLASH_F16, E4M3 = DFLASH_E4M3, F64, I32, U32, OTHER };
#define DTYPES 7

static PyObject *s_shape, *s_stride, *s_data_ptr, *s_dtype, *s_get_device, *s_new_empty, *kw_dtype;
static PyObject* dtypes[DTYPES]; /* torch's, by the codes above */
static PyObject *error_type, *empty_like, *raw_stream, *raw_alloc, *raw_delete;
static __typeof__(&dflash_paged_append) lib_append;
static __typeof__(&dflash_paged_attention) lib_attention;
static __typeof__(&dflash_paged_attention_workspace) lib_attention_workspace;
static __typeof__(&dflash_verify) lib_verify;
static __typeof__(&dflash_verify_workspace) lib_verify_workspace;
static __typeof__(&dflash_last_error) lib_last_error;

typedef struct {
    void* p;
    int64_t shape[4], stride[4];
    int nd, dtype, dev;
} Tensor;

static int raise_error(int code, const char* msg) {
    PyObject* e = PyObject_CallFunction(error_type, "is", code, msg);
    if (e != NULL) {
        PyErr_SetObject(error_type, e);
        Py_DECREF(e);
    }
    return -1;
}
static int refuse(const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return raise_error(DFLASH_EINVAL, buf);
}
/* a library call's code: 0, or its error raised */
static int check(int64_t rc) { return rc < 0 ? raise_error((int)rc, lib_last_error(NULL)) : 0; }

static int numbers(PyObject* tuple, int64_t* out, int nd) {
    for (int i = 0; i < nd; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    return PyErr_Occurred() ? -1 : 0;
}
/* Reads a tensor of 1 to 4 dimensions on device `dev` (-1: any). */
static int read_tensor(PyObject* o, const char* name, int dev, Tensor* t) {
    PyObject* x = PyObject_GetAttr(o, s_shape);
    if (x == NULL) return -1;
    const Py_ssize_t nd = PyTuple_Check(x) ? PyTuple_GET_SIZE(x) : 0;
    t->nd = (int)nd;
    int rc = nd >= 1 && nd <= 4 ? numbers(x, t->shape, t->nd) : refuse("%s has %zd dimensions", name, nd);
    Py_DECREF(x);
    if (rc) return -1;
    x = PyObject_CallMethodNoArgs(o, s_stride);
    if (x == NULL) return -1;
    rc = numbers(x, t->stride, t->nd);
    Py_DECREF(x);
    if (rc) return -1;
    x = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (x == NULL) return -1;
    t->p = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    x = PyObject_GetAttr(o, s_dtype);
    if (x == NULL) return -1;
    for (t->dtype = 0; t->dtype < DTYPES && dtypes[t->dtype] != x; ++t->dtype) {}
    Py_DECREF(x);
    x = PyObject_CallMethodNoArgs(o, s_get_device);
    if (x == NULL) return -1;
    t->dev = (int)PyLong_AsLong(x);
    Py_DECREF(x);
    if (PyErr_Occurred()) return -1;
    if (t->dev < 0 || (dev >= 0 && t->dev != dev)) return refuse("%s is not on the call's CUDA device", name);
    /* the stride of a dimension of one element is anything */
    for (int i = 0; i < t->nd; ++i)
        if (t->shape[i] <= 1) t->stride[i] = i == t->nd - 1 ? 1 : 0;
    return 0;
}
static int written(const Tensor* t, const char* name) {
    for (int i = 0; i < t->nd; ++i)
        if (t->shape[i] > 1 && t->stride[i] == 0) return refuse("%s is written and may not be an expanded tensor", name);
    return 0;
}
/* A contiguous vector of n elements of one type, or None (NULL). */
static int vector(PyObject* o, const char* name, int dev, int64_t n, int dtype, void** out) {
    *out = NULL;
    if (o == Py_None) return 0;
    Tensor t;
    if (read_tensor(o, name, dev, &t)) return -1;
    if (t.nd != 1 || t.shape[0] != n || t.stride[0] != 1 || t.dtype != dtype)
        return refuse("%s has to be a contiguous vector of %lld elements of its type", name, (long long)n);
    *out = t.p;
    return 0;
}
static int head_rows(const Tensor* t, const char* name, int64_t n, int64_t hd, dflash_head_rows* out) {
    if (t->nd != 3 || t->shape[0] != n || t->shape[2] != hd || t->stride[2] != 1)
        return refuse("%s has to be [%lld][heads][%lld] with contiguous columns", name, (long long)n, (long long)hd);
    if (t->shape[1] > INT32_MAX) return refuse("%s has %lld heads", name, (long long)t->shape[1]);
    out->data = t->p;
    out->dtype = t->dtype;
    out->heads = (int32_t)t->shape[1];
    out->row_stride = t->stride[0];
    out->head_stride = t->stride[1];
    return 0;
}
static int read_cache(PyObject* k, PyObject* v, PyObject* k_scale, PyObject* v_scale, int* dev, int writes,
                      dflash_paged_cache* c) {
    Tensor tk, tv;
    if (read_tensor(k, "k_cache", *dev, &tk)) return -1;
    *dev = tk.dev;
    if (read_tensor(v, "v_cache", *dev, &tv)) return -1;
    if (tk.nd != 4 || tv.nd != 4 || tk.dtype != tv.dtype) return refuse("k_cache and v_cache have to be [pages][page_size][kv_heads][head_dim] of one type");
    for (int i = 0; i < 4; ++i)
        if (tk.shape[i] != tv.shape[i]) return refuse("k_cache and v_cache differ in shape");
    if (tk.stride[3] != 1 || tv.stride[3] != 1) return refuse("k_cache and v_cache need contiguous columns");
    if (writes && (written(&tk, "k_cache") || written(&tv, "v_cache"))) return -1;
    if (tk.shape[1] > INT32_MAX || tk.shape[2] > INT32_MAX || tk.shape[3] > INT32_MAX) return refuse("a cache dimension is too large");
    c->k = tk.p;
    c->v = tv.p;
    c->dtype = tk.dtype;
    c->n_pages = tk.shape[0];
    c->page_size = (int32_t)tk.shape[1];
    c->kv_heads = (int32_t)tk.shape[2];
    c->head_dim = (int32_t)tk.shape[3];
    for (int i = 0; i < 3; ++i) {
        c->k_strides[i] = tk.stride[i];
        c->v_strides[i] = tv.stride[i];
    }
    void *ks, *vs;
    if (vector(k_scale, "k_scale", *dev, c->kv_heads, F32, &ks) || vector(v_scale, "v_scale", *dev, c->kv_heads, F32, &vs))
        return -1;
    c->k_scale = ks;
    c->v_scale = vs;
    return 0;
}
static int read_rows(PyObject* table, PyObject* kv_len, PyObject* row_start, int dev, int64_t n_rows, dflash_paged_rows* r) {
    Tensor t;
    void *len, *start;
    if (read_tensor(table, "table", dev, &t)) return -1;
    if (t.nd != 2 || t.dtype != I32 || t.stride[1] != 1 || t.shape[0] > INT32_MAX - 1 || t.shape[1] > INT32_MAX)
        return refuse("table has to be int32 [sequences][pages] with contiguous rows");
    if (vector(kv_len, "kv_len", dev, t.shape[0], I32, &len) || vector(row_start, "row_start", dev, t.shape[0] + 1, I32, &start))
        return -1;
    if (len == NULL && kv_len == Py_None) return refuse("kv_len is None");
    r->n_seqs = (int32_t)t.shape[0];
    r->max_pages = (int32_t)t.shape[1];
    r->n_rows = n_rows;
    r->row_start = start;
    r->kv_len = len;
    r->table = t.p;
    r->table_stride = t.shape[0] > 1 ? t.stride[0] : t.shape[1];
    return 0;
}
static int current_stream(int dev, void** out) {
    PyObject* d = PyLong_FromLong(dev);
    PyObject* s = d != NULL ? PyObject_CallOneArg(raw_stream, d) : NULL;
    Py_XDECREF(d);
    if (s == NULL) return -1;
    *out = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return PyErr_Occurred() ? -1 : 0;
}
/* like.new_empty(n, dtype=dtypes[dtype]) */
static PyObject* new_empty(PyObject* like, int64_t n, int dtype) {
    PyObject* size = PyLong_FromLongLong(n);
    if (size == NULL) return NULL;
    PyObject* args[3] = {like, size, dtypes[dtype]};
    PyObject* t = PyObject_VectorcallMethod(s_new_empty, args, 2 | PY_VECTORCALL_ARGUMENTS_OFFSET, kw_dtype);
    Py_DECREF(size);
    return t;
}
/* The caller's workspace, or `need` bytes of torch's allocator for the call's stream: given back as soon as the call
 * is queued, they are dealt out again to work behind it on that stream alone. */
typedef struct {
    void* p;
    int64_t bytes;
    PyObject* own; /* the address to give back, or NULL */
} Workspace;
static int workspace_of(PyObject* given, int dev, void* stream, int64_t need, Workspace* w) {
    Tensor t;
    static const int size[DTYPES] = {4, 2, 2, 1, 8, 4, 4};
    w->own = NULL;
    if (given != Py_None) {
        if (read_tensor(given, "workspace", dev, &t)) return -1;
        if (t.nd != 1 || t.stride[0] != 1) return refuse("workspace has to be a contiguous vector");
        w->p = t.p;
        w->bytes = (t.dtype < DTYPES ? size[t.dtype] : 1) * t.shape[0]; /* (uint8 is none of the types above) */
        return 0;
    }
    w->own = PyObject_CallFunction(raw_alloc, "LK", (long long)need, (unsigned long long)(uintptr_t)stream);
    if (w->own == NULL) return -1;
    w->p = PyLong_AsVoidPtr(w->own);
    w->bytes = need;
    return PyErr_Occurred() ? -1 : 0;
}
/* Gives an allocated workspace back; keeps the error that is set, if one is. */
static int workspace_end(Workspace* w) {
    if (w->own == NULL) return 0;
    PyObject* err = PyErr_GetRaisedException();
    PyObject* x = PyObject_CallOneArg(raw_delete, w->own);
    const int bad = x == NULL;
    Py_XDECREF(x);
    Py_CLEAR(w->own);
    if (err != NULL) PyErr_SetRaisedException(err);
    return bad ? -1 : 0;
}

/* k_cache, v_cache, k, v, table, kv_len, row_start, q, q_out, inv_freq, interleaved, rope_scale, q_norm, k_norm, eps,
 * k_scale, v_scale */
static PyObject* paged_append(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 17) return PyErr_Format(PyExc_TypeError, "17 arguments, got %zd", na);
    dflash_paged_cache c;
    dflash_paged_rows r;
    dflash_head_rows k, v, q, qo;
    dflash_rotation rot;
    Tensor tk, tv, tq, to;
    int dev = -1;
    void *qn, *kn, *stream;
    if (read_cache(a[0], a[1], a[15], a[16], &dev, 1, &c) || read_tensor(a[2], "k", dev, &tk) || read_tensor(a[3], "v", dev, &tv))
        return NULL;
    const int64_t n = tk.shape[0], hd = c.head_dim;
    if (head_rows(&tk, "k", n, hd, &k) || head_rows(&tv, "v", n, hd, &v) || read_rows(a[4], a[5], a[6], dev, n, &r)) return NULL;
    if (vector(a[12], "q_norm", dev, hd, F32, &qn) || vector(a[13], "k_norm", dev, hd, F32, &kn)) return NULL;
    if (a[9] != Py_None) {
        Tensor f;
        if (read_tensor(a[9], "inv_freq", dev, &f)) return NULL;
        if (f.nd != 1 || f.dtype != F64 || f.stride[0] != 1 || f.shape[0] > 32768) {
            refuse("inv_freq has to be a contiguous float64 vector");
            return NULL;
        }
        const int inter = PyObject_IsTrue(a[10]);
        rot.inv_freq = f.p;
        rot.rotary = (int32_t)(2 * f.shape[0]);
        rot.interleaved = inter;
        rot.scale = (float)PyFloat_AsDouble(a[11]);
    }
    const float eps = (float)PyFloat_AsDouble(a[14]);
    if (PyErr_Occurred()) return NULL;
    PyObject* out = a[8];
    if (a[7] == Py_None && out != Py_None) {
        refuse("q_out without q");
        return NULL;
    }
    if (a[7] != Py_None) {
        if (read_tensor(a[7], "q", dev, &tq) || head_rows(&tq, "q", n, hd, &q)) return NULL;
        if (out == Py_None) {
            out = PyObject_CallOneArg(empty_like, a[7]);
            if (out == NULL) return NULL;
        } else {
            Py_INCREF(out);
        }
        if (read_tensor(out, "q_out", dev, &to) || written(&to, "q_out") || head_rows(&to, "q_out", n, hd, &qo)) goto fail;
    } else {
        Py_INCREF(out);
    }
    if (current_stream(dev, &stream)) goto fail;
    const int with_q = a[7] != Py_None, with_rot = a[9] != Py_None;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = lib_append(&c, &r, &k, &v, with_q ? &q : NULL, with_q ? &qo : NULL, qn, kn, eps, with_rot ? &rot : NULL, stream);
    Py_END_ALLOW_THREADS;
    if (check(rc)) goto fail;
    return out;
fail:
    Py_DECREF(out);
    return NULL;
}

/* q, k_cache, v_cache, table, kv_len, row_start, scale, window, k_scale, v_scale, out, lse, workspace */
static PyObject* paged_attention(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 13) return PyErr_Format(PyExc_TypeError, "13 arguments, got %zd", na);
    dflash_paged_cache c;
    dflash_paged_rows r;
    dflash_head_rows q, o;
    Tensor tq, to, tl;
    int dev = -1;
    void *stream, *lse = NULL;
    if (read_cache(a[1], a[2], a[8], a[9], &dev, 0, &c) || read_tensor(a[0], "q", dev, &tq)) return NULL;
    const int64_t n = tq.shape[0], hd = c.head_dim;
    if (head_rows(&tq, "q", n, hd, &q) || read_rows(a[3], a[4], a[5], dev, n, &r)) return NULL;
    const double scale = PyFloat_AsDouble(a[6]);
    const long window = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) return NULL;
    if (window < 0 || window > INT32_MAX) {
        refuse("window %ld", window);
        return NULL;
    }
    if (a[11] != Py_None) {
        if (read_tensor(a[11], "lse", dev, &tl)) return NULL;
        if (tl.nd != 2 || tl.dtype != F32 || tl.shape[0] != n || tl.shape[1] != q.heads || tl.stride[1] != 1 ||
            (n > 1 && tl.stride[0] != q.heads)) {
            refuse("lse has to be contiguous float32 [%lld][%d]", (long long)n, (int)q.heads);
            return NULL;
        }
        lse = tl.p;
    }
    const int64_t need = lib_attention_workspace(&c, r.n_seqs, n, q.heads);
    if (check(need)) return NULL;
    PyObject* out = a[10];
    if (out == Py_None) {
        out = PyObject_CallOneArg(empty_like, a[0]);
        if (out == NULL) return NULL;
    } else {
        Py_INCREF(out);
    }
    Workspace w = {NULL, 0, NULL};
    int rc = -1;
    if (!read_tensor(out, "out", dev, &to) && !written(&to, "out") && !head_rows(&to, "out", n, hd, &o) &&
        !current_stream(dev, &stream) && !workspace_of(a[12], dev, stream, need, &w)) {
        Py_BEGIN_ALLOW_THREADS;
        rc = lib_attention(&c, &r, &q, &o, lse, (float)scale, (int32_t)window, w.p, w.bytes, stream);
        Py_END_ALLOW_THREADS;
        rc = check(rc);
    }
    rc |= workspace_end(&w);
    if (rc) {
        Py_DECREF(out);
        return NULL;
    }
    return out;
}

/* target_logits, draft_tokens, accept_u, sample_u, draft_logits, draft_start, temperature, accepted, next_token, prob,
 * workspace */
static PyObject* verify_drafts(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 11) return PyErr_Format(PyExc_TypeError, "11 arguments, got %zd", na);
    Tensor t, tok, u, dl;
    if (read_tensor(a[0], "target_logits", -1, &t)) return NULL;
    const int dev = t.dev;
    if (read_tensor(a[1], "draft_tokens", dev, &tok) || read_tensor(a[3], "sample_u", dev, &u)) return NULL;
    if (t.nd != 2 || t.stride[1] != 1) {
        refuse("target_logits has to be [rows][vocab] with contiguous rows");
        return NULL;
    }
    /* [sequences][drafts] or [drafts], contiguous */
    int64_t d = 1;
    int packed = tok.dtype == I32 || tok.dtype == U32;
    for (int i = tok.nd - 1; i >= 0; --i) {
        packed &= tok.shape[i] <= 1 || tok.stride[i] == d;
        d *= tok.shape[i];
    }
    if (!packed) {
        refuse("draft_tokens has to be contiguous int32 or uint32");
        return NULL;
    }
    if (u.nd != 1) {
        refuse("sample_u has to be a vector");
        return NULL;
    }
    const int64_t n = u.shape[0], vocab = t.shape[1];
    if (t.shape[0] != n + d) {
        refuse("%lld drafts of %lld sequences need %lld target rows, got %lld", (long long)d, (long long)n, (long long)(n + d),
               (long long)t.shape[0]);
        return NULL;
    }
    int64_t ds = 0;
    if (a[4] != Py_None) {
        if (read_tensor(a[4], "draft_logits", dev, &dl)) return NULL;
        /* rows of the vocabulary, evenly apart: any leading dimensions that fold into one */
        int ok = dl.dtype == F32 && dl.nd >= 2 && dl.shape[dl.nd - 1] == vocab && dl.stride[dl.nd - 1] == 1;
        int64_t rows = 1;
        ds = vocab;
        for (int i = dl.nd - 2; ok && i >= 0; --i) {
            if (dl.shape[i] > 1) {
                if (rows == 1)
                    ds = dl.stride[i];
                else
                    ok = dl.stride[i] == rows * ds;
            }
            rows *= dl.shape[i];
        }
        if (!ok || rows != d) {
            refuse("draft_logits has to be float32 [%lld][%lld] with evenly spaced, contiguous rows", (long long)d,
                   (long long)vocab);
            return NULL;
        }
    }
    void *start, *temp, *au, *su, *acc, *nxt, *prob, *stream;
    if (a[2] == Py_None || vector(a[2], "accept_u", dev, d, F32, &au) || vector(a[3], "sample_u", dev, n, F32, &su) ||
        vector(a[5], "draft_start", dev, n + 1, I32, &start) || vector(a[6], "temperature", dev, n, F32, &temp)) {
        if (!PyErr_Occurred()) refuse("accept_u is None");
        return NULL;
    }
    const int64_t need = lib_verify_workspace((int32_t)(n > INT32_MAX ? -1 : n), d, vocab);
    if (check(need)) return NULL;
    PyObject* o[3] = {a[7], a[8], a[9]};
    for (int i = 0; i < 3; ++i) {
        if (o[i] == Py_None)
            o[i] = i == 0 ? new_empty(a[3], n, I32) : PyObject_CallOneArg(empty_like, i == 1 ? o[0] : a[2]);
        else
            Py_INCREF(o[i]);
        if (o[i] == NULL) {
            while (i-- > 0) Py_DECREF(o[i]);
            return NULL;
        }
    }
    Workspace w = {NULL, 0, NULL};
    int rc = -1;
    if (!vector(o[0], "accepted", dev, n, I32, &acc) && !vector(o[1], "next_token", dev, n, I32, &nxt) &&
        !vector(o[2], "prob", dev, d, F32, &prob) && !current_stream(dev, &stream) &&
        !workspace_of(a[10], dev, stream, need, &w)) {
        Py_BEGIN_ALLOW_THREADS;
        rc = lib_verify(t.p, t.dtype, t.shape[0] > 1 ? t.stride[0] : vocab, a[4] != Py_None ? (const float*)dl.p : NULL, ds,
                        tok.p, start, temp, au, su, (int32_t)n, d, vocab, acc, nxt, prob, w.p, w.bytes, stream);
        Py_END_ALLOW_THREADS;
        rc = check(rc);
    }
    rc |= workspace_end(&w);
    PyObject* res = rc ? NULL : PyTuple_Pack(3, o[0], o[1], o[2]);
    for (int i = 0; i < 3; ++i) Py_DECREF(o[i]);
    return res;
}

/* init(addresses of the six entry points, torch's dtypes by code, DFlashError, empty_like, the raw stream of a device,
 * torch's allocation of (bytes, stream) and its release) */
static PyObject* init(PyObject* self, PyObject* args) {
    (void)self;
    unsigned long long f[6];
    PyObject *types, *err, *like, *raw, *alloc, *dealloc;
    if (!PyArg_ParseTuple(args, "(KKKKKK)O!OOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &PyTuple_Type, &types, &err,
                          &like, &raw, &alloc, &dealloc))
        return NULL;
    if (PyTuple_GET_SIZE(types) != DTYPES) return PyErr_Format(PyExc_ValueError, "%d types", DTYPES);
    lib_append = (__typeof__(lib_append))(uintptr_t)f[0];
    lib_attention = (__typeof__(lib_attention))(uintptr_t)f[1];
    lib_attention_workspace = (__typeof__(lib_attention_workspace))(uintptr_t)f[2];
    lib_verify = (__typeof__(lib_verify))(uintptr_t)f[3];
    lib_verify_workspace = (__typeof__(lib_verify_workspace))(uintptr_t)f[4];
    lib_last_error = (__typeof__(lib_last_error))(uintptr_t)f[5];
    for (int i = 0; i < DTYPES; ++i) {
        Py_INCREF(PyTuple_GET_ITEM(types, i));
        Py_XSETREF(dtypes[i], PyTuple_GET_ITEM(types, i));
    }
    Py_INCREF(err);
    Py_XSETREF(error_type, err);
    Py_INCREF(like);
    Py_XSETREF(empty_like, like);
    Py_INCREF(raw);
    Py_XSETREF(raw_stream, raw);
    Py_INCREF(alloc);
    Py_XSETREF(raw_alloc, alloc);
    Py_INCREF(dealloc);
    Py_XSETREF(raw_delete, dealloc);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"init", init, METH_VARARGS, NULL},
                                {"paged_append", (PyCFunction)(void (*)(void))paged_append, METH_FASTCALL, NULL},
                                {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, NULL},
                                {"verify_drafts", (PyCFunction)(void (*)(void))verify_drafts, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_new_empty = PyUnicode_InternFromString("new_empty");
    kw_dtype = Py_BuildValue("(s)", "dtype");
    if (!s_shape || !s_stride || !s_data_ptr || !s_dtype || !s_get_device || !s_new_empty || !kw_dtype) return NULL;
    return PyModule_Create(&module);
}
