// The hot half of target.py: what a call of the target's verification pass does
// on the host.  These calls run once a layer and step, where checks and
// allocations through Python's side of torch (4 to 5 us an output tensor, half a
// us a tensor read, on this part's host cores) took longer than the kernels they
// start; here tensors are read and made through torch's C++ side.
//
// The library's entry points come in as addresses (init).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <optional>
#include <string>

#include "../../include/dflash.h"

namespace {

enum { F32 = DFLASH_F32, BF16 = DFLASH_BF16, F16 = DFLASH_F16, E4M3 = DFLASH_E4M3, E2M1 = DFLASH_E2M1, F64 = 64, I32, U32, U8, OTHER };

PyObject *error_type, *memory_error;  // DFlashError, torch's OutOfMemoryError
decltype(&dflash_paged_append_at) lib_append;
decltype(&dflash_paged_read) lib_read;
decltype(&dflash_paged_key_weights) lib_key_weights;
decltype(&dflash_paged_evict) lib_evict;
decltype(&dflash_paged_evict_workspace) lib_evict_workspace;
decltype(&dflash_paged_attention) lib_attention;
decltype(&dflash_paged_attention_workspace) lib_attention_workspace;
decltype(&dflash_verify) lib_verify;
decltype(&dflash_verify_workspace) lib_verify_workspace;
decltype(&dflash_last_error) lib_last_error;

struct Refused {
    int code;
    std::string why;
};
struct PythonError {};  // set already
[[noreturn]] __attribute__((format(printf, 1, 2))) void refuse(const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    throw Refused{DFLASH_EINVAL, buf};
}
// a library call's code: 0 or a size, or its error raised
int64_t checked(int64_t rc) {
    if (rc < 0) throw Refused{(int)rc, lib_last_error(nullptr)};
    return rc;
}
// An entry point's body, its exceptions raised in Python.
template <class F>
PyObject* entry(F f) {
    try {
        return f();
    } catch (const PythonError&) {
    } catch (const Refused& r) {
        if (PyObject* e = PyObject_CallFunction(error_type, "is", r.code, r.why.c_str())) {
            PyErr_SetObject(error_type, e);
            Py_DECREF(e);
        }
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(memory_error, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

int type_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return F32;
        case at::kBFloat16: return BF16;
        case at::kHalf: return F16;
        case at::kFloat8_e4m3fn: return E4M3;
        case at::kDouble: return F64;
        case at::kInt: return I32;
        case at::kUInt32: return U32;
        case at::kByte: return U8;
        case at::ScalarType::Float4_e2m1fn_x2: return E2M1;
        default: return OTHER;
    }
}

// A tensor of 1 to 4 dimensions on the call's device.
struct Tensor {
    void* p;
    int64_t shape[4], stride[4];
    int nd, dtype;
    Tensor(const at::Tensor& t, const char* name, int dev) {
        if (!t.is_cuda() || t.get_device() != dev) refuse("%s is not on the call's CUDA device", name);
        nd = (int)t.dim();
        if (nd < 1 || nd > 4) refuse("%s has %d dimensions", name, nd);
        for (int i = 0; i < nd; ++i) {
            shape[i] = t.size(i);
            // (the stride of a dimension of one element is anything)
            stride[i] = shape[i] > 1 ? t.stride(i) : i == nd - 1 ? 1 : 0;
        }
        if (t.numel() == 0)  // (and so are all of a tensor without elements)
            for (int64_t i = nd - 1, s = 1; i >= 0; s *= shape[i] > 1 ? shape[i] : 1, --i) stride[i] = s;
        dtype = type_of(t.scalar_type());
        p = t.data_ptr();
    }
    void written(const char* name) const {
        for (int i = 0; i < nd; ++i)
            if (shape[i] > 1 && stride[i] == 0) refuse("%s is written and may not be an expanded tensor", name);
    }
};
const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s has to be a tensor, not %s", name, Py_TYPE(o)->tp_name);
        throw PythonError{};
    }
    return THPVariable_Unpack(o);
}

// A call's device and stream, made current: what the call allocates belongs to the stream that is current, so that it
// is not dealt out again before that stream is done with it.
struct Call {
    int dev;
    void* stream;
    std::optional<c10::cuda::CUDAGuard> on_device;
    std::optional<c10::cuda::CUDAStreamGuard> on_stream;
    Call(const at::Tensor& t, PyObject* given) {
        if (!t.is_cuda()) refuse("tensors have to be on a CUDA device");
        dev = t.get_device();
        if (given != Py_None) {
            const unsigned long long handle = PyLong_AsUnsignedLongLong(given);
            if (PyErr_Occurred()) throw PythonError{};
            on_stream.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>((uintptr_t)handle),
                                                               (c10::DeviceIndex)dev));
        } else if (c10::cuda::current_device() != dev) {
            on_device.emplace((c10::DeviceIndex)dev);
        }
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
    Tensor read(PyObject* o, const char* name) const { return Tensor(tensor(o, name), name, dev); }
    // a contiguous vector of n elements of one type, or None (null)
    void* vector(PyObject* o, const char* name, int64_t n, int dtype) const {
        if (o == Py_None) return nullptr;
        const Tensor t = read(o, name);
        if (t.nd != 1 || t.shape[0] != n || t.stride[0] != 1 || t.dtype != dtype)
            refuse("%s has to be a contiguous vector of %lld elements of its type", name, (long long)n);
        return t.p;
    }
    at::Tensor make(at::IntArrayRef size, at::ScalarType type) const {
        return at::empty(size, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev)));
    }
};
// The caller's workspace, or `need` bytes of torch's allocator: given back as soon as the call is queued, they are
// dealt out again to work behind it on its stream alone.
struct Workspace {
    c10::DataPtr own;
    void* p;
    int64_t bytes;
    Workspace(const Call& call, PyObject* given, int64_t need) {
        if (given != Py_None) {
            const Tensor t = call.read(given, "workspace");
            if (t.nd != 1 || t.stride[0] != 1) refuse("workspace has to be a contiguous vector");
            p = t.p;
            bytes = (int64_t)THPVariable_Unpack(given).nbytes();
        } else {
            own = c10::cuda::CUDACachingAllocator::get()->allocate((size_t)need);
            p = own.get();
            bytes = need;
        }
    }
};
template <class F>
int64_t unlocked(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const int64_t rc = f();
    PyEval_RestoreThread(state);
    return rc;
}
double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw PythonError{};
    return x;
}
PyObject* kept(PyObject* o) {
    Py_INCREF(o);
    return o;
}

dflash_head_rows head_rows(const Tensor& t, const char* name, int64_t n, int64_t hd) {
    if (t.nd != 3 || t.shape[0] != n || t.shape[2] != hd || t.stride[2] != 1)
        refuse("%s has to be [%lld][heads][%lld] with contiguous columns", name, (long long)n, (long long)hd);
    if (t.shape[1] > INT32_MAX) refuse("%s has %lld heads", name, (long long)t.shape[1]);
    return {t.p, t.dtype, (int32_t)t.shape[1], t.stride[0], t.stride[1]};
}
// A 4-bit cache's block scales, one an e4m3 byte for 16 columns.
void read_blocks(const Call& call, PyObject* o, const char* name, const dflash_paged_cache& c, bool writes, void** p,
                 int64_t (&strides)[3]) {
    if (o == Py_None) refuse("a 4-bit cache needs %s", name);
    const Tensor t = call.read(o, name);
    if (t.nd != 4 || t.dtype != E4M3 || t.shape[0] != c.n_pages || t.shape[1] != c.page_size ||
        t.shape[2] != c.kv_heads || t.shape[3] != c.head_dim / 16 || t.stride[3] != 1)
        refuse("%s has to be float8_e4m3fn [%lld][%d][%d][%d] with contiguous blocks", name, (long long)c.n_pages,
               (int)c.page_size, (int)c.kv_heads, (int)c.head_dim / 16);
    if (writes) t.written(name);
    *p = t.p;
    for (int i = 0; i < 3; ++i) strides[i] = t.stride[i];
}
// v None: a call that reads keys alone (the values' fields are then the keys').
dflash_paged_cache read_cache(const Call& call, PyObject* k, PyObject* v, PyObject* k_scale, PyObject* v_scale,
                              PyObject* k_block, PyObject* v_block, bool writes) {
    const Tensor tk = call.read(k, "k_cache"), tv = v == Py_None ? tk : call.read(v, "v_cache");
    if (tk.nd != 4 || tv.nd != 4 || tk.dtype != tv.dtype)
        refuse("k_cache and v_cache have to be [pages][page_size][kv_heads][head_dim] of one type");
    for (int i = 0; i < 4; ++i)
        if (tk.shape[i] != tv.shape[i]) refuse("k_cache and v_cache differ in shape");
    if (tk.stride[3] != 1 || tv.stride[3] != 1) refuse("k_cache and v_cache need contiguous columns");
    if (writes) tk.written("k_cache"), tv.written("v_cache");
    for (int i = 1; i < 4; ++i)
        if (tk.shape[i] > INT32_MAX / 2) refuse("a cache dimension is too large");
    dflash_paged_cache c{};
    c.k = tk.p;
    c.v = tv.p;
    c.dtype = tk.dtype == U8 ? E2M1 : tk.dtype;
    c.n_pages = tk.shape[0];
    c.page_size = (int32_t)tk.shape[1];
    c.kv_heads = (int32_t)tk.shape[2];
    c.head_dim = (int32_t)tk.shape[3] * (c.dtype == E2M1 ? 2 : 1);
    for (int i = 0; i < 3; ++i) {
        c.k_strides[i] = tk.stride[i];
        c.v_strides[i] = tv.stride[i];
    }
    c.k_scale = static_cast<const float*>(call.vector(k_scale, "k_scale", c.kv_heads, F32));
    c.v_scale = v == Py_None ? c.k_scale : static_cast<const float*>(call.vector(v_scale, "v_scale", c.kv_heads, F32));
    if (c.dtype == E2M1) {
        read_blocks(call, k_block, "k_block", c, writes, &c.k_block, c.k_block_strides);
        read_blocks(call, v == Py_None ? k_block : v_block, v == Py_None ? "k_block" : "v_block", c, writes, &c.v_block,
                    c.v_block_strides);
    } else if (k_block != Py_None || v_block != Py_None) {
        refuse("block scales need a 4-bit cache");
    }
    return c;
}
dflash_paged_rows read_rows(const Call& call, PyObject* table, PyObject* kv_len, PyObject* row_start, int64_t n_rows) {
    const Tensor t = call.read(table, "table");
    if (t.nd != 2 || t.dtype != I32 || t.stride[1] != 1 || t.shape[0] > INT32_MAX - 1 || t.shape[1] > INT32_MAX)
        refuse("table has to be int32 [sequences][pages] with contiguous rows");
    if (kv_len == Py_None) refuse("kv_len is None");
    dflash_paged_rows r{};
    r.n_seqs = (int32_t)t.shape[0];
    r.max_pages = (int32_t)t.shape[1];
    r.n_rows = n_rows;
    r.row_start = static_cast<const int32_t*>(call.vector(row_start, "row_start", t.shape[0] + 1, I32));
    r.kv_len = static_cast<const int32_t*>(call.vector(kv_len, "kv_len", t.shape[0], I32));
    r.table = static_cast<const int32_t*>(t.p);
    r.table_stride = t.shape[0] > 1 ? t.stride[0] : t.shape[1];
    return r;
}
bool arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, got);
    return got == want;
}

// k_cache, v_cache, k, v, table, kv_len, row_start, q, q_out, inv_freq, interleaved, rope_scale, q_norm, k_norm, eps,
// k_scale, v_scale, stream, k_block, v_block, evicted
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 21)) return nullptr;
    return entry([&]() -> PyObject* {
        const Call call(tensor(a[0], "k_cache"), a[17]);
        const dflash_paged_cache c = read_cache(call, a[0], a[1], a[15], a[16], a[18], a[19], true);
        const Tensor tk = call.read(a[2], "k"), tv = call.read(a[3], "v");
        const int64_t n = tk.shape[0], hd = c.head_dim;
        const dflash_head_rows k = head_rows(tk, "k", n, hd), v = head_rows(tv, "v", n, hd);
        const dflash_paged_rows r = read_rows(call, a[4], a[5], a[6], n);
        const float* qn = static_cast<const float*>(call.vector(a[12], "q_norm", hd, F32));
        const float* kn = static_cast<const float*>(call.vector(a[13], "k_norm", hd, F32));
        const auto* evicted = static_cast<const int32_t*>(call.vector(a[20], "evicted", r.n_seqs, I32));
        dflash_rotation rot{};
        const bool rotates = a[9] != Py_None, with_q = a[7] != Py_None;
        if (rotates) {
            const Tensor f = call.read(a[9], "inv_freq");
            if (f.nd != 1 || f.dtype != F64 || f.stride[0] != 1 || f.shape[0] > 32768)
                refuse("inv_freq has to be a contiguous float64 vector");
            rot.inv_freq = static_cast<const double*>(f.p);
            rot.rotary = (int32_t)(2 * f.shape[0]);
            rot.interleaved = PyObject_IsTrue(a[10]);
            if (rot.interleaved < 0) throw PythonError{};
            rot.scale = (float)number(a[11]);
        }
        const float eps = (float)number(a[14]);
        if (!with_q && a[8] != Py_None) refuse("q_out without q");
        dflash_head_rows q{}, qo{};
        at::Tensor made;
        if (with_q) {
            const at::Tensor& tq = tensor(a[7], "q");
            q = head_rows(Tensor(tq, "q", call.dev), "q", n, hd);
            if (a[8] == Py_None) made = call.make(tq.sizes(), tq.scalar_type());
            const Tensor to(a[8] == Py_None ? made : tensor(a[8], "q_out"), "q_out", call.dev);
            to.written("q_out");
            qo = head_rows(to, "q_out", n, hd);
        }
        checked(unlocked([&] {
            return lib_append(&c, &r, &k, &v, with_q ? &q : nullptr, with_q ? &qo : nullptr, qn, kn, eps,
                              rotates ? &rot : nullptr, evicted, call.stream);
        }));
        return made.defined() ? THPVariable_Wrap(std::move(made)) : kept(a[8]);
    });
}

// The scale of the scores: None is head_dim ** -0.5.
double scale_of(PyObject* o, int64_t hd) { return o == Py_None ? std::pow((double)hd, -0.5) : number(o); }
int32_t window_of(PyObject* o) {
    const long window = PyLong_AsLong(o);
    if (PyErr_Occurred()) throw PythonError{};
    if (window < 0 || window > INT32_MAX) refuse("window %ld", window);
    return (int32_t)window;
}
float* read_lse(const Call& call, PyObject* o, int64_t n, int heads) {
    const Tensor t = call.read(o, "lse");
    if (t.nd != 2 || t.dtype != F32 || t.shape[0] != n || t.shape[1] != heads || t.stride[1] != 1 ||
        (n > 1 && t.stride[0] != heads))
        refuse("lse has to be contiguous float32 [%lld][%d]", (long long)n, heads);
    return static_cast<float*>(t.p);
}

// q, k_cache, v_cache, table, kv_len, row_start, scale, window, k_scale, v_scale, out, lse, workspace, stream, k_block,
// v_block
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 16)) return nullptr;
    return entry([&]() -> PyObject* {
        const at::Tensor& qt = tensor(a[0], "q");
        const Call call(qt, a[13]);
        const dflash_paged_cache c = read_cache(call, a[1], a[2], a[8], a[9], a[14], a[15], false);
        const Tensor tq(qt, "q", call.dev);
        const int64_t n = tq.shape[0], hd = c.head_dim;
        const dflash_head_rows q = head_rows(tq, "q", n, hd);
        const dflash_paged_rows r = read_rows(call, a[3], a[4], a[5], n);
        const double scale = scale_of(a[6], hd);
        const int32_t window = window_of(a[7]);
        float* lse = a[11] == Py_None ? nullptr : read_lse(call, a[11], n, q.heads);
        const int64_t need = checked(lib_attention_workspace(&c, r.n_seqs, n, q.heads));
        at::Tensor made;
        if (a[10] == Py_None) made = call.make(qt.sizes(), qt.scalar_type());
        const Tensor to(a[10] == Py_None ? made : tensor(a[10], "out"), "out", call.dev);
        to.written("out");
        const dflash_head_rows o = head_rows(to, "out", n, hd);
        const Workspace w(call, a[12], need);
        checked(unlocked([&] {
            return lib_attention(&c, &r, &q, &o, lse, (float)scale, window, w.p, w.bytes, call.stream);
        }));
        return made.defined() ? THPVariable_Wrap(std::move(made)) : kept(a[10]);
    });
}

// k_cache, v_cache, table, kv_len, rows, row_start, k_scale, v_scale, k_block, v_block, dtype's name, k_out, v_out, stream
PyObject* paged_read(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 14)) return nullptr;
    return entry([&]() -> PyObject* {
        const Call call(tensor(a[0], "k_cache"), a[13]);
        const dflash_paged_cache c = read_cache(call, a[0], a[1], a[6], a[7], a[8], a[9], false);
        const long long n = PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) throw PythonError{};
        if (n < 0 || n >= 1 << 24) refuse("rows %lld", n);
        const dflash_paged_rows r = read_rows(call, a[2], a[3], a[5], n);
        at::ScalarType type = at::kBFloat16;
        if (a[10] != Py_None) {
            if (!THPDtype_Check(a[10])) {
                PyErr_Format(PyExc_TypeError, "dtype has to be a torch.dtype, not %s", Py_TYPE(a[10])->tp_name);
                throw PythonError{};
            }
            type = reinterpret_cast<THPDtype*>(a[10])->scalar_type;
        } else if (c.dtype == F16) {
            type = at::kHalf;
        }
        at::Tensor made[2];
        dflash_head_rows out[2];
        static const char* const names[2] = {"k_out", "v_out"};
        if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
            refuse("dtype is not float32, bfloat16 or float16");
        for (int i = 0; i < 2; ++i) {
            if (a[11 + i] == Py_None) made[i] = call.make({n, c.kv_heads, c.head_dim}, type);
            const Tensor t(a[11 + i] == Py_None ? made[i] : tensor(a[11 + i], names[i]), names[i], call.dev);
            t.written(names[i]);
            if (a[10] != Py_None && t.dtype != type_of(type)) refuse("%s is not of the dtype asked for", names[i]);
            out[i] = head_rows(t, names[i], n, c.head_dim);
        }
        checked(unlocked([&] { return lib_read(&c, &r, &out[0], &out[1], call.stream); }));
        PyObject* res = PyTuple_New(2);
        for (int i = 0; res != nullptr && i < 2; ++i) {
            PyObject* x = made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : kept(a[11 + i]);
            if (x == nullptr) Py_CLEAR(res);
            if (res != nullptr) PyTuple_SET_ITEM(res, i, x);
        }
        return res;
    });
}

// float32 [sequences][kv_heads][positions] with contiguous positions
dflash_key_weights read_weights(const Call& call, PyObject* o, const char* name, const dflash_paged_rows& r,
                                const dflash_paged_cache& c, bool writes) {
    const Tensor t = call.read(o, name);
    if (t.nd != 3 || t.dtype != F32 || t.shape[0] != r.n_seqs || t.shape[1] != c.kv_heads || t.stride[2] != 1)
        refuse("%s has to be float32 [%d][%d][positions] with contiguous positions", name, (int)r.n_seqs, (int)c.kv_heads);
    if (writes) t.written(name);
    return {static_cast<float*>(t.p), t.shape[2], t.stride[0], t.stride[1]};
}

// weights, q, k_cache, table, kv_len, lse, row_start, scale, window, k_scale, k_block, stream
PyObject* paged_key_weights(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 12)) return nullptr;
    return entry([&]() -> PyObject* {
        const at::Tensor& qt = tensor(a[1], "q");
        const Call call(qt, a[11]);
        const dflash_paged_cache c = read_cache(call, a[2], Py_None, a[9], Py_None, a[10], Py_None, false);
        const Tensor tq(qt, "q", call.dev);
        const int64_t n = tq.shape[0], hd = c.head_dim;
        const dflash_head_rows q = head_rows(tq, "q", n, hd);
        const dflash_paged_rows r = read_rows(call, a[3], a[4], a[6], n);
        const double scale = scale_of(a[7], hd);
        const int32_t window = window_of(a[8]);
        const float* lse = read_lse(call, a[5], n, q.heads);
        const dflash_key_weights w = read_weights(call, a[0], "weights", r, c, true);
        checked(unlocked([&] { return lib_key_weights(&c, &r, &q, lse, (float)scale, window, &w, call.stream); }));
        return kept(a[0]);
    });
}

int32_t whole(PyObject* o, const char* name) {
    const long x = PyLong_AsLong(o);
    if (PyErr_Occurred()) throw PythonError{};
    if (x < 0 || x > INT32_MAX) refuse("%s %ld", name, x);
    return (int32_t)x;
}
// k_cache, v_cache, weights, table, kv_len, keep, first, recent, k_block, v_block, weights_out, new_len, kept, evicted,
// workspace, stream
PyObject* paged_evict(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 16)) return nullptr;
    return entry([&]() -> PyObject* {
        const Call call(tensor(a[0], "k_cache"), a[15]);
        const dflash_paged_cache c = read_cache(call, a[0], a[1], Py_None, Py_None, a[8], a[9], true);
        const dflash_paged_rows r = read_rows(call, a[3], a[4], Py_None, 0);
        const int32_t keep = whole(a[5], "keep"), first = whole(a[6], "first"), recent = whole(a[7], "recent");
        const bool aside = a[10] != Py_None && a[10] != a[2];
        const dflash_key_weights w = read_weights(call, a[2], "weights", r, c, !aside);
        const dflash_key_weights o = aside ? read_weights(call, a[10], "weights_out", r, c, true) : w;
        int32_t* kept_slots = nullptr;
        if (a[12] != Py_None) {
            const Tensor t = call.read(a[12], "kept");
            if (t.nd != 3 || t.dtype != I32 || t.shape[0] != r.n_seqs || t.shape[1] != c.kv_heads || t.shape[2] != keep ||
                (keep > 1 && t.stride[2] != 1) || (c.kv_heads > 1 && t.stride[1] != keep) ||
                (r.n_seqs > 1 && t.stride[0] != (int64_t)c.kv_heads * keep))
                refuse("kept has to be contiguous int32 [%d][%d][%d]", (int)r.n_seqs, (int)c.kv_heads, (int)keep);
            kept_slots = static_cast<int32_t*>(t.p);
        }
        auto* evicted = static_cast<int32_t*>(call.vector(a[13], "evicted", r.n_seqs, I32));
        const int64_t need = checked(lib_evict_workspace(r.n_seqs, c.kv_heads, keep, kept_slots == nullptr));
        at::Tensor made;
        if (a[11] == Py_None) made = call.make({r.n_seqs}, at::kInt);
        auto* new_len = static_cast<int32_t*>(a[11] == Py_None ? made.data_ptr() : call.vector(a[11], "new_len", r.n_seqs, I32));
        const Workspace ws(call, a[14], need);
        checked(unlocked([&] {
            return lib_evict(&c, &r, keep, first, recent, &w, &o, new_len, kept_slots, evicted, ws.p, ws.bytes, call.stream);
        }));
        return made.defined() ? THPVariable_Wrap(std::move(made)) : kept(a[11]);
    });
}

// target_logits, draft_tokens, accept_u, sample_u, draft_logits, draft_start, temperature, accepted, next_token, prob,
// workspace, stream
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!arguments(na, 12)) return nullptr;
    return entry([&]() -> PyObject* {
        const at::Tensor& tt = tensor(a[0], "target_logits");
        const Call call(tt, a[11]);
        const Tensor t(tt, "target_logits", call.dev), tok = call.read(a[1], "draft_tokens"),
            u = call.read(a[3], "sample_u");
        if (t.nd != 2 || t.stride[1] != 1) refuse("target_logits has to be [rows][vocab] with contiguous rows");
        // [sequences][drafts] or [drafts], contiguous
        int64_t d = 1;
        bool packed = tok.dtype == I32 || tok.dtype == U32;
        for (int i = tok.nd - 1; i >= 0; --i) {
            packed &= tok.shape[i] <= 1 || tok.stride[i] == d;
            d *= tok.shape[i];
        }
        if (!packed) refuse("draft_tokens has to be contiguous int32 or uint32");
        if (u.nd != 1) refuse("sample_u has to be a vector");
        const int64_t n = u.shape[0], vocab = t.shape[1];
        if (t.shape[0] != n + d)
            refuse("%lld drafts of %lld sequences need %lld target rows, got %lld", (long long)d, (long long)n,
                   (long long)(n + d), (long long)t.shape[0]);
        int64_t ds = 0;
        const float* draft = nullptr;
        if (a[4] != Py_None) {
            const Tensor dl = call.read(a[4], "draft_logits");
            // rows of the vocabulary, evenly apart: any leading dimensions that fold into one
            bool ok = dl.dtype == F32 && dl.nd >= 2 && dl.shape[dl.nd - 1] == vocab && dl.stride[dl.nd - 1] == 1;
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
            if (!ok || rows != d)
                refuse("draft_logits has to be float32 [%lld][%lld] with evenly spaced, contiguous rows", (long long)d,
                       (long long)vocab);
            draft = static_cast<const float*>(dl.p);
        }
        if (a[2] == Py_None) refuse("accept_u is None");
        const auto* au = static_cast<const float*>(call.vector(a[2], "accept_u", d, F32));
        const auto* su = static_cast<const float*>(call.vector(a[3], "sample_u", n, F32));
        const auto* start = static_cast<const int32_t*>(call.vector(a[5], "draft_start", n + 1, I32));
        const auto* temp = static_cast<const float*>(call.vector(a[6], "temperature", n, F32));
        const int64_t need = checked(lib_verify_workspace((int32_t)(n > INT32_MAX ? -1 : n), d, vocab));
        static const char* const names[3] = {"accepted", "next_token", "prob"};
        at::Tensor made[3];
        void* out[3];
        for (int i = 0; i < 3; ++i) {
            const int64_t size = i < 2 ? n : d;
            if (a[7 + i] == Py_None) {
                made[i] = call.make({size}, i < 2 ? at::kInt : at::kFloat);
                out[i] = made[i].data_ptr();
            } else {
                out[i] = call.vector(a[7 + i], names[i], size, i < 2 ? I32 : F32);
            }
        }
        const Workspace w(call, a[10], need);
        checked(unlocked([&] {
            return lib_verify(t.p, t.dtype, t.shape[0] > 1 ? t.stride[0] : vocab, draft, ds,
                              static_cast<const uint32_t*>(tok.p), start, temp, au, su, (int32_t)n, d, vocab,
                              static_cast<int32_t*>(out[0]), static_cast<int32_t*>(out[1]), static_cast<float*>(out[2]),
                              w.p, w.bytes, call.stream);
        }));
        PyObject* res = PyTuple_New(3);
        for (int i = 0; res != nullptr && i < 3; ++i) {
            PyObject* x = made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : kept(a[7 + i]);
            if (x == nullptr) Py_CLEAR(res);
            if (res != nullptr) PyTuple_SET_ITEM(res, i, x);
        }
        return res;
    });
}

// init(addresses of the entry points, DFlashError, torch's OutOfMemoryError)
PyObject* init(PyObject*, PyObject* args) {
    unsigned long long f[10];
    PyObject *err, *memory;
    if (!PyArg_ParseTuple(args, "(KKKKKKKKKK)OO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9],
                          &err, &memory))
        return nullptr;
    lib_append = reinterpret_cast<decltype(lib_append)>((uintptr_t)f[0]);
    lib_attention = reinterpret_cast<decltype(lib_attention)>((uintptr_t)f[1]);
    lib_attention_workspace = reinterpret_cast<decltype(lib_attention_workspace)>((uintptr_t)f[2]);
    lib_verify = reinterpret_cast<decltype(lib_verify)>((uintptr_t)f[3]);
    lib_verify_workspace = reinterpret_cast<decltype(lib_verify_workspace)>((uintptr_t)f[4]);
    lib_last_error = reinterpret_cast<decltype(lib_last_error)>((uintptr_t)f[5]);
    lib_read = reinterpret_cast<decltype(lib_read)>((uintptr_t)f[6]);
    lib_key_weights = reinterpret_cast<decltype(lib_key_weights)>((uintptr_t)f[7]);
    lib_evict = reinterpret_cast<decltype(lib_evict)>((uintptr_t)f[8]);
    lib_evict_workspace = reinterpret_cast<decltype(lib_evict_workspace)>((uintptr_t)f[9]);
    Py_INCREF(err);
    Py_XSETREF(error_type, err);
    Py_INCREF(memory);
    Py_XSETREF(memory_error, memory);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}
PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"paged_append", fast(paged_append), METH_FASTCALL, nullptr},
                         {"paged_attention", fast(paged_attention), METH_FASTCALL, nullptr},
                         {"paged_read", fast(paged_read), METH_FASTCALL, nullptr},
                         {"paged_key_weights", fast(paged_key_weights), METH_FASTCALL, nullptr},
                         {"paged_evict", fast(paged_evict), METH_FASTCALL, nullptr},
                         {"verify_drafts", fast(verify_drafts), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
