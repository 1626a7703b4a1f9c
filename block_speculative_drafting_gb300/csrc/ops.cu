// The C entry points of the target's verification pass (include/dflash.h): the
// checks of their arguments, and the hand-over to the kernels' launchers.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/dflash.h"
#include "common.cuh"
#include "kernels.cuh"
#include "paged_attn.cuh"

using namespace dflash;

namespace {

__attribute__((format(printf, 2, 3))) int fail(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_thread_error(code, buf);
}
int launched(int e, const char* what) {
    if (e == 0) return DFLASH_OK;
    cudaGetLastError();  // the error is reported here, not by the next call that looks
    return fail(e == (int)cudaErrorMemoryAllocation ? DFLASH_ENOMEM : DFLASH_ECUDA, "%s: %s", what,
                cudaGetErrorString((cudaError_t)e));
}
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
// (of a 4-bit cache: of the two codes that its strides count)
int64_t size_of(int dtype) { return dtype == DFLASH_F32 ? 4 : dtype == DFLASH_E4M3 || dtype == DFLASH_E2M1 ? 1 : 2; }

// The current device's SM count (asked of the driver once a device).
int sms(int* out) {
    static std::mutex mu;
    static int known[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return launched((int)e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(DFLASH_EINVAL, "device %d", dev);
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        int n = 0;
        if (cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev))
            return launched((int)e, "cudaDeviceGetAttribute");
        known[dev] = n;
    }
    *out = known[dev];
    return DFLASH_OK;
}

int check_cache(const dflash_paged_cache* c, PagedCache* out) {
    if (c == nullptr) return fail(DFLASH_EINVAL, "cache is NULL");
    if (c->dtype != DFLASH_BF16 && c->dtype != DFLASH_F16 && c->dtype != DFLASH_E4M3 && c->dtype != DFLASH_E2M1)
        return fail(DFLASH_EINVAL, "cache dtype %d is not BF16, F16, E4M3 or E2M1", c->dtype);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(DFLASH_EGEOM, "head_dim %d is not 64 or 128", c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > 65536) return fail(DFLASH_EINVAL, "kv_heads %d", c->kv_heads);
    if (c->page_size < 1 || c->page_size > 65536) return fail(DFLASH_EINVAL, "page_size %d", c->page_size);
    if (c->n_pages < 0 || c->n_pages > INT32_MAX) return fail(DFLASH_EINVAL, "n_pages %lld", (long long)c->n_pages);
    if (c->n_pages > 0 && (c->k == nullptr || c->v == nullptr)) return fail(DFLASH_EINVAL, "cache k or v is NULL");
    if (!al16(c->k) || !al16(c->v)) return fail(DFLASH_EINVAL, "cache k and v need 16-byte alignment");
    if ((c->k_scale == nullptr) != (c->v_scale == nullptr))
        return fail(DFLASH_EINVAL, "k_scale and v_scale come together");
    if (c->k_scale != nullptr && c->dtype != DFLASH_E4M3 && c->dtype != DFLASH_E2M1)
        return fail(DFLASH_EINVAL, "scales need an E4M3 cache or an E2M1 one");
    if (!al4(c->k_scale) || !al4(c->v_scale)) return fail(DFLASH_EINVAL, "scales need 4-byte alignment");
    const int64_t e = size_of(c->dtype);
    *out = PagedCache{};
    out->k = static_cast<unsigned char*>(c->k);
    out->v = static_cast<unsigned char*>(c->v);
    for (int i = 0; i < 3; ++i) {
        out->ks[i] = c->k_strides[i] * e;
        out->vs[i] = c->v_strides[i] * e;
        if (c->k_strides[i] < 0 || c->v_strides[i] < 0 || out->ks[i] % 16 || out->vs[i] % 16)
            return fail(DFLASH_EINVAL, "cache strides must be multiples of 16 bytes and not negative");
    }
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->n_pages = c->n_pages;
    out->kv_heads = c->kv_heads;
    if (c->dtype == DFLASH_E2M1) {
        const int64_t row = c->head_dim / 16;
        const auto apart = [row](const void* p) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)row == 0; };
        if (c->n_pages > 0 && (c->k_block == nullptr || c->v_block == nullptr))
            return fail(DFLASH_EINVAL, "an E2M1 cache needs k_block and v_block");
        bool ok = apart(c->k_block) && apart(c->v_block);
        for (int i = 0; i < 3; ++i) {
            out->kbs[i] = c->k_block_strides[i];
            out->vbs[i] = c->v_block_strides[i];
            ok = ok && out->kbs[i] >= 0 && out->vbs[i] >= 0 && out->kbs[i] % row == 0 && out->vbs[i] % row == 0;
            if (out->ks[i] > INT32_MAX || out->vs[i] > INT32_MAX || out->kbs[i] > INT32_MAX || out->vbs[i] > INT32_MAX)
                return fail(DFLASH_EINVAL, "strides of an E2M1 cache must be below 2^31 bytes");
        }
        if (!ok)
            return fail(DFLASH_EINVAL, "block scales: base and strides must be multiples of %d bytes, strides not negative",
                        (int)row);
        out->kb = static_cast<unsigned char*>(c->k_block);
        out->vb = static_cast<unsigned char*>(c->v_block);
    }
    return DFLASH_OK;
}

int check_rows(const dflash_paged_rows* r, const dflash_paged_cache* c, PagedRows* out) {
    if (r == nullptr) return fail(DFLASH_EINVAL, "rows is NULL");
    if (r->n_seqs < 0 || r->n_seqs >= 1 << 24) return fail(DFLASH_EINVAL, "n_seqs %d", r->n_seqs);
    if (r->n_rows < 0 || r->n_rows >= 1 << 24) return fail(DFLASH_EINVAL, "n_rows %lld", (long long)r->n_rows);
    if (r->n_rows > 0 && r->n_seqs == 0) return fail(DFLASH_EINVAL, "rows without a sequence");
    if (r->max_pages < 0 || (int64_t)r->max_pages * c->page_size > INT32_MAX - 65536)
        return fail(DFLASH_EINVAL, "max_pages %d of %d slots", r->max_pages, c->page_size);
    if (r->row_start == nullptr && r->n_seqs > 0 && r->n_rows % r->n_seqs)
        return fail(DFLASH_EINVAL, "%lld rows do not divide over %d sequences", (long long)r->n_rows, r->n_seqs);
    if (r->n_rows > 0 && r->kv_len == nullptr) return fail(DFLASH_EINVAL, "kv_len is NULL");
    if (r->n_rows > 0 && r->max_pages > 0 && r->table == nullptr) return fail(DFLASH_EINVAL, "table is NULL");
    if (r->table_stride < 0 || (r->n_seqs > 1 && r->table_stride > 0 && r->table_stride < r->max_pages))
        return fail(DFLASH_EINVAL, "table_stride %lld under its %d columns", (long long)r->table_stride, r->max_pages);
    if (!al4(r->row_start) || !al4(r->kv_len) || !al4(r->table))
        return fail(DFLASH_EINVAL, "row_start, kv_len and table need 4-byte alignment");
    *out = PagedRows{};
    out->n_seqs = r->n_seqs;
    out->max_pages = r->max_pages;
    out->per = r->row_start == nullptr && r->n_seqs > 0 ? (int)(r->n_rows / r->n_seqs) : 0;
    out->n_rows = (int)r->n_rows;
    out->cap = r->max_pages * c->page_size;
    out->row_start = r->row_start;
    out->kv_len = r->kv_len;
    out->table = r->table;
    out->table_stride = r->table_stride;
    out->page = fast_div(c->page_size);
    return DFLASH_OK;
}

// Rows of `heads` heads (0: any number that is a multiple of `kv_heads`).
int check_heads(const dflash_head_rows* h, const char* name, int heads, int kv_heads, int64_t n_rows, HeadRows* out) {
    if (h == nullptr) return fail(DFLASH_EINVAL, "%s is NULL", name);
    if (h->dtype != DFLASH_F32 && h->dtype != DFLASH_BF16 && h->dtype != DFLASH_F16)
        return fail(DFLASH_EINVAL, "%s dtype %d is not F32, BF16 or F16", name, h->dtype);
    if (heads > 0 ? h->heads != heads : h->heads < 1 || h->heads > 65536 || h->heads % kv_heads != 0)
        return fail(DFLASH_EINVAL, "%s has %d heads for %d key/value heads", name, h->heads, kv_heads);
    if (n_rows * h->heads > INT32_MAX) return fail(DFLASH_EINVAL, "%s: too many rows x heads", name);
    if (n_rows > 0 && h->data == nullptr) return fail(DFLASH_EINVAL, "%s data is NULL", name);
    const int64_t e = size_of(h->dtype);
    if (!al16(h->data) || h->row_stride < 0 || h->head_stride < 0 || h->row_stride * e % 16 || h->head_stride * e % 16)
        return fail(DFLASH_EINVAL, "%s: base and strides must be multiples of 16 bytes, strides not negative", name);
    *out = HeadRows{static_cast<unsigned char*>(h->data), h->row_stride * e, h->head_stride * e, h->dtype, h->heads};
    return DFLASH_OK;
}

int check_weights(const dflash_key_weights* w, const char* name, const PagedRows& R, KeyWeights* out) {
    if (w == nullptr) return fail(DFLASH_EINVAL, "%s is NULL", name);
    if ((w->data == nullptr && R.n_seqs > 0 && R.cap > 0) || !al4(w->data)) return fail(DFLASH_EINVAL, "%s data is NULL or not 4-byte aligned", name);
    if (w->positions < R.cap)
        return fail(DFLASH_EINVAL, "%s of %lld positions, the table names %d", name, (long long)w->positions, R.cap);
    if (w->seq_stride < 0 || w->head_stride < 0) return fail(DFLASH_EINVAL, "%s: strides must not be negative", name);
    *out = KeyWeights{w->data, w->seq_stride, w->head_stride};
    return DFLASH_OK;
}

#define TRY(expr)                   \
    do {                            \
        const int e__ = (expr);     \
        if (e__ != 0) return e__;   \
    } while (0)

}  // namespace

extern "C" {

int dflash_paged_append_at(const dflash_paged_cache* cache, const dflash_paged_rows* rows, const dflash_head_rows* k,
                           const dflash_head_rows* v, const dflash_head_rows* q, const dflash_head_rows* q_out,
                           const float* q_norm, const float* k_norm, float eps, const dflash_rotation* rotation,
                           const int32_t* evicted, void* stream) {
    PagedCache C;
    PagedRows R;
    HeadRows K, V, Q{}, QO{};
    TRY(check_cache(cache, &C));
    TRY(check_rows(rows, cache, &R));
    TRY(check_heads(k, "k", cache->kv_heads, 1, R.n_rows, &K));
    TRY(check_heads(v, "v", cache->kv_heads, 1, R.n_rows, &V));
    if ((q == nullptr) != (q_out == nullptr)) return fail(DFLASH_EINVAL, "q and q_out come together");
    if (q != nullptr) {
        TRY(check_heads(q, "q", 0, cache->kv_heads, R.n_rows, &Q));
        TRY(check_heads(q_out, "q_out", q->heads, 1, R.n_rows, &QO));
        if (q->data == q_out->data && R.n_rows > 0 &&
            (q->dtype != q_out->dtype || q->row_stride != q_out->row_stride || q->head_stride != q_out->head_stride))
            return fail(DFLASH_EINVAL, "q_out in q's place needs q's type and strides");
    }
    if (v->dtype != k->dtype || (q != nullptr && q->dtype != k->dtype))
        return fail(DFLASH_EINVAL, "q, k and v need one type");
    if (!al16(q_norm) || !al16(k_norm)) return fail(DFLASH_EINVAL, "norm gains need 16-byte alignment");
    if ((q_norm != nullptr || k_norm != nullptr) && !(eps >= 0.f && std::isfinite(eps)))
        return fail(DFLASH_EINVAL, "eps %g", (double)eps);
    Rotation rot{};
    if (rotation != nullptr) {
        if (rotation->rotary < 16 || rotation->rotary > cache->head_dim || rotation->rotary % 16)
            return fail(DFLASH_EINVAL, "rotary %d is not a multiple of 16 up to %d", rotation->rotary, cache->head_dim);
        if (rotation->inv_freq == nullptr || (reinterpret_cast<uintptr_t>(rotation->inv_freq) & 7))
            return fail(DFLASH_EINVAL, "inv_freq is NULL or not 8-byte aligned");
        if (!std::isfinite(rotation->scale)) return fail(DFLASH_EINVAL, "rotation scale %g", (double)rotation->scale);
        rot = Rotation{rotation->inv_freq, rotation->rotary, rotation->interleaved != 0, rotation->scale};
    }
    if (!al4(evicted)) return fail(DFLASH_EINVAL, "evicted needs 4-byte alignment");
    if (R.n_rows == 0) return DFLASH_OK;
    int n = 0;
    TRY(sms(&n));
    return launched(paged_append(C, cache->dtype, cache->head_dim, R, K, V, Q, QO, q_norm, k_norm, eps, rot, evicted, n,
                                 static_cast<cudaStream_t>(stream)),
                    "dflash_paged_append");
}

int dflash_paged_append(const dflash_paged_cache* cache, const dflash_paged_rows* rows, const dflash_head_rows* k,
                        const dflash_head_rows* v, const dflash_head_rows* q, const dflash_head_rows* q_out,
                        const float* q_norm, const float* k_norm, float eps, const dflash_rotation* rotation,
                        void* stream) {
    return dflash_paged_append_at(cache, rows, k, v, q, q_out, q_norm, k_norm, eps, rotation, nullptr, stream);
}

int dflash_paged_read(const dflash_paged_cache* cache, const dflash_paged_rows* rows, const dflash_head_rows* k_out,
                      const dflash_head_rows* v_out, void* stream) {
    PagedCache C;
    PagedRows R;
    HeadRows K{}, V{};
    TRY(check_cache(cache, &C));
    TRY(check_rows(rows, cache, &R));
    if (k_out == nullptr && v_out == nullptr) return fail(DFLASH_EINVAL, "k_out and v_out are NULL");
    if (k_out != nullptr) TRY(check_heads(k_out, "k_out", cache->kv_heads, 1, R.n_rows, &K));
    if (v_out != nullptr) TRY(check_heads(v_out, "v_out", cache->kv_heads, 1, R.n_rows, &V));
    if (k_out != nullptr && v_out != nullptr && k_out->dtype != v_out->dtype)
        return fail(DFLASH_EINVAL, "k_out and v_out need one type");
    if (k_out != nullptr && v_out != nullptr && R.n_rows > 0 && k_out->data == v_out->data)
        return fail(DFLASH_EINVAL, "k_out and v_out are one memory");
    if (R.n_rows == 0) return DFLASH_OK;
    int n = 0;
    TRY(sms(&n));
    return launched(paged_read(C, cache->dtype, cache->head_dim, R, K, V, n, static_cast<cudaStream_t>(stream)),
                    "dflash_paged_read");
}

int dflash_paged_key_weights(const dflash_paged_cache* cache, const dflash_paged_rows* rows, const dflash_head_rows* q,
                             const float* lse, float scale, int32_t window, const dflash_key_weights* weights,
                             void* stream) {
    PagedCache C;
    PagedRows R;
    HeadRows Q;
    KeyWeights W;
    TRY(check_cache(cache, &C));
    TRY(check_rows(rows, cache, &R));
    TRY(check_heads(q, "q", 0, cache->kv_heads, R.n_rows, &Q));
    if (q->dtype == DFLASH_F32 || (size_of(cache->dtype) == 2 && q->dtype != cache->dtype))
        return fail(DFLASH_EINVAL, "q needs the cache's type (BF16 or F16 for an E4M3 or E2M1 cache)");
    if (!(scale >= 1e-30f && scale <= 1e30f)) return fail(DFLASH_EINVAL, "scale %g", (double)scale);
    if (window < 0 || window > 1 << 30) return fail(DFLASH_EINVAL, "window %d", window);
    if (!al4(lse) || (lse == nullptr && R.n_rows > 0)) return fail(DFLASH_EINVAL, "lse is NULL or not 4-byte aligned");
    TRY(check_weights(weights, "weights", R, &W));
    if (!pa_line_fits(R, q->heads, cache->kv_heads, DFLASH_E2M1))
        return fail(DFLASH_EINVAL, "%d sequences of %d positions: too many tiles of keys", R.n_seqs, R.cap);
    if (R.n_rows == 0) return DFLASH_OK;
    int n = 0;
    TRY(sms(&n));
    return launched(paged_key_weights(C, cache->dtype, cache->head_dim, R, Q, lse, scale, window, W, n,
                                      static_cast<cudaStream_t>(stream)),
                    "dflash_paged_key_weights");
}

int64_t dflash_paged_evict_workspace(int32_t n_seqs, int32_t kv_heads, int32_t keep, int32_t own_kept) {
    if (n_seqs < 0 || n_seqs >= 1 << 24 || kv_heads < 1 || kv_heads > 65536 || keep < 1 ||
        (int64_t)n_seqs * kv_heads > INT32_MAX / 16)
        return fail(DFLASH_EINVAL, "n_seqs %d, kv_heads %d, keep %d", n_seqs, kv_heads, keep);
    return paged_evict_workspace(n_seqs, kv_heads, keep, own_kept != 0);
}

int dflash_paged_evict(const dflash_paged_cache* cache, const dflash_paged_rows* seqs, int32_t keep, int32_t first,
                       int32_t recent, const dflash_key_weights* weights, const dflash_key_weights* out,
                       int32_t* new_len, int32_t* kept, int32_t* evicted, void* workspace, int64_t workspace_bytes,
                       void* stream) {
    EvictArgs A{};
    TRY(check_cache(cache, &A.C));
    TRY(check_rows(seqs, cache, &A.R));
    if (A.R.n_rows != 0 || A.R.row_start != nullptr) return fail(DFLASH_EINVAL, "an eviction has no rows");
    if (keep < 1 || first < 0 || recent < 0 || (int64_t)first + recent > keep)
        return fail(DFLASH_EINVAL, "keep %d, first %d, recent %d", keep, first, recent);
    const int64_t need = dflash_paged_evict_workspace(A.R.n_seqs, cache->kv_heads, keep, kept == nullptr);
    if (need < 0) return (int)need;
    if (A.R.n_seqs == 0) return DFLASH_OK;
    if (A.R.kv_len == nullptr || (A.R.max_pages > 0 && A.R.table == nullptr))
        return fail(DFLASH_EINVAL, "kv_len or table is NULL");
    // (rows of both would be moved at once)
    if (A.C.n_pages > 0 && (A.C.k == A.C.v || (cache->dtype == DFLASH_E2M1 && A.C.kb == A.C.vb)))
        return fail(DFLASH_EINVAL, "k and v of the cache are one memory");
    TRY(check_weights(weights, "weights", A.R, &A.in));
    TRY(check_weights(out, "out", A.R, &A.out));
    if (A.in.p == A.out.p && (A.in.ss != A.out.ss || A.in.hs != A.out.hs))
        return fail(DFLASH_EINVAL, "out in weights' place needs its strides");
    if (new_len == nullptr || !al4(new_len) || !al4(kept) || !al4(evicted))
        return fail(DFLASH_EINVAL, "new_len is NULL, or new_len, kept or evicted not 4-byte aligned");
    if (new_len == evicted) return fail(DFLASH_EINVAL, "new_len and evicted are one memory");
    if (workspace == nullptr || !al16(workspace))
        return fail(DFLASH_EINVAL, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < need)
        return fail(DFLASH_ECAPACITY, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                    (long long)need);
    int n = 0;
    TRY(sms(&n));
    A.keep = keep, A.first = first, A.recent = recent;
    A.new_len = new_len, A.evicted = evicted;
    A.lens = static_cast<int2*>(workspace);
    A.kept = kept != nullptr ? kept
                             : reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) +
                                                          paged_evict_workspace(A.R.n_seqs, cache->kv_heads, keep, false));
    return launched(paged_evict(A, cache->dtype, cache->head_dim, n, static_cast<cudaStream_t>(stream)),
                    "dflash_paged_evict");
}

int64_t dflash_paged_attention_workspace(const dflash_paged_cache* cache, int32_t n_seqs, int64_t n_rows,
                                         int32_t heads) {
    PagedCache C;
    TRY(check_cache(cache, &C));
    if (n_seqs < 0 || n_rows < 0 || n_rows >= 1 << 24 || heads < 1 || heads % cache->kv_heads)
        return fail(DFLASH_EINVAL, "n_seqs %d, n_rows %lld, heads %d", n_seqs, (long long)n_rows, heads);
    int n = 0;
    TRY(sms(&n));
    return paged_attention_workspace(cache->dtype, cache->head_dim, n_seqs, n_rows, heads, cache->kv_heads, n);
}

int dflash_paged_attention(const dflash_paged_cache* cache, const dflash_paged_rows* rows, const dflash_head_rows* q,
                           const dflash_head_rows* out, float* lse, float scale, int32_t window, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    PagedCache C;
    PagedRows R;
    HeadRows Q, O;
    TRY(check_cache(cache, &C));
    TRY(check_rows(rows, cache, &R));
    TRY(check_heads(q, "q", 0, cache->kv_heads, R.n_rows, &Q));
    TRY(check_heads(out, "out", q->heads, 1, R.n_rows, &O));
    if (q->dtype == DFLASH_F32 || out->dtype != q->dtype || (size_of(cache->dtype) == 2 && q->dtype != cache->dtype))
        return fail(DFLASH_EINVAL, "q and out need the cache's type (BF16 or F16 for an E4M3 or E2M1 cache)");
    if (q->data == out->data && R.n_rows > 0 && (q->row_stride != out->row_stride || q->head_stride != out->head_stride))
        return fail(DFLASH_EINVAL, "out in q's place needs q's strides");
    if (!(scale >= 1e-30f && scale <= 1e30f)) return fail(DFLASH_EINVAL, "scale %g", (double)scale);
    if (window < 0 || window > 1 << 30) return fail(DFLASH_EINVAL, "window %d", window);
    if (!al4(lse)) return fail(DFLASH_EINVAL, "lse needs 4-byte alignment");
    if (!pa_line_fits(R, q->heads, cache->kv_heads, cache->dtype))
        return fail(DFLASH_EINVAL, "%d sequences of %d positions: too many tiles of keys", R.n_seqs, R.cap);
    if (R.n_rows == 0) return DFLASH_OK;
    int n = 0;
    TRY(sms(&n));
    const int64_t need =
        paged_attention_workspace(cache->dtype, cache->head_dim, R.n_seqs, R.n_rows, q->heads, cache->kv_heads, n);
    if (workspace == nullptr || !al16(workspace))
        return fail(DFLASH_EINVAL, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < need)
        return fail(DFLASH_ECAPACITY, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                    (long long)need);
    return launched(paged_attention(C, cache->dtype, cache->head_dim, R, Q, O, lse, scale, window, workspace, n,
                                    static_cast<cudaStream_t>(stream)),
                    "dflash_paged_attention");
}

int64_t dflash_verify_workspace(int32_t n_seqs, int64_t n_drafts, int64_t vocab) {
    if (n_seqs < 0 || n_drafts < 0 || n_drafts + n_seqs >= 1 << 24 || vocab < 1 || vocab >= 1 << 30)
        return fail(DFLASH_EINVAL, "n_seqs %d, n_drafts %lld, vocab %lld", n_seqs, (long long)n_drafts,
                    (long long)vocab);
    int n = 0;
    TRY(sms(&n));
    return verify_workspace(n_seqs, n_drafts, vocab, n);
}

int dflash_verify(const void* target, int32_t target_dtype, int64_t target_stride, const float* draft_logits,
                  int64_t draft_stride, const uint32_t* draft_tok, const int32_t* draft_start, const float* temperature,
                  const float* accept_u, const float* sample_u, int32_t n_seqs, int64_t n_drafts, int64_t vocab,
                  int32_t* accepted, int32_t* next_tok, float* prob, void* workspace, int64_t workspace_bytes,
                  void* stream) {
    if (n_seqs < 0 || n_drafts < 0 || n_drafts + n_seqs >= 1 << 24)
        return fail(DFLASH_EINVAL, "n_seqs %d, n_drafts %lld", n_seqs, (long long)n_drafts);
    if (vocab < 1 || vocab >= 1 << 30) return fail(DFLASH_EINVAL, "vocab %lld", (long long)vocab);
    if (target_dtype != DFLASH_F32 && target_dtype != DFLASH_BF16 && target_dtype != DFLASH_F16)
        return fail(DFLASH_EINVAL, "target dtype %d is not F32, BF16 or F16", target_dtype);
    if (n_drafts > 0 && n_seqs == 0) return fail(DFLASH_EINVAL, "drafts without a sequence");
    if (n_seqs == 0) return DFLASH_OK;
    if (draft_start == nullptr && n_drafts % n_seqs)
        return fail(DFLASH_EINVAL, "%lld drafts do not divide over %d sequences", (long long)n_drafts, n_seqs);
    if (target == nullptr || sample_u == nullptr || accepted == nullptr || next_tok == nullptr)
        return fail(DFLASH_EINVAL, "target, sample_u, accepted or next_tok is NULL");
    if (n_drafts > 0 && (draft_tok == nullptr || accept_u == nullptr))
        return fail(DFLASH_EINVAL, "draft_tok or accept_u is NULL");
    if (target_stride < vocab || (draft_logits != nullptr && n_drafts > 0 && draft_stride < vocab))
        return fail(DFLASH_EINVAL, "a row stride is under the vocabulary");
    if (reinterpret_cast<uintptr_t>(target) % (uintptr_t)size_of(target_dtype) || !al4(draft_logits) ||
        !al4(draft_tok) || !al4(draft_start) || !al4(temperature) || !al4(accept_u) || !al4(sample_u) ||
        !al4(accepted) || !al4(next_tok) || !al4(prob))
        return fail(DFLASH_EINVAL, "a pointer is not aligned to its elements");
    int n = 0;
    TRY(sms(&n));
    const int64_t need = verify_workspace(n_seqs, n_drafts, vocab, n);
    if (workspace == nullptr || !al16(workspace))
        return fail(DFLASH_EINVAL, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < need)
        return fail(DFLASH_ECAPACITY, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                    (long long)need);
    VerifyArgs A{};
    A.target = target, A.target_dtype = target_dtype, A.target_stride = target_stride;
    A.draft = n_drafts > 0 ? draft_logits : nullptr, A.draft_stride = draft_stride;
    A.draft_tok = draft_tok, A.draft_start = draft_start;
    A.temperature = temperature, A.accept_u = accept_u, A.sample_u = sample_u;
    A.n_seqs = n_seqs, A.n_drafts = (int)n_drafts, A.vocab = (int)vocab;
    A.per = draft_start == nullptr ? (int)(n_drafts / n_seqs) : 0;
    A.accepted = accepted, A.next_tok = next_tok, A.prob = prob;
    return launched(verify(A, workspace, n, static_cast<cudaStream_t>(stream)), "dflash_verify");
}

}  // extern "C"
