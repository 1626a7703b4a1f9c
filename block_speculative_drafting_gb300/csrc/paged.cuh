// What the kernels of the target's verification pass share: the paged cache
// and the call's rows as kernel parameters, the walk from a row to its
// sequence and position, element conversions, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dflash {

// element types: the values of DFLASH_F32 .. DFLASH_E2M1
constexpr int kF32 = 0, kBF16 = 1, kF16 = 2, kE4M3 = 3, kE2M1 = 4;

constexpr int kMaxDevices = 64;

// Division of 0 <= n < 2^31 by a fixed d: one high product, one addition and
// a shift (T. Granlund and P. L. Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994; a page size is any number, and every key row divides
// by it).
struct FastDiv {
    uint32_t mul, shift;
    int d;
};
inline FastDiv fast_div(int d) {
    uint32_t s = 0;
    while ((1ull << s) < (uint64_t)d) ++s;
    return {(uint32_t)((((1ull << s) - (uint64_t)d) << 32) / (uint64_t)d + 1), s, d};
}
// (the walk from rows to pages also runs on the host, for its tests)
#define DF_HD __host__ __device__ __forceinline__
DF_HD int lowest(int a, int b) { return a < b ? a : b; }
DF_HD int highest(int a, int b) { return a > b ? a : b; }
DF_HD int div_by(const FastDiv& f, int n) {
    return (int)(((uint32_t)(((uint64_t)(uint32_t)n * f.mul) >> 32) + (uint32_t)n) >> f.shift);
}

struct PagedCache {
    unsigned char *k, *v;
    int64_t ks[3], vs[3];  // page, slot, head strides in bytes
    const float *k_scale, *v_scale;
    int64_t n_pages;
    int kv_heads;
    // 4-bit caches: a row's block scales, one e4m3 byte for 16 columns
    unsigned char *kb, *vb;
    int64_t kbs[3], vbs[3];  // page, slot, head strides in bytes
};
struct PagedRows {
    int n_seqs, max_pages, per;  // per: rows of every sequence where row_start is null
    int n_rows, cap;             // cap: max_pages * page size
    const int32_t *row_start, *kv_len, *table;
    int64_t table_stride;
    FastDiv page;
};
struct HeadRows {
    unsigned char* p;
    int64_t rs, hs;  // row, head strides in bytes
    int dtype, heads;
};

// A row start as it is read: inside [0, n_rows], and not before any start ahead of it (the largest so far counts), so
// that the sequences' rows are apart and in order whatever the array holds.  On the device the two walks below are a
// warp's: 32 starts at once, every lane with the same s or r and the same answer.
DF_HD int row_start_at(const PagedRows& R, int j) { return lowest(highest(R.row_start[j], 0), R.n_rows); }
#ifdef __CUDA_ARCH__
constexpr int kWalk = 32;
DF_DEV int walk_lane() { return (int)(threadIdx.x & 31); }
DF_DEV int walk_max(int x) {
    for (int o = 16; o > 0; o >>= 1) x = highest(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
DF_DEV int walk_first(bool x) { return __ffs(__ballot_sync(0xffffffffu, x)) - 1; }  // the first lane with x, or -1
#else
constexpr int kWalk = 1;
inline int walk_lane() { return 0; }
inline int walk_max(int x) { return x; }
inline int walk_first(bool x) { return x ? 0 : -1; }
#endif
// Rows [a, b) of sequence s.
DF_HD void rows_of(const PagedRows& R, int s, int& a, int& b) {
    if (R.row_start == nullptr) {
        a = s * R.per;
        b = a + R.per;
        return;
    }
    int m = 0;
    for (int j = walk_lane(); j <= s; j += kWalk) m = highest(m, row_start_at(R, j));
    a = walk_max(m);
    b = highest(row_start_at(R, s + 1), a);
}
// The sequence that holds row r, or -1: the one before the first start past r.
DF_HD int seq_of(const PagedRows& R, int r) {
    if (R.row_start == nullptr) return R.per > 0 ? r / R.per : -1;
    for (int j0 = 0; j0 <= R.n_seqs; j0 += kWalk) {
        const int j = j0 + walk_lane();
        const int past = walk_first(j <= R.n_seqs && row_start_at(R, j) > r);
        if (past >= 0) return j0 + past - 1;
    }
    return -1;
}
// The table's entry for position p of sequence s, -1 outside the table.
DF_HD int page_entry(const PagedRows& R, int s, int p, int& slot) {
    slot = 0;
    if (p < 0 || p >= R.cap) return -1;
    const int idx = div_by(R.page, p);
    slot = p - idx * R.page.d;
    return R.table[(int64_t)s * R.table_stride + idx];
}
DF_HD bool page_held(int id, int64_t n_pages) { return id >= 0 && id < n_pages; }
// The page of position p of sequence s, or -1 where it is not held.
DF_HD int64_t page_of(const PagedRows& R, int64_t n_pages, int s, int p, int& slot) {
    const int id = page_entry(R, s, p, slot);
    return page_held(id, n_pages) ? id : -1;
}

// ---- launchers (0 = queued fine, else a cudaError_t)
struct Rotation {
    const double* inv_freq;
    int rotary, interleaved;
    float scale;
};
int paged_append(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& k, const HeadRows& v,
                 const HeadRows& q, const HeadRows& qo, const float* q_norm, const float* k_norm, float eps,
                 const Rotation& rot, const int32_t* evicted, int num_sms, cudaStream_t st);
int paged_read(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& ko, const HeadRows& vo,
               int num_sms, cudaStream_t st);
// weights: [sequence][key/value head][position] f32, the strides of the first two in elements
struct KeyWeights {
    float* p;
    int64_t ss, hs;
};
int paged_key_weights(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                      const float* lse, float scale, int window, const KeyWeights& W, int num_sms, cudaStream_t st);
struct EvictArgs {
    PagedCache C;
    PagedRows R;
    KeyWeights in, out;
    int keep, first, recent;
    int32_t *new_len, *evicted;
    int32_t* kept;   // [sequence][head][keep]: the slots that stay, -1 from the new length on
    int2* lens;      // [sequence]: the length before and after
};
int64_t paged_evict_workspace(int n_seqs, int kv_heads, int keep, bool own_kept);
int paged_evict(const EvictArgs& A, int cache_dtype, int hd, int num_sms, cudaStream_t st);

int64_t paged_attention_workspace(int cache_dtype, int hd, int n_seqs, int64_t n_rows, int heads, int kv_heads,
                                  int num_sms);
int paged_attention(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                    const HeadRows& out, float* lse, float scale, int window, void* ws, int num_sms, cudaStream_t st);

struct VerifyArgs {
    const void* target;
    int target_dtype;
    int64_t target_stride, draft_stride;  // elements
    const float* draft;                   // nullptr: all of q at the draft
    const uint32_t* draft_tok;
    const int32_t* draft_start;
    const float *temperature, *accept_u, *sample_u;
    int n_seqs, n_drafts, per, vocab;
    int32_t *accepted, *next_tok;
    float* prob;
};
int64_t verify_workspace(int n_seqs, int64_t n_drafts, int64_t vocab, int num_sms);
int verify(const VerifyArgs& A, void* ws, int num_sms, cudaStream_t st);

}  // namespace dflash
