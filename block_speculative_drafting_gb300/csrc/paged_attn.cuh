// What the two kernels of the attention over a paged cache share: the line of
// work that the CTAs cut into equal parts and the walk along it, asynchronous
// copies, and conversions of 16-bit and 8-bit floats.
#pragma once

#include "paged.cuh"

namespace dflash {

constexpr int kPaTile = 128;     // keys a CTA takes at once: 16 a warp
// A row's reference m: its largest score in log2 units less kPaUnder when m is set, moved only where a score passes
// that by more than kPaLazy.  P = 2^(score - m) in f16 loses bits below 2^-14: set 7 under the maximum (P is then at
// most 2^15) it loses none that weigh 2^-21 of the largest.  (bf16 has f32's exponents, and values near f32's end.)
template <bool BF>
constexpr float kPaUnder = BF ? 0.f : 7.f;
constexpr float kPaLazy = 8.f;

struct PaArgs {
    PagedCache C;
    PagedRows R;
    HeadRows q, out;
    float* lse;
    float* ws_o;     // [2 CTAs][MT][HD]
    float2* ws_ml;   // [2 CTAs][MT]
    struct PaJoin* ws_join;  // [CTAs]
    int32_t* ws_odd;         // [CTAs]: outputs of the CTA's whole units wait for pa_odd_row
    float scale_log2;
    int window, group;
};

// A unit that starts in a CTA's share and ends in another's, for the join:
// its parts are this CTA's second slot and the first slots of the CTAs up to
// `last` (below 0: this CTA starts no such unit).
struct __align__(16) PaJoin {
    int32_t last, row0, m0, rows, head, seq, pad[2];  // rows from m0 on of sequence seq, whose rows start at row0; kv head
};

// What the walk needs of one sequence.
struct PaSeq {
    int row0, rows, p0;  // its rows of the call; the position of the first
    int lo, hi;          // keys that any of its rows may see
    int ntiles, nunits;
};

// of sequence s with rows [a, b)
DF_DEV PaSeq pa_seq(const PaArgs& A, int s, int a, int b, int mt) {
    PaSeq q;
    q.row0 = a;
    q.rows = b - a;
    const int len = A.R.kv_len[s];
    q.p0 = max(len, -1) - q.rows;  // a length below 0 reads as -1: no position of any row is held
    q.hi = min(max(len, 0), A.R.cap);
    q.lo = A.window > 0 ? max(0, q.p0 - A.window + 1) : 0;
    q.ntiles = max(1, (q.hi - q.lo + kPaTile - 1) / kPaTile);  // a sequence with rows but no keys: one tile of nothing
    q.nunits = (int)(((int64_t)q.rows * A.group + mt - 1) / mt) * A.C.kv_heads;
    return q;
}

// The line: the units' tiles in order (sequence, row tile, key/value head),
// each unit led by `ov` places without a tile, which stand for what it costs a
// CTA to end one unit and begin another, so that shares of equal length take
// equal time.  ov is 0 where most CTAs hold a tile or two: there a place
// without a tile would be an idle CTA.  (The line is shorter than 2^31: pa_line_fits.)
struct PaCur {
    PaSeq q;
    int s, u, tile;  // tile `tile` of unit `u` of sequence `s`
    int ov;
    int left;  // places of the CTA's share from here on (0: none)
};
// The end of sequence s's rows, which start at a.
DF_DEV int pa_rows_end(const PaArgs& A, int s, int a) {
    return A.R.row_start == nullptr ? a + A.R.per : max(row_start_at(A.R, s + 1), a);
}
// Rows [a, b) of sequence s0 + lane (warp-wide; none past the last sequence); `from`: where sequence s0's start.
DF_DEV void pa_rows_of_lane(const PaArgs& A, int s0, int from, int lane, int& a, int& b) {
    const int s = min(s0 + lane, A.R.n_seqs - 1);
    if (A.R.row_start == nullptr) {
        a = s * A.R.per;
        b = a + A.R.per;
    } else {
        b = max(row_start_at(A.R, s + 1), from);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) b = max(b, y);
        }
        a = __shfl_up_sync(0xffffffffu, b, 1);
        if (lane == 0) a = from;
    }
}
// This CTA's share (warp-wide); `chunk`: the places of a share.
DF_DEV PaCur pa_share(const PaArgs& A, int mt, int ovh, int lane, int& chunk) {
    int64_t t64 = 0, v64 = 0;
    int w0 = 0, u0 = 0;
    const int first = A.R.row_start == nullptr ? 0 : row_start_at(A.R, 0);
    for (int s0 = 0, from = first; s0 < A.R.n_seqs; s0 += 32) {
        int a, b;
        pa_rows_of_lane(A, s0, from, lane, a, b);
        from = __shfl_sync(0xffffffffu, b, 31);
        if (s0 + lane >= A.R.n_seqs) continue;
        const PaSeq q = pa_seq(A, s0 + lane, a, b, mt);
        const int64_t w = (int64_t)q.ntiles * q.nunits;
        if (s0 == 0) w0 = (int)w, u0 = q.nunits;
        t64 = min(t64 + w, (int64_t)1 << 40);
        v64 = min(v64 + q.nunits, (int64_t)1 << 40);
    }
    PaCur c{};
    chunk = 1;
    auto sum = [](int64_t x) {
        return ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)(x >> 20)) << 20) +
               __reduce_add_sync(0xffffffffu, (unsigned)(x & 0xfffff));
    };
    t64 = sum(t64);
    v64 = sum(v64);
    if (t64 + ovh * v64 >= 1ll << 31) return c;  // (never: pa_line_fits)
    const int tiles = (int)t64, units = (int)v64;
    c.ov = tiles > 2 * (int)gridDim.x ? ovh : 0;
    const int total = tiles + c.ov * units, grid = (int)gridDim.x;
    chunk = total / grid + (total % grid != 0);
    if ((int64_t)blockIdx.x * chunk >= total) return c;
    const int t = (int)blockIdx.x * chunk;
    int run = 0;
    for (int s0 = 0, from = first; s0 < A.R.n_seqs; s0 += 32) {
        int w = w0 + c.ov * u0, a, b;
        pa_rows_of_lane(A, s0, from, lane, a, b);
        from = __shfl_sync(0xffffffffu, b, 31);
        if (s0 > 0) {
            const PaSeq q = pa_seq(A, min(s0 + lane, A.R.n_seqs - 1), a, b, mt);
            w = s0 + lane < A.R.n_seqs ? (q.ntiles + c.ov) * q.nunits : 0;
        }
        int in = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + in > t);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int x = t - (run + __shfl_sync(0xffffffffu, in - w, l));
            c.s = s0 + l;
            c.q = pa_seq(A, c.s, __shfl_sync(0xffffffffu, a, l), __shfl_sync(0xffffffffu, b, l), mt);
            const int per = c.q.ntiles + c.ov;
            c.u = x / per;
            const int v = x - c.u * per;
            c.left = min(chunk, total - t);
            if (v < c.ov)
                c.left = max(c.left - (c.ov - v), 0);
            else
                c.tile = v - c.ov;
            return c;
        }
        run += __shfl_sync(0xffffffffu, in, 31);
    }
    return c;
}
DF_DEV void pa_next(const PaArgs& A, int mt, PaCur& c) {
    --c.left;
    if (++c.tile < c.q.ntiles) return;
    c.tile = 0;
    c.left -= c.ov;
    if (c.left <= 0) {
        c.left = 0;
        return;
    }
    if (++c.u < c.q.nunits) return;
    c.u = 0;
    do {
        if (++c.s >= A.R.n_seqs) {  // (never, while the lengths stay as they were counted)
            c.left = 0;
            return;
        }
        const int a = c.q.row0 + c.q.rows;
        c.q = pa_seq(A, c.s, a, pa_rows_end(A, c.s, a), mt);
    } while (c.q.nunits == 0);
}
// The entry of a unit that begins in this CTA's share and has `rest` tiles after it.
DF_DEV PaJoin pa_join_entry(const PaCur& c, int rt, int mt, int rows, int head, int rest, int chunk) {
    PaJoin e{};
    e.last = (int)(blockIdx.x + (rest + chunk - 1) / chunk);
    e.row0 = c.q.row0;
    e.m0 = rt * mt;
    e.rows = rows;
    e.head = head;
    e.seq = c.s;
    return e;
}

DF_DEV void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
DF_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DF_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 2^x by the special-function unit (relative error about 2^-22: the level of f32 rounding)
DF_DEV float pa_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two e4m3 codes -> two f16 (exact)
DF_DEV uint32_t e4m3x2_f16x2(uint32_t codes) {
    uint32_t y;
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(y) : "r"(codes));
    return y;
}
// four codes -> four f16
DF_DEV void e4m3x4_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
// (a, b) -> a pair of 16-bit floats, and what the rounding left
template <bool BF>
DF_DEV uint32_t pack2(float a, float b) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool BF>
DF_DEV float2 unpack2(uint32_t u) {
    if constexpr (BF)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// A value that is infinite, at a key in a row's view, makes that column of the row infinite (NaN where both signs meet, or
// where the key's weight is 0 because its score is -inf).  The products do not see to that: a weight goes in as a hi + lo
// pair, whose lo may be 0 or below, a row on two lanes multiplies the other lane's keys by 0, and a moved reference may
// multiply by 0.  All of these give NaN, so outputs that are NaN though the row's weights are not are kept apart by a NaN of
// their own (FMA gives 0x7fff) until the join's kernel looks over the row's keys for values that are not finite (pa_odd_row).
template <bool BF>
constexpr uint32_t kPaOdd = BF ? 0x7fc1u : 0x7e01u;
template <bool BF>
DF_DEV bool finite16(uint32_t h) {
    return BF ? (h & 0x7f80u) != 0x7f80u : (h & 0x7c00u) != 0x7c00u;
}
// whether a sum of weights is one (not 0, NaN or infinite)
DF_DEV bool pa_weighs(float l) { return l > 0.f && l < INFINITY; }
// An output row's NaN made the one kept apart, by one thread.
template <bool BF>
DF_DEV void pa_mark_odd(unsigned char* row, int hd) {
    uint16_t* x = reinterpret_cast<uint16_t*>(row);
#pragma unroll 1
    for (int d = 0; d < hd; ++d)
        if ((x[d] & 0x7fffu) > (BF ? 0x7f80u : 0x7c00u)) x[d] = (uint16_t)kPaOdd<BF>;
}

// Whether the places of any line of such a call stay below 2^31.
inline bool pa_line_fits(const PagedRows& R, int heads, int kv_heads) {
    const double units = (double)R.n_rows * heads / 16 + (double)R.n_seqs * kv_heads;
    return units * ((double)R.cap / kPaTile + 8) < 2147483648.0;
}
// tiles' time that a unit's end and the next one's beginning take in the tcgen05 kernel (32 blocks over a
// bf16 cache: 0 81.7 us, 2 73.3, 4 71.1)
constexpr int kPtOver = 4;
// The tcgen05 kernel (k_paged_attn_tc.cu): units of up to mt = 64 or 128 rows.
int paged_attention_tc(const PaArgs& A, int cache_dtype, int hd, int mt, int num_sms, cudaStream_t st);

}  // namespace dflash
