// Verification of drafted tokens against the target's probabilities.
//
// Two kernels.  verify_stats_kernel reads every logit row once: a CTA takes
// one part of one row's vocabulary and leaves what softmax needs of it, the sum
// of 2^(x c - R) with c = log2(e) / T and an integer reference R (or, of a
// greedy sequence, the largest logit and the lowest index that has it).
// verify_pick_kernel then takes a sequence per cluster: the parts of its rows
// are joined, each draft's p and q formed in 64 bits and compared with the
// given number, and one row -- the first refused, or the last -- is read again
// to sample the next token: the cluster's warps sum what is left of equal
// parts of the vocabulary, and the CTA in which the running sum passes the
// given number's share of the whole finds the part and, by 32nds, the entry.  That kernel runs once through its code, so its
// code is kept small (rolled loops): what it waits for most is instructions.
//
// Arithmetic.  A softmax sum is a tree of f32 additions of exponentials within
// 2^-22 each; c is a pair (hi, lo), so that its rounding does not tilt the
// distribution, and R is an integer, so that moving a sum to another reference
// is exact and x c - R is rounded once.  The running sum over a vocabulary
// decides which of 10^5 entries is drawn: it is carried in pairs of f32 by
// error-free additions, about 48 bits, since the 64-bit units of this part are
// few (two lanes a clock and SM: 64-bit sums in every warp took 30 us of a
// 40 us call).  The drafts' p and q are formed in 64 bits, a lane a draft.
//
// Memory bound: the logits, once (the re-read row comes out of L2).  32 blocks of
// up to 16 drafts, 151936 bf16 logits against f32 ones: 88 us, of which the
// statistics 55 (5.5 TB/s, 81 % of a copy) and the picking kernel 22 and its
// launch; one block 16 us, greedy 6.7, most of it latency.
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "paged.cuh"

namespace dflash {

namespace cg = cooperative_groups;

constexpr int kVsThreads = 256;
constexpr int kVpCluster = 8;
constexpr int kVpKept = 24576;  // entries of a CTA's parts whose weights are kept in shared memory
constexpr float kRefNone = -3e38f;               // the reference of a sum of nothing

// A sum as an unevaluated pair, about 48 bits.
struct Pair {
    float hi = 0.f, lo = 0.f;
};
DF_DEV Pair operator+(Pair a, Pair b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
DF_DEV Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
DF_DEV bool positive(Pair a) { return a.hi > 0.f; }  // (normalised: lo cannot turn the sign)
DF_DEV Pair shfl_xor(Pair a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
DF_DEV Pair shfl(Pair a, int l) { return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)}; }
// sums of the lanes up to and with this one
DF_DEV Pair warp_running(Pair a, int lane) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const Pair b{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if (lane >= o) a = a + b;
    }
    return a;
}
DF_DEV Pair warp_sum(Pair a) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) a = a + shfl_xor(a, o);
    return a;
}
// 2^d for an integer d <= 0 (0 under the normal range)
DF_DEV float pow2(float d) { return d < -126.f ? 0.f : __int_as_float(((int)d + 127) << 23); }
DF_DEV float ex2(float z) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(z));
    return y;
}

// What a part of a row (or a row) leaves.  Plain: the sum of 2^(x c - ref).
// Careful, where that form does not hold (a NaN, an infinite logit, entries so
// far apart that x c overflows or every weight underflows): the sum of
// 2^((x - max) c), 1 at the largest, 0 at NaN.
struct __align__(16) VerifyStat {
    float sum, ref, max;
    int32_t tag;  // a greedy sequence's: the lowest index of the largest logit; else 1: careful
};

struct VerifyParams {
    VerifyArgs A;
    VerifyStat* stats;  // [target rows, then draft rows][parts]
    int parts;
};

// A start as it is read: inside [0, n_drafts], and not before any start ahead of it, so that the sequences' drafts are
// apart and in order whatever the array holds.
DF_DEV int draft_start_at(const VerifyArgs& A, int j) { return min(max(A.draft_start[j], 0), A.n_drafts); }
// Drafts [a, b) of sequence s.  By a warp.
DF_DEV void draft_range(const VerifyArgs& A, int s, int lane, int& a, int& b) {
    if (A.draft_start == nullptr) {
        a = s * A.per;
        b = a + A.per;
        return;
    }
    int m = 0;
    for (int j = lane; j <= s; j += 32) m = max(m, draft_start_at(A, j));
    a = __reduce_max_sync(0xffffffffu, m);
    b = max(draft_start_at(A, s + 1), a);
}
// The sequence that holds draft (shift 0) or target row (shift 1) i, or -1: the last whose drafts or target rows start
// at or before it, unless they end there.  By a warp, 32 starts at once.
DF_DEV int verify_seq(const VerifyArgs& A, int i, int shift, int lane) {
    if (A.draft_start == nullptr) return i / (A.per + shift);
    int run = 0;  // the largest start so far
    for (int b = 0; b <= A.n_seqs; b += 32) {
        const int j = b + lane;
        int at = j <= A.n_seqs ? draft_start_at(A, j) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at = max(at, y);
        }
        at = max(at, run);
        // (starts ascend from here on: the first one past row i ends the search; sequence j has target rows at + j ..)
        const uint32_t past = __ballot_sync(0xffffffffu, j <= A.n_seqs && (int64_t)at + shift * (int64_t)j > i);
        if (past != 0) return b + __ffs(past) - 2;
        run = __shfl_sync(0xffffffffu, at, 31);
    }
    return -1;
}

// c = log2(e) / T as hi + lo, lo > 0 (so that -inf * lo is -inf); hi = 0
// for a greedy sequence (T <= 0 or NaN).  T is held to where both are finite.
struct Scale {
    float hi, lo;
    DF_DEV bool greedy() const { return hi == 0.f; }
    DF_DEV double wide() const { return (double)hi + (double)lo; }
};
DF_DEV Scale scale_of(const VerifyArgs& A, int s) {
    const float t0 = A.temperature != nullptr ? A.temperature[s] : 1.f;
    if (!(t0 > 0.f)) return {0.f, 0.f};
    const float t = fminf(fmaxf(t0, 1e-30f), 1e30f);
    const float lh = 1.44269502162933f, ll = 1.92596299e-8f;  // log2(e)
    const float ih = 1.f / t, il = fmaf(-t, ih, 1.f) * ih;    // 1 / T
    Scale c;
    c.hi = ih * lh;
    c.lo = fmaf(ih, lh, -c.hi) + fmaf(ih, ll, il * lh);
    if (c.lo < 0.f) {
        const float down = __int_as_float(__float_as_int(c.hi) - 1);
        c.lo += c.hi - down;
        c.hi = down;
    }
    c.lo = fmaxf(c.lo, 1e-37f);  // (-inf * 0 would be NaN)
    return c;
}
// 2^(x c - ref)
DF_DEV float weight(float x, Scale c, float ref) { return ex2(fmaf(x, c.lo, fmaf(x, c.hi, -ref))); }
// 2^((x - m) c): 1 at the largest (an infinite one too), 0 at NaN and far below
DF_DEV float weight_careful(float x, Scale c, float m) {
    const float t = fmaxf(x, -INFINITY) - m, z = fmaf(t, c.lo, t * c.hi);
    return x == m ? 1.f : z > -200.f ? ex2(z) : 0.f;
}

template <int DT>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<kF32> {
    static constexpr int N = 4;
    using T = float;
    DF_DEV static void split(uint4 v, float* x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    DF_DEV static float one(const float* p) { return __ldg(p); }
};
template <bool BF>
struct Vec16 {
    static constexpr int N = 8;
    using T = uint16_t;
    DF_DEV static float2 two(uint32_t u) {
        if constexpr (BF) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
    DF_DEV static void split(uint4 v, float* x) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = two(u[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    DF_DEV static float one(const uint16_t* p) { return two(__ldg(p)).x; }
};
template <>
struct Vec<kBF16> : Vec16<true> {};
template <>
struct Vec<kF16> : Vec16<false> {};

// The batches of a thread: f(x[4 N], first indices) over [v0, v1) of a row, absent entries -inf.  The entries
// up to the first 16-byte boundary and the last few come as a batch of their own.  A batch's four 16-byte
// loads are in flight while the one before it is worked on.
template <int DT>
struct Batches {
    using V = Vec<DT>;
    using T = typename V::T;
    static constexpr int N = V::N, U = 4, M = U * N;
    const T* row;
    const uint4* vec;
    int v0, v1, a, b, nv, i;
    uint4 next[U];
    DF_DEV Batches(const T* r, int from, int to) : row(r), v0(from), v1(to) {
        const int mis = (int)((reinterpret_cast<uintptr_t>(row + v0) & 15) / sizeof(T));
        a = min(v1, v0 + (mis ? N - mis : 0));
        nv = (v1 - a) / N;
        b = a + nv * N;
        vec = reinterpret_cast<const uint4*>(row + a);
        start();
    }
    DF_DEV void start() {
        i = threadIdx.x;
        load();
    }
    DF_DEV void load() {
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * kVsThreads < nv) next[k] = __ldg(vec + i + k * kVsThreads);
    }
    template <class F>
    DF_DEV void each(F f) {
        float x[M];
        int at[U];
        if (a > v0 || v1 > b) {
#pragma unroll
            for (int j = 0; j < M; ++j) x[j] = -INFINITY;
#pragma unroll
            for (int k = 0; k < U; ++k) at[k] = v0;
            const int h = v0 + threadIdx.x, t = b + threadIdx.x;
            if (h < a) x[0] = V::one(row + h), at[0] = h;
            if (t < v1) x[N] = V::one(row + t), at[1] = t;
            if (h < a || t < v1) f(x, at);
        }
        while (i < nv) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int j = i + k * kVsThreads;
                at[k] = a + j * N;
                if (j < nv) {
                    V::split(next[k], x + k * N);
                } else {
#pragma unroll
                    for (int n = 0; n < N; ++n) x[k * N + n] = -INFINITY;
                }
            }
            i += U * kVsThreads;
            load();
            f(x, at);
        }
    }
};
template <int M>
DF_DEV float max_of(const float* x) {
    float m = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < M; i += 2) m = fmaxf(m, fmaxf(x[i], x[i + 1]));
    return m;
}

// One part of one row, by the whole CTA: target row or (drafter) draft row `entry`.
template <int DT>
DF_DEV void row_part(const typename Vec<DT>::T* row, int v0, int v1, const VerifyArgs& A, int entry, int drafter,
                     VerifyStat* warps, VerifyStat* out) {
    constexpr int M = Batches<DT>::M, N = Vec<DT>::N, W = kVsThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first loads go out before the sequence and its temperature are looked up
    Batches<DT> batches(row, v0, v1);
    const int s = verify_seq(A, entry, 1 - drafter, lane);
    if (s < 0) return;
    const Scale c = scale_of(A, s);
    if (drafter && c.greedy()) return;  // a greedy sequence's drafter is not asked
    VerifyStat r{0.f, kRefNone, -INFINITY, 0x7fffffff};
    if (c.greedy()) {
        auto join = [&](float m, int arg) {
            if (m > r.max || (m == r.max && arg < r.tag)) r.max = m, r.tag = arg;
        };
        batches.each([&](const float* x, const int* at) {
            const float m = max_of<M>(x);
            if (m >= r.max && m > -INFINITY) {
                int arg = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < M; ++i)
                    if (x[i] == m) arg = min(arg, at[i / N] + i % N);
                join(m, arg);
            }
        });
        auto fold = [&](int from) {
#pragma unroll
            for (int o = from; o > 0; o >>= 1)
                join(__shfl_xor_sync(0xffffffffu, r.max, o), __shfl_xor_sync(0xffffffffu, r.tag, o));
        };
        fold(16);
        if (lane == 0) warps[warp] = r;
        __syncthreads();
        r = warps[lane % W];
        fold(W / 2);
        if (threadIdx.x == 0) *out = r;
        return;
    }
    batches.each([&](const float* x, const int*) {
        const float m = max_of<M>(x);
        r.max = fmaxf(r.max, m);
        const float ref = fmaxf(r.ref, ceilf(m * c.hi));
        float s[4] = {r.sum * pow2(r.ref - ref), 0.f, 0.f, 0.f};
        r.ref = ref;
#pragma unroll
        for (int i = 0; i < M; ++i) s[(i + 1) & 3] += weight(x[i], c, ref);
        r.sum = (s[0] + s[1]) + (s[2] + s[3]);
    });
    auto fold = [&](int from) {
        float to = r.ref;
#pragma unroll
        for (int o = from; o > 0; o >>= 1) {
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
            r.max = fmaxf(r.max, __shfl_xor_sync(0xffffffffu, r.max, o));
        }
        r.sum *= pow2(r.ref - to);
        r.ref = to;
#pragma unroll
        for (int o = from; o > 0; o >>= 1) r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
    };
    fold(16);
    r.tag = 0;
    if (lane == 0) warps[warp] = r;
    __syncthreads();
    r = warps[lane % W];
    fold(W / 2);
    // (a NaN or an infinite entry makes the sum NaN; no weight at all although there are entries: too far apart)
    if (r.sum < INFINITY && (r.sum > 0.f || r.max == -INFINITY)) {
        if (threadIdx.x == 0) *out = r;
        return;
    }
    // again, with the part's largest logit taken off first
    const float m = fmaxf(r.max, -INFINITY);
    r = VerifyStat{0.f, kRefNone, m, 1};
    batches.start();
    if (m > -INFINITY)
        batches.each([&](const float* x, const int*) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < M; ++i) s += weight_careful(x[i], c, m);
            r.sum += s;
        });
    r.sum = warp_sum(r.sum);
    __syncthreads();
    if (lane == 0) warps[warp].sum = r.sum;
    __syncthreads();
    r.sum = 0.f;
    for (int w = 0; w < W; ++w) r.sum += warps[w].sum;
    if (threadIdx.x == 0) *out = r;
}

__global__ void __launch_bounds__(kVsThreads, 4) verify_stats_kernel(const __grid_constant__ VerifyParams P) {
    const VerifyArgs& A = P.A;
    __shared__ VerifyStat warps[kVsThreads / 32];
    const int part = blockIdx.x % P.parts, row = blockIdx.x / P.parts;
    const int nt = A.n_drafts + A.n_seqs;
    pdl_wait();
    pdl_trigger();
    const int v0 = (int)((int64_t)A.vocab * part / P.parts), v1 = (int)((int64_t)A.vocab * (part + 1) / P.parts);
    VerifyStat* out = P.stats + (int64_t)row * P.parts + part;
    if (row >= nt)
        row_part<kF32>(A.draft + (int64_t)(row - nt) * A.draft_stride, v0, v1, A, row - nt, 1, warps, out);
    else if (A.target_dtype == kF32)
        row_part<kF32>(static_cast<const float*>(A.target) + (int64_t)row * A.target_stride, v0, v1, A, row, 0, warps, out);
    else if (A.target_dtype == kBF16)
        row_part<kBF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, A, row, 0, warps,
                        out);
    else
        row_part<kF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, A, row, 0, warps,
                       out);
}

// A row's parts joined (warp-wide, every lane gets the answer).  A row with a
// careful part is careful as a whole.
DF_DEV VerifyStat row_stat(const VerifyParams& P, int64_t row, Scale c, int lane) {
    const VerifyStat* st = P.stats + row * P.parts;
    VerifyStat r{0.f, kRefNone, -INFINITY, 0};
    if (c.greedy()) {
        r.tag = 0x7fffffff;
        auto join = [&](float m, int arg) {
            if (m > r.max || (m == r.max && arg < r.tag)) r.max = m, r.tag = arg;
        };
        for (int i = lane; i < P.parts; i += 32) join(st[i].max, st[i].tag);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(__shfl_xor_sync(0xffffffffu, r.max, o), __shfl_xor_sync(0xffffffffu, r.tag, o));
        return r;
    }
    for (int i = lane; i < P.parts; i += 32) {
        const VerifyStat x = st[i];
        const float to = fmaxf(r.ref, x.ref);
        r.sum = r.sum * pow2(r.ref - to) + x.sum * pow2(x.ref - to);
        r.ref = to;
        r.max = fmaxf(r.max, x.max);
        r.tag |= x.tag;
    }
    r.tag = __any_sync(0xffffffffu, r.tag);
    r.max = warp_max(r.max);
    if (!r.tag) {
        const float to = warp_max(r.ref);
        r.sum *= pow2(r.ref - to);
        r.ref = to;
    } else {
        // in 64 bits: every part's sum to the row's largest logit
        double sum = 0.0;
        for (int i = lane; i < P.parts; i += 32) {
            const VerifyStat x = st[i];
            if (x.sum == 0.f) continue;
            double f = 1.0;
            if (!x.tag)
                f = exp2((double)x.ref - (double)r.max * c.wide());
            else if (x.max != r.max)
                f = exp2(((double)x.max - (double)r.max) * c.wide());
            sum += (double)x.sum * f;
        }
        r.sum = (float)sum;
    }
    r.sum = warp_sum(r.sum);
    return r;
}
DF_DEV float logit_at(const void* base, int dtype, int64_t i) {
    return dtype == kF32    ? Vec<kF32>::one(static_cast<const float*>(base) + i)
           : dtype == kBF16 ? Vec<kBF16>::one(static_cast<const uint16_t*>(base) + i)
                            : Vec<kF16>::one(static_cast<const uint16_t*>(base) + i);
}
// The weight of one entry of a row (its probability times the row's sum) to about 2^-22 however small it is,
// for the numbers that accept a draft: the exponent as a pair, its whole part apart.
DF_DEV float weight_exact(float x, const VerifyStat& r, Scale c) {
    if (r.max == -INFINITY || !(x > -INFINITY)) return 0.f;
    if (x == r.max && r.tag) return 1.f;
    float y = x, yl = 0.f, ref = r.ref;
    if (r.tag) {
        y = x - r.max;
        if (!(y > -INFINITY)) return 0.f;
        const float t = y - x;
        yl = (x - (y - t)) + (-r.max - t);
        ref = 0.f;
    }
    const float p = y * c.hi, s = p - ref, t = s - p;
    if (!(s > -1e9f)) return 0.f;
    const float n = rintf(s), f = (s - n) + (fmaf(y, c.hi, -p) + ((p - (s - t)) + (-ref - t)) + fmaf(y, c.lo, yl * c.hi));
    return ldexpf(exp2f(f), (int)n);
}

// The weight of an entry of a row.  A row without any probability has an infinite reference.
DF_DEV float weight_any(float x, const VerifyStat& r, Scale c) {
    return r.tag ? weight_careful(x, c, r.max) : weight(x, c, r.ref);
}

// What is left at the entries of the sampled row: mode 0 the target's
// probability (unnormalised), 1 with the draft taken out, 2 max(p - q, 0).
struct Left {
    const unsigned char* target;
    const float* draft;
    int dtype, mode, x;
    VerifyStat t, q;
    float tz, qz;  // 1 / the rows' sums
    Scale c;
    // entries i, i + 32, .. (N of them, 0 from `end` on): all loads first
    template <int N>
    DF_DEV void get(int i, int end, float (&w)[N]) const {
        float y[N];
        if (dtype == kF32) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                w[k] = i + 32 * k < end ? __ldg(reinterpret_cast<const float*>(target) + i + 32 * k) : -INFINITY;
        } else {
            uint32_t u[N];
#pragma unroll
            for (int k = 0; k < N; ++k)
                u[k] = i + 32 * k < end ? __ldg(reinterpret_cast<const uint16_t*>(target) + i + 32 * k)
                       : dtype == kBF16 ? 0xff80u
                                        : 0xfc00u;
#pragma unroll
            for (int k = 0; k < N; ++k)
                w[k] = dtype == kBF16 ? __uint_as_float(u[k] << 16) : __half2float(__ushort_as_half((uint16_t)u[k]));
        }
        if (mode == 2) {
#pragma unroll
            for (int k = 0; k < N; ++k) y[k] = i + 32 * k < end ? __ldg(draft + i + 32 * k) : -INFINITY;
        }
        // (plain rows, nearly all there are, first: a weight is three instructions)
        if (!t.tag && !q.tag) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                w[k] = weight(w[k], c, t.ref);
                if (mode == 2) w[k] = fmaxf(fmaf(w[k], tz, -weight(y[k], c, q.ref) * qz), 0.f);
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                w[k] = weight_any(w[k], t, c);
                if (mode == 2) w[k] = fmaxf(fmaf(w[k], tz, -weight_any(y[k], q, c) * qz), 0.f);
            }
        }
        // (absent entries are logits of -inf: no weight)
        if (mode == 1) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (i + 32 * k == x) w[k] = 0.f;
        }
    }
};

// A CTA's shared memory may be written from its cluster only once it runs: every CTA says so as it starts, and none
// writes before all have (the wait falls into the statistics' time).
DF_DEV void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
DF_DEV void cluster_wait_started() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

template <int WARPS>
__global__ void __cluster_dims__(kVpCluster, 1, 1) __launch_bounds__(WARPS * 32)
    verify_pick_kernel(const __grid_constant__ VerifyParams P) {
    constexpr int kParts = kVpCluster * WARPS;  // vocabulary parts of the sampled row
    constexpr int kKept = kVpKept / WARPS;      // entries of a warp's part that are kept
    const VerifyArgs& A = P.A;
    // a round of 32 rows of the sequence: the target's statistics and the drafter's, the draft's logits
    __shared__ VerifyStat stat[2][32];
    __shared__ float logit[2][32];
    __shared__ int refused;
    __shared__ float2 part_sum[WARPS];           // the warps' sums
    __shared__ float2 cta_sum[2][kVpCluster];    // the CTAs' (two passes at most: each has its own)
    extern __shared__ float kept[];         // [WARPS][kKept]
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), s = blockIdx.x / kVpCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cluster_started();
    pdl_wait();
    int a, b;
    draft_range(A, s, lane, a, b);
    const int d = b - a;
    const Scale c = scale_of(A, s);
    const bool drawn = A.draft != nullptr && !c.greedy();  // q is the drafter's distribution, not one token
    const int64_t nt = (int64_t)A.n_drafts + A.n_seqs, row0 = (int64_t)a + s;
    const float u_token = A.sample_u[s];

    // every CTA of the cluster decides alike; the first one writes
    if (threadIdx.x == 0) refused = 0x7fffffff;
    int i0 = 0;
    for (;; i0 += 32) {
        const int n = min(32, d + 1 - i0);  // rows of the round, the one after the last draft among them
        for (int j = warp; j < (drawn ? 2 : 1) * n; j += WARPS) {
            const int i = i0 + j % n, side = j / n;
            float l = -INFINITY;
            if (i < d) {
                const uint32_t x = A.draft_tok[a + i];
                if (x < (uint32_t)A.vocab)
                    l = side ? __ldg(A.draft + (int64_t)(a + i) * A.draft_stride + x)
                             : logit_at(A.target, A.target_dtype, (row0 + i) * A.target_stride + x);
            }
            if (side && i == d) continue;
            const VerifyStat t = row_stat(P, side ? nt + a + i : row0 + i, c, lane);
            if (lane == 0) {
                stat[side][i - i0] = t;
                logit[side][i - i0] = l;
            }
        }
        __syncthreads();
        if (warp == 0 && i0 + lane < d) {
            const int i = i0 + lane;
            // p = wp / sp and q = wq / sq: compared as u wq sp < wp sq
            const VerifyStat t = stat[0][lane];
            float wp, sp = 1.f, wq = 1.f, sq = 1.f;
            if (c.greedy()) {
                wp = t.max > -INFINITY && t.tag == (int)A.draft_tok[a + i] ? 1.f : 0.f;
            } else {
                wp = weight_exact(logit[0][lane], t, c);
                if (t.max > -INFINITY) sp = t.sum;
            }
            if (drawn) {
                const VerifyStat g = stat[1][lane];
                wq = weight_exact(logit[1][lane], g, c);
                if (g.max > -INFINITY) sq = g.sum;
            }
            const double p = (double)wp * (double)sq, q = (double)wq * (double)sp;
            if (!((double)A.accept_u[a + i] * q < p)) atomicMin(&refused, i);
            // (q = 0: a draft the drafter could not make; kept when p is not 0)
            if (rank == 0 && A.prob != nullptr) A.prob[a + i] = p < q ? (wp / sp) / (wq / sq) : wp > 0.f ? 1.f : 0.f;
        }
        __syncthreads();
        if (i0 + 32 > d) break;
    }
    const int acc = min(refused, d);
    const int64_t row = row0 + acc;
    const VerifyStat t = acc >= i0 ? stat[0][acc - i0] : row_stat(P, row, c, lane);
    int token = t.max == -INFINITY ? -1 : t.tag;
    bool writes = rank == 0 && threadIdx.x == 0;
    const bool sampled = !c.greedy() && t.max > -INFINITY;
    cluster_wait_started();
    if (sampled) {
        writes = false;
        Left L;
        L.target = static_cast<const unsigned char*>(A.target) + row * A.target_stride * (A.target_dtype == kF32 ? 4 : 2);
        L.draft = nullptr;
        L.dtype = A.target_dtype;
        L.c = c;
        L.t = t;
        L.q = t;
        L.tz = 1.f / t.sum;
        L.qz = 0.f;
        L.x = -1;
        L.mode = 0;
        if (acc < d) {
            L.x = (int)min(A.draft_tok[a + acc], 0x7fffffffu);
            L.mode = 1;
            if (drawn) {
                const VerifyStat g = acc >= i0 ? stat[1][acc - i0] : row_stat(P, nt + a + acc, c, lane);
                L.q = g;
                if (g.max == -INFINITY) L.q.ref = INFINITY;
                L.draft = A.draft + (int64_t)(a + acc) * A.draft_stride;
                L.mode = 2;
                L.qz = g.max == -INFINITY ? 0.f : 1.f / g.sum;
            }
        }
        // this warp's part of the vocabulary
        const int w = rank * WARPS + warp;
        const int v0 = (int)((int64_t)A.vocab * w / kParts), v1 = (int)((int64_t)A.vocab * (w + 1) / kParts);
        float* mine_kept = kept + warp * kKept;
        for (int pass = 0; pass < 2; ++pass) {
            Pair mine;
            constexpr int N = 8;
#pragma unroll 1
            for (int i = v0 + lane; i < v1; i += 32 * N) {
                float x[N];
                L.get<N>(i, v1, x);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (i - v0 + 32 * k < kKept) mine_kept[i - v0 + 32 * k] = x[k];
                mine = mine + Pair{((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])), 0.f};
            }
            mine = warp_sum(mine);
            if (lane == 0) part_sum[warp] = make_float2(mine.hi, mine.lo);
            __syncthreads();
            // the running sums of the CTA's parts (warp 0; the others keep pace), its whole sum to every CTA
            Pair own, up;
            if (warp == 0) {
                if (lane < WARPS) own = Pair{part_sum[lane].x, part_sum[lane].y};
                up = warp_running(own, lane);
                const Pair sum = shfl(up, 31);
                if (lane < kVpCluster) *cl.map_shared_rank(&cta_sum[pass][rank], lane) = make_float2(sum.hi, sum.lo);
            }
            cl.sync();
            Pair cta;
            if (lane < kVpCluster) cta = Pair{cta_sum[pass][lane].x, cta_sum[pass][lane].y};
            const Pair to = warp_running(cta, lane), whole = shfl(to, 31);
            if (!positive(whole) && L.mode != 0) {
                L.mode = 0;  // the draft had all of it: the target's own distribution
                continue;
            }
            if (warp != 0) break;
            Pair rest;  // u * whole
            rest.hi = u_token * whole.hi;
            rest.lo = fmaf(u_token, whole.hi, -rest.hi) + u_token * whole.lo;
            // the first CTA whose running sum passes `rest`, then its first warp, a 32nd of that warp's part and
            // so on to the entry; where none passes (rounding, or a number of 1), the last that has any weight
            bool inside = true;
            auto narrow = [&](Pair piece, Pair upto) -> int {
                const uint32_t any = __ballot_sync(0xffffffffu, positive(piece));
                const uint32_t over = __ballot_sync(0xffffffffu, inside && positive(piece) && positive(upto - rest));
                const int l = over ? __ffs(over) - 1 : 31 - __clz(any);
                inside = over != 0;
                if (inside) rest = rest - shfl(upto - piece, l);
                return l;
            };
            if (narrow(cta, to) != rank) break;
            const int part = rank * WARPS + narrow(own, up);
            const float* its_kept = kept + (part % WARPS) * kKept;
            const int f0 = (int)((int64_t)A.vocab * part / kParts);
            int p0 = f0, p1 = (int)((int64_t)A.vocab * (part + 1) / kParts);
#pragma unroll 1
            while (p1 - p0 > 1) {
                const int per = (p1 - p0 + 31) / 32, q0 = min(p0 + lane * per, p1), q1 = min(q0 + per, p1);
                float sum = 0.f;
#pragma unroll 2
                for (int i = q0; i < q1; ++i) {
                    float x[1];
                    if (i - f0 < kKept)
                        x[0] = its_kept[i - f0];
                    else
                        L.get<1>(i, q1, x);
                    sum += x[0];
                }
                const Pair piece{sum, 0.f};
                const int l = narrow(piece, warp_running(piece, lane));
                p0 = __shfl_sync(0xffffffffu, q0, l);
                p1 = __shfl_sync(0xffffffffu, q1, l);
            }
            token = p0;
            writes = lane == 0;
            break;
        }
    }
    if (writes) {
        A.accepted[s] = acc;
        A.next_tok[s] = token;
    }
    // (a CTA's sums are written before the last meeting and read by itself alone: none has to wait to leave)
}

// Parts of a row: of up to 32K entries and at least 4K.  Where 32K entries a part leave all CTAs resident at once (four
// an SM), as many as give two CTAs an SM (3 blocks of 16 rows against f32 logits: 24.9 us, with 16 CTAs an SM 29.2; one
// block 16.1, 18.2); beyond, 16 CTAs an SM, whose last wave is the shorter (4 blocks: 29.5, with 32K entries a part
// 31.2).
static int verify_parts(int64_t rows, int64_t vocab, int num_sms) {
    const int64_t most = (vocab + 4095) / 4096, least = (vocab + 32767) / 32768, n = rows > 0 ? rows : 1;
    const int64_t want = ((least * n <= 4 * (int64_t)num_sms ? 2 : 16) * (int64_t)num_sms + n - 1) / n;
    const int64_t p = want < least ? least : want;
    return (int)(p > most ? most : p);
}
static int64_t verify_rows(int n_seqs, int64_t n_drafts, bool drawn) { return n_seqs + (drawn ? 2 : 1) * n_drafts; }

int64_t verify_workspace(int n_seqs, int64_t n_drafts, int64_t vocab, int num_sms) {
    int64_t most = 0;
    for (bool drawn : {false, true}) {
        const int64_t rows = verify_rows(n_seqs, n_drafts, drawn);
        const int64_t n = rows * verify_parts(rows, vocab, num_sms);
        if (n > most) most = n;
    }
    return most * (int64_t)sizeof(VerifyStat);
}

template <int WARPS>
static int launch_pick(const VerifyParams& P, cudaStream_t st) {
    constexpr size_t smem = kVpKept * sizeof(float);
    static size_t limit[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(verify_pick_kernel<WARPS>, smem, &limit[dev])) return (int)e;
    return (int)launch(verify_pick_kernel<WARPS>, dim3((unsigned)P.A.n_seqs * kVpCluster), dim3(WARPS * 32), smem, st, P);
}

int verify(const VerifyArgs& A, void* ws, int num_sms, cudaStream_t st) {
    VerifyParams P;
    P.A = A;
    P.stats = static_cast<VerifyStat*>(ws);
    const int64_t rows = verify_rows(A.n_seqs, A.n_drafts, A.draft != nullptr);
    P.parts = verify_parts(rows, A.vocab, num_sms);
    if (cudaError_t e = launch(verify_stats_kernel, dim3((unsigned)(rows * P.parts)), dim3(kVsThreads), 0, st, P))
        return (int)e;
    // 32 warps a CTA while every CTA has an SM to itself (one block: 18.2 us, with 16 warps 19.9), else 16, two CTAs an
    // SM (32 blocks: 87.5 us, with 32 warps 94.3)
    return A.n_seqs * kVpCluster <= num_sms ? launch_pick<32>(P, st) : launch_pick<16>(P, st);
}

}  // namespace dflash
