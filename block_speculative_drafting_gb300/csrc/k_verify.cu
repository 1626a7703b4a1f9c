// Verification of drafted tokens against the target's probabilities.
//
// Two kernels.  verify_stats_kernel reads every logit row once: a CTA takes
// one part of one row's vocabulary and leaves what softmax needs of it, the sum
// of 2^(x c - R) with c = log2(e) / T and an integer reference R (or, of a
// greedy sequence, the largest logit and the lowest index that has it).
// verify_pick_kernel then takes a sequence per cluster: the parts of its rows
// are joined, each draft's p and q compared with the given number, and one row
// -- the first refused, or the last -- is read again to sample the next token:
// the cluster's warps sum what is left of equal parts of the vocabulary, and the
// CTA in which the running sum passes the given number's share of the whole finds
// the part and the entry.  That kernel runs once through its code, so its code is
// kept small (rolled loops, one copy of each part): what it waits for most is
// instructions, and code that does not run costs it time as well (without the exact
// form's, one block 17.6 -> 16.9 us).
//
// Arithmetic.  A softmax sum of the statistics is a tree of f32 additions of
// exponentials within 2^-22 each; c is a pair (hi, lo), so that its rounding does
// not tilt the distribution, and R is an integer, so that moving a sum to another
// reference is exact and x c - R is rounded once: off by 2^-18 at most (prob was
// seen within 2^-21 of its value).  A draft whose number lies within that of p / q, and a
// token whose share of the whole lies within the 32-bit form's bound of a border
// (below), are decided again in 64 bits: every decision is the definition's.
//
// Memory bound: the logits, once (the re-read row comes out of L2).  32 blocks of
// up to 16 drafts, 151936 bf16 logits against f32 ones: 80 us, of which the
// statistics 55 (5.5 TB/s, 81 % of a copy) and the picking kernel the rest; one
// block 17.6 us, 13.7 of chosen drafts, greedy 6.7, most of it latency.
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "paged.cuh"

namespace dflash {

namespace cg = cooperative_groups;

constexpr int kVsThreads = 256;
constexpr int kVpCluster = 8;
constexpr int kVpPiece = 128;       // a warp's step through the sampled row
constexpr float kRefNone = -3e38f;  // the reference of a sum of nothing

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
#pragma unroll 1
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
__device__ __noinline__ VerifyStat row_stat(const VerifyParams& P, int64_t row, Scale c, int lane) {
    const VerifyStat* st = P.stats + row * P.parts;
    VerifyStat r{0.f, kRefNone, -INFINITY, 0};
    if (c.greedy()) {
        r.tag = 0x7fffffff;
        auto join = [&](float m, int arg) {
            if (m > r.max || (m == r.max && arg < r.tag)) r.max = m, r.tag = arg;
        };
#pragma unroll 1
        for (int i = lane; i < P.parts; i += 32) join(st[i].max, st[i].tag);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(__shfl_xor_sync(0xffffffffu, r.max, o), __shfl_xor_sync(0xffffffffu, r.tag, o));
        return r;
    }
#pragma unroll 1
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
#pragma unroll 1
        for (int i = lane; i < P.parts; i += 32) {
            const VerifyStat x = st[i];
            if (x.sum == 0.f) continue;
            // (an infinite largest logit has nothing but itself)
            const double by = x.tag ? x.max == r.max ? 0.0 : ((double)x.max - (double)r.max) * c.wide()
                                    : (double)x.ref - (double)r.max * c.wide();
            sum += (double)x.sum * exp2(by);
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


// The weight of an entry of a row that has any, off by its exponent's two roundings.
DF_DEV float weight_any(float x, const VerifyStat& r, Scale c) {
    return r.tag ? weight_careful(x, c, r.max) : weight(x, c, r.ref);
}

// ---------------------------------------------------------------- the sampled row
// The entry drawn is the first whose running sum passes the given number's share of the whole, so an error anywhere
// ahead of it moves its border.  Shares are whole numbers in units of 2^-60 of a row: their sums are exact, in any order.
//
// 2^z by a table of 2^(i / 128) and a polynomial (P. T. P. Tang, "Table-driven implementation of the exponential function
// in IEEE floating-point arithmetic", ACM TOMS 15, 1989), first in 32 bits: z = x c to the nearest 128th, the remainder
// r, |r| <= 2^-8 + 2^-10, by two roundings; the table, normalised by the row's sum as the statistics have it, rounded to
// 2^-32; 257 (2^r - 1) + 3 in f32, whose 32 bits from 2.0 to 4.0 are 0x40400000 2^r (257 = 0x40400000 / 2^22), rounded to
// 2^-31; their product in 64 bits.  Together under kVpEps.  The pass also sums the rows themselves, whose statistics are
// off by about 2^-20: with g = sum of (p' - q'), p' and q' as computed, p - q is p' - q' - g q' (of p' + ..), where a
// change of sign matters only in entries whose p' and q' agree to within g; those are summed (`tie`).
//
// The entry's distance from both of its borders is compared with the bound that all this gives.  Where it is within the
// bound, or the exponents are past that form's range, the row is gone through again with exponents in 64 bits, table and
// polynomial in 64-bit fixed point, and p and q by exactly normalised sums: the definition in 64 bits, with sums that do
// not round.  Of 2048 refused rows over 151936 entries: none where a third of the mass is refused, 13 at 5 %, 238 at
// 0.05 %; 108 us more for one sequence.  (Weights of 22 bits, in sums of 48, drew another token in up to 7 % of such rows;
// one pass in 64-bit floats would take 0.6 ms: two lanes of them a clock and SM.)
constexpr int kVpSteps = 128;
// 2.7 2^-31: the last rounding 1, the table 1/2, r's two 2 (1/2 ln 2 past 2^-8), the polynomial's two 2 / 2^2.5 of it
// (c's own error is every entry's, and goes with the normaliser)
constexpr float kVpEps = 1.26e-9f;
constexpr long long kVpOne = 1ll << 60;
constexpr float kVpMagic = 98304.f;  // 1.5 * 2^16: a sum with it is rounded to 128ths
constexpr uint32_t kVpZero = 0x47C00000;  // its bits
__device__ const unsigned long long kTwoTo[kVpSteps] = {  // 2^(i / 128 + 63)
    0x8000000000000000ull, 0x80b1ed4fd999ab6cull, 0x8164d1f3bc030773ull, 0x8218af4373fc25ecull, 0x82cd8698ac2ba1d7ull,
    0x8383594eefb6ee37ull, 0x843a28c3acde4046ull, 0x84f1f656379c1a29ull, 0x85aac367cc487b15ull, 0x8664915b923fba04ull,
    0x871f61969e8d1010ull, 0x87db357ff698d792ull, 0x88980e8092da8527ull, 0x8955ee03618e5fddull, 0x8a14d575496efd9aull,
    0x8ad4c6452c728924ull, 0x8b95c1e3ea8bd6e7ull, 0x8c57c9c4646f4ddeull, 0x8d1adf5b7e5ba9e6ull, 0x8ddf042022e69cd6ull,
    0x8ea4398b45cd53c0ull, 0x8f6a8117e6c8e5c4ull, 0x9031dc431466b1dcull, 0x90fa4c8beee4b12bull, 0x91c3d373ab11c336ull,
    0x928e727d9531f9acull, 0x935a2b2f13e6e92cull, 0x9426ff0fab1c04b6ull, 0x94f4efa8fef70961ull, 0x95c3fe86d6cc7fefull,
    0x96942d3720185a00ull, 0x97657d49f17ab08eull, 0x9837f0518db8a96full, 0x990b87e266c189aaull, 0x99e0459320b7fa65ull,
    0x9ab62afc94ff864aull, 0x9b8d39b9d54e5539ull, 0x9c6573682ec32c2dull, 0x9d3ed9a72cffb751ull, 0x9e196e189d472420ull,
    0x9ef5326091a111aeull, 0x9fd228256400dd06ull, 0xa0b0510fb9714fc2ull, 0xa18faeca8544b6e4ull, 0xa27043030c496819ull,
    0xa3520f68e802bb93ull, 0xa43515ae09e6809eull, 0xa5195786be9ef339ull, 0xa5fed6a9b15138eaull, 0xa6e594cfeee86b1eull,
    0xa7cd93b4e965356aull, 0xa8b6d5167b320e09ull, 0xa9a15ab4ea7c0ef8ull, 0xaa8d2652ec907629ull, 0xab7a39b5a93ed337ull,
    0xac6896a4be3fe929ull, 0xad583eea42a14ac6ull, 0xae493452ca35b80eull, 0xaf3b78ad690a4375ull, 0xb02f0dcbb6e04584ull,
    0xb123f581d2ac2590ull, 0xb21a31a66618fe3bull, 0xb311c412a9112489ull, 0xb40aaea2654b9841ull, 0xb504f333f9de6484ull,
    0xb60093a85ed5f76cull, 0xb6fd91e328d17791ull, 0xb7fbefca8ca41e7cull, 0xb8fbaf4762fb9ee9ull, 0xb9fcd2452c0b9debull,
    0xbaff5ab2133e45fbull, 0xbc034a7ef2e9fb0dull, 0xbd08a39f580c36bfull, 0xbe0f6809860993e2ull, 0xbf1799b67a731083ull,
    0xc0213aa1f0d08db0ull, 0xc12c4cca66709456ull, 0xc238d2311e3d6673ull, 0xc346ccda24976407ull, 0xc4563ecc5334cb33ull,
    0xc5672a115506daddull, 0xc67990b5aa245f79ull, 0xc78d74c8abb9b15dull, 0xc8a2d85c8ffe2c45ull, 0xc9b9bd866e2f27a3ull,
    0xcad2265e4290774eull, 0xcbec14fef2727c5dull, 0xcd078b86503dcdd2ull, 0xce248c151f8480e4ull, 0xcf4318cf191918c1ull,
    0xd06333daef2b2595ull, 0xd184df6251699ac6ull, 0xd2a81d91f12ae45aull, 0xd3ccf099859ac379ull, 0xd4f35aabcfedfa1full,
    0xd61b5dfe9f9bce07ull, 0xd744fccad69d6af4ull, 0xd870394c6db32c84ull, 0xd99d15c278afd7b6ull, 0xdacb946f2ac9cc72ull,
    0xdbfbb797daf23755ull, 0xdd2d818508324c20ull, 0xde60f4825e0e9124ull, 0xdf9612deb8f04420ull, 0xe0ccdeec2a94e111ull,
    0xe2055afffe83d369ull, 0xe33f8972be8a5a51ull, 0xe47b6ca0373da88dull, 0xe5b906e77c8348a8ull, 0xe6f85aaaee1fce22ull,
    0xe8396a503c4bdc68ull, 0xe97c38406c4f8c57ull, 0xeac0c6e7dd24392full, 0xec0718b64c1cbddcull, 0xed4f301ed9942b84ull,
    0xee990f980da3025bull, 0xefe4b99bdcdaf5cbull, 0xf13230a7ad094509ull, 0xf281773c59ffb13aull, 0xf3d28fde3a641a5bull,
    0xf5257d152486cc2cull, 0xf67a416c733f846eull, 0xf7d0df730ad13bb9ull, 0xf92959bb5dd4ba74ull, 0xfa83b2db722a033aull,
    0xfbdfed6ce5f09c49ull, 0xfd3e0c0cf486c175ull, 0xfe9e115c7b8f884cull,
};

// What is summed: lanes', warps', CTAs' shares of a pass.
struct __align__(8) Sums {
    long long d;   // what is left (positive p' - q', or p'); first pass of the exact form: p'
    long long g;   // p' - q' over all entries; first pass of the exact form: q'
    uint32_t q;    // q' where p' - q' is positive, in units of 2^-28
    uint32_t tie;  // q' where p' and q' nearly agree, likewise
};
// (the 32-lane sums of 22-bit pieces fit 32 bits)
DF_DEV long long warp_sum(long long x) {
    const uint32_t m = (1u << 22) - 1;
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)x & m),
                   b = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 22) & m),
                   c = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 44));
    return (long long)(a + ((unsigned long long)b << 22) + ((unsigned long long)c << 44));
}
DF_DEV Sums warp_sum(Sums a) {
    a.d = warp_sum(a.d);
    a.g = warp_sum(a.g);
    a.q = __reduce_add_sync(0xffffffffu, a.q);
    a.tie = __reduce_add_sync(0xffffffffu, a.tie);
    return a;
}
// sums of the lanes up to and with this one
template <int N = 32>
DF_DEV long long warp_running(long long x, int lane) {
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// log2(e) / T to the nearest f32, with what that leaves.
DF_DEV Scale nearest(Scale c) {
    Scale n;
    n.hi = c.hi + c.lo;
    n.lo = c.lo - (n.hi - c.hi);
    return n;
}
// A row's exponents and normaliser in the 32-bit form.
// (approximate as it is: any common factor of a row's shares near its sum will do)
struct Norm {
    float magic;  // kVpMagic and the row's log2 sum to the nearest 128th
    float log;          // of the log2 sum: what its whole part (below) leaves
    float whole;
    uint32_t mul;  // 2^(what the 128th left) / 1.00390625, by 2^32
    bool fits;     // |x c| under 2^14 where it counts
};
DF_DEV Norm norm_of(const VerifyStat& r, Scale c) {
    Norm n;
    n.whole = r.ref;
    n.log = __log2f(r.sum);
    if (r.tag) {  // (its sum is relative to the largest)
        n.whole = rintf(r.max * c.hi);
        n.log += fmaf(r.max, c.hi, -n.whole) + r.max * c.lo;
    }
    const float j = rintf(n.log * 128.f) * 0.0078125f, l = n.whole + j;
    n.magic = kVpMagic + l;
    n.mul = __float2uint_rn(ex2(j - n.log) * (4294967296.f / 1.00390625f));
    n.fits = fabsf(l) + 64.f < 16384.f && fabsf(r.max * c.hi) < 16384.f;
    return n;
}
// two f32 at once
struct Two {
    unsigned long long v;
    DF_DEV Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    DF_DEV void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
DF_DEV Two fma2(Two a, Two b, Two c) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c.v) : "l"(a.v), "l"(b.v));
    return c;
}
// 2^60 times the probabilities of logits xa and xb, about, by their rows' magic and tables (far below, -inf and NaN: the
// shift is past 63, which leaves 0).  Of t's bits the lowest seven are -z's 128ths, the ones above them its whole part.
DF_DEV void shares(float xa, float xb, Scale c, float ma, float mb, const uint32_t* ta, const uint32_t* tb,
                   unsigned long long& a, unsigned long long& b) {
    const Two x(xa, xb), hi(c.hi, c.hi), t = fma2(x, Two(-c.hi, -c.hi), Two(ma, mb));
    const Two r = fma2(x, Two(c.lo, c.lo), fma2(x, hi, fma2(t, Two(1.f, 1.f), Two(-ma, -mb))));
    // 257 (ln 2)^k / k!
    const Two y = fma2(r, fma2(fma2(r, Two(14.2646017f, 14.2646017f), Two(61.7385330f, 61.7385330f)), r,
                               Two(178.138824f, 178.138824f)),
                       Two(3.f, 3.f));
    float t0, t1, y0, y1;
    t.get(t0, t1);
    y.get(y0, y1);
    const auto part = [](float t, float y, const uint32_t* table) {
        const uint32_t i = __float_as_uint(t);
        unsigned long long p = (unsigned long long)table[i & (kVpSteps - 1)] * __float_as_uint(y);
        asm("shr.u64 %0, %0, %1;" : "+l"(p) : "r"((i >> 7) - ((kVpZero >> 7) - 2)));
        return p;
    };
    a = part(t0, y0, ta);
    b = part(t1, y1, tb);
}

// The sampled row, for the 32-bit form.  mode 0: the target's probability, 1: with the draft taken out, 2: max(p - q, 0)
struct Sampled {
    const unsigned char* target;
    const float* draft;
    int dtype, mode, x;  // x: the draft that is taken out (mode 1), or -1
    Scale c;
    float tm, qm;       // the two rows' magic
    float apart, tol;   // the rows' log2 sums: the drafter's less the target's; what counts as agreeing
    // N entries, 32 apart
    template <int N>
    DF_DEV void add(int from, Sums& a, const uint32_t (*table)[kVpSteps]) const {
        float w[N], y[N];
        if (dtype == kF32) {
            const float* p = reinterpret_cast<const float*>(target) + from;
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = __ldg(p + 32 * k);
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(target) + from;
            uint32_t u[N];
#pragma unroll
            for (int k = 0; k < N; ++k) u[k] = __ldg(p + 32 * k);
#pragma unroll
            for (int k = 0; k < N; ++k)
                w[k] = dtype == kBF16 ? __uint_as_float(u[k] << 16) : __half2float(__ushort_as_half((uint16_t)u[k]));
        }
        if (mode == 2) {
#pragma unroll
            for (int k = 0; k < N; ++k) y[k] = __ldg(draft + from + 32 * k);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                unsigned long long p, q;
                shares(w[k], y[k], c, tm, qm, table[0], table[1], p, q);
                const long long d = (long long)(p - q);
                const uint32_t high = (uint32_t)(q >> 32);
                a.g += d;
                if ((int)(d >> 32) >= 0) {
                    a.d += d;
                    a.q += high;
                }
                if (fabsf(fmaf(w[k] - y[k], c.hi, apart)) < tol) a.tie += high;
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 2) {
                unsigned long long p, p1;
                shares(w[k], k + 1 < N ? w[k + 1 < N ? k + 1 : 0] : -INFINITY, c, tm, tm, table[0], table[0], p, p1);
                if (from + 32 * k != x) a.d += (long long)p;
                if (from + 32 * k + 32 != x) a.d += (long long)p1;
            }
        }
    }
    // entries [i0, end)
    DF_DEV Sums sums(int i0, int end, int lane, const uint32_t (*table)[kVpSteps]) const {
        Sums a{};
        int i = i0 + lane;
#pragma unroll 1
        for (; i + kVpPiece - lane <= end; i += kVpPiece) add<kVpPiece / 32>(i, a, table);
#pragma unroll 1
        for (; i < end; i += 32) add<1>(i, a, table);
        return a;
    }
    // what is left of one entry
    DF_DEV long long left(int i, long long g, const uint32_t (*table)[kVpSteps]) const {
        unsigned long long p, q;
        shares(logit_at(target, dtype, i), mode == 2 ? __ldg(draft + i) : -INFINITY, c, tm, qm, table[0], table[1], p, q);
        if (mode == 2) return p > q ? max((long long)(p - q) - (((g >> 14) * (long long)(q >> 32)) >> 14), 0ll) : 0ll;
        return i == x ? 0ll : (long long)p;
    }
};

// A target row and a draft row for the exact form, in shared memory.
struct Exact {
    const void* target;
    const float* draft;  // nullptr: the target's row alone
    int dtype, mode, x;
    bool first;  // the number is 0: every entry with any probability at all counts
    float max[2];
    double c;           // log2(e) / T
    float c1, c2, c3;   // the same in three parts
    long long log[2];   // the rows' log2 sums relative to their largest logits, by 2^56
    long long over[2];  // the rows' sums less one, in units of 2^-60
};
// 2^60 times the probability of logit x of a row (side 0 the target's, 1 the drafter's), about: the exponent as a whole
// number of 2^-56 (x less the largest as an error-free pair, times c's parts; few 64-bit floats: two lanes of them a clock
// and SM), then the table and the polynomial
DF_DEV long long exact_share(const Exact& E, int side, float x) {
    const float m = E.max[side], s = x - m;
    long long z = -E.log[side];
    if (x != m) {
        if (!(s * E.c1 > -64.f)) return 0;
        const float v = s - x, e = (x - (s - v)) - (m + v);
        const float p1 = s * E.c1, p2 = s * E.c2, p3 = e * E.c1;
        const float low = fmaf(s, E.c2, -p2) + fmaf(e, E.c1, -p3) + fmaf(s, E.c3, e * E.c2);
        const auto whole = [](float y) { return __float2ll_rn(y * 72057594037927936.f); };  // 2^56
        z += whole(p1) + whole(fmaf(s, E.c1, -p1)) + whole(p2) + whole(p3) + whole(low);
    }
    if (z < -(62ll << 56)) return 0;
    const unsigned long long r = (unsigned long long)(z & ((1ll << 49) - 1)) << 8;
    // 2^r - 1 by (ln 2)^k / k!, k = 1 .. 6, the last four in 32 bits
    const uint32_t rh = (uint32_t)(r >> 32);
    uint32_t h = __umulhi(rh, 0x000a1848u) + 0x005761ffu;
    h = __umulhi(rh, h) + 0x0276556du;
    h = __umulhi(rh, h) + 0x0e35846bu;
    unsigned long long p = __umul64hi(r, (unsigned long long)h << 32) + 0x3d7f7bff058b1d51ull;
    p = __umul64hi(r, p) + 0xb17217f7d1cf79acull;
    p = __umul64hi(r, p);
    const unsigned long long two = kTwoTo[(z >> 49) & (kVpSteps - 1)] >> 1, y = two + __umul64hi(two, p);
    const int down = 2 - (int)(z >> 56);
    return (long long)((y + (1ull << (down - 1))) >> down);
}
DF_DEV float exact_logit(const Exact& E, int side, int i) {
    return side ? __ldg(E.draft + i) : logit_at(E.target, E.dtype, i);
}
// of an entry that the number 0 may draw although its share is under a unit: whether it has any probability (left)
__device__ __noinline__ bool exact_any(const Exact& E, int i) {
    double z[2];
    for (int side = 0; side < (E.mode == 2 ? 2 : 1); ++side) {
        const float x = exact_logit(E, side, i);
        z[side] = (x == E.max[side] ? 0.0 : x > -INFINITY ? ((double)x - (double)E.max[side]) * E.c : -INFINITY) -
                  (double)E.log[side] * 1.3877787807814457e-17;
    }
    const double one = (double)kVpOne;
    return z[0] > -1074.0 && (E.mode < 2 || z[0] - z[1] > log2(1.0 + (double)E.over[0] / one) - log2(1.0 + (double)E.over[1] / one));
}
// what is left of one entry, in units of 2^-60
DF_DEV long long exact_entry(const Exact& E, int i) {
    if (E.mode == 1 && i == E.x) return 0;
    long long p = exact_share(E, 0, exact_logit(E, 0, i));
    if (E.mode == 2) {
        long long q = exact_share(E, 1, exact_logit(E, 1, i));
        // each by the other's sum: p' S_q - q' S_p
        p += __mul64hi(p << 2, E.over[1] << 2);
        q += __mul64hi(q << 2, E.over[0] << 2);
        p -= q;
    }
    return p > 0 ? p : E.first && p > -4 ? (long long)exact_any(E, i) : 0;
}
__device__ __noinline__ long long exact_left(const Exact& E, int i) { return exact_entry(E, i); }
// Entries [i0, end), by a warp: what is left of them, or (`rows`) p' and, with a drafter, q'.
__device__ __noinline__ Sums exact_sums(const Exact& E, int i0, int end, bool rows) {
    Sums a{};
#pragma unroll 1
    for (int i = i0 + (int)(threadIdx.x & 31); i < end; i += 32) {
        if (!rows) {
            a.d += exact_entry(E, i);
        } else {
            a.d += exact_share(E, 0, exact_logit(E, 0, i));
            if (E.mode == 2) a.g += exact_share(E, 1, exact_logit(E, 1, i));
        }
    }
    return a;
}

// A CTA's shared memory may be written from its cluster only once it runs: every CTA says so as it starts, and none
// writes before all have (the wait falls into the statistics' time).
DF_DEV void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
DF_DEV void cluster_wait_started() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// Which part of the sampled row is drawn from.
struct Picked {
    int v0, v1;       // in this CTA; v1 = 0: in another
    bool inside;      // its running sums pass the number's share
    long long rest;   // what of that share is left for it
    long long whole, g;
};
template <int WARPS>
struct PickShared {
    // a round of 32 rows of the sequence: the target's statistics and the drafter's, the draft's logits, which drafts are
    // refused, and which are too near to say
    VerifyStat stat[2][32];
    float logit[2][32];
    uint32_t refused, unsure;
    Norm norm[2][32];  // the rows' normalisers
    uint32_t table[2][kVpSteps];
    Sums part[WARPS], cta[2][kVpCluster];  // the warps' sums; the CTAs', of every other meeting
    int again[2];                          // likewise: whether the row has to be gone through in the exact form
    Picked picked;
    Exact exact;
};
// The warps' sums to every CTA of the cluster (S.cta), by all of it.
template <int WARPS>
DF_DEV void cluster_meet(PickShared<WARPS>& S, cg::cluster_group cl, Sums a, int turn) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_sum(a);
    if (lane == 0) S.part[warp] = a;
    __syncthreads();
    if (warp == 0) {
        Sums x{};
        if (lane < WARPS) x = S.part[lane];
        x = warp_sum(x);
        if (lane < kVpCluster) *cl.map_shared_rank(&S.cta[turn & 1][cl.block_rank()], lane) = x;
    }
    cl.sync();
}
// Entries [v0, v1) of part `part` of `parts` of n: whole steps, the last part with what they leave.
DF_DEV void row_share(int n, int part, int parts, int& v0, int& v1) {
    const int steps = n / kVpPiece;
    v0 = (int)((int64_t)steps * part / parts) * kVpPiece;
    v1 = part == parts - 1 ? n : (int)((int64_t)steps * (part + 1) / parts) * kVpPiece;
}
// The first of the lanes' pieces whose running sum passes `rest`; where none does (a number of 1, or a sum cut shorter
// than its parts'), the last that has any weight.  By a warp.
DF_DEV int narrow(long long piece, int lane, long long& rest, bool& inside) {
    const long long upto = warp_running(piece, lane);
    const uint32_t any = __ballot_sync(0xffffffffu, piece > 0);
    const uint32_t over = __ballot_sync(0xffffffffu, inside && piece > 0 && upto > rest);
    const int l = over ? __ffs(over) - 1 : any ? 31 - __clz(any) : 0;
    inside = over != 0;
    if (inside) rest -= __shfl_sync(0xffffffffu, upto - piece, l);
    return l;
}
// what a piece leaves of max(p - q, 0)
DF_DEV long long left_of(const Sums& x, long long g) { return x.d - (((g >> 14) * (long long)x.q) >> 14); }
// The exact form's description of target row `row` and, in mode 2, draft row `drow` (statistics in S.stat[..][slot]), and
// their sums.  By all of the cluster; a meeting.
template <int WARPS>
__device__ __noinline__ void exact_rows(PickShared<WARPS>& S, const VerifyArgs& A, int s, int slot, int64_t row, int64_t drow,
                                        int mode, int turn) {
    cg::cluster_group cl = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Exact& E = S.exact;
    __syncthreads();
    if (threadIdx.x == 0) {
        E.target = static_cast<const unsigned char*>(A.target) + row * A.target_stride * (A.target_dtype == kF32 ? 4 : 2);
        E.draft = mode == 2 ? A.draft + drow * A.draft_stride : nullptr;
        E.dtype = A.target_dtype;
        E.mode = mode;
        E.first = !(A.sample_u[s] > 0.f);
        E.c = 1.4426950408889634074 / (A.temperature != nullptr ? (double)fminf(fmaxf(A.temperature[s], 1e-30f), 1e30f) : 1.0);
        E.c1 = (float)E.c;
        E.c2 = (float)(E.c - (double)E.c1);
        E.c3 = (float)(E.c - (double)E.c1 - (double)E.c2);
        for (int side = 0; side < (mode == 2 ? 2 : 1); ++side) {
            const VerifyStat& r = S.stat[side][slot];
            E.max[side] = r.max;
            E.log[side] = __double2ll_rn(((double)log2f(r.sum) + (r.tag ? 0.0 : (double)r.ref - (double)r.max * E.c)) * 7.2057594037927936e16);
        }
    }
    __syncthreads();
    int v0, v1;
    row_share(A.vocab, (int)cl.block_rank() * WARPS + warp, kVpCluster * WARPS, v0, v1);
    Sums a = exact_sums(E, v0, v1, true);
    cluster_meet(S, cl, a, turn);
    if (warp == 0) {
        a = Sums{};
        if (lane < kVpCluster) a = S.cta[turn & 1][lane];
        a = warp_sum(a);
        if (lane == 0) E.over[0] = a.d - kVpOne, E.over[1] = a.g - kVpOne;
    }
    __syncthreads();
}
// Whether the draft of those rows, with logits lp and lq, stays: u q < p.
__device__ __noinline__ bool exact_keeps(const Exact& E, float u, float lp, float lq) {
    const auto weight = [&](int side, float x) {
        return exp2((x == E.max[side] ? 0.0 : ((double)x - (double)E.max[side]) * E.c) - (double)E.log[side] * 1.3877787807814457e-17);
    };
    const double one = (double)kVpOne, sp = one + (double)E.over[0], sq = one + (double)E.over[1];
    return E.mode == 2 ? (double)u * weight(1, lq) * sp < weight(0, lp) * sq : (double)u * sp < weight(0, lp) * one;
}

template <int WARPS>
__global__ void __cluster_dims__(kVpCluster, 1, 1) __launch_bounds__(WARPS * 32)
    verify_pick_kernel(const __grid_constant__ VerifyParams P) {
    constexpr int kParts = kVpCluster * WARPS;  // vocabulary parts of the sampled row
    const VerifyArgs& A = P.A;
    __shared__ PickShared<WARPS> S;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), s = blockIdx.x / kVpCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int turn = 0;  // meetings of the cluster
    cluster_started();
    // 2^63 times 2^(-i / 128)
    const int step = threadIdx.x & (kVpSteps - 1);
    const unsigned long long two = kTwoTo[(kVpSteps - step) & (kVpSteps - 1)] >> (step != 0);
    pdl_wait();
    int a, b;
    draft_range(A, s, lane, a, b);
    const int d = b - a;
    const Scale c = scale_of(A, s);
    const bool drawn = A.draft != nullptr && !c.greedy();  // q is the drafter's distribution, not one token
    const int64_t nt = (int64_t)A.n_drafts + A.n_seqs, row0 = (int64_t)a + s;
    // how far what decides on a draft may be off: the rows' sums of exponentials, in chains of up to 64 f32 additions and
    // the join of their parts
    const float tol = 1.6e-5f + P.parts * 4e-9f;
    bool met = false;
    auto meet_first = [&]() {
        if (!met) cluster_wait_started();
        met = true;
    };

    // every CTA of the cluster decides alike; the first one writes
    int refused = 0x7fffffff, i0 = 0;
    for (;; i0 += 32) {
        const int n = min(32, d + 1 - i0);  // rows of the round, the one after the last draft among them
        float u = 0.f;
        if (warp == 0 && i0 + lane < d) u = __ldg(A.accept_u + a + i0 + lane);
#pragma unroll 1
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
                S.stat[side][i - i0] = t;
                S.logit[side][i - i0] = l;
            }
        }
        __syncthreads();
        // warp 0 decides on the drafts, warp 1 writes their probabilities; warps 2 and 3 normalise the rows
        const int i = i0 + lane;
        if (warp == 0) {
            bool refuse = false, unsure = false;
            if (i < d) {
                const VerifyStat t = S.stat[0][lane];
                if (c.greedy()) {
                    refuse = t.max == -INFINITY || t.tag != (int)A.draft_tok[a + i];
                } else {
                    // p = wp / sp and q = wq / sq: compared as u wq sp < wp sq
                    const VerifyStat g = S.stat[1][lane];
                    const float lp = S.logit[0][lane], lq = S.logit[1][lane];
                    const bool some = t.max > -INFINITY && lp > -INFINITY, other = drawn && g.max > -INFINITY && lq > -INFINITY;
                    const float wp = some ? weight_any(lp, t, c) : 0.f, sp = t.max > -INFINITY ? t.sum : 1.f,
                                wq = !drawn ? 1.f : other ? weight_any(lq, g, c) : 0.f, sq = drawn && g.max > -INFINITY ? g.sum : 1.f;
                    const float p = wp * sq, uq = u * (wq * sp);
                    refuse = !(uq < p);
                    // (a weight's exponent, rounded twice, may be 2^-23 of it off, and so may those of the sums, which
                    // the low part of c can move; weights under f32's range count as 0)
                    const float far = fabsf(lp * c.hi - (t.tag ? t.max * c.hi : t.ref)) + fabsf(t.max * c.lo) +
                                      (other ? fabsf(lq * c.hi - (g.tag ? g.max * c.hi : g.ref)) + fabsf(g.max * c.lo) : 0.f);
                    unsure = some && (!drawn || other) &&
                             fabsf(uq - p) <= fmaf(fmaf(fminf(far, 300.f), 3e-7f, tol), fmaxf(uq, p), 1e-35f * (sp * sq));
                }
            }
            const uint32_t r = __ballot_sync(0xffffffffu, refuse && !unsure), m = __ballot_sync(0xffffffffu, unsure);
            if (lane == 0) S.refused = r, S.unsure = m;
        } else if (warp == 1) {
            if (rank == 0 && A.prob != nullptr && i < d) {
                const VerifyStat t = S.stat[0][lane], g = S.stat[1][lane];
                float wp, sp = 1.f, wq = 1.f, sq = 1.f;
                if (c.greedy()) {
                    wp = t.max > -INFINITY && t.tag == (int)A.draft_tok[a + i] ? 1.f : 0.f;
                } else {
                    wp = weight_exact(S.logit[0][lane], t, c);
                    if (t.max > -INFINITY) sp = t.sum;
                }
                if (drawn) {
                    wq = weight_exact(S.logit[1][lane], g, c);
                    if (g.max > -INFINITY) sq = g.sum;
                }
                // (q = 0: a draft the drafter could not make; kept when p is not 0)
                A.prob[a + i] = wp * sq < wq * sp ? (wp / sp) / (wq / sq) : wp > 0.f ? 1.f : 0.f;
            }
        } else if (warp < (drawn ? 4 : 3) && !c.greedy() && lane < n) {
            if (S.stat[warp - 2][lane].max > -INFINITY) S.norm[warp - 2][lane] = norm_of(S.stat[warp - 2][lane], nearest(c));
        }
        __syncthreads();
        uint32_t open = S.unsure;
        const uint32_t certain = S.refused;
        while (refused == 0x7fffffff && (open | certain) != 0) {
            const int j = __ffs(open | certain) - 1;
            bool keep = false;
            if ((open >> j) & 1u) {
                meet_first();
                exact_rows<WARPS>(S, A, s, j, row0 + i0 + j, a + i0 + j, drawn ? 2 : 0, turn++);
                keep = __syncthreads_or(threadIdx.x == 0 &&
                                        exact_keeps(S.exact, __ldg(A.accept_u + a + i0 + j), S.logit[0][j], S.logit[1][j]));
                open &= ~(1u << j);
            }
            if (!keep) refused = i0 + j;
        }
        if (i0 + 32 > d) break;
        __syncthreads();
    }
    const int acc = min(refused, d);
    const int64_t row = row0 + acc;
    int slot = acc - i0;
    if (slot < 0) {  // (refused more than a round ago)
        slot = 0;
        __syncthreads();
        if (warp < (drawn ? 2 : 1)) {
            const VerifyStat t = row_stat(P, warp ? nt + a + acc : row, c, lane);
            if (lane == 0) {
                S.stat[warp][0] = t;
                if (!c.greedy() && t.max > -INFINITY) S.norm[warp][0] = norm_of(t, nearest(c));
            }
        }
        __syncthreads();
    }
    const float most = S.stat[0][slot].max;
    meet_first();
    if (c.greedy() || most == -INFINITY) {
        if (rank == 0 && threadIdx.x == 0) {
            A.accepted[s] = acc;
            A.next_tok[s] = most == -INFINITY ? -1 : S.stat[0][slot].tag;
        }
        return;
    }
    // (a drafter without any probability takes nothing off)
    const int mode = acc == d ? 0 : !drawn ? 1 : S.stat[1][slot].max > -INFINITY ? 2 : 0;
    if (threadIdx.x < (mode == 2 ? 2 : 1) * kVpSteps)
        S.table[threadIdx.x >> 7][step] =
            (uint32_t)((__umul64hi(two, (unsigned long long)S.norm[threadIdx.x >> 7][slot].mul << 32) + (1ull << 30)) >> 31);
    __syncthreads();
    Sampled L;
    L.target = static_cast<const unsigned char*>(A.target) + row * A.target_stride * (A.target_dtype == kF32 ? 4 : 2);
    L.draft = mode == 2 ? A.draft + (int64_t)(a + acc) * A.draft_stride : nullptr;
    L.dtype = A.target_dtype;
    L.mode = mode;
    L.x = mode == 1 ? (int)min(A.draft_tok[a + acc], 0x7fffffffu) : -1;
    L.c = nearest(c);
    const Norm &pn = S.norm[0][slot], &qn = S.norm[mode == 2][slot];
    L.tm = pn.magic;
    L.qm = qn.magic;
    L.apart = (qn.whole - pn.whole) + (qn.log - pn.log);
    L.tol = 1.6e-5f + fabsf(L.apart) * 5e-7f;
    const bool fits = pn.fits && qn.fits;
    bool exact = !fits, known = false;  // known: the exact form's description stands
    for (;;) {
        if (exact) {
            if (!known) exact_rows<WARPS>(S, A, s, slot, row, a + acc, L.mode, turn++);
            known = true;
            __syncthreads();
            if (threadIdx.x == 0) S.exact.mode = L.mode, S.exact.x = L.x;
            __syncthreads();
        }
        auto sums_of = [&](int p0, int p1) -> Sums {
            return exact ? exact_sums(S.exact, p0, p1, false) : L.sums(p0, p1, lane, S.table);
        };
        int v0, v1;
        row_share(A.vocab, rank * WARPS + warp, kParts, v0, v1);
        cluster_meet(S, cl, sums_of(v0, v1), turn++);
        const Sums* ctas = S.cta[(turn - 1) & 1];
        // the first CTA whose running sum passes the number's share of the whole, then its first warp
        if (warp == 0) {
            Sums x{};
            if (lane < kVpCluster) x = ctas[lane];
            Picked k;
            k.g = L.mode == 2 && !exact ? warp_sum(x.g) : 0;  // (under 2^42, or nothing below counts)
            const long long own = left_of(x, k.g);
            k.whole = warp_sum(own);
            // (the whole part of u times the whole; of nothing, nothing)
            const unsigned long long u = __float2ull_rz(fmaxf(__ldg(A.sample_u + s), 0.f) * 18446744073709551616.f);
            k.rest = (long long)__umul64hi((unsigned long long)max(k.whole, 0ll), u);
            k.inside = true;
            k.v0 = k.v1 = 0;
            if (narrow(own, lane, k.rest, k.inside) == rank) {
                const int l = narrow(lane < WARPS ? left_of(S.part[lane], k.g) : 0, lane, k.rest, k.inside);
                row_share(A.vocab, rank * WARPS + l, kParts, k.v0, k.v1);
            }
            if (lane == 0) S.picked = k;
        }
        __syncthreads();
        Picked k = S.picked;
        if (exact && k.whole <= 0 && L.mode != 0) {
            L.mode = 0;  // the draft had all of it: the target's own distribution
            L.x = -1;
            exact = !fits;
            __syncthreads();
            continue;
        }
        // (about nothing, or normalisers further off than what `tie` takes for agreeing: the exact form says what)
        if (!exact && (k.whole <= 0 || llabs(k.g) >= 1ll << 42)) {
            exact = true;
            __syncthreads();
            continue;
        }
        if (k.v1 > 0) {
            constexpr int kEach = 4;  // entries of a lane at the last step
            while (k.v1 - k.v0 > kEach * WARPS * 32) {  // (a vocabulary of more than 260 000: by warps again)
                row_share(k.v1 - k.v0, warp, WARPS, v0, v1);
                const Sums x = warp_sum(sums_of(k.v0 + v0, k.v0 + v1));
                __syncthreads();
                if (lane == 0) S.part[warp] = x;
                __syncthreads();
                const int l = narrow(lane < WARPS ? left_of(S.part[lane], k.g) : 0, lane, k.rest, k.inside);
                row_share(k.v1 - k.v0, l, WARPS, v0, v1);
                k.v1 = k.v0 + v1;
                k.v0 += v0;
            }
            // entry by entry: a lane's in a row
            const int each = (k.v1 - k.v0 + WARPS * 32 - 1) / (WARPS * 32), first = k.v0 + (int)threadIdx.x * each;
            long long left[kEach] = {}, mine = 0;
#pragma unroll 1
            for (int j = 0; j < each && first + j < k.v1; ++j) {
                const long long x = exact ? exact_left(S.exact, first + j) : L.left(first + j, k.g, S.table);
#pragma unroll
                for (int n = 0; n < kEach; ++n)
                    if (n == j) left[n] = x;
                mine += x;
            }
            const long long all = warp_sum(mine);
            __syncthreads();
            if (lane == 0) S.part[warp].d = all;
            __syncthreads();
            if (narrow(lane < WARPS ? S.part[lane].d : 0, lane, k.rest, k.inside) == warp) {
                const int l = narrow(mine, lane, k.rest, k.inside);
                Sums sum{};
                if (lane < kVpCluster) sum = ctas[lane];
                sum = warp_sum(sum);
                bool sure = false;
                if (lane == l) {
                    int at = -1, last = 0;
                    long long below = 0, above = 0;  // distances from the entry's borders
#pragma unroll
                    for (int j = 0; j < kEach; ++j) {
                        if (left[j] > 0) last = j;
                        if (k.inside && at < 0 && left[j] > k.rest) at = j, below = k.rest, above = left[j] - k.rest;
                        k.rest -= left[j];
                    }
                    // What a border may be off by: the shares ahead of it count 1 - u times, those behind it u times.
                    // After a refusal p' and q' where p' - q' is positive, and q' there times the error of g, which is
                    // both rows'; entries of uncertain sign; the units that shifts cut off.
                    const float u = __ldg(A.sample_u + s), entries = (float)A.vocab, g = fabsf((float)k.g);
                    const float eps = kVpEps * fmaxf(u, 1.f - u);
                    float off = eps * (float)k.whole + 2.f * entries;
                    if (L.mode == 2)
                        off = eps * ((float)k.whole + 4.f * 4294967296.f * (float)sum.q) +
                              2.1f * g * (3.7252903e-9f * (float)sum.tie) + entries * (4.f + 1.5e-8f * g) + 65536.f;
                    sure = at >= 0 && (float)below > off && (float)above > off;
                    if (exact || sure) {
                        A.accepted[s] = acc;
                        A.next_tok[s] = first + (at < 0 ? last : at);
                    }
                }
                sure = __shfl_sync(0xffffffffu, sure, l);
                if (!exact && lane < kVpCluster) *cl.map_shared_rank(&S.again[turn & 1], lane) = !sure;
            }
        }
        if (exact) break;
        cl.sync();
        const bool again = S.again[turn & 1];
        ++turn;
        if (!again) break;
        exact = true;
    }
    // (the last that is written into a CTA is written before the last meeting: none has to wait to leave)
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
    return (int)launch(verify_pick_kernel<WARPS>, dim3((unsigned)P.A.n_seqs * kVpCluster), dim3(WARPS * 32), 0, st, P);
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
