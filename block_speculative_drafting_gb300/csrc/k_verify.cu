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
// parts of the vocabulary, every CTA finds the part in which the running sum
// passes the given number's share of the whole, and the warp that owns it
// finds the chunk and the entry.
//
// Arithmetic.  The sums decide whole numbers, so they carry about 48 bits: f32
// batches of 16 or 32 exponentials (each within 2^-22) are added to a pair
// (hi, lo) by error-free additions -- the 64-bit units of this part are too
// few for that (two lanes a clock and SM).  c is a pair too, so that its
// rounding does not tilt the distribution, and R is an integer, so that moving
// a sum to another reference is exact and x c - R is rounded once.
//
// Memory bound: the logits, once (the re-read row comes out of L2).
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "paged.cuh"

namespace dflash {

namespace cg = cooperative_groups;

constexpr int kVsThreads = 256;
constexpr int kVpThreads = 512, kVpWarps = kVpThreads / 32;
constexpr int kVpCluster = 8;
constexpr int kVpParts = kVpCluster * kVpWarps;  // vocabulary parts of the sampled row
constexpr int kVpChunks = 64;                    // chunks of a part, at most
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
DF_DEV Pair scaled(Pair a, float f) { return {a.hi * f, a.lo * f}; }  // (f a power of two: exact)
DF_DEV double wide(Pair a) { return (double)a.hi + (double)a.lo; }
DF_DEV Pair shfl_xor(Pair a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
DF_DEV Pair warp_sum(Pair a) {
#pragma unroll
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
struct VerifyStat {
    Pair sum;
    float ref, max;
    int32_t arg;  // (greedy) the lowest index of the largest logit
    int32_t careful;
};

struct VerifyParams {
    VerifyArgs A;
    VerifyStat* stats;  // [target rows, then draft rows][parts]
    int parts;
};

DF_DEV void draft_range(const VerifyArgs& A, int s, int& a, int& b) {
    if (A.draft_start == nullptr) {
        a = s * A.per;
        b = a + A.per;
    } else {
        a = min(max(A.draft_start[s], 0), A.n_drafts);
        b = min(max(A.draft_start[s + 1], a), A.n_drafts);
    }
}
// The last sequence whose drafts (shift 0) or target rows (shift 1) start at
// or before entry i; -1 where no sequence holds it.
DF_DEV int verify_seq(const VerifyArgs& A, int i, int shift) {
    if (A.draft_start == nullptr) return i / (A.per + shift);
    int lo = 0, hi = A.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.draft_start[mid] + shift * mid <= i)
            lo = mid;
        else
            hi = mid;
    }
    int a, b;
    draft_range(A, lo, a, b);
    return i >= a + shift * lo && i < b + shift * (lo + 1) ? lo : -1;
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
    DF_DEV static void get(const float* p, float* x) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
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
    DF_DEV static void get(const uint16_t* p, float* x) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
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
// up to the first 16-byte boundary and the last few come as a batch of their own.
template <int DT, class F>
DF_DEV void each_batch(const typename Vec<DT>::T* row, int v0, int v1, F f) {
    using V = Vec<DT>;
    constexpr int N = V::N, U = 4;
    const int mis = (int)((reinterpret_cast<uintptr_t>(row + v0) & 15) / sizeof(typename V::T));
    const int a = min(v1, v0 + (mis ? N - mis : 0)), nv = (v1 - a) / N, b = a + nv * N;
    float x[U * N];
    int at[U];
    if (a > v0 || v1 > b) {
#pragma unroll
        for (int i = 0; i < U * N; ++i) x[i] = -INFINITY;
#pragma unroll
        for (int k = 0; k < U; ++k) at[k] = v0;
        const int h = v0 + threadIdx.x, t = b + threadIdx.x;
        if (h < a) x[0] = V::one(row + h), at[0] = h;
        if (t < v1) x[N] = V::one(row + t), at[1] = t;
        if (h < a || t < v1) f(x, at);
    }
    for (int i = threadIdx.x; i < nv; i += U * kVsThreads) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = i + k * kVsThreads;
            at[k] = a + j * N;
            if (j < nv) {
                V::get(row + at[k], x + k * N);
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n) x[k * N + n] = -INFINITY;
            }
        }
        f(x, at);
    }
}
template <int M>
DF_DEV float max_of(const float* x) {
    float m = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < M; i += 2) m = fmaxf(m, fmaxf(x[i], x[i + 1]));
    return m;
}

// One part of one row, by the whole CTA; thread 0 has the answer.
template <int DT>
DF_DEV VerifyStat row_part(const typename Vec<DT>::T* row, int v0, int v1, Scale c, VerifyStat* warps) {
    constexpr int N = Vec<DT>::N, M = 4 * N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    VerifyStat r{{0.f, 0.f}, kRefNone, -INFINITY, 0x7fffffff, 0};
    if (c.greedy()) {
        auto join = [&](float m, int arg) {
            if (m > r.max || (m == r.max && arg < r.arg)) r.max = m, r.arg = arg;
        };
        each_batch<DT>(row, v0, v1, [&](const float* x, const int* at) {
            const float m = max_of<M>(x);
            if (m >= r.max && m > -INFINITY) {
                int arg = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < M; ++i)
                    if (x[i] == m) arg = min(arg, at[i / N] + i % N);
                join(m, arg);
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(__shfl_xor_sync(0xffffffffu, r.max, o), __shfl_xor_sync(0xffffffffu, r.arg, o));
        if (lane == 0) warps[warp] = r;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 1; w < kVsThreads / 32; ++w) join(warps[w].max, warps[w].arg);
        return r;
    }
    each_batch<DT>(row, v0, v1, [&](const float* x, const int*) {
        const float m = max_of<M>(x);
        r.max = fmaxf(r.max, m);
        const float ref = fmaxf(r.ref, ceilf(m * c.hi));
        r.sum = scaled(r.sum, pow2(r.ref - ref));
        r.ref = ref;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < M; ++i) s[i & 3] += weight(x[i], c, ref);
        r.sum = r.sum + Pair{(s[0] + s[1]) + (s[2] + s[3]), 0.f};
    });
    bool plain = !__syncthreads_or(!(r.sum.hi < INFINITY));
    if (plain) {
        auto join = [&](Pair s, float ref, float m) {
            const float to = fmaxf(r.ref, ref);
            r.sum = scaled(r.sum, pow2(r.ref - to)) + scaled(s, pow2(ref - to));
            r.ref = to;
            r.max = fmaxf(r.max, m);
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(shfl_xor(r.sum, o), __shfl_xor_sync(0xffffffffu, r.ref, o), __shfl_xor_sync(0xffffffffu, r.max, o));
        if (lane == 0) warps[warp] = r;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 1; w < kVsThreads / 32; ++w) join(warps[w].sum, warps[w].ref, warps[w].max);
        plain = !__syncthreads_or(threadIdx.x == 0 && r.sum.hi == 0.f && r.max > -INFINITY);
        if (plain) return r;
    }
    // again, with the part's largest logit taken off first
    float m = warp_max(fmaxf(r.max, -INFINITY));
    if (lane == 0) warps[warp].max = m;
    __syncthreads();
    for (int w = 0; w < kVsThreads / 32; ++w) m = fmaxf(m, warps[w].max);
    __syncthreads();
    r = VerifyStat{{0.f, 0.f}, kRefNone, m, 0x7fffffff, 1};
    if (m > -INFINITY)
        each_batch<DT>(row, v0, v1, [&](const float* x, const int*) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < M; ++i) s += weight_careful(x[i], c, m);
            r.sum = r.sum + Pair{s, 0.f};
        });
    r.sum = warp_sum(r.sum);
    if (lane == 0) warps[warp] = r;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kVsThreads / 32; ++w) r.sum = r.sum + warps[w].sum;
    return r;
}

__global__ void __launch_bounds__(kVsThreads) verify_stats_kernel(const __grid_constant__ VerifyParams P) {
    const VerifyArgs& A = P.A;
    __shared__ VerifyStat warps[kVsThreads / 32];
    const int part = blockIdx.x % P.parts, row = blockIdx.x / P.parts;
    const int nt = A.n_drafts + A.n_seqs;
    pdl_wait();
    pdl_trigger();
    const int s = row < nt ? verify_seq(A, row, 1) : verify_seq(A, row - nt, 0);
    if (s < 0) return;
    const Scale c = scale_of(A, s);
    if (row >= nt && c.greedy()) return;  // a greedy sequence's drafter is not asked
    const int v0 = (int)((int64_t)A.vocab * part / P.parts), v1 = (int)((int64_t)A.vocab * (part + 1) / P.parts);
    VerifyStat r;
    if (row >= nt)
        r = row_part<kF32>(A.draft + (int64_t)(row - nt) * A.draft_stride, v0, v1, c, warps);
    else if (A.target_dtype == kF32)
        r = row_part<kF32>(static_cast<const float*>(A.target) + (int64_t)row * A.target_stride, v0, v1, c, warps);
    else if (A.target_dtype == kBF16)
        r = row_part<kBF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, c, warps);
    else
        r = row_part<kF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, c, warps);
    if (threadIdx.x == 0) P.stats[(int64_t)row * P.parts + part] = r;
}

// A row's parts joined (warp-wide, every lane gets the answer).  A row with a
// careful part is careful as a whole.
DF_DEV VerifyStat row_stat(const VerifyParams& P, int64_t row, Scale c, int lane) {
    const VerifyStat* st = P.stats + row * P.parts;
    VerifyStat r{{0.f, 0.f}, kRefNone, -INFINITY, 0x7fffffff, 0};
    if (c.greedy()) {
        for (int i = lane; i < P.parts; i += 32)
            if (st[i].max > r.max || (st[i].max == r.max && st[i].arg < r.arg)) r.max = st[i].max, r.arg = st[i].arg;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, r.max, o);
            const int arg = __shfl_xor_sync(0xffffffffu, r.arg, o);
            if (m > r.max || (m == r.max && arg < r.arg)) r.max = m, r.arg = arg;
        }
        return r;
    }
    for (int i = lane; i < P.parts; i += 32) {
        r.ref = fmaxf(r.ref, st[i].ref);
        r.max = fmaxf(r.max, st[i].max);
        r.careful |= st[i].careful;
    }
    r.ref = warp_max(r.ref);
    r.max = warp_max(r.max);
    r.careful = __any_sync(0xffffffffu, r.careful);
    if (!r.careful) {
        for (int i = lane; i < P.parts; i += 32) r.sum = r.sum + scaled(st[i].sum, pow2(st[i].ref - r.ref));
    } else {
        // in 64 bits: every part's sum to the row's largest logit
        for (int i = lane; i < P.parts; i += 32) {
            const VerifyStat x = st[i];
            if (x.sum.hi == 0.f) continue;
            double f = 1.0;
            if (x.careful) {
                if (x.max != r.max) f = exp2(((double)x.max - (double)r.max) * c.wide());
            } else {
                f = exp2((double)x.ref - (double)r.max * c.wide());
            }
            const double y = wide(x.sum) * f;
            const float hi = (float)y;
            r.sum = r.sum + Pair{hi, (float)(y - (double)hi)};
        }
    }
    r.sum = warp_sum(r.sum);
    return r;
}
DF_DEV float logit_at(const void* base, int dtype, int64_t i) {
    return dtype == kF32    ? Vec<kF32>::one(static_cast<const float*>(base) + i)
           : dtype == kBF16 ? Vec<kBF16>::one(static_cast<const uint16_t*>(base) + i)
                            : Vec<kF16>::one(static_cast<const uint16_t*>(base) + i);
}
// p(x) of one entry, in 64 bits.
DF_DEV double prob_at(float x, const VerifyStat& r, Scale c) {
    if (r.max == -INFINITY || !(x > -INFINITY)) return 0.0;
    const double w = !r.careful     ? exp2((double)x * c.wide() - (double)r.ref)
                     : x == r.max ? 1.0
                                  : exp2(((double)x - (double)r.max) * c.wide());
    return w / wide(r.sum);
}

// What is left at the entries of the sampled row: mode 0 the target's
// probability (unnormalised), 1 with the draft taken out, 2 max(p - q, 0).
struct Left {
    const unsigned char* target;
    const float* draft;
    int dtype, mode, x;
    bool aligned;  // both rows start at 16-byte boundaries
    VerifyStat t, q;
    float tz, qz;  // 1 / the rows' sums
    Scale c;
    // the eight entries from i on (i a multiple of 8), 0 from `end` on
    DF_DEV void eight(int i, int end, float (&w)[8]) const {
        float a[8], b[8];
        const bool vec = aligned && i + 8 <= end;
        if (vec) {
            if (dtype == kF32) {
                Vec<kF32>::get(reinterpret_cast<const float*>(target) + i, a);
                Vec<kF32>::get(reinterpret_cast<const float*>(target) + i + 4, a + 4);
            } else if (dtype == kBF16) {
                Vec<kBF16>::get(reinterpret_cast<const uint16_t*>(target) + i, a);
            } else {
                Vec<kF16>::get(reinterpret_cast<const uint16_t*>(target) + i, a);
            }
            if (mode == 2) {
                Vec<kF32>::get(draft + i, b);
                Vec<kF32>::get(draft + i + 4, b + 4);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] = i + k < end ? logit_at(target, dtype, i + k) : -INFINITY;
                if (mode == 2) b[k] = i + k < end ? __ldg(draft + i + k) : -INFINITY;
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            w[k] = t.careful ? weight_careful(a[k], c, t.max) : weight(a[k], c, t.ref);
            if (mode == 1 && i + k == x) w[k] = 0.f;
            if (mode == 2) {
                float y = 0.f;
                if (q.max > -INFINITY) y = (q.careful ? weight_careful(b[k], c, q.max) : weight(b[k], c, q.ref)) * qz;
                w[k] = fmaxf(fmaf(w[k], tz, -y), 0.f);
            }
            if (i + k >= end) w[k] = 0.f;
        }
    }
    // their sums over [p0, p1), warp-wide: lane l holds the entries p0 + 8 l .. of every 256
    DF_DEV float lane_sum(int i, int end, float (&w)[8]) const {
        eight(i, end, w);
        return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    }
};

__global__ void __cluster_dims__(kVpCluster, 1, 1) __launch_bounds__(kVpThreads)
    verify_pick_kernel(const __grid_constant__ VerifyParams P) {
    const VerifyArgs& A = P.A;
    __shared__ int refused;
    __shared__ double part_sum[2][kVpWarps];  // (two passes at most: each has its own)
    __shared__ double chunk_sum[kVpWarps][kVpChunks];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), s = blockIdx.x / kVpCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) refused = 0x7fffffff;
    __syncthreads();
    // the inputs are final before the statistics kernel lets this one start
    int a, b;
    draft_range(A, s, a, b);
    const int d = b - a;
    const Scale c = scale_of(A, s);
    const bool drawn = A.draft != nullptr && !c.greedy();  // q is the drafter's distribution, not one token
    const int64_t nt = (int64_t)A.n_drafts + A.n_seqs;

    // every CTA of the cluster decides alike; the first one writes
    for (int i = warp; i < d; i += kVpWarps) {
        const int64_t row = (int64_t)a + s + i;
        const uint32_t x = A.draft_tok[a + i];
        const bool known = x < (uint32_t)A.vocab;
        const float u = A.accept_u[a + i];
        const float lt = known ? logit_at(A.target, A.target_dtype, row * A.target_stride + x) : -INFINITY;
        const float ld = known && drawn ? __ldg(A.draft + (int64_t)(a + i) * A.draft_stride + x) : -INFINITY;
        pdl_wait();
        const VerifyStat t = row_stat(P, row, c, lane);
        double p, q = 1.0;
        if (c.greedy())
            p = known && t.max > -INFINITY && t.arg == (int)x ? 1.0 : 0.0;
        else
            p = known ? prob_at(lt, t, c) : 0.0;
        if (drawn) {
            const VerifyStat g = row_stat(P, nt + a + i, c, lane);
            q = known ? prob_at(ld, g, c) : 0.0;
        }
        if (lane == 0) {
            if (!((double)u * q < p)) atomicMin(&refused, i);
            // (q = 0: a draft the drafter could not make; kept when p is not 0)
            if (rank == 0 && A.prob != nullptr) A.prob[a + i] = (float)(p < q ? p / q : p > 0.0 ? 1.0 : 0.0);
        }
    }
    pdl_wait();
    __syncthreads();
    const int acc = min(refused, d);
    const int64_t row = (int64_t)a + s + acc;
    const VerifyStat t = row_stat(P, row, c, lane);
    int token = t.max == -INFINITY ? -1 : t.arg;
    bool writes = rank == 0 && threadIdx.x == 0;
    const bool sampled = !c.greedy() && t.max > -INFINITY;
    if (sampled) {
        writes = false;
        Left L;
        L.target = static_cast<const unsigned char*>(A.target) + row * A.target_stride * (A.target_dtype == kF32 ? 4 : 2);
        L.draft = nullptr;
        L.dtype = A.target_dtype;
        L.c = c;
        L.t = L.q = t;
        L.tz = (float)(1.0 / wide(t.sum));
        L.qz = 0.f;
        L.x = -1;
        L.mode = 0;
        if (acc < d) {
            L.x = (int)min(A.draft_tok[a + acc], 0x7fffffffu);
            L.mode = 1;
            if (drawn) {
                L.q = row_stat(P, nt + a + acc, c, lane);
                L.draft = A.draft + (int64_t)(a + acc) * A.draft_stride;
                L.mode = 2;
                L.qz = L.q.max == -INFINITY ? 0.f : (float)(1.0 / wide(L.q.sum));
            }
        }
        L.aligned = ((reinterpret_cast<uintptr_t>(L.target) | reinterpret_cast<uintptr_t>(L.draft)) & 15) == 0;
        // this warp's part of the vocabulary, in chunks of a multiple of 256 entries
        const int w = rank * kVpWarps + warp;
        const int64_t v8 = ((int64_t)A.vocab + 7) / 8;
        const int v0 = (int)(v8 * w / kVpParts) * 8, v1 = min((int)(v8 * (w + 1) / kVpParts) * 8, A.vocab);
        const int chunk = 256 * max(1, (v1 - v0 + 256 * kVpChunks - 1) / (256 * kVpChunks));
        const int nchunks = (max(v1 - v0, 0) + chunk - 1) / chunk;
        const float u = A.sample_u[s];
        for (int pass = 0; pass < 2; ++pass) {
            double mine = 0.0;
            for (int k = 0; k < nchunks; ++k) {
                const int e = min(v0 + (k + 1) * chunk, v1);
                Pair sum;
#pragma unroll 2
                for (int i = v0 + k * chunk + 8 * lane; i < e; i += 256) {
                    float x[8];
                    sum = sum + Pair{L.lane_sum(i, e, x), 0.f};
                }
                const double y = wide(warp_sum(sum));
                if (lane == 0) chunk_sum[warp][k] = y;
                mine += y;
            }
            if (lane == 0) part_sum[pass][warp] = mine;
            cl.sync();
            // the cluster's sums, kVpParts / 32 a lane in order, and their running sums
            constexpr int PL = kVpParts / 32;
            double sum[PL], run = 0.0;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                const int j = lane * PL + k;
                sum[k] = *cl.map_shared_rank(&part_sum[pass][j % kVpWarps], j / kVpWarps);
                run += sum[k];
            }
            double in = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += y;
            }
            const double whole = __shfl_sync(0xffffffffu, in, 31);
            if (whole == 0.0 && L.mode != 0) {
                L.mode = 0;  // the draft had all of it: the target's own distribution
                continue;
            }
            double rest = (double)u * whole;
            // the first part whose running sum passes the number's share (the last with any of it, should
            // rounding or a number of 1 leave none)
            int hit = 0x7fffffff, some = -1;
            double before = in - run, hit_before = 0.0;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                if (sum[k] > 0.0) {
                    some = lane * PL + k;
                    if (hit == 0x7fffffff && before + sum[k] > rest) hit = lane * PL + k, hit_before = before;
                }
                before += sum[k];
            }
            const int first = (int)__reduce_min_sync(0xffffffffu, (unsigned)hit);
            const int last = __reduce_max_sync(0xffffffffu, some);
            if ((first != 0x7fffffff ? first : last) != w) break;
            rest = first != 0x7fffffff ? rest - __shfl_sync(0xffffffffu, hit_before, first / PL) : INFINITY;
            // the chunk, in order, the same way
            int at = 0, k = 0;
            for (; k < nchunks; ++k) {
                const double y = chunk_sum[warp][k];
                if (y <= 0.0) continue;
                at = k;
                if (y > rest) break;
                rest -= y;
            }
            if (k == nchunks) rest = INFINITY;
            // and the entry: 256 at a time, eight neighbours a lane
            const int e = min(v0 + (at + 1) * chunk, v1);
            int found = -1;
            for (int i0 = v0 + at * chunk; i0 < e; i0 += 256) {
                float x[8];
                const double y = (double)L.lane_sum(i0 + 8 * lane, e, x);
                double up = y;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double z = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += z;
                }
                const uint32_t any = __ballot_sync(0xffffffffu, y > 0.0);
                const uint32_t over = __ballot_sync(0xffffffffu, y > 0.0 && up > rest);
                if (any) {
                    const int l = over ? __ffs(over) - 1 : 31 - __clz(any);
                    // the lane's own entries: the first over what remains, else its last with any of it
                    double r = over ? rest - (up - y) : INFINITY;
                    int mine_at = -1;
                    bool done = false;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        if (!done && x[n] > 0.f) {
                            mine_at = i0 + 8 * lane + n;
                            if ((double)x[n] > r) done = true;
                            r -= (double)x[n];
                        }
                    }
                    found = __shfl_sync(0xffffffffu, mine_at, l);
                }
                if (over) break;
                rest -= __shfl_sync(0xffffffffu, up, 31);
            }
            token = found;
            writes = lane == 0;
            break;
        }
    }
    if (writes) {
        A.accepted[s] = acc;
        A.next_tok[s] = token;
    }
    if (sampled) cl.sync();  // no CTA leaves while its sums may be read
}

// Parts of a row: of at least 16 KB each, and where there are few rows enough
// of them for a few CTAs an SM.
static int verify_parts(int64_t rows, int64_t vocab, int num_sms) {
    const int64_t want = (16 * (int64_t)num_sms + rows - 1) / (rows > 0 ? rows : 1);
    const int64_t most = (vocab + 4095) / 4096, least = (vocab + 16383) / 16384;
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

int verify(const VerifyArgs& A, void* ws, int num_sms, cudaStream_t st) {
    VerifyParams P;
    P.A = A;
    P.stats = static_cast<VerifyStat*>(ws);
    const int64_t rows = verify_rows(A.n_seqs, A.n_drafts, A.draft != nullptr);
    P.parts = verify_parts(rows, A.vocab, num_sms);
    if (cudaError_t e = launch(verify_stats_kernel, dim3((unsigned)(rows * P.parts)), dim3(kVsThreads), 0, st, P))
        return (int)e;
    return (int)launch(verify_pick_kernel, dim3((unsigned)A.n_seqs * kVpCluster), dim3(kVpThreads), 0, st, P);
}

}  // namespace dflash
