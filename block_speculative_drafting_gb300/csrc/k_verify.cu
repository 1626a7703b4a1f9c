// Verification of drafted tokens against the target's probabilities.
//
// Two kernels.  verify_stats_kernel reads every logit row once: a CTA takes
// one part of one row's vocabulary and leaves its largest logit (with the
// lowest index that has it) and the sum of exp((x - largest) / T).  The sum
// decides whole numbers, so it is kept in 64 bits: every thread adds short
// f32 batches of exponentials (each within 2^-21 of its value) to a 64-bit
// sum.  verify_pick_kernel then takes a sequence per cluster: the parts of
// its rows are joined, each draft's p and q formed in 64 bits and compared
// with the given number, and one row -- the first refused, or the last -- is
// read again to sample the next token: the cluster's warps sum what is left
// of their equal parts of the vocabulary in 64 bits, every CTA finds the part
// in which the running sum passes the given number's share of the whole, and
// the warp that owns the part finds the lane's piece and the entry in it.
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

struct VerifyStat {
    double sum;  // of exp((x - max) / T) over the part; 0 where max is -inf
    float max;
    int32_t arg;  // the lowest index that has it
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
// T <= 0 and NaN: greedy (0).  Otherwise 1 / T, T held to where both are finite.
DF_DEV float inverse_temperature(const VerifyArgs& A, int s) {
    const float t = A.temperature != nullptr ? A.temperature[s] : 1.f;
    return t > 0.f ? 1.f / fminf(fmaxf(t, 1e-30f), 1e30f) : 0.f;
}
// exp(t * it), t <= 0: 2^(t c) with c = it log2(e) in two parts, so that the
// constant's rounding does not tilt the distribution; ex2 is within 2^-22.
struct ExpScale {
    float hi, lo;
};
// (a greedy sequence, it = 0, has no use for its sums: any scale)
DF_DEV ExpScale exp_scale(float it) {
    const double c = (double)(it > 0.f ? it : 1.f) * 1.4426950408889634074;
    const float hi = (float)c;
    return {hi, (float)(c - (double)hi)};
}
DF_DEV float exp_of(float t, ExpScale e) {
    const float z = fmaf(t, e.lo, t * e.hi);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(z));
    return z > -200.f ? y : 0.f;  // (t = -inf: z is -inf or NaN)
}
// x against the row's largest: 0 at it (an infinite one too); a NaN counts as -inf
DF_DEV float below(float x, float m) { return x == m ? 0.f : fmaxf(x, -INFINITY) - m; }

template <int DT>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<kF32> {
    static constexpr int N = 4;
    using T = float;
    DF_DEV static void get(const float* p, float (&x)[4]) {
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
    DF_DEV static void get(const uint16_t* p, float (&x)[8]) {
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

// A thread's (largest, its index, sum) of what it has seen.
struct Running {
    float m = -INFINITY;
    int arg = 0x7fffffff;
    double s = 0.0;
};
DF_DEV void join(Running& a, float m, int arg, double s, ExpScale e) {
    if (m > a.m) {
        a.s = s + a.s * (double)exp_of(a.m - m, e);  // (a.m = -inf: a.s is 0 and so is the factor)
        a.m = m;
        a.arg = arg;
    } else if (m == a.m) {
        a.s += s;
        a.arg = min(a.arg, arg);
    } else {
        a.s += s * (double)exp_of(m - a.m, e);
    }
}
template <int N>
DF_DEV void take(Running& r, const float (&x)[N], int i0, ExpScale e) {
    float m = fmaxf(x[0], -INFINITY);
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    if (m > r.m) {
        r.s = r.m == -INFINITY ? 0.0 : r.s * (double)exp_of(r.m - m, e);
        r.m = m;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (x[i] == m) r.arg = i0 + i;
    }
    if (r.m == -INFINITY) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += exp_of(below(x[i], r.m), e);
    r.s += (double)s;
}

// One part of one row.
template <int DT>
DF_DEV Running row_part(const typename Vec<DT>::T* row, int v0, int v1, ExpScale e) {
    using V = Vec<DT>;
    constexpr int N = V::N;
    Running r;
    // up to the next 16-byte boundary one by one, then vectors, then the rest
    const int mis = (int)((reinterpret_cast<uintptr_t>(row + v0) & 15) / sizeof(typename V::T));
    const int a = min(v1, v0 + (mis ? N - mis : 0)), nv = (v1 - a) / N, b = a + nv * N;
    float one[1];
    if ((int)threadIdx.x < a - v0) {
        one[0] = V::one(row + v0 + threadIdx.x);
        take<1>(r, one, v0 + threadIdx.x, e);
    }
    constexpr int U = 4;
    int i = threadIdx.x;
    for (; i + (U - 1) * kVsThreads < nv; i += U * kVsThreads) {
        float x[U][N];
#pragma unroll
        for (int k = 0; k < U; ++k) V::get(row + a + (i + k * kVsThreads) * N, x[k]);
#pragma unroll
        for (int k = 0; k < U; ++k) take<N>(r, x[k], a + (i + k * kVsThreads) * N, e);
    }
    for (; i < nv; i += kVsThreads) {
        float x[N];
        V::get(row + a + i * N, x);
        take<N>(r, x, a + i * N, e);
    }
    if ((int)threadIdx.x < v1 - b) {
        one[0] = V::one(row + b + threadIdx.x);
        take<1>(r, one, b + threadIdx.x, e);
    }
    return r;
}

__global__ void __launch_bounds__(kVsThreads) verify_stats_kernel(const __grid_constant__ VerifyParams P) {
    const VerifyArgs& A = P.A;
    __shared__ VerifyStat wst[kVsThreads / 32];
    const int part = blockIdx.x % P.parts, row = blockIdx.x / P.parts;
    const int nt = A.n_drafts + A.n_seqs;
    pdl_wait();
    pdl_trigger();
    const int s = row < nt ? verify_seq(A, row, 1) : verify_seq(A, row - nt, 0);
    if (s < 0) return;
    const float it = inverse_temperature(A, s);
    if (row >= nt && it == 0.f) return;  // a greedy sequence's drafter is not asked
    const ExpScale e = exp_scale(it);
    const int v0 = (int)((int64_t)A.vocab * part / P.parts), v1 = (int)((int64_t)A.vocab * (part + 1) / P.parts);
    Running r;
    if (row >= nt)
        r = row_part<kF32>(A.draft + (int64_t)(row - nt) * A.draft_stride, v0, v1, e);
    else if (A.target_dtype == kF32)
        r = row_part<kF32>(static_cast<const float*>(A.target) + (int64_t)row * A.target_stride, v0, v1, e);
    else if (A.target_dtype == kBF16)
        r = row_part<kBF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, e);
    else
        r = row_part<kF16>(static_cast<const uint16_t*>(A.target) + (int64_t)row * A.target_stride, v0, v1, e);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, r.m, o);
        const int arg = __shfl_xor_sync(0xffffffffu, r.arg, o);
        const double sum = __shfl_xor_sync(0xffffffffu, r.s, o);
        join(r, m, arg, sum, e);
    }
    if (lane == 0) wst[warp] = {r.s, r.m, r.arg};
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kVsThreads / 32; ++w) join(r, wst[w].max, wst[w].arg, wst[w].sum, e);
        P.stats[(int64_t)row * P.parts + part] = {r.s, r.m, r.arg};
    }
}

// A row's parts joined (warp-wide, every lane gets the answer).
DF_DEV Running row_stat(const VerifyParams& P, int64_t row, ExpScale e, int lane) {
    Running r;
    for (int i = lane; i < P.parts; i += 32) {
        const VerifyStat x = P.stats[row * P.parts + i];
        join(r, x.max, x.arg, x.sum, e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, r.m, o);
        const int arg = __shfl_xor_sync(0xffffffffu, r.arg, o);
        const double sum = __shfl_xor_sync(0xffffffffu, r.s, o);
        join(r, m, arg, sum, e);
    }
    return r;
}
DF_DEV float logit_at(const void* base, int dtype, int64_t i) {
    return dtype == kF32    ? Vec<kF32>::one(static_cast<const float*>(base) + i)
           : dtype == kBF16 ? Vec<kBF16>::one(static_cast<const uint16_t*>(base) + i)
                            : Vec<kF16>::one(static_cast<const uint16_t*>(base) + i);
}
// p(x) of one entry, in 64 bits.
DF_DEV double prob_at(float x, const Running& r, float it) {
    if (r.m == -INFINITY || !(x > -INFINITY)) return 0.0;
    return (x == r.m ? 1.0 : exp(((double)x - (double)r.m) * (double)it)) / r.s;
}

// What is left at one entry of the sampled row: mode 0 the target's
// probability (unnormalised), 1 with the draft taken out, 2 max(p - q, 0).
struct Left {
    const unsigned char* target;
    const float* draft;
    int dtype, mode, x;
    float tm, qm, tz, qz;  // the rows' largest logits, 1 / their sums
    ExpScale e;
    DF_DEV float at(int i) const {
        const float t = logit_at(target, dtype, i);
        float w = tm == -INFINITY ? 0.f : exp_of(below(t, tm), e);
        if (mode == 1) return i == x ? 0.f : w;
        if (mode == 2) {
            const float q = qm == -INFINITY ? 0.f : exp_of(below(__ldg(draft + i), qm), e) * qz;
            w = fmaxf(fmaf(w, tz, -q), 0.f);
        }
        return w;
    }
};

__global__ void __cluster_dims__(kVpCluster, 1, 1) __launch_bounds__(kVpThreads)
    verify_pick_kernel(const __grid_constant__ VerifyParams P) {
    const VerifyArgs& A = P.A;
    __shared__ int refused;
    __shared__ double part_sum[2][kVpWarps];  // (two passes at most: each has its own)
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), s = blockIdx.x / kVpCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) refused = 0x7fffffff;
    __syncthreads();
    pdl_wait();
    int a, b;
    draft_range(A, s, a, b);
    const int d = b - a;
    const float it = inverse_temperature(A, s);
    const ExpScale e = exp_scale(it);
    const bool drawn = A.draft != nullptr && it > 0.f;  // q is the drafter's distribution, not one token
    const int64_t nt = (int64_t)A.n_drafts + A.n_seqs;

    // every CTA of the cluster decides alike; the first one writes
    for (int i = warp; i < d; i += kVpWarps) {
        const int64_t row = (int64_t)a + s + i;
        const uint32_t x = A.draft_tok[a + i];
        const bool known = x < (uint32_t)A.vocab;
        const Running t = row_stat(P, row, e, lane);
        double p, q = 1.0;
        if (it > 0.f)
            p = known ? prob_at(logit_at(A.target, A.target_dtype, row * A.target_stride + x), t, it) : 0.0;
        else
            p = known && t.m > -INFINITY && t.arg == (int)x ? 1.0 : 0.0;
        if (drawn) {
            const Running g = row_stat(P, nt + a + i, e, lane);
            q = known ? prob_at(__ldg(A.draft + (int64_t)(a + i) * A.draft_stride + x), g, it) : 0.0;
        }
        if (lane == 0) {
            if (!((double)A.accept_u[a + i] * q < p)) atomicMin(&refused, i);
            // (q = 0: a draft the drafter could not make; kept when p is not 0)
            if (rank == 0 && A.prob != nullptr) A.prob[a + i] = (float)(p < q ? p / q : p > 0.0 ? 1.0 : 0.0);
        }
    }
    __syncthreads();
    const int acc = min(refused, d);
    const int64_t row = (int64_t)a + s + acc;
    const Running t = row_stat(P, row, e, lane);
    int token = t.m == -INFINITY ? -1 : t.arg;
    const int w = rank * kVpWarps + warp;  // this warp's part of the vocabulary
    bool writes = rank == 0 && threadIdx.x == 0;
    if (it > 0.f && t.m > -INFINITY) {
        Left L;
        L.target = static_cast<const unsigned char*>(A.target) + row * A.target_stride * (A.target_dtype == kF32 ? 4 : 2);
        L.draft = nullptr;
        L.dtype = A.target_dtype;
        L.e = e;
        L.tm = t.m;
        L.tz = (float)(1.0 / t.s);
        L.qm = L.qz = 0.f;
        L.x = -1;
        L.mode = 0;
        if (acc < d) {
            L.x = (int)min(A.draft_tok[a + acc], 0x7fffffffu);
            L.mode = 1;
            if (drawn) {
                const Running g = row_stat(P, nt + a + acc, e, lane);
                L.draft = A.draft + (int64_t)(a + acc) * A.draft_stride;
                L.mode = 2;
                L.qm = g.m;
                L.qz = g.m == -INFINITY ? 0.f : (float)(1.0 / g.s);
            }
        }
        const int v0 = (int)((int64_t)A.vocab * w / kVpParts), v1 = (int)((int64_t)A.vocab * (w + 1) / kVpParts);
        writes = false;
        for (int pass = 0; pass < 2; ++pass) {
            double mine = 0.0;
            for (int i = v0 + lane; i < v1; i += 4 * 32) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + 32 * k < v1) x += L.at(i + 32 * k);
                mine += (double)x;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
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
            const double want = (double)A.sample_u[s] * whole;
            // the first part whose running sum passes `want` (the last with any of it, should rounding
            // or a number of 1 leave none), and the sum before it
            int hit = 0x7fffffff, some = -1;
            double before = in - run, hit_before = 0.0;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                if (sum[k] > 0.0) {
                    some = lane * PL + k;
                    if (hit == 0x7fffffff && before + sum[k] > want) hit = lane * PL + k, hit_before = before;
                }
                before += sum[k];
            }
            const int first = (int)__reduce_min_sync(0xffffffffu, (unsigned)hit);
            const int last = __reduce_max_sync(0xffffffffu, some);
            const int owner = first != 0x7fffffff ? first : last;
            if (owner != w) break;
            double rest = first != 0x7fffffff
                              ? want - __shfl_sync(0xffffffffu, hit_before, owner / PL)
                              : INFINITY;
            // the part's lanes, a piece of neighbouring entries each, then the entries of one piece
            const int n = v1 - v0, per = (n + 31) / 32;
            int p0 = min(v0 + lane * per, v1), p1 = min(p0 + per, v1);
            double piece = 0.0;
            for (int i = p0; i < p1; ++i) piece += (double)L.at(i);
            for (int level = 0;; ++level) {
                double up = piece;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += y;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, piece > 0.0 && up > rest);
                const uint32_t any = __ballot_sync(0xffffffffu, piece > 0.0);
                // (no entry over it, by the rounding of another order of sums: the last that has any)
                const int l = over ? __ffs(over) - 1 : 31 - __clz(any);
                const int q0 = __shfl_sync(0xffffffffu, p0, l), q1 = __shfl_sync(0xffffffffu, p1, l);
                if (any == 0) break;
                if (q1 - q0 == 1) {
                    token = q0;
                    writes = lane == 0;
                    break;
                }
                if (over) rest -= __shfl_sync(0xffffffffu, up - piece, l);
                else rest = INFINITY;
                const int m = q1 - q0, pp = (m + 31) / 32;
                p0 = min(q0 + lane * pp, q1), p1 = min(p0 + pp, q1);
                piece = 0.0;
                for (int i = p0; i < p1; ++i) piece += (double)L.at(i);
            }
            break;
        }
    }
    if (writes) {
        A.accepted[s] = acc;
        A.next_tok[s] = token;
    }
    if (it > 0.f && t.m > -INFINITY) cl.sync();  // no CTA leaves while its sums may be read
}

// Parts of a row: enough CTAs for the card to stay busy with a few an SM, of at
// least a few KB of logits each.
static int verify_parts(int64_t rows, int64_t vocab, int num_sms) {
    const int64_t want = (16 * (int64_t)num_sms + rows - 1) / (rows > 0 ? rows : 1);
    const int64_t most = (vocab + 4095) / 4096;
    return (int)(want < 1 ? 1 : want > most ? most : want);
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
