// The attention weight that each cached key receives, for few rows (one token a
// sequence, or a drafted block): k_paged_weights.cu's sums on warp MMAs.
//
// A warp takes 32 keys on its own: S = K Q^T with keys as the 16 rows of
// m16n8k16 MMAs (the tile's operands stay in registers) and the queries that share the
// head, eight at a time, as their columns (in shared memory, in the order that the
// MMAs take them).  A key's weights then lie in four lanes, which add them up: no sum
// leaves the warp, one order, equal bits.  The line of work and its cut into shares
// are k_paged_attn.cu's, a unit being a (sequence, key/value head) with all its
// rows; each warp has its own ring of stages, filled by asynchronous copies.
//
// With one token a sequence the keys' bytes bound it (32 sequences of 1024 to 4096
// bf16 keys, 8 heads of 128: 33 us, 4.9 TB/s, where k_paged_weights.cu takes 40), with a
// block the MMAs and, over 4 bits, the conversions (16 rows of four query heads over
// 32768 keys: 22 us and 28; the MMAs alone, one of 16 x 8 x 16 every two clocks and SM, 7).  Rows beyond 64 go by in sets of 64, the CTA's
// warps in step (a sequence that has many more rows than the call's average); its tiles count once for each set in the
// line (400 rows and 31 single ones over 4096 keys each: 200 us; with tiles alike, a few CTAs had all of those rows' work, 1956).
//
// Keys that only some rows see, rows of lse -inf and columns without a row are
// left out of a tile's sums one by one.
#include <type_traits>

#include "kernels.cuh"
#include "paged_attn.cuh"

namespace dflash {

constexpr int kPfKeys = 32, kPfRows = 64;  // keys of a warp's stage, rows that shared memory holds at once
// tiles' time that a unit's end and the next one's beginning take
constexpr int kPfOver = 8;

struct PfArgs {
    PaArgs A;
    KeyWeights W;
    const float* lse;
    FastDiv by_group;
};

// CB: bits of a cache's element.  BF: 16-bit ones are bf16
template <int CB, int HD>
struct PfShape {
    static constexpr int W = CB == 16 ? 8 : 12, kThreads = W * 32;
    static constexpr int RB = HD * CB / 8, CH = RB / 16, SB = CB == 4 ? HD / 16 : 0;  // a row's bytes, chunks, block scales
    static constexpr int kCodes = kPfKeys * RB, kStage = kCodes + kPfKeys * SB;
    static constexpr int NST = (CB == 16 ? 3 : 4) * (128 / HD);
    static constexpr int kQueries = kPfRows * HD * 2;
    static constexpr size_t kSmem = (size_t)W * NST * kStage + kQueries;
    static_assert(kSmem <= 220 * 1024, "shared memory");
};
// byte offset of chunk c of row r, so that eight rows' chunks of one column sit in different banks
template <int CH>
DF_DEV uint32_t pf_off(int r, int c) {
    return (uint32_t)(r * CH * 16 + ((CH >= 8 ? c ^ (r & 7) : CH == 4 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4));
}
DF_DEV void pf_ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF>
DF_DEV void pf_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF, int CB, int HD>
__global__ void __launch_bounds__((PfShape<CB, HD>::kThreads), 1) paged_weights_few_kernel(const __grid_constant__ PfArgs P) {
    using S = PfShape<CB, HD>;
    constexpr int W = S::W, NST = S::NST, CH = S::CH, SB = S::SB, KS = HD / 16;  // MMAs along a row
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ uint32_t vbits[W][NST];  // a stage's held keys
    // a set's rows: exp2(s c + nl) of the keys from `see`.x to .y (none: a row that is not there, or of lse -inf)
    __shared__ __align__(8) float2 num[kPfRows];
    __shared__ __align__(8) int2 see[kPfRows];
    __shared__ int odd[2];  // whether a set has rows without keys; of every other set
    const PaArgs& A = P.A;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint32_t base = smem_addr(sm) + warp * NST * S::kStage;
    const uint32_t queries = smem_addr(sm) + W * NST * S::kStage;
    constexpr int kAll = 1 << 30;  // rows of a unit: all of a sequence's
    pdl_wait();
    pdl_trigger();

    int chunk;
    PaCur cur = pa_share<kPfKeys, false, kPfRows>(A, kAll, kPfOver, lane, chunk);
    if (cur.left <= 0) return;
    auto tiles_of = [&](const PaCur& c) { return pa_tiles<kPfRows>(A, c); };
    auto skip = [&](PaCur& c, int n) {
        c.left -= (n - 1) * pa_places<kPfRows>(A, c.q);
        c.tile += n - 1;
        pa_next<kPfKeys, false, kPfRows>(A, kAll, c);
    };

    // Rows 64 x .. of a unit to shared memory, in the MMAs' order: a warp takes eight rows, lane (gq, tq) of row gq the columns
    // in the order in which the codes of a key come.  Fetched into registers while the unit before goes on.
    static_assert(8 * W >= kPfRows, "a warp has eight rows at most");
    uint32_t w[2 * KS];
    float lse = 0.f;
    auto fetch = [&](const PaCur& c, int x) {
        const int all = c.q.rows * A.group, mm = x * kPfRows + 8 * warp + gq;
        if (8 * warp >= min(kPfRows, all - x * kPfRows)) return;
        const int i = div_by(P.by_group, mm), hq = c.u * A.group + mm - i * A.group;
        const bool in = mm < all;
        const unsigned char* p = A.q.p + (int64_t)(c.q.row0 + i) * A.q.rs + (int64_t)hq * A.q.hs;
        lse = in ? P.lse[(int64_t)(c.q.row0 + i) * A.q.heads + hq] : -INFINITY;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            // two pairs of MMA j
            const int c0 = CB == 16 ? 16 * j + 2 * tq : CB == 8 ? 16 * j + 4 * tq : 32 * (j >> 1) + 8 * tq + 4 * (j & 1);
            const int c1 = c0 + (CB == 16 ? 8 : 2);
            w[2 * j] = in ? *reinterpret_cast<const uint32_t*>(p + 2 * c0) : 0u;
            w[2 * j + 1] = in ? *reinterpret_cast<const uint32_t*>(p + 2 * c1) : 0u;
        }
    };
    int turn = 0;
    auto place = [&](float ks, int rows, const PaCur& c, int x) {
        __syncthreads();  // (the set before has been read)
        turn ^= 1;
        if (8 * warp < rows) {
            float rf = 1.f;
            if (CB < 16 && A.q.dtype == kBF16) {
                // a row times 2^-x, its largest element in [1, 2): what f16 cannot hold of it then is under 2^-25 of that
                float mx = 0.f, down = 1.f;
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j) {
                    const float2 f = unpack2<true>(w[j]);
                    mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (mx > 0.f && mx < INFINITY) {
                    const int e = min(max(ilogbf(mx), -120), 120);
                    down = ldexpf(1.f, -e);
                    rf = ldexpf(1.f, e);
                }
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j) {
                    const float2 f = unpack2<true>(w[j]);
                    w[j] = pack2<false>(f.x * down, f.y * down);
                }
            }
#pragma unroll
            for (int j = 0; j < KS / 2; ++j)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(queries + (uint32_t)((warp * (KS / 2) + j) * 512 + lane * 16)),
                             "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                             : "memory");
            if (tq == 0) {
                const int m = 8 * warp + gq;
                const bool none = lse == -INFINITY;
                const int pos = c.q.p0 + div_by(P.by_group, x * kPfRows + m);
                num[m] = make_float2(fminf(fmaxf(ks * rf, 1e-37f), 3e38f), none ? 0.f : -1.4426950408889634f * lse);
                see[m] = none ? make_int2(0, -1) : make_int2(A.window > 0 ? max(pos - A.window + 1, 0) : 0, pos);
                if (none) odd[turn] = 1;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) odd[turn ^ 1] = 0;
    };
    fetch(cur, 0);

    // ---------------------------------------------------------------- copies
    // Lane l holds the place of a stage's key l; `ahead` belongs to the stage to copy next.
    struct Look {
        int id, slot, h;
    };
    PaCur put = cur;
    int put_n = tiles_of(put), put_t = warp;  // this warp's tile among the unit's
    auto settle = [&]() {                     // to the next unit with a tile for this warp
        while (put.left > 0 && put_t >= put_n) {
            skip(put, put_n);
            put_n = tiles_of(put);
            put_t = warp;
        }
    };
    auto look = [&]() -> Look {
        Look k{-1, 0, put.u};
        const int key = put.q.lo + (put.tile + put_t) * kPfKeys + lane;
        if (key < put.q.hi) k.id = page_entry(A.R, put.s, key, k.slot);
        return k;
    };
    Look ahead{-1, 0, 0};
    if (put_t >= put_n) settle();
    if (put.left > 0) ahead = look();
    int stage_put = 0;
    auto copy = [&]() {
        if (put.left > 0) {
            const uint32_t st = base + stage_put * S::kStage;
            const bool held = page_held(ahead.id, A.C.n_pages);
            const unsigned char *kp = A.q.p, *kb = A.q.p;  // (nothing is read)
            if (held) {
                kp = A.C.k + ahead.id * A.C.ks[0] + ahead.slot * A.C.ks[1] + ahead.h * A.C.ks[2];
                if constexpr (CB == 4) kb = A.C.kb + ahead.id * A.C.kbs[0] + ahead.slot * A.C.kbs[1] + ahead.h * A.C.kbs[2];
            }
            const uint32_t bits = __ballot_sync(0xffffffffu, held);
            if (lane == 0) vbits[warp][stage_put] = bits;
            put_t += W;
            if (put_t >= put_n) settle();
            if (put.left > 0) ahead = look();
            constexpr int RPI = 32 / CH;  // rows a copy instruction covers
#pragma unroll
            for (int i = 0; i < kPfKeys / RPI; ++i) {
                const int r = i * RPI + lane / CH;
                const uint64_t k = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(kp), r);
                cp16(st + pf_off<CH>(r, lane % CH), reinterpret_cast<const unsigned char*>(k) + 16 * (lane % CH), (bits >> r & 1u) << 4);
            }
            if constexpr (SB == 8) cp8(st + S::kCodes + lane * SB, kb, held ? 8 : 0);
            if constexpr (SB == 4) cp4(st + S::kCodes + lane * SB, kb, held ? 4 : 0);
            stage_put = stage_put + 1 == NST ? 0 : stage_put + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) copy();

    const int lrow = ((lane >> 3) & 1) * 8 + (lane & 7), lch = lane >> 4;  // this lane's row and chunk of an ldmatrix
    int stage = 0;
    if (threadIdx.x < 2) odd[threadIdx.x] = 0;
    while (cur.left > 0) {
        // ------------------------------------------------------------ a unit
        const PaCur unit = cur;
        const PaSeq& sq = unit.q;
        const int tiles = tiles_of(unit), h = unit.u, all = sq.rows * A.group, sets = (all + kPfRows - 1) / kPfRows;
        const float ks = A.scale_log2 * (CB < 16 && A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f);
        float* const weights = P.W.p + (int64_t)unit.s * P.W.ss + (int64_t)h * P.W.hs;
        if (sets == 1) place(ks, min(kPfRows, all), unit, 0);
        const PaCur next = [&] {
            PaCur x = cur;
            skip(x, tiles);
            return x;
        }();
        if (next.left > 0) fetch(next, 0);
        // keys up to `clear` and from `wtop` on are seen by every row of the sequence
        const int clear = sq.p0, wtop = A.window > 0 ? sq.p0 + sq.rows - A.window : 0;

        // (where rows come in sets, every warp goes through every round)
#pragma unroll 1
        for (int t0 = 0; t0 < tiles; t0 += W) {
            const int t = t0 + warp;
            const bool mine = t < tiles;
            if (!mine && sets == 1) break;
            uint32_t a[2][KS][4];
            uint32_t bits = 0;
            int kfirst = 0;
            float old = 0.f;
            if (mine) {
                cp_wait<NST - 2>();
                __syncwarp();
                copy();
                const uint32_t sk = base + stage * S::kStage;
                bits = vbits[warp][stage];
                kfirst = sq.lo + (unit.tile + t) * kPfKeys;
                stage = stage + 1 == NST ? 0 : stage + 1;
                const int key = kfirst + 16 * (tq >> 1) + 8 * (tq & 1) + gq;  // the key whose sum this lane writes
                if (key < sq.hi && key < sq.p0) old = weights[key];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (CB == 16) {
#pragma unroll
                        for (int j = 0; j < KS; ++j) pf_ldsm(a[k][j], sk + pf_off<CH>(16 * k + lrow, 2 * j + lch));
                    } else if constexpr (CB == 8) {
#pragma unroll
                        for (int j = 0; j < KS; j += 2) {
                            uint32_t r[4];  // codes of keys gq and gq + 8, chunks j and j + 1
                            pf_ldsm(r, sk + pf_off<CH>(16 * k + lrow, j + lch));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                e4m3x4_f16x4(r[2 * i], a[k][j + i][0], a[k][j + i][2]);
                                e4m3x4_f16x4(r[2 * i + 1], a[k][j + i][1], a[k][j + i][3]);
                            }
                        }
                    } else {
                        uint32_t s[2][2];  // the keys' scales of this lane's block of chunks 0, 1 and 2, 3
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t lo, hi;
                            const uint32_t at = sk + S::kCodes + (16 * k + gq + 8 * e) * SB;
                            if constexpr (SB == 8)
                                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(at));
                            else {
                                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(at));
                                hi = lo;
                            }
                            e4m3x4_f16x4(__byte_perm(lo, hi, tq & 2 ? (SB == 8 ? 0x7531 : 0x3131) : (SB == 8 ? 0x6420 : 0x2020)), s[e][0], s[e][1]);
                        }
#pragma unroll
                        for (int j = 0; j < CH; j += 2) {
                            uint32_t r[4];
                            pf_ldsm(r, sk + pf_off<CH>(16 * k + lrow, j + lch));
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    uint32_t y[4];
                                    e2m1x8_f16x8(r[2 * i + e], y);
                                    const uint32_t f = __byte_perm(s[e][j >> 1], 0, i ? 0x3232 : 0x1010);
                                    a[k][2 * (j + i)][e] = mul_f16x2(y[0], f);
                                    a[k][2 * (j + i)][2 + e] = mul_f16x2(y[1], f);
                                    a[k][2 * (j + i) + 1][e] = mul_f16x2(y[2], f);
                                    a[k][2 * (j + i) + 1][2 + e] = mul_f16x2(y[3], f);
                                }
                        }
                    }
                }
            }
            float sum[2][2] = {};
#pragma unroll 1
            for (int x = 0; x < sets; ++x) {
                if (sets > 1) {
                    fetch(unit, x);
                    place(ks, min(kPfRows, all - x * kPfRows), unit, x);
                }
                if (bits == 0) continue;
                const int rows = min(kPfRows, all - x * kPfRows);
                const bool plain = kfirst + kPfKeys - 1 <= clear && kfirst >= wtop && odd[turn] == 0;
                // eights of rows n .. n + N - 1: two at a time, whose chains of MMAs go on side by side
                auto eights = [&](int n, auto count) {
                    constexpr int N = decltype(count)::value;
                    float sc[N][2][4] = {};
#pragma unroll
                    for (int j = 0; j < KS / 2; ++j)
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            uint32_t b[4];
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                                         : "r"(queries + (uint32_t)(((n + i) * (KS / 2) + j) * 512 + lane * 16)));
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                pf_mma<BF>(sc[i][k], a[k][2 * j], b[0], b[1]);
                                pf_mma<BF>(sc[i][k], a[k][2 * j + 1], b[2], b[3]);
                            }
                        }
#pragma unroll
                    for (int i = 0; i < N; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * (n + i) + 2 * tq + e;
                            const float2 f = num[row];
                            const int2 v = plain ? make_int2(0, 0) : see[row];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    float z = fmaf(sc[i][k][2 * y + e], f.x, f.y);
                                    if (!plain) {
                                        const int key = kfirst + 16 * k + 8 * y + gq;
                                        z = key >= v.x && key <= v.y ? z : -INFINITY;
                                    }
                                    sum[k][y] += pa_exp2(z);
                                }
                        }
                };
                int n = 0;
#pragma unroll 1
                for (; 8 * n + 8 < rows; n += 2) eights(n, std::integral_constant<int, 2>());
                if (8 * n < rows) eights(n, std::integral_constant<int, 1>());
            }
            if (mine) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        sum[k][y] += __shfl_xor_sync(0xffffffffu, sum[k][y], 1);
                        sum[k][y] += __shfl_xor_sync(0xffffffffu, sum[k][y], 2);
                    }
                const int place = 16 * (tq >> 1) + 8 * (tq & 1) + gq, key = kfirst + place;
                const float got = tq & 2 ? (tq & 1 ? sum[1][1] : sum[1][0]) : (tq & 1 ? sum[0][1] : sum[0][0]);
                if (key < sq.hi && (bits >> place & 1u)) weights[key] = old + got;
            }
        }
        if (sets > 1 && next.left > 0) fetch(next, 0);  // (the last set's rows were fetched over it)
        cur = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool BF, int CB, int HD>
static int pf_launch(const PfArgs& P, int num_sms, cudaStream_t st) {
    using S = PfShape<CB, HD>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_weights_few_kernel<BF, CB, HD>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(S::kThreads), S::kSmem, st, P);
}
template <int HD>
static int pf_type(const PfArgs& P, int cd, int num_sms, cudaStream_t st) {
    return cd == kBF16   ? pf_launch<true, 16, HD>(P, num_sms, st)
           : cd == kF16  ? pf_launch<false, 16, HD>(P, num_sms, st)
           : cd == kE4M3 ? pf_launch<false, 8, HD>(P, num_sms, st)
                         : pf_launch<false, 4, HD>(P, num_sms, st);
}
int paged_key_weights_few(const PaArgs& A, const KeyWeights& W, const float* lse, int cache_dtype, int hd, int num_sms,
                          cudaStream_t st) {
    PfArgs P{A, W, lse, fast_div(A.group)};
    return hd == 64 ? pf_type<64>(P, cache_dtype, num_sms, st) : pf_type<128>(P, cache_dtype, num_sms, st);
}

}  // namespace dflash
