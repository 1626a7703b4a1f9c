// Attention of a pass's new rows (one token a sequence, or a drafted block)
// over a paged key/value cache.
//
// The query heads that share a key/value head share its reads: the unit of
// work is a (sequence, key/value head, tile of MT rows of the sequence's rows x
// group heads), its keys go by in tiles of 128, and softmax runs online in one
// pass (a running reference m and sum l a row, the output rescaled when m
// moves).  The memory it cannot do without is each key and value once.
//
// Work split.  All tiles of all units, in order, are one line that the CTAs
// (one an SM) cut into equal parts: a CTA takes whole units, and the head and
// tail of units that its neighbours share.  The line's length comes from
// kv_len on the device, so sequences of any mix of lengths are balanced and a
// captured call follows the lengths of its replay.  A unit that one CTA holds
// whole is written out at once; a shared one leaves (m, l, O) per part in the
// workspace, and a second small kernel joins the parts.
//
// In a CTA, each of 8 warps takes 16 of a tile's 128 keys against the unit's (at
// most 16) rows on its own: m16n8k16 MMAs (scores from K by ldmatrix, P from
// the scores' registers, values by transposed ldmatrix), its own reference and
// sum, its own ring of stages filled by 16-byte asynchronous copies.  The warps
// meet once a unit, to join.  The page of a key is looked up a stage before
// its copy.  Units of more rows go to the tcgen05 kernel (k_paged_attn_tc.cu).
//
// Memory bound: 16 streams of 32768 keys x 8 heads of 128 in bf16, one token of
// 32 heads each, 320 us = 6.7 TB/s (99 % of a copy; with an e4m3 cache 245 us, the
// conversions' and MMAs' latency in 8 warps); 32 streams of 1100 to 4000 keys 59 us
// (79 %: ramps, two to three unit ends an SM, the join); one stream of 2048: 9.2 us,
// of two launches' and one tile's latency.
//
// Masking.  Keys that no row may see (past the end, pages not held) are not
// read: their slots are zero-filled and a bit mask sends their scores to -inf.
// A key that some rows see and others do not (the new rows among themselves, a
// window's edge) is masked per row; P is then 0 there, and 0 times an infinite
// or NaN value would not be, so such stages look for non-finite values and,
// where there are any, add P V row by row with the hidden keys left out.  What
// an infinite value that every row sees makes of the products, the join's kernel
// mends (pa_odd_row).
#include "kernels.cuh"
#include "paged_attn.cuh"

namespace dflash {

constexpr int kPaThreads = 256, kPaWarps = 8;
// tiles' time that a unit's end and the next one's beginning take (32 streams of one token: 0 61.0 us, 1 58.5, 2 58.3)
constexpr int kPaOver = 2;

DF_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DF_DEV void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF>
DF_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// BF: MMAs and cache in bf16 (else f16).  E8: an e4m3 cache; its codes become
// f16 exactly, and a query row is brought into f16 by a power of two.
// P goes through the MMAs as hi + lo pairs, so that they add no rounding of
// their own to the output's: two more MMAs a value fragment, which the memory
// leaves time for.
constexpr int kPaM = 16, kPaKeys = 16;  // rows of a unit's tile, keys of a warp's stage
template <bool BF, bool E8, int HD>
struct PaShape {
    static constexpr int RB = HD * (E8 ? 1 : 2);  // bytes of a key row
    static constexpr int CH = RB / 16;            // its 16-byte chunks
    static constexpr int kStage = 2 * kPaKeys * RB;  // a warp's stage: keys, then values
    static constexpr int kRound = kPaWarps * kStage;
    static constexpr int NST = 196608 / kRound < 6 ? 196608 / kRound : 6;
    static constexpr int NF = HD / 8;  // output fragments of a warp
    static constexpr int kMerge = kPaWarps / 2 * kPaM * HD * 4;
    static constexpr size_t kSmem = (size_t)NST * kRound + kMerge;
};

// byte offset of chunk c of key row r, so that eight rows' chunks of one column sit in different banks
template <int CH>
DF_DEV uint32_t pa_off(int r, int c) {
    return (uint32_t)(r * CH * 16 + ((CH >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
}

template <bool BF, bool E8, int HD>
__global__ void __launch_bounds__(kPaThreads, 1) paged_attn_kernel(const __grid_constant__ PaArgs A) {
    using S = PaShape<BF, E8, HD>;
    constexpr int NST = S::NST, CH = S::CH, MT = kPaM, NF = S::NF, KG = kPaWarps;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ uint32_t vbits[kPaWarps][NST];  // a stage's valid keys
    __shared__ float2 ml[KG][MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint32_t base = smem_addr(sm) + warp * NST * S::kStage;
    pdl_wait();
    pdl_trigger();

    int chunk;
    PaCur cur = pa_share(A, MT, kPaOver, lane, chunk);
    if (threadIdx.x == 0) A.ws_join[blockIdx.x].last = -1, A.ws_odd[blockIdx.x] = 0;
    if (cur.left <= 0) return;

    // ---------------------------------------------------------------- copies
    // Lanes 0-15 hold the places of a stage's 16 key rows of this warp, lanes
    // 16-31 those of its value rows; `ahead` belongs to the stage to copy next.
    // (the page's number alone: a pointer made of it here would wait for it)
    struct Look {
        int id, slot, h;
    };
    PaCur put = cur;
    Look ahead{-1, 0, 0};
    auto look = [&](const PaCur& c) -> Look {
        Look k{-1, 0, c.u % A.C.kv_heads};
        const int key = c.q.lo + c.tile * kPaTile + warp * kPaKeys + (lane & 15);
        if (key < c.q.hi) k.id = page_entry(A.R, c.s, key, k.slot);
        return k;
    };
    const unsigned char* tensor = lane < 16 ? A.C.k : A.C.v;
    const int64_t sp = lane < 16 ? A.C.ks[0] : A.C.vs[0], ss = lane < 16 ? A.C.ks[1] : A.C.vs[1],
                  sh = lane < 16 ? A.C.ks[2] : A.C.vs[2];
    if (put.left > 0) ahead = look(put);
    int stage_put = 0;
    auto copy = [&]() {
        if (put.left > 0) {
            const uint32_t st = base + stage_put * S::kStage;
            const unsigned char* now =
                page_held(ahead.id, A.C.n_pages) ? tensor + ahead.id * sp + ahead.slot * ss + ahead.h * sh : nullptr;
            const uint32_t bits = __ballot_sync(0xffffffffu, now != nullptr) & 0xffffu;
            if (lane == 0) vbits[warp][stage_put] = bits;
            pa_next(A, MT, put);
            if (put.left > 0) ahead = look(put);
            constexpr int RPI = 32 / CH;  // rows a copy instruction covers
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
                const int r = i * RPI + lane / CH, c = lane % CH;
                const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(now), r);
                const uint32_t dst = st + (r >> 4) * (kPaKeys * S::RB) + pa_off<CH>(r & 15, c);
                const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * c : A.q.p;  // (nothing is read)
                cp16(dst, src, p ? 16 : 0);
            }
            stage_put = stage_put + 1 == NST ? 0 : stage_put + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) copy();

    int stage = 0;
    while (cur.left > 0) {
        // ------------------------------------------------------------ a unit
        const PaCur unit = cur;
        const PaSeq& sq = unit.q;
        const int u = cur.u, tile0 = cur.tile;
        const int h = u % A.C.kv_heads, rt = u / A.C.kv_heads;
        const int mvalid = min(MT, sq.rows * A.group - rt * MT);
        // this thread's rows gq and gq + 8: positions (-1: no row)
        int pos[2], wlo[2];
        uint32_t qf[HD / 16][4];
        float rf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = gq + 8 * e;
            const bool in = m < mvalid;
            const int mm = rt * MT + m, r = mm / A.group, hq = h * A.group + mm % A.group;
            pos[e] = in ? sq.p0 + r : -1;
            wlo[e] = A.window > 0 ? pos[e] - A.window + 1 : 0;
            const unsigned char* p = A.q.p + (int64_t)(sq.row0 + r) * A.q.rs + (int64_t)hq * A.q.hs;
            rf[e] = 1.f;
            if constexpr (!E8) {
#pragma unroll
                for (int j = 0; j < HD / 16; ++j) {
                    qf[j][e] = in ? *reinterpret_cast<const uint32_t*>(p + (16 * j + 2 * tq) * 2) : 0u;
                    qf[j][2 + e] = in ? *reinterpret_cast<const uint32_t*>(p + (16 * j + 8 + 2 * tq) * 2) : 0u;
                }
            } else {
                // columns 16 j + 4 tq + {0, 1, 2, 3}: the order in which the codes come (below)
                uint2 w[HD / 16];
                float mx = 0.f;
                const bool qb = A.q.dtype == kBF16;
#pragma unroll
                for (int j = 0; j < HD / 16; ++j) {
                    w[j] = in ? *reinterpret_cast<const uint2*>(p + (16 * j + 4 * tq) * 2) : make_uint2(0u, 0u);
                    if (qb) {
                        const float2 a = unpack2<true>(w[j].x), b = unpack2<true>(w[j].y);
                        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // a bf16 row times 2^-x, its largest element in [1, 2): what f16 cannot hold of it then
                // is under 2^-25 of that element
                float down = 1.f;
                if (qb && mx > 0.f && mx < INFINITY) {
                    const int x = min(max(ilogbf(mx), -120), 120);
                    down = ldexpf(1.f, -x);
                    rf[e] = ldexpf(1.f, x);
                }
#pragma unroll
                for (int j = 0; j < HD / 16; ++j) {
                    if (qb) {
                        const float2 a = unpack2<true>(w[j].x), b = unpack2<true>(w[j].y);
                        qf[j][e] = pack2<false>(a.x * down, a.y * down);
                        qf[j][2 + e] = pack2<false>(b.x * down, b.y * down);
                    } else {
                        qf[j][e] = w[j].x;
                        qf[j][2 + e] = w[j].y;
                    }
                }
            }
        }
        // scores in log2 units: (S rf) * c; never 0, so that -inf stays -inf
        float c[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float ks = E8 && A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f;
            c[e] = fminf(fmaxf(A.scale_log2 * ks * rf[e], 1e-37f), 3e38f);
        }
        // positions between which every row of the unit's tile sees every key
        const int pmin = sq.p0 + (rt * MT) / A.group;
        const int pmax = sq.p0 + (rt * MT + mvalid - 1) / A.group;
        const int wtop = A.window > 0 ? pmax - A.window + 1 : 0;

        float o[NF][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[f][e] = 0.f;

        bool last_tile;
        int done = tile0;  // tiles of the unit behind us
        do {
            cp_wait<NST - 2>();
            __syncwarp();
            copy();
            const uint32_t st = base + stage * S::kStage;
            const uint32_t sv = st + kPaKeys * S::RB;
            const int kfirst = sq.lo + cur.tile * kPaTile + warp * kPaKeys, klast = kfirst + kPaKeys - 1;
            const uint32_t bits = vbits[warp][stage];
            if (bits != 0) {
                constexpr int NT = kPaKeys / 8;
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
                if constexpr (!E8) {
#pragma unroll
                    for (int j = 0; j < HD / 32; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t b[4];
                            ldsm4(b, st + pa_off<CH>(n * 8 + (lane & 7), 4 * j + (lane >> 3)));
                            mma16816<BF>(sc[n], qf[2 * j], b[0], b[1]);
                            mma16816<BF>(sc[n], qf[2 * j + 1], b[2], b[3]);
                        }
                } else {
                    // a chunk is 16 codes; lane 4 gq + tq receives codes 4 tq .. 4 tq + 3 of key gq
#pragma unroll
                    for (int j = 0; j < HD / 64; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t b[4];
                            ldsm4(b, st + pa_off<CH>(n * 8 + (lane & 7), 4 * j + (lane >> 3)));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t b0, b1;
                                e4m3x4_f16x4(b[i], b0, b1);
                                mma16816<false>(sc[n], qf[4 * j + i], b0, b1);
                            }
                        }
                }
                const bool full = bits == 0xffffu && klast <= pmin && kfirst >= wtop;
                // bit 4 n + e of `hid`: this thread's score sc[n][e] is not in its row's view
                uint32_t hid = 0;
                if (!full) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int kk = n * 8 + 2 * tq + (e & 1), key = kfirst + kk;
                            const bool see = ((bits >> kk) & 1u) && key <= pos[e >> 1] && key >= wlo[e >> 1];
                            if (!see) {
                                sc[n][e] = -INFINITY;
                                hid |= 1u << (4 * n + e);
                            }
                        }
                }
                float mx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(sc[0][2 * e], sc[0][2 * e + 1]);
#pragma unroll
                    for (int n = 1; n < NT; ++n) mx[e] = fmaxf(mx[e], fmaxf(sc[n][2 * e], sc[n][2 * e + 1]));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                    mx[e] *= c[e];
                }
                constexpr float under = kPaUnder<BF && !E8>;
                const bool move = mx[0] > m[0] + (kPaLazy + under) || mx[1] > m[1] + (kPaLazy + under);
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float to = mx[e] > m[e] + (kPaLazy + under) ? mx[e] - under : m[e];
                        const float f = to == m[e] ? 1.f : pa_exp2(m[e] - to);
                        m[e] = to;
                        l[e] *= f;
#pragma unroll
                        for (int i = 0; i < NF; ++i) {
                            o[i][2 * e] *= f;
                            o[i][2 * e + 1] *= f;
                        }
                    }
                }
                const float mr[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[n][e] = pa_exp2(fmaf(sc[n][e], c[e >> 1], -mr[e >> 1]));
                        l[e >> 1] += sc[n][e];
                    }
                // keys that some row of the tile sees and another does not: are their values finite?
                bool plain = true;
                if (!full && (klast > pmin || kfirst < wtop)) {
                    uint32_t bad = 0;
                    for (int i = lane; i < kPaKeys * CH; i += 32) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(sv + pa_off<CH>(i / CH, i % CH)));
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if constexpr (E8) {
                                // only S.1111.111 is not finite
                                const uint32_t y = (w[x] & 0x7f7f7f7fu) + 0x01010101u;
                                bad |= y & 0x80808080u;
                            } else {
                                constexpr uint32_t ex = BF ? 0x7f80u : 0x7c00u;
                                bad |= (w[x] & ex) == ex;
                                bad |= ((w[x] >> 16) & ex) == ex;
                            }
                        }
                    }
                    plain = !__any_sync(0xffffffffu, bad != 0);
                }
                if (plain) {
                    uint32_t ph[4], pl[4];
                    constexpr bool PB = BF && !E8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = sc[i >> 1][2 * (i & 1)], y = sc[i >> 1][2 * (i & 1) + 1];
                        ph[i] = pack2<PB>(x, y);
                        const float2 r = unpack2<PB>(ph[i]);
                        pl[i] = pack2<PB>(x - r.x, y - r.y);
                    }
#pragma unroll
                    for (int j = 0; j < CH / 2; ++j) {
                        uint32_t b[4];
                        ldsm4t(b, sv + pa_off<CH>(lane & 15, 2 * j + (lane >> 4)));
                        if constexpr (!E8) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                mma16816<BF>(o[2 * j + i], ph, b[2 * i], b[2 * i + 1]);
                                mma16816<BF>(o[2 * j + i], pl, b[2 * i], b[2 * i + 1]);
                            }
                        } else {
                            // a register: two neighbouring columns of keys 2 tq, 2 tq + 1 -> even
                            // columns to fragment 2 ch, odd ones to 2 ch + 1 (chunk ch)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x0 = __byte_perm(b[2 * i], 0, 0x3120),
                                               x1 = __byte_perm(b[2 * i + 1], 0, 0x3120);
                                uint32_t e0, e1, d0, d1;
                                e4m3x4_f16x4(x0, e0, d0);
                                e4m3x4_f16x4(x1, e1, d1);
                                const int f = 2 * (2 * j + i);
                                mma16816<false>(o[f], ph, e0, e1);
                                mma16816<false>(o[f + 1], ph, d0, d1);
                                mma16816<false>(o[f], pl, e0, e1);
                                mma16816<false>(o[f + 1], pl, d0, d1);
                            }
                        }
                    }
                } else {
                    // key by key, the hidden ones left out
#pragma unroll 1
                    for (int kk = 0; kk < kPaKeys; ++kk) {
                        const int n = kk >> 3, src = (lane & ~3) | ((kk & 7) >> 1);
                        float p[2];
                        bool out[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = 0.f;
#pragma unroll
                            for (int i = 0; i < NT; ++i)
                                if (i == n) x = (kk & 1) ? sc[i][2 * e + 1] : sc[i][2 * e];
                            p[e] = __shfl_sync(0xffffffffu, x, src);
                            const uint32_t hb = __shfl_sync(0xffffffffu, hid, src);
                            out[e] = (hb >> (4 * n + 2 * e + (kk & 1))) & 1u;
                        }
#pragma unroll
                        for (int f = 0; f < NF; ++f)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                // the column of this thread's o[f][y] and o[f][2 + y]
                                const int col = E8 ? 16 * (f >> 1) + 4 * tq + 2 * y + (f & 1) : 8 * f + 2 * tq + y;
                                float val;
                                const uint32_t at = sv + pa_off<CH>(kk, col * (E8 ? 1 : 2) / 16) +
                                                    (col * (E8 ? 1 : 2)) % 16;
                                if constexpr (E8) {
                                    uint32_t w;
                                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w) : "r"(at));
                                    val = unpack2<false>(e4m3x2_f16x2(w)).x;
                                } else {
                                    uint16_t w;
                                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at));
                                    val = unpack2<BF>(w).x;
                                }
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!out[e]) o[f][2 * e + y] = fmaf(p[e], val, o[f][2 * e + y]);
                            }
                    }
                }
            }
            stage = stage + 1 == NST ? 0 : stage + 1;
            last_tile = ++done == sq.ntiles;
            pa_next(A, MT, cur);
        } while (!last_tile && cur.left > 0);

        // ------------------------------------------------------------ the unit's end
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }
        const bool whole = tile0 == 0 && last_tile;
        if (!whole && tile0 == 0 && threadIdx.x == 0)
            A.ws_join[blockIdx.x] = pa_join_entry(unit, rt, MT, mvalid, h, sq.ntiles - done, chunk);
        // a part of a shared unit: its start goes to the CTA's second slot, any other part to the first
        const int part = blockIdx.x * 2 + (tile0 == 0 ? 1 : 0);
        float big[2];
        {
            if (tq == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) ml[warp][gq + 8 * e] = make_float2(m[e], l[e]);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = gq + 8 * e;
                big[e] = -INFINITY;
#pragma unroll
                for (int g = 0; g < KG; ++g) big[e] = fmaxf(big[e], ml[g][r].x);
                float sum = 0.f;
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    const float2 x = ml[g][r];
                    sum += x.x == -INFINITY ? x.y : x.y * pa_exp2(x.x - big[e]);  // (a NaN sum without a maximum stays)
                }
                const float f = m[e] == -INFINITY ? 1.f : pa_exp2(m[e] - big[e]);
                l[e] = sum;
                m[e] = big[e];
#pragma unroll
                for (int i = 0; i < NF; ++i) {
                    o[i][2 * e] *= f;
                    o[i][2 * e + 1] *= f;
                }
            }
            // the upper half of the groups hand their sums to the lower half
            float* mg = reinterpret_cast<float*>(sm + (size_t)NST * S::kRound);
            constexpr int H = KG / 2;
            auto at = [&](int g, int i) { return mg + ((size_t)g * (NF * 4) + i) * 32 + lane; };
            if (warp >= H) {
#pragma unroll
                for (int i = 0; i < NF * 4; ++i) *at(warp - H, i) = o[i / 4][i % 4];
            }
            __syncthreads();
            if (warp < H) {
#pragma unroll
                for (int i = 0; i < NF * 4; ++i) o[i / 4][i % 4] += *at(warp, i);
            }
            if (warp > 0 && warp < H) {
#pragma unroll
                for (int i = 0; i < NF * 4; ++i) *at(warp, i) = o[i / 4][i % 4];
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int g = 1; g < H; ++g)
#pragma unroll
                    for (int i = 0; i < NF * 4; ++i) o[i / 4][i % 4] += *at(g, i);
            }
        }
        if (warp == 0) {
            const float vs = E8 && A.C.v_scale != nullptr ? A.C.v_scale[h] : 1.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int mrow = gq + 8 * e;
                if (mrow >= mvalid) continue;
                if (whole) {
                    const int mm = rt * MT + mrow, r = sq.row0 + mm / A.group, hq = h * A.group + mm % A.group;
                    const float inv = l[e] == 0.f ? 0.f : vs / l[e];
                    unsigned char* p = A.out.p + (int64_t)r * A.out.rs + (int64_t)hq * A.out.hs;
                    const bool ob = A.out.dtype == kBF16;
                    bool odd = false;
#pragma unroll
                    for (int f = 0; f < NF; f += E8 ? 2 : 1) {
                        auto w2 = [&](int col, float x, float y) {
                            *reinterpret_cast<uint32_t*>(p + col * 2) =
                                ob ? pack2<true>(x * inv, y * inv) : pack2<false>(x * inv, y * inv);
                            if constexpr (!E8) odd |= x != x || y != y;
                        };
                        if constexpr (E8) {
                            w2(8 * f + 4 * tq, o[f][2 * e], o[f + 1][2 * e]);
                            w2(8 * f + 4 * tq + 2, o[f][2 * e + 1], o[f + 1][2 * e + 1]);
                        } else {
                            w2(8 * f + 2 * tq, o[f][2 * e], o[f][2 * e + 1]);
                        }
                    }
                    if (!E8 && odd && pa_weighs(l[e])) {  // (columns of the other lanes' too: they wrote NaN, or will mark it)
                        pa_mark_odd<BF>(p, HD);
                        A.ws_odd[blockIdx.x] = 1;
                    }
                    if (A.lse != nullptr && tq == 0)
                        A.lse[(int64_t)r * A.q.heads + hq] =
                            l[e] == 0.f ? -INFINITY : (m[e] == -INFINITY ? l[e] : (m[e] + log2f(l[e])) * 0.69314718056f);
                } else {
                    float* p = A.ws_o + ((int64_t)part * MT + mrow) * HD;
#pragma unroll
                    for (int f = 0; f < NF; f += E8 ? 2 : 1) {
                        if constexpr (E8)
                            *reinterpret_cast<float4*>(p + 8 * f + 4 * tq) =
                                make_float4(o[f][2 * e], o[f + 1][2 * e], o[f][2 * e + 1], o[f + 1][2 * e + 1]);
                        else
                            *reinterpret_cast<float2*>(p + 8 * f + 2 * tq) = make_float2(o[f][2 * e], o[f][2 * e + 1]);
                    }
                    if (tq == 0) A.ws_ml[(int64_t)part * MT + mrow] = make_float2(m[e], l[e]);
                }
            }
        }
    }
}

// Row r, head hq of the output: NaN that is kept apart becomes the sum of the column's values that are not finite over
// the keys in the row's view.  By a warp; in little code, which all calls carry and few run (with its loops unrolled and a
// form for each type it took 6 us of a call's 40, one block over 32768 keys, though nothing of it ran).
// `mine`: this warp has joined the row; else rows that are joined are left alone, which their own warps may not have
// written yet (what the buffer held before may look like that NaN).
template <int HD>
DF_DEV void pa_odd_row(const PaArgs& A, int r, int hq, bool mine) {
    constexpr int V = HD / 32;  // columns a lane
    const int lane = threadIdx.x & 31, h = hq / A.group;
    const bool bf = A.out.dtype == kBF16;
    const uint32_t top = bf ? 0x7f807f80u : 0x7c007c00u, mark = bf ? kPaOdd<true> : kPaOdd<false>;
    uint16_t* out = reinterpret_cast<uint16_t*>(A.out.p + (int64_t)r * A.out.rs + (int64_t)hq * A.out.hs) + V * lane;
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) which |= (uint32_t)(out[i] == mark) << i;
    if (!__any_sync(0xffffffffu, which)) return;
    const int s = seq_of(A.R, r);
    if (s < 0) return;
    int a, b;
    rows_of(A.R, s, a, b);
    if (!mine) {
        const int mm = (r - a) * A.group + hq % A.group;
        bool joined = false;
#pragma unroll 1
        for (int c = lane; c < (int)gridDim.x; c += 32) {
            const PaJoin e = A.ws_join[c];
            joined |= e.last > c && e.seq == s && e.head == h && mm >= e.m0 && mm - e.m0 < e.rows;
        }
        if (__any_sync(0xffffffffu, joined)) return;
    }
    const int pos = pa_seq(A, s, a, b, kPaM).p0 + r - a;
    float sum[V] = {};
#pragma unroll 1
    for (int j0 = A.window > 0 ? max(0, pos - A.window + 1) : 0; j0 <= pos && j0 < A.R.cap; j0 += 32) {
        int slot = 0;
        const int64_t page = j0 + lane <= pos ? page_of(A.R, A.C.n_pages, s, j0 + lane, slot) : -1;
        const int64_t at = page < 0 ? -1 : page * A.C.vs[0] + slot * A.C.vs[1] + h * A.C.vs[2];
        const int64_t key = page * A.C.ks[0] + slot * A.C.ks[1] + h * A.C.ks[2];
        bool odd = false;
        if (page >= 0) {
#pragma unroll 2
            for (int c = 0; c < HD / 2; ++c) {
                const uint32_t x = ~reinterpret_cast<const uint32_t*>(A.C.v + at)[c] & top;
                odd |= (x & 0xffffu) == 0 || x < 0x10000u;
            }
        }
#pragma unroll 1
        for (uint32_t found = __ballot_sync(0xffffffffu, odd); found != 0; found &= found - 1) {
            const int l = __ffs(found) - 1;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(A.C.v + __shfl_sync(0xffffffffu, at, l)) + V * lane;
            const uint16_t* k = reinterpret_cast<const uint16_t*>(A.C.k + __shfl_sync(0xffffffffu, key, l)) + V * lane;
            // (the row's weights are finite: with a key that is not, the score was -inf)
            bool fine = true;
#pragma unroll
            for (int i = 0; i < V; ++i) fine &= (~k[i] & top & 0xffffu) != 0;
            const float times = __all_sync(0xffffffffu, fine) ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((~v[i] & top & 0xffffu) == 0)
                    sum[i] += times * (v[i] & ~top & 0x7fffu ? NAN : v[i] & 0x8000u ? -INFINITY : INFINITY);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((which >> i) & 1u)
            out[i] = (uint16_t)(sum[i] == 0.f || sum[i] != sum[i] ? 0x7fffu : (top & 0xffffu) | (sum[i] < 0.f ? 0x8000u : 0u));
}
// The shared units' parts joined: CTA (c, y) takes rows 16 y .. of the unit that
// starts in share c and ends in another, a warp a row.
template <int HD>
__global__ void __launch_bounds__(kPaThreads) paged_join_kernel(const __grid_constant__ PaArgs A, int mt, int e8) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int odd = A.ws_odd[blockIdx.x];
    bool any = false;
    const PaJoin e = A.ws_join[blockIdx.x];
    const int c0 = blockIdx.x, c1 = e.last, h = e.head;
    if (c1 > c0) {
#pragma unroll 1
    for (int mrow = 16 * blockIdx.y + warp; mrow < min(e.rows, 16 * (int)blockIdx.y + 16); mrow += kPaWarps) {
    const int mm = e.m0 + mrow, row = e.row0 + mm / A.group, hq = h * A.group + mm % A.group;
    constexpr int V = HD / 32;  // columns a lane
    float m = -INFINITY, l = 0.f, o[V] = {};
    // parts in order, 32 references and sums at a time, 8 outputs in flight (16 are more code: 40.3 -> 42.6 us, one block
    // over 32768 keys)
    for (int b = c0; b <= c1; b += 32) {
        const int n = min(32, c1 - b + 1);
        float2 x = make_float2(-INFINITY, 0.f);
        auto slot = [&](int c) { return (int64_t)(c * 2 + (c == c0 ? 1 : 0)) * mt + mrow; };
        if (lane < n) x = A.ws_ml[slot(b + lane)];
        constexpr int U = 8;
        float y[U][V];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (k0 + k < n) {
                    const float* p = A.ws_o + slot(b + k0 + k) * HD + V * lane;
                    if constexpr (V == 4) {
                        const float4 q = *reinterpret_cast<const float4*>(p);
                        y[k][0] = q.x, y[k][1] = q.y, y[k][2] = q.z, y[k][3] = q.w;
                    } else {
                        const float2 q = *reinterpret_cast<const float2*>(p);
                        y[k][0] = q.x, y[k][1] = q.y;
                    }
                }
        };
        load(0);
        const float to = fmaxf(m, warp_max(x.x));
        const float fm = m == to ? 1.f : pa_exp2(m - to);
        const float f = x.x == -INFINITY ? 1.f : pa_exp2(x.x - to);  // (without a maximum the sums are 0 or NaN)
        m = to;
        l = l * fm + warp_sum(x.y * f);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= fm;
        for (int k0 = 0; k0 < n; k0 += U) {
            if (k0 > 0) load(k0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const float w = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
                if (k0 + k < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = fmaf(w, y[k][i], o[i]);
                }
            }
        }
    }
    const float inv = l == 0.f ? 0.f : (e8 && A.C.v_scale != nullptr ? A.C.v_scale[h] : 1.f) / l;
    unsigned char* p = A.out.p + (int64_t)row * A.out.rs + (int64_t)hq * A.out.hs + V * lane * 2;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint32_t*>(p + 2 * i) = A.out.dtype == kBF16 ? pack2<true>(o[i] * inv, o[i + 1] * inv)
                                                                       : pack2<false>(o[i] * inv, o[i + 1] * inv);
    if (A.lse != nullptr && lane == 0)
        A.lse[(int64_t)row * A.q.heads + hq] =
            l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + log2f(l)) * 0.69314718056f);
    if (!e8 && pa_weighs(l)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (o[i] != o[i]) {
                reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(A.out.dtype == kBF16 ? kPaOdd<true> : kPaOdd<false>);
                any = true;
            }
    }
    }
    }
    // this warp's joined rows with NaN that is kept apart; then, where the share's whole units have some, all of the call's
    // rows, dealt out over the warps of all such shares
    any = __any_sync(0xffffffffu, any);
    if (!any && odd == 0) return;
    uint32_t shares = 0, before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < (int)gridDim.x; c0 += 32) {
        const uint32_t w = __ballot_sync(0xffffffffu, c0 + lane < (int)gridDim.x && A.ws_odd[c0 + lane] != 0);
        shares += __popc(w);
        before += __popc(c0 + 32 <= (int)blockIdx.x ? w : c0 > (int)blockIdx.x ? 0u : w & ((1u << (blockIdx.x - c0)) - 1));
    }
    const uint32_t joined = any ? min(16, e.rows - 16 * (int)blockIdx.y) : 0,
                   all = odd != 0 ? (uint32_t)A.R.n_rows * A.q.heads : 0,  // (under 2^31: check_heads)
                   by = shares * gridDim.y * kPaWarps;
    uint32_t i = warp;
    bool mine = true;
#pragma unroll 1
    for (;;) {
        if (mine && i >= joined) {
            mine = false;
            i = (before * gridDim.y + blockIdx.y) * kPaWarps + warp;
        }
        if (!mine && i >= all) break;
        // rows of a unit are group by group, rows of the call heads by heads
        const uint32_t per = mine ? A.group : A.q.heads, at = mine ? e.m0 + 16 * blockIdx.y + i : i, r = at / per;
        pa_odd_row<HD>(A, (int)r + (mine ? e.row0 : 0), (int)(at - r * per) + (mine ? h * A.group : 0), mine);
        i += mine ? kPaWarps : by;
    }
}

// Rows a unit's tile holds, by what a sequence of average length brings: 16 on
// the warp MMAs; beyond that the tcgen05 kernel's 64 or 128.  (A warp-MMA
// kernel of 32 rows took 71.7 us where the tcgen05 kernel's 64 take 67.4, 32
// sequences of 8 rows x 4 heads, and 12.6 against 14.7 us on one sequence of
// 2048 keys; with 16 rows, 32 sequences, the warp MMAs take 58 us, tcgen05 64.
// 64 rows in a tile of 128: 41.0 for 40.1 us, one block over 32768 keys.)
static int pa_tile_rows(int n_seqs, int64_t n_rows, int group) {
    const int64_t per = n_seqs > 0 ? (n_rows + n_seqs - 1) / n_seqs : 0;
    const int64_t m = per * group;
    return m <= kPaM ? kPaM : m <= 64 ? 64 : 128;
}

int64_t paged_attention_workspace(int hd, int n_seqs, int64_t n_rows, int heads, int kv_heads, int num_sms) {
    const int64_t mt = pa_tile_rows(n_seqs, n_rows, heads / kv_heads);
    return num_sms * (2 * mt * (hd * 4 + 8) + (int64_t)sizeof(PaJoin) + (int64_t)sizeof(int32_t));
}

template <bool BF, bool E8, int HD>
static int pa_launch(const PaArgs& A, int num_sms, cudaStream_t st) {
    using S = PaShape<BF, E8, HD>;
    // the limit is a device's own: one record each
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_attn_kernel<BF, E8, HD>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(kPaThreads), S::kSmem, st, A);
}
template <int HD>
static int pa_type(const PaArgs& A, int cache_dtype, int num_sms, cudaStream_t st) {
    return cache_dtype == kBF16  ? pa_launch<true, false, HD>(A, num_sms, st)
           : cache_dtype == kF16 ? pa_launch<false, false, HD>(A, num_sms, st)
                                 : pa_launch<false, true, HD>(A, num_sms, st);
}

int paged_attention(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                    const HeadRows& out, float* lse, float scale, int window, void* ws, int num_sms, cudaStream_t st) {
    PaArgs A{};
    A.C = C, A.R = R, A.q = q, A.out = out, A.lse = lse, A.window = window;
    A.scale_log2 = scale * 1.4426950408889634f;
    A.group = q.heads / C.kv_heads;
    const int mt = pa_tile_rows(R.n_seqs, R.n_rows, A.group);
    A.ws_o = static_cast<float*>(ws);
    A.ws_ml = reinterpret_cast<float2*>(A.ws_o + 2 * (int64_t)num_sms * mt * hd);
    A.ws_join = reinterpret_cast<PaJoin*>(A.ws_ml + 2 * (int64_t)num_sms * mt);
    A.ws_odd = reinterpret_cast<int32_t*>(A.ws_join + num_sms);
    const int e = mt > kPaM ? paged_attention_tc(A, cache_dtype, hd, mt, num_sms, st)
                  : hd == 64 ? pa_type<64>(A, cache_dtype, num_sms, st)
                             : pa_type<128>(A, cache_dtype, num_sms, st);
    if (e != 0) return e;
    const dim3 grid(num_sms, mt / 16);
    const int e8 = cache_dtype == kE4M3;
    return hd == 64 ? (int)launch(paged_join_kernel<64>, grid, dim3(kPaThreads), 0, st, A, mt, e8)
                    : (int)launch(paged_join_kernel<128>, grid, dim3(kPaThreads), 0, st, A, mt, e8);
}

}  // namespace dflash
