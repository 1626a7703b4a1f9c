// Attention of few rows (one token a sequence, mostly) over a 4-bit paged cache.
// The line of work, its cut into equal shares and the join of shared units are
// k_paged_attn.cu's, in tiles of 32 keys: a tile is one warp's, and a CTA's warps
// deal a unit's tiles out among them.
//
// A byte of this cache is two elements, so the elements' way through the
// registers is what costs: at the memory's rate an SM would have 42 of them a
// clock.  The products are therefore the other way round than
// k_paged_attn.cu's: S^T = K Q^T and O^T = V^T P^T, with keys (or a value's
// columns) as the 16 rows of an m16n8k16 MMA and the unit's rows as its 8
// columns: half the MMAs, half the exponentials and half the output registers
// where a unit has up to 8 rows (two such halves where it has up to 16).  Codes come by
// ldmatrix, four bytes a lane: of a key row those are eight columns, two MMAs'
// operands in any order that the queries follow; of values, transposed in
// two-byte units, four columns of two keys each.  A code is converted by the
// hardware (e2m1 pairs -> f16 pairs) and multiplied by its block's scale in
// f16, exactly.  The weights go from rows of S^T to columns of P^T by movmatrix.
//
// P is one f16 for bf16 outputs, off by 2^-11 of each key's part at most, an
// eighth of the output's own 2^-8, and a hi + lo pair for f16 outputs.  (A pair for
// bf16 outputs, too: 16 sequences of 32768 keys are then 1.664e-3 of the outputs' norm
// from 64 bits, the rounding to bf16, for 1.677e-3, and take 158 us for 146; 32 tokens 43
// for 41; 32 sequences of 4 rows 66 for 57.)
//
// With enough units, or keys beyond what L2 holds, a unit is all (up to eight) heads
// of a key, each with its own warps: the heads' bytes share their lines (kP4Far).
//
// 16 sequences of 32768 keys, 8 heads of 128: 146 us, 4.15 TB/s (61 % of a copy); 32 of
// 1024 to 4096 keys, four query heads each: 41 us.  Bound by issue: a tile's chain of some
// 900 instructions in the four warps of an SM quarter, 0.67 of them a clock (half of them the
// ALU pipe's; twice the value MMAs for fewer of those took 148 us), and by a unit's
// ends (about 4 us, one or two a CTA with the shorter ones).  One sequence of 2048
// keys: 9.2 us, launch, share, first tiles and join one after the other.
//
// Masking: as in k_paged_attn.cu.  Codes are finite, so a value that is not can
// only be a block scale of NaN: where rows see different keys, such tiles add P V key by
// key with the hidden ones left out.
#include "kernels.cuh"
#include "paged_attn.cuh"

namespace dflash {

// tiles' time that a unit's end and the next one's beginning take
constexpr int kP4Over = 8;
// Bytes of keys and values from which on a unit is the heads of a key together, about twice what L2 holds: a head's 64
// bytes of a key and 8 of its scales share their lines with the other heads', and heads that go by at their own times
// fetch those again (16 sequences of 32768 keys read 1530 MB for 605: 228 -> 146 us; of 8192 keys, which L2 holds: 53 and 54).
// It is so, too, where each CTA would begin a unit of its own and end others (32 sequences of 4096 keys 60 -> 53 us, 128 of
// 512 52 -> 41); with few units all CTAs have parts of every head, and the join takes longer (one sequence of 131072 keys
// 46 us head by head, 71 together).
constexpr double kP4Far = 256e6;

DF_DEV void p4_ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DF_DEV void p4_ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DF_DEV void p4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
DF_DEV uint32_t p4_transposed(uint32_t x) {  // an 8 x 8 matrix of 16-bit elements, two of a row a lane
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// a pair times the lower (upper) half of another
DF_DEV uint32_t p4_times(uint32_t a, uint32_t s, bool upper) {
    const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&s);
    const __half2 z = __hmul2(x, upper ? __high2half2(y) : __low2half2(y));
    return *reinterpret_cast<const uint32_t*>(&z);
}
template <int N>
struct P4Words {
    uint32_t w[N];
};
// N words of a row's (or two rows') block scales
template <int N>
DF_DEV P4Words<N> p4_scales(uint32_t addr) {
    P4Words<N> r;
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(addr));
    return r;
}

// PAIR: weights as a hi + lo pair; NT: eights of a unit's rows
template <bool PAIR, int HD, int NT>
struct P4Shape {
    static constexpr int W = NT == 1 ? 16 : 12, kThreads = W * 32;
    static constexpr int RB = HD / 2, CH = RB / 16, SB = HD / 16;  // a row's bytes, 16-byte chunks, block scales
    static constexpr int kCodes = kP4Keys * RB, kScales = kP4Keys * SB;
    static constexpr int kStage = 2 * (kCodes + kScales);  // a warp's stage: keys, values, their scales
    static constexpr int NST = HD == 64 ? 4 : 2;
    static constexpr int kRow = HD + 4;  // f32 of a row's sums on their way through shared memory (four apart: other banks)
    static constexpr int kMerge = W * 8 * NT * kRow * 4;
    static constexpr size_t kSmem = (size_t)W * NST * kStage + kMerge;
};
// byte offset of chunk c of code row r, so that eight rows' chunks of one column sit in different banks
template <int CH>
DF_DEV uint32_t p4_off(int r, int c) {
    return (uint32_t)(r * CH * 16 + ((CH == 4 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4));
}

// TOGETHER: a unit may be several heads
template <bool PAIR, int HD, int NT, bool TOGETHER>
__global__ void __launch_bounds__((P4Shape<PAIR, HD, NT>::kThreads), 1)
    paged_attn4_kernel(const __grid_constant__ PaArgs A) {
    using S = P4Shape<PAIR, HD, NT>;
    constexpr int W = S::W, NST = S::NST, CH = S::CH, SB = S::SB, MT = 8 * NT, SW = SB / 4;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ uint32_t vbits[W][NST];  // a stage's held keys
    __shared__ float2 ml[2][W][MT], sums[W][MT];  // the warps' references and sums at a unit's end, and those to one reference
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint32_t base = smem_addr(sm) + warp * NST * S::kStage;
    float* merge = reinterpret_cast<float*>(sm + (size_t)W * NST * S::kStage);
    pdl_wait();
    pdl_trigger();

    int chunk, heads = 1;
    PaCur cur = pa_share<kP4Keys, TOGETHER>(A, MT, kP4Over, lane, chunk, (int)(kP4Far / S::kStage), &heads);
    const int G = TOGETHER ? heads : 1;
    // heads hg G .. of a unit u = (row tile, hg): this warp's among them, and its turn among the P warps of that head
    const int groups = A.C.kv_heads / G, P = W / G, wg = warp % G, wk = warp / G;
    if (threadIdx.x == 0) A.ws_join[blockIdx.x].last = -1, A.ws_odd[blockIdx.x] = 0;
    if (cur.left <= 0) return;
    // the part of a unit that the share holds, and the unit after it
    auto tiles_of = [](const PaCur& c) { return min(c.q.ntiles - c.tile, c.left); };
    auto skip = [&](PaCur& c, int n) {
        c.left -= n - 1;
        c.tile += n - 1;
        pa_next<kP4Keys, TOGETHER>(A, MT, c, G);
    };

    // Queries of row gq (and gq + 8), columns 32 j + 8 tq .., as they are: fetched before the first copies, and as the unit
    // before ends.
    uint4 qf[NT][CH];
    auto fetch = [&](const PaCur& c) {
        const int h = c.u % groups * G + wg, rt = c.u / groups;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int mm = rt * MT + gq + 8 * n, r = mm / A.group, hq = h * A.group + mm - r * A.group;
            const unsigned char* p = A.q.p + (int64_t)(c.q.row0 + r) * A.q.rs + (int64_t)hq * A.q.hs + 16 * tq;
#pragma unroll
            for (int j = 0; j < CH; ++j)
                qf[n][j] = mm < c.q.rows * A.group ? *reinterpret_cast<const uint4*>(p + 64 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    fetch(cur);

    // ---------------------------------------------------------------- copies
    // Lane l holds the place of a stage's key l; `ahead` belongs to the stage to copy next.
    struct Look {
        int id, slot, h;
    };
    PaCur put = cur;
    int put_n = tiles_of(put), put_t = wk;  // this warp's tile among the unit's
    auto settle = [&]() {  // to the next unit with a tile for this warp
        while (put.left > 0 && put_t >= put_n) {
            skip(put, put_n);
            put_n = tiles_of(put);
            put_t = wk;
        }
    };
    auto look = [&]() -> Look {
        Look k{-1, 0, put.u % groups * G + wg};
        const int key = put.q.lo + (put.tile + put_t) * kP4Keys + lane;
        if (key < put.q.hi) k.id = page_entry(A.R, put.s, key, k.slot);
        return k;
    };
    Look ahead{-1, 0, 0};
    settle();
    if (put.left > 0) ahead = look();
    int stage_put = 0;
    auto copy = [&]() {
        if (put.left > 0) {
            const uint32_t st = base + stage_put * S::kStage;
            const bool held = page_held(ahead.id, A.C.n_pages);
            // (strides of a 4-bit cache are below 2^31)
            auto at = [&](unsigned char* p, const int64_t* strides) -> const unsigned char* {
                const unsigned char* x = p + (int64_t)ahead.id * (int)strides[0] + (int64_t)ahead.slot * (int)strides[1] +
                                         (int64_t)ahead.h * (int)strides[2];
                return held ? x : A.q.p;  // (nothing is read)
            };
            const unsigned char *kp = at(A.C.k, A.C.ks), *vp = at(A.C.v, A.C.vs), *kb = at(A.C.kb, A.C.kbs), *vb = at(A.C.vb, A.C.vbs);
            const uint32_t bits = __ballot_sync(0xffffffffu, held);
            if (lane == 0) vbits[warp][stage_put] = bits;
            put_t += P;
            if (put_t >= put_n) settle();
            if (put.left > 0) ahead = look();
            constexpr int RPI = 32 / CH;  // rows a copy instruction covers
            const uint32_t to = st + p4_off<CH>(lane / CH, lane % CH);
            const uint32_t mine = bits >> (lane / CH);
#pragma unroll
            for (int i = 0; i < kP4Keys / RPI; ++i) {
                const uint64_t k = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(kp), i * RPI + lane / CH);
                const uint64_t v = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(vp), i * RPI + lane / CH);
                const uint32_t bytes = (mine >> (i * RPI) & 1u) << 4;
                cp16(to + i * RPI * S::RB, reinterpret_cast<const unsigned char*>(k) + 16 * (lane % CH), bytes);
                cp16(to + i * RPI * S::RB + S::kCodes, reinterpret_cast<const unsigned char*>(v) + 16 * (lane % CH), bytes);
            }
            if constexpr (SB == 8) {
                cp8(st + 2 * S::kCodes + lane * SB, kb, held ? 8 : 0);
                cp8(st + 2 * S::kCodes + S::kScales + lane * SB, vb, held ? 8 : 0);
            } else {
                cp4(st + 2 * S::kCodes + lane * SB, kb, held ? 4 : 0);
                cp4(st + 2 * S::kCodes + S::kScales + lane * SB, vb, held ? 4 : 0);
            }
            stage_put = stage_put + 1 == NST ? 0 : stage_put + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) copy();

    // this lane's row and chunk of an ldmatrix of 16 rows by two chunks (the next two: 32 bytes on, as an exclusive or)
    const uint32_t mat = p4_off<CH>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4);
    int stage = 0, turn = 0;
    while (cur.left > 0) {
        // ------------------------------------------------------------ a unit
        const PaCur unit = cur;
        const PaSeq& sq = unit.q;
        const int tiles = tiles_of(unit);
        const int h0 = unit.u % groups * G, h = h0 + wg, rt = unit.u / groups;
        const int mvalid = min(MT, sq.rows * A.group - rt * MT);
        // the queries in f16, by a power of two where they are bf16
        float c[NT][2];  // scores of rows 2 tq, 2 tq + 1 in log2 units: S c; never 0, so that -inf stays -inf
        const float ks = A.scale_log2 * (A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float rf = 1.f;
            if (A.q.dtype == kBF16) {
                // a row times 2^-x, its largest element in [1, 2): what f16 cannot hold of it then is under 2^-25 of that
                uint32_t(&w)[4 * CH] = *reinterpret_cast<uint32_t(*)[4 * CH]>(qf[n]);
                float mx = 0.f, down = 1.f;
#pragma unroll
                for (int i = 0; i < 4 * CH; ++i) {
                    const float2 f = unpack2<true>(w[i]);
                    mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (mx > 0.f && mx < INFINITY) {
                    const int x = min(max(ilogbf(mx), -120), 120);
                    down = ldexpf(1.f, -x);
                    rf = ldexpf(1.f, x);
                }
#pragma unroll
                for (int i = 0; i < 4 * CH; ++i) {
                    const float2 f = unpack2<true>(w[i]);
                    w[i] = pack2<false>(f.x * down, f.y * down);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                c[n][e] = fminf(fmaxf(ks * __shfl_sync(0xffffffffu, rf, 4 * (2 * tq + e)), 1e-37f), 3e38f);
        }
        // positions between which every row of the unit's tile sees every key
        const int pmin = sq.p0 + (rt * MT) / A.group;
        const int pmax = sq.p0 + (rt * MT + mvalid - 1) / A.group;
        const int wtop = A.window > 0 ? pmax - A.window + 1 : 0;

        float o[NT][CH][2][4];  // columns 32 c + 4 gq + 2 t + {0, 1} of rows 8 n + 2 tq + {0, 1}
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) m[n][e] = -INFINITY, l[n][e] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][j][t][e] = 0.f;
        }

#pragma unroll 1
        for (int t = wk; t < tiles; t += P) {
            cp_wait<NST - 2>();
            __syncwarp();
            copy();
            const uint32_t sk = base + stage * S::kStage, sv = sk + S::kCodes, bk = sk + 2 * S::kCodes, bv = bk + S::kScales;
            const uint32_t bits = vbits[warp][stage];
            const int kfirst = sq.lo + (unit.tile + t) * kP4Keys, klast = kfirst + kP4Keys - 1;
            stage = stage + 1 == NST ? 0 : stage + 1;
            if (bits == 0) continue;
            // ---- scores: keys 16 k + gq (+ 8) of rows 2 tq, 2 tq + 1
            float sc[2][NT][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[k][n][e] = 0.f;
                uint32_t s[2][2];  // the keys' scales of this lane's block of chunks 0, 1 and 2, 3
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const auto x = p4_scales<SW>(bk + (16 * k + gq + 8 * e) * SB);
                    const uint32_t y = __byte_perm(x.w[0], x.w[SW - 1], tq & 2 ? (SW == 2 ? 0x7531 : 0x3131) : (SW == 2 ? 0x6420 : 0x2020));
                    e4m3x4_f16x4(y, s[e][0], s[e][1]);
                }
#pragma unroll
                for (int j = 0; j < CH; j += 2) {
                    uint32_t r[4];
                    p4_ldsm(r, (sk + 16 * k * S::RB + mat) ^ (16 * j));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t a[4], b[4];
                        e2m1x8_f16x8(r[2 * i], a);
                        e2m1x8_f16x8(r[2 * i + 1], b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = p4_times(a[e], s[0][j >> 1], i), b[e] = p4_times(b[e], s[1][j >> 1], i);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4& q = qf[n][j + i];
                            p4_mma(sc[k][n], a[0], b[0], a[1], b[1], q.x, q.y);
                            p4_mma(sc[k][n], a[2], b[2], a[3], b[3], q.z, q.w);
                        }
                    }
                }
            }
            // ---- softmax
            const bool full = bits == 0xffffffffu && klast <= pmin && kfirst >= wtop;
            uint32_t hid = 0;  // bit 8 n + 4 k + e: sc[k][n][e] is not in its row's view
            if (!full) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * n + 2 * tq + e, mm = rt * MT + row;
                        const int pos = row < mvalid ? sq.p0 + mm / A.group : -1;
                        const int wlo = A.window > 0 ? pos - A.window + 1 : 0;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int kk = 16 * k + gq + 8 * y, key = kfirst + kk;
                                if (!((bits >> kk) & 1u) || key > pos || key < wlo) {
                                    sc[k][n][2 * y + e] = -INFINITY;
                                    hid |= 1u << (8 * n + 4 * k + 2 * y + e);
                                }
                            }
                    }
            }
            constexpr float over = kPaLazy + kPaUnder<false>;
            float mx[NT][2];
            bool move = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[n][e] = fmaxf(fmaxf(sc[0][n][e], sc[0][n][2 + e]), fmaxf(sc[1][n][e], sc[1][n][2 + e])) * c[n][e];
                    move |= mx[n][e] > m[n][e] + over;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = mx[n][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        const float to = x > m[n][e] + over ? x - kPaUnder<false> : m[n][e];
                        const float f = to == m[n][e] ? 1.f : pa_exp2(m[n][e] - to);
                        m[n][e] = to;
                        l[n][e] *= f;
#pragma unroll
                        for (int j = 0; j < CH; ++j)
#pragma unroll
                            for (int t2 = 0; t2 < 2; ++t2) o[n][j][t2][e] *= f, o[n][j][t2][2 + e] *= f;
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mr = m[n][e] == -INFINITY ? 0.f : m[n][e];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float& p = sc[k][n][2 * y + e];
                            p = pa_exp2(fmaf(p, c[n][e], -mr));
                            l[n][e] += p;
                        }
                }
            // keys that some row of the tile sees and another does not: are their values' scales numbers?
            if (!full && (klast > pmin || kfirst < wtop)) {
                const auto x = p4_scales<SW>(bv + lane * SB);
                bool nan = false;
#pragma unroll
                for (int i = 0; i < SW; ++i) nan |= (((x.w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                if (__any_sync(0xffffffffu, nan)) {
                    // key by key, the hidden ones left out
#pragma unroll 1
                    for (int kk = 0; kk < kP4Keys; ++kk) {
                        const int src = 4 * (kk & 7) + tq, at = 4 * (kk >> 4) + 2 * ((kk >> 3) & 1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float p[2] = {0.f, 0.f};
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int y = 0; y < 2; ++y)
                                    if (4 * k + 2 * y == at) p[0] = sc[k][n][2 * y], p[1] = sc[k][n][2 * y + 1];
                            p[0] = __shfl_sync(0xffffffffu, p[0], src);
                            p[1] = __shfl_sync(0xffffffffu, p[1], src);
                            const uint32_t hb = __shfl_sync(0xffffffffu, hid, src) >> (8 * n + at);
#pragma unroll
                            for (int j = 0; j < CH; ++j) {
                                uint32_t w, b;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w) : "r"(sv + p4_off<CH>(kk, j) + 2 * gq));
                                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(bv + kk * SB + 2 * j + (gq >> 2)));
                                uint32_t v[4];
                                e2m1x8_f16x8(w, v);
                                const float s = unpack2<false>(e4m3x2_f16x2(b)).x;
#pragma unroll
                                for (int t2 = 0; t2 < 2; ++t2) {
                                    const float2 f = unpack2<false>(v[t2]);
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (!((hb >> e) & 1u)) {
                                            o[n][j][t2][e] = fmaf(p[e], f.x * s, o[n][j][t2][e]);
                                            o[n][j][t2][2 + e] = fmaf(p[e], f.y * s, o[n][j][t2][2 + e]);
                                        }
                                }
                            }
                        }
                    }
                    continue;
                }
            }
            // ---- values: O^T += V^T P^T
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t hi = pack2<false>(sc[k][n][2 * y], sc[k][n][2 * y + 1]);
                        ph[n][y] = p4_transposed(hi);
                        if constexpr (PAIR) {
                            const float2 f = unpack2<false>(hi);
                            pl[n][y] = p4_transposed(pack2<false>(sc[k][n][2 * y] - f.x, sc[k][n][2 * y + 1] - f.y));
                        }
                    }
                uint32_t s[2][4];  // scales of keys 2 tq, 2 tq + 1 (and 8 on), of this lane's block of each chunk
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const auto x = p4_scales<2 * SW>(bv + (16 * k + 8 * y + 2 * tq) * SB);
                    const uint32_t pick = gq & 4 ? (SW == 2 ? 0x7531 : 0x3131) : (SW == 2 ? 0x6420 : 0x2020);
                    const uint32_t k0 = __byte_perm(x.w[0], x.w[SW - 1], pick), k1 = __byte_perm(x.w[SW], x.w[2 * SW - 1], pick);
                    e4m3x4_f16x4(__byte_perm(k0, k1, 0x5140), s[y][0], s[y][1]);
                    if constexpr (CH == 4) e4m3x4_f16x4(__byte_perm(k0, k1, 0x7362), s[y][2], s[y][3]);
                }
#pragma unroll
                for (int j = 0; j < CH; j += 2) {
                    uint32_t r[4];
                    p4_ldsm_t(r, (sv + 16 * k * S::RB + mat) ^ (16 * j));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t v[2][4];  // columns 0 .. 3 of keys 2 tq, 2 tq + 1 and of keys 8 on
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t x[4];
                            e2m1x8_f16x8(r[2 * i + y], x);
                            const uint32_t sy = s[y][j + i];
                            v[y][0] = mul_f16x2(__byte_perm(x[0], x[2], 0x5410), sy);
                            v[y][1] = mul_f16x2(__byte_perm(x[0], x[2], 0x7632), sy);
                            v[y][2] = mul_f16x2(__byte_perm(x[1], x[3], 0x5410), sy);
                            v[y][3] = mul_f16x2(__byte_perm(x[1], x[3], 0x7632), sy);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int t2 = 0; t2 < 2; ++t2) {
                                p4_mma(o[n][j + i][t2], v[0][2 * t2], v[0][2 * t2 + 1], v[1][2 * t2], v[1][2 * t2 + 1], ph[n][0], ph[n][1]);
                                if constexpr (PAIR)
                                    p4_mma(o[n][j + i][t2], v[0][2 * t2], v[0][2 * t2 + 1], v[1][2 * t2], v[1][2 * t2 + 1], pl[n][0], pl[n][1]);
                            }
                    }
                }
            }
        }

        // ------------------------------------------------------------ the unit's end: the warps of a head that had tiles join
        const int active = min(P, tiles);
        float2(&part)[W][MT] = ml[turn & 1];
        ++turn;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                if (gq == 0) part[warp][8 * n + 2 * tq + e] = make_float2(m[n][e], l[n][e]);
            }
        __syncthreads();
        if (wk < active) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // to the largest reference of the warps
                    const int row = 8 * n + 2 * tq + e;
                    float big = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W; ++w) big = w < active ? fmaxf(big, part[wg + w * G][row].x) : big;
                    const float f = m[n][e] == -INFINITY ? 1.f : pa_exp2(m[n][e] - big);  // (a NaN sum without a maximum stays)
                    float* to = merge + (size_t)(warp * MT + row) * S::kRow + 4 * gq;
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        *reinterpret_cast<float4*>(to + 32 * j) = make_float4(o[n][j][0][e] * f, o[n][j][0][2 + e] * f,
                                                                              o[n][j][1][e] * f, o[n][j][1][2 + e] * f);
                    if (gq == 0) sums[warp][row] = make_float2(big, l[n][e] * f);
                }
        }
        const bool whole = unit.tile == 0 && tiles == sq.ntiles;
        // a part of a shared unit: its start goes to the CTA's second slot, any other part to the first
        const int slot = blockIdx.x * 2 + (unit.tile == 0 ? 1 : 0);
        const int row0 = sq.row0;
        if (!whole && unit.tile == 0 && threadIdx.x == 0) {
            PaJoin e = pa_join_entry(unit, rt, MT, mvalid, h0, sq.ntiles - tiles, chunk);
            e.together = G, e.mt = MT;
            A.ws_join[blockIdx.x] = e;
        }
        skip(cur, tiles);
        if (cur.left > 0) fetch(cur);
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x; i < G * mvalid * (HD / 4); i += S::kThreads) {
            const int at = i / (HD / 4), col = 4 * (i % (HD / 4)), g = G > 1 ? at / mvalid : 0, row = at - g * mvalid;
            const float big = sums[g][row].x;
            float sum = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (w < active) {
                    const float4 z = *reinterpret_cast<const float4*>(merge + (size_t)((g + w * G) * MT + row) * S::kRow + col);
                    y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                    sum += sums[g + w * G][row].y;
                }
            if (whole) {
                const int mm = rt * MT + row, r = row0 + mm / A.group, hq = (h0 + g) * A.group + mm % A.group;
                const float inv = sum == 0.f ? 0.f : (A.C.v_scale != nullptr ? A.C.v_scale[h0 + g] : 1.f) / sum;
                uint2 w;
                if (A.out.dtype == kBF16)
                    w = make_uint2(pack2<true>(y.x * inv, y.y * inv), pack2<true>(y.z * inv, y.w * inv));
                else
                    w = make_uint2(pack2<false>(y.x * inv, y.y * inv), pack2<false>(y.z * inv, y.w * inv));
                *reinterpret_cast<uint2*>(A.out.p + (int64_t)r * A.out.rs + (int64_t)hq * A.out.hs + 2 * col) = w;
                if (A.lse != nullptr && col == 0)
                    A.lse[(int64_t)r * A.q.heads + hq] =
                        sum == 0.f ? -INFINITY : (big == -INFINITY ? sum : (big + log2f(sum)) * 0.69314718056f);
            } else {
                const int64_t place = (int64_t)slot * MT * A.together + g * MT + row;
                *reinterpret_cast<float4*>(A.ws_o + place * HD + col) = y;
                if (col == 0) A.ws_ml[place] = make_float2(big, sum);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool PAIR, int HD, int NT, bool TOGETHER>
static int p4_launch(const PaArgs& A, int num_sms, cudaStream_t st) {
    using S = P4Shape<PAIR, HD, NT>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_attn4_kernel<PAIR, HD, NT, TOGETHER>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(S::kThreads), S::kSmem, st, A);
}
template <bool PAIR, int HD, int NT>
static int p4_launch(const PaArgs& A, int num_sms, cudaStream_t st) {
    return A.together > 1 ? p4_launch<PAIR, HD, NT, true>(A, num_sms, st) : p4_launch<PAIR, HD, NT, false>(A, num_sms, st);
}
template <bool PAIR>
static int p4_shape(const PaArgs& A, int hd, int mt, int num_sms, cudaStream_t st) {
    if (mt == 8) return hd == 64 ? p4_launch<PAIR, 64, 1>(A, num_sms, st) : p4_launch<PAIR, 128, 1>(A, num_sms, st);
    return hd == 64 ? p4_launch<PAIR, 64, 2>(A, num_sms, st) : p4_launch<PAIR, 128, 2>(A, num_sms, st);
}
bool p4_many(const PaArgs& A, int mt, int num_sms) {
    const double units = ((double)A.R.n_rows * A.group / mt + A.R.n_seqs) * A.C.kv_heads;
    return units >= num_sms || units * (A.R.cap / kP4Keys + 1) >= kP4Far / P4Shape<false, 128, 1>::kStage;
}
int paged_attention4(const PaArgs& A, int hd, int mt, int num_sms, cudaStream_t st) {
    return A.out.dtype == kF16 ? p4_shape<true>(A, hd, mt, num_sms, st) : p4_shape<false>(A, hd, mt, num_sms, st);
}

}  // namespace dflash
