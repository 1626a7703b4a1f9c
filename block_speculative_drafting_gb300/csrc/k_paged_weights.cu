// The attention weight that each cached key receives: for every (sequence,
// key/value head) and key j the sum of exp(scale q . k_j - lse) over the rows that
// see j and the query heads that share the head, added to what is there.
//
// The scores are multiplied the other way round than the attention's: S = K Q^T
// (tcgen05.mma, M 128 keys, N up to 64 or 128 rows, both operands in shared memory,
// f32 in tensor memory), so that a key is a tensor-memory lane, the thread that
// owns the lane adds its key's weights up in registers, and no sum crosses
// threads: one order, equal bits, no atomics.
//
// Work.  All key tiles of all (sequence, head)s, in order, are one line, cut into
// a share a CTA (one an SM) of about equal cost, a tile's cost being the query rows that
// see it.  A CTA takes its tiles in pairs and each pair against the tiles of
// queries that see it: few rows are one query tile, which stays while the keys go by
// (memory bound); many rows go by in tiles under a pair of keys that stays (each
// exponential is needed once and costs its turn in the special-function
// unit, 32 a clock and SM; a pair, because each query tile then is fetched from L2 for
// 256 keys).
//
// Warps: 0-3 and 4-7 the sums of a pair's first and second tile, 8 issues the
// MMAs, 9-12 load keys (asynchronous copies; codes become f16, exact, in the
// same ring), 13-16 queries with their columns' scale, lse and position.  Two
// score buffers of 256 columns: the next step's products run while
// this one's exponentials do.  bf16 queries over a cache of codes are brought into f16 by a
// power of two a row.
//
// Keys that only some of a tile's rows see, and rows of lse -inf, take a path
// that looks at each column; keys past the end or not held are zeros whose sums
// are not written.  Every wait is bounded (1 s); a role whose wait expires stops, and sums
// that were not made are NaN.
#include "kernels.cuh"
#include "paged_tile.cuh"

namespace dflash {

constexpr int kPwSum = 8, kPwMma = 8, kPwKeys = 9, kPwQueries = 13, kPwThreads = 17 * 32;  // warps
constexpr int kPwBits = 32;  // tiles whose key masks are kept: more than the loaders can be ahead of the sums
constexpr uint64_t kPwWait = 1000000000ull;

struct PwArgs {
    PagedCache C;
    PagedRows R;
    HeadRows q;
    KeyWeights W;
    const float* lse;
    float scale_log2;
    int window, group;
};

// CB: bits of a cache's element; NQ: rows of a query tile
template <int CB, int HD, int NQ>
struct PwShape {
    static constexpr bool E8 = CB < 16;
    static constexpr int kLoaders = 128, KPW = 32;  // threads of the keys, keys of a warp: one a lane
    static constexpr int kItem = kPaTile * HD * 2, kQItem = NQ * HD * 2;
    static constexpr int kSlots = (E8 ? 3 : NQ == 64 ? 5 : 4) * (128 / HD);
    // half tiles of codes on their way, as in the attention (k_paged_attn_tc.cu)
    static constexpr int kRawCh = HD * CB / 128;
    static constexpr int kRaw = E8 ? 4 * (128 / HD) * 8 / CB : 0, kRawLd = KPW * kRawCh / 64;
    static constexpr int kRawCodes = kRaw * kRawLd * 16 * kLoaders;
    static constexpr int kRawBytes = kRawCodes + (CB == 4 ? kRawCodes / 4 : 0);
    static constexpr int kCtl = 5 * 1024;
    static constexpr size_t kSmem = 1024 /*alignment*/ + kCtl + (size_t)kSlots * kItem + 2 * kQItem + kRawBytes;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct PwCtl {
    uint64_t k_full[10], k_empty[10], q_full[2], q_empty[2], d_full[2], d_empty[2], fin;
    uint32_t tmem;
    int seq, head, tile, left, row0, rows;  // where this CTA's share begins
    uint32_t bits[kPwBits][4];              // a tile's held keys
    uint32_t dead[2][4];                    // a query tile's rows of lse -inf
    alignas(16) float c[2][128], nl[2][128];  // a query tile's columns: exp2(s c - nl)
    alignas(16) int pos[2][128];
};

template <int NQ>
DF_DEV PaSeq pw_seq(const PwArgs& A, int s, int a, int b) {
    PaSeq q;
    q.row0 = a;
    q.rows = b - a;
    const int len = A.R.kv_len[s];
    q.p0 = max(len, -1) - q.rows;
    q.hi = min(max(len, 0), A.R.cap);
    q.lo = A.window > 0 ? max(0, q.p0 - A.window + 1) : 0;
    q.ntiles = q.rows > 0 && q.hi > q.lo ? (q.hi - q.lo + kPaTile - 1) / kPaTile : 0;
    q.nunits = (int)(((int64_t)q.rows * A.group + NQ - 1) / NQ);  // query tiles
    return q;
}

// A step: key tiles kt .. kt + nt - 1 of head h of sequence s against query tile qt (the last of the pair: qe).
struct PwCur {
    PaSeq q;
    int s, h, kt, nt, qt, qe;
    int left;  // key tiles of the share from kt on (0: none)
};
template <int NQ>
DF_DEV void pw_pair(const PwArgs& A, PwCur& c) {
    c.nt = c.kt + 1 < c.q.ntiles && c.left > 1 ? 2 : 1;
    const int kf = c.q.lo + c.kt * kPaTile, kl = min(kf + c.nt * kPaTile, c.q.hi) - 1;
    const int r0 = max(0, kf - c.q.p0);
    const int r1 = A.window > 0 ? (int)min((int64_t)c.q.rows - 1, (int64_t)kl + A.window - 1 - c.q.p0) : c.q.rows - 1;
    c.qt = r0 * A.group / NQ;
    c.qe = (r1 * A.group + A.group - 1) / NQ;
}
template <int NQ>
DF_DEV void pw_next(const PwArgs& A, PwCur& c) {
    if (c.qt < c.qe) {
        ++c.qt;
        return;
    }
    c.left -= c.nt;
    c.kt += c.nt;
    if (c.left <= 0) {
        c.left = 0;
        return;
    }
    if (c.kt >= c.q.ntiles) {
        c.kt = 0;
        if (++c.h == A.C.kv_heads) {
            c.h = 0;
            do {
                if (++c.s >= A.R.n_seqs) {  // (never, while the lengths stay as they were counted)
                    c.left = 0;
                    return;
                }
                const int a = c.q.row0 + c.q.rows;
                c.q = pw_seq<NQ>(A, c.s, a, rows_end(A.R, c.s, a));
            } while (c.q.ntiles == 0);
        }
    }
    pw_pair<NQ>(A, c);
}
DF_DEV bool pw_same_queries(const PwCur& a, const PwCur& b) {
    return b.left > 0 && a.s == b.s && a.h == b.h && a.qt == b.qt;
}

// Cost of a head's first k tiles, in rows' worth of work: the rows that see a tile (exactly but for the rounding to query
// tiles; with a window all of them, which then is alike for all tiles) and a little for the tile itself.
template <int NQ>
DF_DEV int64_t pw_cost(const PwArgs& A, const PaSeq& q, int k) {
    const int64_t all = (int64_t)NQ * q.nunits + NQ / 4;
    int64_t c = all * k;
    if (A.window == 0) {
        const int from = q.p0 >= q.lo ? (q.p0 - q.lo) / kPaTile + 1 : 0;  // tiles before this one: every row sees them
        if (k > from) {
            const int64_t n = k - from;
            c -= A.group * (kPaTile * (n * (from + k - 1) / 2) + (int64_t)(q.lo - q.p0) * n);
        }
    }
    return c;
}
// This CTA's share (one warp): tiles of the line whose cost so far lies in the CTA's part of the whole.
template <int NQ>
DF_DEV void pw_share(const PwArgs& A, PwCtl& ctl, int lane) {
    const PagedRows& R = A.R;
    const int first = R.row_start == nullptr ? 0 : row_start_at(R, 0);
    // a sweep over the sequences, 32 at a time: f(sequence of this lane, its line, its cost a head, whether it is one)
    auto sweep = [&](auto f) {
        for (int s0 = 0, from = first; s0 < R.n_seqs; s0 += 32) {
            int a, b;
            rows_of_lane(R, s0, from, lane, a, b);
            from = __shfl_sync(0xffffffffu, b, 31);
            const bool in = s0 + lane < R.n_seqs;
            const PaSeq q = pw_seq<NQ>(A, min(s0 + lane, R.n_seqs - 1), a, b);
            const int64_t heads = in ? A.C.kv_heads : 0;
            if (!f(s0, q, heads * pw_cost<NQ>(A, q, q.ntiles), heads * q.ntiles)) break;
        }
    };
    auto scan = [&](int64_t x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, (long long)x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    int64_t total = 0, tiles = 0;
    sweep([&](int, const PaSeq&, int64_t cost, int64_t n) {
        total += __shfl_sync(0xffffffffu, (long long)scan(cost), 31);
        tiles += __shfl_sync(0xffffffffu, (long long)scan(n), 31);
        return true;
    });
    // the first tile at which the cost so far reaches a target
    auto tile_at = [&](int64_t target) {
        int64_t c0 = 0, t0 = 0, at = tiles;
        sweep([&](int, const PaSeq& q, int64_t cost, int64_t n) {
            const int64_t ce = c0 + scan(cost), te = t0 + scan(n);
            const uint32_t hit = __ballot_sync(0xffffffffu, ce > target);
            if (hit != 0) {
                const int l = __ffs(hit) - 1;
                int64_t mine = te;
                if (lane == l) {
                    const int64_t per = pw_cost<NQ>(A, q, q.ntiles), rest = max(target - (ce - cost), (int64_t)0), h = rest / per;
                    int lo = 0, hi = q.ntiles;  // the fewest tiles that cost `rest` of a head
                    while (lo < hi) {
                        const int m = (lo + hi) / 2;
                        if (pw_cost<NQ>(A, q, m) >= rest - h * per)
                            hi = m;
                        else
                            lo = m + 1;
                    }
                    mine = te - n + h * q.ntiles + lo;
                }
                at = __shfl_sync(0xffffffffu, (long long)mine, l);
                return false;
            }
            c0 = __shfl_sync(0xffffffffu, (long long)ce, 31);
            t0 = __shfl_sync(0xffffffffu, (long long)te, 31);
            return true;
        });
        return at;
    };
    const int64_t begin = tile_at(total * (int64_t)blockIdx.x / gridDim.x);
    const int64_t end = (int)blockIdx.x + 1 == (int)gridDim.x ? tiles : tile_at(total * ((int64_t)blockIdx.x + 1) / gridDim.x);
    if (lane == 0) ctl.left = (int)max(end - begin, (int64_t)0);
    int64_t t0 = 0;
    sweep([&](int s0, const PaSeq& q, int64_t, int64_t n) {
        const int64_t te = t0 + scan(n);
        const uint32_t hit = __ballot_sync(0xffffffffu, te > begin);
        if (hit != 0) {
            if (lane == __ffs(hit) - 1) {
                const int x = (int)(begin - (te - n));
                ctl.seq = s0 + lane;
                ctl.head = x / q.ntiles;
                ctl.tile = x - ctl.head * q.ntiles;
                ctl.row0 = q.row0;
                ctl.rows = q.rows;
            }
            return false;
        }
        t0 = __shfl_sync(0xffffffffu, (long long)te, 31);
        return true;
    });
}

// kind::f16 products of two shared-memory operands by the one lane with `on`
DF_DEV void pw_mma(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"((uint32_t)on)
        : "memory");
}
DF_DEV void cp_arrive(uint64_t* bar) {  // once this thread's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// BF: 16-bit operands are bf16 (a bf16 cache)
template <bool BF, int CB, int HD, int NQ>
__global__ void __launch_bounds__(kPwThreads, 1) paged_weights_kernel(const __grid_constant__ PwArgs A) {
    using S = PwShape<CB, HD, NQ>;
    constexpr bool E8 = S::E8;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    unsigned char* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
    PwCtl& ctl = *reinterpret_cast<PwCtl*>(sm);
    static_assert(sizeof(PwCtl) <= S::kCtl && S::kSlots <= 10, "control block");
    unsigned char *ring = sm + S::kCtl, *qring = ring + S::kSlots * S::kItem, *rawring = qring + 2 * S::kQItem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // queries in the MMAs' type are copied as they are
    const bool qcopy = !E8 || A.q.dtype == kF16;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            // (16-bit keys' copies arrive by themselves; their warps arrive beside them for the key masks)
            mbar_init(&ctl.k_full[i], S::kLoaders + (E8 ? 0 : 4));
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.q_full[i], qcopy ? 256 : 128);
            mbar_init(&ctl.q_empty[i], 1 + kPwSum);
            mbar_init(&ctl.d_full[i], 2);
            mbar_init(&ctl.d_empty[i], kPwSum);
        }
        mbar_init(&ctl.fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPwMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&ctl.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 0) pw_share<NQ>(A, ctl, lane);
    at_fence_before();
    __syncthreads();
    at_fence_after();
    const uint32_t tmem = ctl.tmem;
    PwCur cur{};
    cur.left = ctl.left;
    if (cur.left > 0) {
        cur.s = ctl.seq, cur.h = ctl.head, cur.kt = ctl.tile;
        cur.q = pw_seq<NQ>(A, cur.s, ctl.row0, ctl.row0 + ctl.rows);
        pw_pair<NQ>(A, cur);
    }

    if (warp >= kPwQueries) {
        // ------------------------------------------------------------ queries
        constexpr int CH = HD / 8, RPP = 128 / CH, PASSES = NQ / RPP;  // 16-byte chunks of a row, rows of a pass
        const int t = threadIdx.x - kPwQueries * 32, ch = t % CH, qw = warp - kPwQueries;
        int qn = 0;
        PwCur before{};
        for (PwCur c = cur; c.left > 0; before = c, pw_next<NQ>(A, c)) {
            if (qn > 0 && pw_same_queries(before, c)) continue;
            const int slot = qn & 1, all = c.q.rows * A.group;
            if (qn >= 2 && !__all_sync(0xffffffffu, mbar_wait(&ctl.q_empty[slot], ((qn >> 1) - 1) & 1, kPwWait))) break;
            unsigned char* dst = qring + slot * S::kQItem;
            const float cs = A.scale_log2 * (E8 && A.C.k_scale != nullptr ? A.C.k_scale[c.h] : 1.f);
            const auto at = [&](int r, bool& in, int& row, int& hq) {
                const int mm = c.qt * NQ + r, i = mm / A.group;
                in = mm < all;
                row = c.q.row0 + i;
                hq = c.h * A.group + mm - i * A.group;
            };
            if (t < NQ) {
                bool in;
                int row, hq;
                at(t, in, row, hq);
                const float lse = in ? A.lse[(int64_t)row * A.q.heads + hq] : 0.f;
                ctl.nl[slot][t] = lse * 1.4426950408889634f;
                ctl.pos[slot][t] = c.q.p0 + row - c.q.row0;
                if (qcopy) ctl.c[slot][t] = fminf(fmaxf(cs, 1e-37f), 3e38f);
                const uint32_t dead = __ballot_sync(0xffffffffu, in && lse == -INFINITY);
                if (lane == 0) ctl.dead[slot][qw] = dead;
            } else if (lane == 0) {
                ctl.dead[slot][qw] = 0;
            }
            if (qcopy) {
#pragma unroll 4
                for (int p = 0; p < PASSES; ++p) {
                    const int r = p * RPP + t / CH;
                    bool in;
                    int row, hq;
                    at(r, in, row, hq);
                    const unsigned char* src =
                        in ? A.q.p + (int64_t)row * A.q.rs + (int64_t)hq * A.q.hs + 16 * ch : A.q.p;  // (else nothing is read)
                    cp16(smem_addr(dst) + (ch >> 3) * (NQ * 128) + at_swz(r, ch & 7), src, in ? 16 : 0);
                }
                cp_arrive(&ctl.q_full[slot]);
            } else {
                // a bf16 row times 2^-x, its largest element in [1, 2): what f16 cannot hold of it then is
                // under 2^-25 of that element
#pragma unroll 4
                for (int p = 0; p < PASSES; ++p) {
                    const int r = p * RPP + t / CH;
                    bool in;
                    int row, hq;
                    at(r, in, row, hq);
                    const uint4 x = in ? *reinterpret_cast<const uint4*>(A.q.p + (int64_t)row * A.q.rs + (int64_t)hq * A.q.hs + 16 * ch)
                                       : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    float mx = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<true>(w[j]);
                        mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
                    for (int o = CH / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    float down = 1.f, rf = 1.f;
                    if (mx > 0.f && mx < INFINITY) {
                        const int e = min(max(ilogbf(mx), -120), 120);
                        down = ldexpf(1.f, -e);
                        rf = ldexpf(1.f, e);
                    }
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<true>(w[j]);
                        y[j] = pack2<false>(f.x * down, f.y * down);
                    }
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * (NQ * 128) + at_swz(r, ch & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                    if (ch == 0) ctl.c[slot][r] = fminf(fmaxf(cs * rf, 1e-37f), 3e38f);
                }
            }
            mbar_arrive(&ctl.q_full[slot]);
            ++qn;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= kPwKeys) {
        // ------------------------------------------------------------ keys
        const int lw = warp - kPwKeys;
        int n = 0;  // the next tile
        struct Look {
            int id, slot, h;
        };
        // the share's tiles one by one: this lane's key's page, looked up a tile ahead
        PwCur c = cur;
        auto look = [&]() -> Look {
            Look k{-1, 0, c.h};
            const int key = c.q.lo + c.kt * kPaTile + lw * S::KPW + lane;
            if (key < c.q.hi) k.id = page_entry(A.R, c.s, key, k.slot);
            return k;
        };
        auto next_tile = [&]() {  // (as pw_next, a single tile and no queries)
            c.nt = 1;
            c.qt = c.qe;
            pw_next<NQ>(A, c);
        };
        auto wait_empty = [&](int tile) -> bool {
            return tile < S::kSlots ||
                   __all_sync(0xffffffffu, mbar_wait(&ctl.k_empty[tile % S::kSlots], ((tile / S::kSlots) - 1) & 1, kPwWait));
        };
        auto walk = [&](auto emit) {
            Look ahead{-1, 0, 0};
            if (c.left > 0) ahead = look();
            while (c.left > 0) {
                const unsigned char *row = nullptr, *blocks = nullptr;
                if (page_held(ahead.id, A.C.n_pages)) {
                    row = A.C.k + ahead.id * A.C.ks[0] + ahead.slot * A.C.ks[1] + ahead.h * A.C.ks[2];
                    if constexpr (CB == 4) blocks = A.C.kb + ahead.id * A.C.kbs[0] + ahead.slot * A.C.kbs[1] + ahead.h * A.C.kbs[2];
                }
                const uint32_t b = __ballot_sync(0xffffffffu, row != nullptr);
                if (lane == 0) ctl.bits[n % kPwBits][lw] = b;
                next_tile();
                if (c.left > 0) ahead = look();
                if (!emit(row, blocks)) return;
            }
        };
        if constexpr (!E8) {
            constexpr int CH = HD / 8, RPI = 32 / CH;
            walk([&](const unsigned char* rows, const unsigned char*) -> bool {
                if (!wait_empty(n)) return false;
                const uint32_t dst = smem_addr(ring) + (n % S::kSlots) * S::kItem;
#pragma unroll
                for (int i = 0; i < S::KPW / RPI; ++i) {
                    const int r = i * RPI + lane / CH, ch = lane % CH;
                    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                    const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * ch : A.q.p;  // (nothing is read)
                    cp16(dst + (ch >> 3) * (kPaTile * 128) + at_swz(lw * S::KPW + r, ch & 7), src, p ? 16 : 0);
                }
                cp_arrive(&ctl.k_full[n % S::kSlots]);
                // (that follows the copies alone: the tile's key mask, written by this lane, takes an arrival of its own)
                if (lane == 0) mbar_arrive(&ctl.k_full[n % S::kSlots]);
                ++n;
                return true;
            });
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            constexpr int CH = S::kRawCh, RPI = 32 / CH, LD = S::kRawLd;  // copies of a lane a half tile
            const int ch = lane % CH, self = threadIdx.x - kPwKeys * 32;
            unsigned char *raw = rawring + self * 16, *raw_scale = rawring + S::kRawCodes + self * 4;
            constexpr int kPlace = S::kLoaders * 16;  // from one of a thread's places to the next
            auto write = [&](int half) -> bool {
                const int tile = half >> 1, slot = tile % S::kSlots;
                if ((half & 1) == 0 && !wait_empty(tile)) return false;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int key = lw * S::KPW + ((half & 1) * LD + i) * RPI + lane / CH;
                    const uint4 x = *reinterpret_cast<const uint4*>(raw + ((half % S::kRaw) * LD + i) * kPlace);
                    uint32_t scales = 0;
                    if constexpr (CB == 4)
                        scales = *reinterpret_cast<const uint32_t*>(raw_scale + ((half % S::kRaw) * LD + i) * (kPlace / 4)) >>
                                 ((2 * ch & 3) * 8);
                    tile_place<CB, HD>(ring + slot * S::kItem, key, ch, x, scales);
                }
                if (half & 1) mbar_arrive(&ctl.k_full[slot]);
                return true;
            };
            walk([&](const unsigned char* rows, const unsigned char* blocks) -> bool {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int half = 2 * n + hf;
#pragma unroll
                    for (int i = 0; i < LD; ++i) {
                        const int r = (hf * LD + i) * RPI + lane / CH;
                        const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                        const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * ch : A.q.p;  // (nothing is read)
                        cp16(smem_addr(raw) + ((half % S::kRaw) * LD + i) * kPlace, src, p ? 16 : 0);
                        if constexpr (CB == 4) {
                            const uint64_t b = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(blocks), r);
                            const void* bs = b ? reinterpret_cast<const unsigned char*>(b) + (2 * ch & ~3) : A.q.p;
                            cp4(smem_addr(raw_scale) + ((half % S::kRaw) * LD + i) * (kPlace / 4), bs, b ? 4 : 0);
                        }
                    }
                    cp_commit();
                    cp_wait<S::kRaw - 1>();
                    if (half >= S::kRaw - 1 && !write(half - (S::kRaw - 1))) return false;
                }
                ++n;
                return true;
            });
            asm volatile("cp.async.wait_all;" ::: "memory");
            for (int half = max(0, 2 * n - (S::kRaw - 1)); half < 2 * n; ++half)
                if (!write(half)) break;
        }
    } else if (warp == kPwMma) {
        // ------------------------------------------------------------ MMAs
        auto whole_warp = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // (said so to the compiler)
        auto wait = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, kPwWait)); };
        const bool on = lane == 0;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;  // A, B: bf16, or f16
        const uint64_t dk0 = at_desc(smem_addr(ring), 16), dq0 = at_desc(smem_addr(qring), 16);
        int st = 0, kn = 0, qn = 0;  // steps, key tiles before this pair, query tiles so far
        bool first = true, ok = true;
        PwCur before{};
        for (PwCur c = cur; ok && whole_warp((int)(c.left > 0)) != 0; ++st) {
            const int nt = whole_warp(c.nt);
            if (first)
                for (int i = 0; ok && i < nt; ++i) ok = wait(&ctl.k_full[(kn + i) % S::kSlots], (kn + i) / S::kSlots);
            if (ok && (qn == 0 || !pw_same_queries(before, c))) {
                ok = wait(&ctl.q_full[qn & 1], qn >> 1);
                ++qn;
            }
            const int qs = whole_warp((qn - 1) & 1);
            if (ok && st >= 2) ok = wait(&ctl.d_empty[st & 1], (st >> 1) - 1);
            if (!ok) break;
            fence_proxy_async_smem();
            at_fence_after();
            const int nv = min(NQ, c.q.rows * A.group - c.qt * NQ);
            const uint32_t idesc = (uint32_t)whole_warp((int)(at_idesc(128, (nv + 15) & ~15, false) | kType));
            const uint64_t qd = dq0 + (uint64_t)(qs * S::kQItem >> 4);
            for (int i = 0; i < nt; ++i) {
                const uint64_t kd = dk0 + (uint64_t)(whole_warp((kn + i) % S::kSlots) * (S::kItem >> 4));
                const uint32_t d = tm + (uint32_t)((st & 1) * 256 + i * 128);
#pragma unroll
                for (int j = 0; j < HD / 16; ++j)
                    pw_mma(on, d, kd + (uint64_t)(((j >> 2) * (kPaTile * 128) + (j & 3) * 32) >> 4),
                           qd + (uint64_t)(((j >> 2) * (NQ * 128) + (j & 3) * 32) >> 4), idesc, j > 0 ? 1u : 0u);
            }
            before = c;
            pw_next<NQ>(A, c);
            first = before.qt == before.qe;
            if (first) {
                for (int i = 0; i < nt; ++i) pt_commit(on, &ctl.k_empty[(kn + i) % S::kSlots]);
                kn += nt;
            }
            if (!pw_same_queries(before, c)) pt_commit(on, &ctl.q_empty[qs]);
            pt_commit(on, &ctl.d_full[st & 1]);
            // (an arrival of this thread's own, which orders the key masks and the columns' numbers)
            if (on) mbar_arrive(&ctl.d_full[st & 1]);
        }
        // every MMA issued has completed before the CTA moves on
        pt_commit(on, &ctl.fin);
        mbar_wait(&ctl.fin, 0, kPwWait);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ sums
        const int half = warp >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        bool ok = true;
        int st = 0, kn = 0, qn = 0;
        PwCur before{};
        for (PwCur c = cur; c.left > 0;) {
            const PaSeq sq = c.q;
            const int nt = c.nt, kfirst = sq.lo + (c.kt + half) * kPaTile, j = kfirst + (warp & 3) * 32 + lane;
            const bool mine = half < nt;
            float* w = A.W.p + (int64_t)c.s * A.W.ss + (int64_t)c.h * A.W.hs + j;
            const bool adds = mine && j < sq.hi && j < sq.p0;
            const float old = adds ? *w : 0.f;  // (a position that the call brings starts at 0)
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            bool last;
            do {
                if (qn == 0 || !pw_same_queries(before, c)) ++qn;
                const int qs = (qn - 1) & 1;
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl.d_full[st & 1], (st >> 1) & 1, kPwWait));
                if (ok && mine) {
                    at_fence_after();
                    const int nv = min(NQ, sq.rows * A.group - c.qt * NQ);
                    const int pmin = sq.p0 + c.qt * NQ / A.group, pmax = sq.p0 + (c.qt * NQ + nv - 1) / A.group;
                    const bool plain = kfirst + kPaTile - 1 <= pmin && (A.window == 0 || kfirst > pmax - A.window) &&
                                       (ctl.dead[qs][0] | ctl.dead[qs][1] | ctl.dead[qs][2] | ctl.dead[qs][3]) == 0;
                    const uint32_t sb = lane_addr + (uint32_t)((st & 1) * 256);
                    const float cs0 = ctl.c[qs][0];
#pragma unroll 1
                    for (int x = 0; x < nv; x += 32) {
                        float v[32];
                        pt_ld32(sb + x, *reinterpret_cast<uint32_t(*)[32]>(v));
                        at_wait_ld();
                        if (plain && x + 32 <= nv) {
#pragma unroll
                            for (int y = 0; y < 32; y += 4) {
                                const float4 nl = *reinterpret_cast<const float4*>(&ctl.nl[qs][x + y]);
                                float4 cs = make_float4(cs0, cs0, cs0, cs0);  // (16-bit queries: one scale)
                                if constexpr (E8) cs = *reinterpret_cast<const float4*>(&ctl.c[qs][x + y]);
                                sum[0] += pa_exp2(fmaf(v[y], cs.x, -nl.x));
                                sum[1] += pa_exp2(fmaf(v[y + 1], cs.y, -nl.y));
                                sum[2] += pa_exp2(fmaf(v[y + 2], cs.z, -nl.z));
                                sum[3] += pa_exp2(fmaf(v[y + 3], cs.w, -nl.w));
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                if (x + y >= nv) break;
                                const int p = ctl.pos[qs][x + y];
                                const float nl = ctl.nl[qs][x + y];
                                const bool see = j <= p && (A.window == 0 || j > p - A.window) && nl != -INFINITY;
                                if (see) sum[y & 3] += pa_exp2(fmaf(v[y], ctl.c[qs][x + y], -nl));
                            }
                        }
                    }
                    at_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.d_empty[st & 1]);
                ++st;
                before = c;
                last = c.qt == c.qe;
                pw_next<NQ>(A, c);
                if (!pw_same_queries(before, c) && lane == 0) mbar_arrive(&ctl.q_empty[qs]);
            } while (!last);
            const uint32_t held = ctl.bits[(kn + half) % kPwBits][warp & 3];
            if (mine && j < sq.hi && (!ok || ((held >> lane) & 1u))) *w = ok ? old + ((sum[0] + sum[1]) + (sum[2] + sum[3])) : NAN;
            kn += nt;
        }
    }
    at_fence_before();
    __syncthreads();
    if (warp == kPwMma) {
        at_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <bool BF, int CB, int HD, int NQ>
static int pw_launch(const PwArgs& A, int num_sms, cudaStream_t st) {
    using S = PwShape<CB, HD, NQ>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_weights_kernel<BF, CB, HD, NQ>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(kPwThreads), S::kSmem, st, A);
}
template <int HD, int NQ>
static int pw_type(const PwArgs& A, int cd, int num_sms, cudaStream_t st) {
    return cd == kBF16   ? pw_launch<true, 16, HD, NQ>(A, num_sms, st)
           : cd == kF16  ? pw_launch<false, 16, HD, NQ>(A, num_sms, st)
           : cd == kE4M3 ? pw_launch<false, 8, HD, NQ>(A, num_sms, st)
                         : pw_launch<false, 4, HD, NQ>(A, num_sms, st);
}
int paged_key_weights(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                      const float* lse, float scale, int window, const KeyWeights& W, int num_sms, cudaStream_t st) {
    PwArgs A{};
    A.C = C, A.R = R, A.q = q, A.W = W, A.lse = lse, A.window = window;
    A.scale_log2 = scale * 1.4426950408889634f;
    A.group = q.heads / C.kv_heads;
    if (R.cap == 0) return 0;
    const int64_t per = ((int64_t)R.n_rows + R.n_seqs - 1) / R.n_seqs * A.group;  // rows of an average sequence's head
    if (per <= 64) return hd == 64 ? pw_type<64, 64>(A, cache_dtype, num_sms, st) : pw_type<128, 64>(A, cache_dtype, num_sms, st);
    return hd == 64 ? pw_type<64, 128>(A, cache_dtype, num_sms, st) : pw_type<128, 128>(A, cache_dtype, num_sms, st);
}

}  // namespace dflash
