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
// see it.  A CTA takes its tiles in pairs and each pair against the tiles of 128 query rows
// that see it: rows of one or two tiles go against keys in shared memory, one
// tile staying while the keys go by; more rows go by in tiles under a pair of keys that stays (each
// exponential is needed once and costs its turn in the special-function
// unit, 32 a clock and SM; a pair, because each query tile then is fetched from L2 for
// 256 keys).  Keys that stay are moved to tensor memory: with both operands in
// shared memory an MMA reads it at its full 128 bytes a clock.
//
// Warps: 0-3 and 4-7 the sums of a pair's first and second tile, 8 issues the
// MMAs, 9-11 load queries with their columns' scale, lse and position, 12-15 keys
// (asynchronous copies; codes become f16, exact, in the same ring).  Three
// score buffers of 128 columns go round: the next products run while the last ones'
// exponentials do.  Codes and bf16 queries meet in f16 where the keys go by (a
// query row is brought into it by a power of two), and in bf16 where they stay (codes
// times block scales, of 6 bits at most, are exact in either).  (Up to 64 rows a head, on average, are k_paged_weights_few.cu's.)
//
// 2048 rows of four query heads over 16384 bf16 keys x 8 heads: 289 us, 0.89 PFLOP/s, 47 % of
// a large product's rate.  The sums bound it: two warps a quarter of an SM take some 2000 clocks for
// a step's 256 x 128 scores, whose exponentials alone are 1024; the CTAs' shares end 15 % apart.
//
// Keys that only some of a tile's rows see, and rows of lse -inf, take a path
// with a mask of columns; keys past the end or not held are zeros whose sums
// are not written.  Every wait is bounded (1 s); a role whose wait expires stops, and sums
// that were not made are NaN.
#include <climits>

#include "kernels.cuh"
#include "paged_tile.cuh"

namespace dflash {

constexpr int kPwSum = 8, kPwMma = 8, kPwQueries = 9, kPwKeys = 12, kPwWarps = 16;  // warps
constexpr int kPwThreads = kPwWarps * 32, kPwQThreads = (kPwKeys - kPwQueries) * 32;
constexpr int kPwN = 128, kPwQSlots = 3, kPwScores = 3;  // rows of a query tile, tiles in their ring, score buffers
// Barriers on which a half waits for its score buffers, in its own order, and for the end of a pair without a tile for it
// (else it could run so far ahead that a barrier's last phase but one would look like the one it waits for): more than can be
// open at once, three buffers and as many pairs' ends as there are query tiles in the ring.
constexpr int kPwFull = 8;
// Query tiles from which on a pair of keys goes to tensor memory.  bf16 queries over codes need no conversion then, so for
// them two (64 rows of four query heads over 32768 e2m1 keys 66 -> 43 us); else three (over bf16 keys
// 33.9 us from three on, 35.1 from two).
constexpr int kPwStay = 3, kPwStayMixed = 2;
constexpr int kPwBits = 32;  // tiles whose key masks are kept: more than the loaders can be ahead of the sums
constexpr uint64_t kPwWait = 1000000000ull;

struct PwArgs {
    PagedCache C;
    PagedRows R;
    HeadRows q;
    KeyWeights W;
    const float* lse;
    float scale_log2;
    int window, group, stay;
    FastDiv by_group;
};

// CB: bits of a cache's element
template <int CB, int HD>
struct PwShape {
    static constexpr bool E8 = CB < 16;
    static constexpr int kLoaders = (kPwWarps - kPwKeys) * 32, KPW = kPaTile * 32 / kLoaders;  // threads of the keys, a warp's keys
    static constexpr int kItem = kPaTile * HD * 2, kQItem = kPwN * HD * 2;
    static constexpr int kSlots = (E8 ? 2 : 3) * (128 / HD);
    // tiles of codes on their way, 16 bytes a place, each place copied and read by one thread; beside a place of e2m1
    // codes the four bytes of the row's block scales that hold its two
    static constexpr int kRawCh = HD * CB / 128, kRawLd = KPW * kRawCh / 32;  // places of a row, of a lane and tile
    static constexpr int kRaw = !E8 ? 0 : (CB == 4 ? 5 : 3) * (128 / HD);
    static constexpr int kRawCodes = kRaw * kRawLd * 16 * kLoaders;
    static constexpr int kRawBytes = kRawCodes + (CB == 4 ? kRawCodes / 4 : 0);
    static constexpr int kCtl = 6 * 1024;
    static constexpr size_t kSmem = 1024 /*alignment*/ + kCtl + (size_t)kSlots * kItem + kPwQSlots * kQItem + kRawBytes;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    // tensor memory: score buffers, that the halves of the sums take in turn, and the keys that stay
    static constexpr int kColS = 0, kColK = kPwScores * kPwN;
};

struct PwCtl {
    uint64_t k_full[8], k_empty[8], q_full[kPwQSlots], q_empty[kPwQSlots], d_full[2][kPwFull], d_empty[kPwScores], stay[2], fin;
    uint32_t tmem;
    int seq, head, tile, left, row0, rows;  // where this CTA's share begins
    uint32_t bits[kPwBits][4];              // a tile's held keys
    uint64_t dead[kPwQSlots][2];            // a query tile's rows of lse -inf
    alignas(16) float c[kPwQSlots][kPwN], nl[kPwQSlots][kPwN];  // a query tile's columns: exp2(s c + nl)
};

DF_DEV PaSeq pw_seq(const PwArgs& A, int s, int a, int b) {
    PaSeq q;
    q.row0 = a;
    q.rows = b - a;
    const int len = A.R.kv_len[s];
    q.p0 = max(len, -1) - q.rows;
    q.hi = min(max(len, 0), A.R.cap);
    q.lo = A.window > 0 ? max(0, q.p0 - A.window + 1) : 0;
    q.ntiles = q.rows > 0 && q.hi > q.lo ? (q.hi - q.lo + kPaTile - 1) / kPaTile : 0;
    q.nunits = (int)(((int64_t)q.rows * A.group + kPwN - 1) / kPwN);  // query tiles
    return q;
}

// A pair: key tiles kt .. kt + nt - 1 of head h of sequence s against query tiles qt .. qe.
struct PwCur {
    PaSeq q;
    int s, h, kt, nt, qt, qe;
    int left;  // key tiles of the share from kt on (0: none)
};
DF_DEV void pw_pair(const PwArgs& A, PwCur& c) {
    c.nt = c.kt + 1 < c.q.ntiles && c.left > 1 ? 2 : 1;
    const int kf = c.q.lo + c.kt * kPaTile, kl = min(kf + c.nt * kPaTile, c.q.hi) - 1;
    const int r0 = max(0, kf - c.q.p0);
    const int r1 = A.window > 0 ? (int)min((int64_t)c.q.rows - 1, (int64_t)kl + A.window - 1 - c.q.p0) : c.q.rows - 1;
    c.qt = r0 * A.group / kPwN;
    c.qe = (r1 * A.group + A.group - 1) / kPwN;
}
// (out of line, as is what waits: the kernel's code is fetched once a call, and 180 KB of it took longer than the work)
__device__ __noinline__ void pw_next_head(const PwArgs& A, PwCur& c) {
    c.kt = 0;
    if (++c.h < A.C.kv_heads) return;
    c.h = 0;
    do {
        if (++c.s >= A.R.n_seqs) {  // (never, while the lengths stay as they were counted)
            c.left = 0;
            return;
        }
        const int a = c.q.row0 + c.q.rows;
        c.q = pw_seq(A, c.s, a, rows_end(A.R, c.s, a));
    } while (c.q.ntiles == 0);
}
DF_DEV void pw_next(const PwArgs& A, PwCur& c) {
    c.left -= c.nt;
    c.kt += c.nt;
    if (c.left <= 0) {
        c.left = 0;
        return;
    }
    if (c.kt >= c.q.ntiles) {
        PwCur x = c;  // (the copy alone is in memory)
        pw_next_head(A, x);
        c = x;
        if (c.left == 0) return;
    }
    pw_pair(A, c);
}
DF_DEV bool pw_stays(const PwArgs& A, const PwCur& c) { return c.qe - c.qt + 1 >= A.stay; }
// whether b, the pair after a, begins with the query tile that a ends with (in the form that it has there)
DF_DEV bool pw_keeps(const PwArgs& A, const PwCur& a, const PwCur& b) {
    return b.left > 0 && a.s == b.s && a.h == b.h && a.qe == b.qt && pw_stays(A, a) == pw_stays(A, b);
}

// Cost of a head's first k tiles: the query tiles that see each (but for the rounding; with a window all of them, which
// then is alike for all tiles).  (The whole line's is below 2^31: pa_line_fits.)
DF_DEV int pw_cost(const PwArgs& A, const PaSeq& q, int k) {
    const int from = q.p0 >= q.lo ? (q.p0 - q.lo) / kPaTile + 1 : 0;  // tiles before this one: every row sees them
    int64_t hidden = 0;
    if (A.window == 0 && k > from) {
        const int64_t n = k - from;
        hidden = A.group * (kPaTile * (n * (from + k - 1) / 2) + (int64_t)(q.lo - q.p0) * n) / kPwN;
    }
    return (int)((int64_t)k * q.nunits - hidden);
}
// Sequences s0 + lane (warp-wide), whose rows start at `from`; the tiles and the cost of each lane's with all before it
// in the 32; returns where the next 32's rows start.
struct PwLook {
    PaSeq q;
    int tiles, cost, tiles_to, cost_to;
};
__device__ __noinline__ int pw_look(const PwArgs& A, int s0, int from, int lane, PwLook& x) {
    int a, b;
    rows_of_lane(A.R, s0, from, lane, a, b);
    x.q = pw_seq(A, min(s0 + lane, A.R.n_seqs - 1), a, b);
    const int heads = s0 + lane < A.R.n_seqs ? A.C.kv_heads : 0;
    x.tiles_to = x.tiles = heads * x.q.ntiles;
    x.cost_to = x.cost = heads * pw_cost(A, x.q, x.q.ntiles);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, x.tiles_to, o), c = __shfl_up_sync(0xffffffffu, x.cost_to, o);
        if (lane >= o) x.tiles_to += t, x.cost_to += c;
    }
    return __shfl_sync(0xffffffffu, b, 31);
}
// This CTA's share (one warp): tiles of the line whose cost so far lies in the CTA's part of the whole.
DF_DEV void pw_share(const PwArgs& A, PwCtl& ctl, int lane) {
    const int first = A.R.row_start == nullptr ? 0 : row_start_at(A.R, 0);
    PwLook x;
    int total = 0, tiles = 0;
    bool again = true;
#pragma unroll 1
    for (int s0 = 0, from = first; s0 < A.R.n_seqs; s0 += 32) {
        from = pw_look(A, s0, from, lane, x);
        total += __shfl_sync(0xffffffffu, x.cost_to, 31);
        tiles += __shfl_sync(0xffffffffu, x.tiles_to, 31);
        again = s0 > 0;  // (one look serves where there are no more than 32)
    }
    // the first tiles at which the cost so far reaches this CTA's target, and the next one's
    int at[2] = {0, tiles};
    const int grid = gridDim.x, cta = blockIdx.x;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        if (cta + e == 0 || cta + e == grid) continue;
        const int target = (int)((int64_t)total * (cta + e) / grid);
        int c0 = 0, t0 = 0, found = tiles;
#pragma unroll 1
        for (int s0 = 0, from = first; s0 < A.R.n_seqs; s0 += 32) {
            if (again) from = pw_look(A, s0, from, lane, x);
            const uint32_t hit = __ballot_sync(0xffffffffu, c0 + x.cost_to > target);
            if (hit != 0) {
                const int l = __ffs(hit) - 1;
                if (lane == l) {
                    const int rest = target - (c0 + x.cost_to - x.cost), per = x.cost / A.C.kv_heads, h = rest / per;
                    int lo = 0, hi = x.q.ntiles;  // the fewest tiles that cost `rest` of a head
#pragma unroll 1
                    while (lo < hi) {
                        const int m = (lo + hi) / 2;
                        if (pw_cost(A, x.q, m) >= rest - h * per)
                            hi = m;
                        else
                            lo = m + 1;
                    }
                    found = t0 + x.tiles_to - x.tiles + h * x.q.ntiles + lo;
                }
                found = __shfl_sync(0xffffffffu, found, l);
                break;
            }
            c0 += __shfl_sync(0xffffffffu, x.cost_to, 31);
            t0 += __shfl_sync(0xffffffffu, x.tiles_to, 31);
        }
        at[e] = found;
    }
    if (lane == 0) ctl.left = max(at[1] - at[0], 0);
    int t0 = 0;
#pragma unroll 1
    for (int s0 = 0, from = first; s0 < A.R.n_seqs; s0 += 32) {
        if (again) from = pw_look(A, s0, from, lane, x);
        const uint32_t hit = __ballot_sync(0xffffffffu, t0 + x.tiles_to > at[0]);
        if (hit != 0) {
            if (lane == __ffs(hit) - 1) {
                const int y = at[0] - (t0 + x.tiles_to - x.tiles);
                ctl.seq = s0 + lane;
                ctl.head = y / x.q.ntiles;
                ctl.tile = y - ctl.head * x.q.ntiles;
                ctl.row0 = x.q.row0;
                ctl.rows = x.q.rows;
            }
            break;
        }
        t0 += __shfl_sync(0xffffffffu, x.tiles_to, 31);
    }
}

// A whole warp's bounded wait.
__device__ __noinline__ bool pw_wait_long(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, kPwWait));
}
DF_DEV bool pw_wait(uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1)) || pw_wait_long(bar, phase & 1);
}

// kind::f16 products of two shared-memory operands (by pt_elect's lane)
DF_DEV void pw_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// pairs of f32 in one register pair
DF_DEV uint64_t pw_pair2(uint32_t a, uint32_t b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "r"(a), "r"(b));
    return y;
}
DF_DEV uint64_t pw_pair2(float a, float b) { return pw_pair2(__float_as_uint(a), __float_as_uint(b)); }
DF_DEV uint64_t pw_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
DF_DEV void pw_add2(uint64_t& a, uint64_t b) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b)); }
DF_DEV uint64_t pw_exp2(uint64_t x) {
    return pw_pair2(pa_exp2(__uint_as_float((uint32_t)x)), pa_exp2(__uint_as_float((uint32_t)(x >> 32))));
}
DF_DEV void cp_arrive(uint64_t* bar) {  // once this thread's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// BF: 16-bit operands are bf16 (a bf16 cache)
template <bool BF, int CB, int HD>
__global__ void __launch_bounds__(kPwThreads, 1) paged_weights_kernel(const __grid_constant__ PwArgs A) {
    using S = PwShape<CB, HD>;
    constexpr bool E8 = S::E8;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    unsigned char* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
    PwCtl& ctl = *reinterpret_cast<PwCtl*>(sm);
    static_assert(sizeof(PwCtl) <= S::kCtl && S::kSlots <= 8, "control block");
    unsigned char *ring = sm + S::kCtl, *qring = ring + S::kSlots * S::kItem, *rawring = qring + kPwQSlots * S::kQItem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool mixed = E8 && A.q.dtype == kBF16;  // codes and bf16 queries

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            // (16-bit keys' copies arrive by themselves; their warps arrive beside them for the key masks)
            mbar_init(&ctl.k_full[i], S::kLoaders + (E8 ? 0 : kPwWarps - kPwKeys));
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < kPwQSlots; ++i) {
            mbar_init(&ctl.q_full[i], 2 * kPwQThreads);  // (the copies, and their threads beside them)
            mbar_init(&ctl.q_empty[i], 1 + kPwSum);
        }
        for (int i = 0; i < kPwScores; ++i) mbar_init(&ctl.d_empty[i], 4);
        // (the commit, and an arrival of the MMA thread's own that orders the key masks)
        for (int i = 0; i < kPwFull; ++i) {
            mbar_init(&ctl.d_full[0][i], 2);
            mbar_init(&ctl.d_full[1][i], 2);
        }
        mbar_init(&ctl.stay[0], 4);
        mbar_init(&ctl.stay[1], 4);
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
    if (warp == 0) pw_share(A, ctl, lane);
    at_fence_before();
    __syncthreads();
    at_fence_after();
    const uint32_t tmem = ctl.tmem;
    PwCur cur{};
    cur.left = ctl.left;
    if (cur.left > 0) {
        cur.s = ctl.seq, cur.h = ctl.head, cur.kt = ctl.tile;
        cur.q = pw_seq(A, cur.s, ctl.row0, ctl.row0 + ctl.rows);
        pw_pair(A, cur);
    }

    if (warp >= kPwKeys) {
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
        auto next_tile = [&]() {  // (as pw_next, a single tile)
            c.nt = 1;
            pw_next(A, c);
        };
        auto wait_empty = [&](int tile) -> bool {
            return tile < S::kSlots ||
                   pw_wait(&ctl.k_empty[tile % S::kSlots], tile / S::kSlots - 1);
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
        static_assert(S::KPW == 32, "a key a lane");
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
            using Lanes = TileLanes<CB, HD>;
            constexpr int RPI = Lanes::RPI, LD = S::kRawLd;  // copies of a lane a tile
            const int ch = Lanes::place(lane), lane_row = Lanes::row(lane), self = threadIdx.x - kPwKeys * 32;
            unsigned char *raw = rawring + self * 16, *raw_scale = rawring + S::kRawCodes + self * 4;
            constexpr int kPlace = S::kLoaders * 16;  // from one of a thread's places to the next
            auto write = [&](int tile) -> bool {
                const int slot = tile % S::kSlots;
                if (!wait_empty(tile)) return false;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int key = lw * S::KPW + i * RPI + lane_row;
                    const uint4 x = *reinterpret_cast<const uint4*>(raw + ((tile % S::kRaw) * LD + i) * kPlace);
                    uint32_t scales = 0;
                    if constexpr (CB == 4)
                        scales = *reinterpret_cast<const uint32_t*>(raw_scale + ((tile % S::kRaw) * LD + i) * (kPlace / 4)) >>
                                 ((2 * ch & 3) * 8);
                    tile_place<CB, HD>(ring + slot * S::kItem, key, ch, x, scales);
                }
                mbar_arrive(&ctl.k_full[slot]);
                return true;
            };
            walk([&](const unsigned char* rows, const unsigned char* blocks) -> bool {
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int r = i * RPI + lane_row;
                    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                    const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * ch : A.q.p;  // (nothing is read)
                    cp16(smem_addr(raw) + ((n % S::kRaw) * LD + i) * kPlace, src, p ? 16 : 0);
                    if constexpr (CB == 4) {
                        const uint64_t b = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(blocks), r);
                        const void* bs = b ? reinterpret_cast<const unsigned char*>(b) + (2 * ch & ~3) : A.q.p;
                        cp4(smem_addr(raw_scale) + ((n % S::kRaw) * LD + i) * (kPlace / 4), bs, b ? 4 : 0);
                    }
                }
                cp_commit();
                cp_wait<S::kRaw - 1>();
                if (n >= S::kRaw - 1 && !write(n - (S::kRaw - 1))) return false;
                ++n;
                return true;
            });
            asm volatile("cp.async.wait_all;" ::: "memory");
            for (int tile = max(0, n - (S::kRaw - 1)); tile < n; ++tile)
                if (!write(tile)) break;
        }
    } else if (warp >= kPwQueries) {
        // ------------------------------------------------------------ queries
        // four lanes a row, each every fourth of its 16-byte chunks
        constexpr int CH = HD / 8, ITEMS = kPwN * 4, PASSES = (ITEMS + kPwQThreads - 1) / kPwQThreads;
        const int t = threadIdx.x - kPwQueries * 32;
        int qn = 0;
        constexpr int NL = (kPwN + kPwQThreads - 1) / kPwQThreads;  // rows of a thread's lse
        float lse[NL] = {};
        bool in[NL] = {}, kept = false, ok = true;
        // a tile's numbers, written once the next one's copies are on their way (its lse has arrived by then)
        auto finish = [&](int n) {
            const int slot = n % kPwQSlots;
#pragma unroll
            for (int x = 0; x < NL; ++x) {
                const int r = t + x * kPwQThreads;
                if (r < kPwN) {  // (whole warps)
                    ctl.nl[slot][r] = -1.4426950408889634f * lse[x];
                    const uint32_t dead = __ballot_sync(0xffffffffu, in[x] && lse[x] == -INFINITY);
                    if (lane == 0) reinterpret_cast<uint32_t*>(ctl.dead[slot])[r >> 5] = dead;
                }
            }
            mbar_arrive(&ctl.q_full[slot]);
        };
        for (PwCur c = cur; ok && c.left > 0;) {
            PwCur nx = c;
            pw_next(A, nx);
            const bool keeps = pw_keeps(A, c, nx);
            const float cs = A.scale_log2 * (E8 && A.C.k_scale != nullptr ? A.C.k_scale[c.h] : 1.f);
            const int all = c.q.rows * A.group;
            const bool qcopy = !mixed || pw_stays(A, c);
            const unsigned char* base = A.q.p + (int64_t)c.q.row0 * A.q.rs + (int64_t)(c.h * A.group) * A.q.hs;
#pragma unroll 1
            for (int qt = c.qt + (kept ? 1 : 0); qt <= c.qe; ++qt) {
                const int slot = qn % kPwQSlots, turn = qn / kPwQSlots;
                if (qn > 0) finish(qn - 1);
#pragma unroll
                for (int x = 0; x < NL; ++x) {
                    const int r = t + x * kPwQThreads, mm = qt * kPwN + r, i = div_by(A.by_group, mm);
                    in[x] = r < kPwN && mm < all;
                    lse[x] = in[x] ? A.lse[(int64_t)(c.q.row0 + i) * A.q.heads + c.h * A.group + (mm - i * A.group)] : 0.f;
                }
                if (turn > 0 && !(ok = pw_wait(&ctl.q_empty[slot], turn - 1))) break;
                unsigned char* dst = qring + slot * S::kQItem;
                if (qcopy) {
#pragma unroll
                    for (int p = 0; p < PASSES; ++p) {
                        const int item = p * kPwQThreads + t, r = item >> 2, m = qt * kPwN + r, j = div_by(A.by_group, m);
                        if (ITEMS % kPwQThreads != 0 && item >= ITEMS) break;  // (whole warps)
                        const bool use = m < all;
                        const unsigned char* src = base + (int64_t)j * A.q.rs + (int64_t)(m - j * A.group) * A.q.hs;
#pragma unroll
                        for (int k = 0; k < CH / 4; ++k) {
                            const int ch = 4 * k + (t & 3);
                            cp16(smem_addr(dst) + (ch >> 3) * (kPwN * 128) + at_swz(r, ch & 7), use ? src + 16 * ch : A.q.p,
                                 use ? 16 : 0);
                        }
                        if ((t & 3) == 0) ctl.c[slot][r] = fminf(fmaxf(cs, 1e-37f), 3e38f);
                    }
                } else {
                    // a bf16 row times 2^-x, its largest element in [1, 2): what f16 cannot hold of it then is
                    // under 2^-25 of that element
#pragma unroll 1
                    for (int p = 0; p < PASSES; ++p) {
                        const int item = p * kPwQThreads + t, r = item >> 2, m = qt * kPwN + r, j = div_by(A.by_group, m);
                        if (ITEMS % kPwQThreads != 0 && item >= ITEMS) break;
                        const unsigned char* src = base + (int64_t)j * A.q.rs + (int64_t)(m - j * A.group) * A.q.hs;
                        uint4 v[CH / 4];
                        uint32_t (&w)[CH] = *reinterpret_cast<uint32_t(*)[CH]>(v);
#pragma unroll
                        for (int k = 0; k < CH / 4; ++k)
                            v[k] = m < all ? *reinterpret_cast<const uint4*>(src + 16 * (4 * k + (t & 3))) : make_uint4(0u, 0u, 0u, 0u);
                        float mx = 0.f;
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const float2 f = unpack2<true>(w[k]);
                            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        float down = 1.f, rf = 1.f;
                        if (mx > 0.f && mx < INFINITY) {
                            const int e = min(max(ilogbf(mx), -120), 120);
                            down = ldexpf(1.f, -e);
                            rf = ldexpf(1.f, e);
                        }
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const float2 f = unpack2<true>(w[k]);
                            w[k] = pack2<false>(f.x * down, f.y * down);
                        }
#pragma unroll
                        for (int k = 0; k < CH / 4; ++k) {
                            const int ch = 4 * k + (t & 3);
                            *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kPwN * 128) + at_swz(r, ch & 7)) = v[k];
                        }
                        if ((t & 3) == 0) ctl.c[slot][r] = fminf(fmaxf(cs * rf, 1e-37f), 3e38f);
                    }
                }
                if (qcopy)
                    cp_arrive(&ctl.q_full[slot]);
                else
                    mbar_arrive(&ctl.q_full[slot]);  // (in the copies' place)
                ++qn;
            }
            kept = keeps;
            c = nx;
        }
        if (ok && qn > 0) finish(qn - 1);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kPwMma) {
        // ------------------------------------------------------------ MMAs
        // (whole-warp values, said so to the compiler: the operands then stay in uniform registers)
        auto whole_warp = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dk0 = at_desc(smem_addr(ring), 16), dq0 = at_desc(smem_addr(qring), 16);
        int kn = 0, qn = 0;       // key tiles before this pair, query tiles so far
        int dn = 0, hn[2] = {}, sn[2] = {};  // score buffers filled; of each half what it waits for, and pairs that stayed
        bool ok = true, kept = false;
        PwCur c = cur;
        while (ok && whole_warp((int)(c.left > 0)) != 0) {
            const int nt = whole_warp(c.nt), q0 = whole_warp(c.qt), qe = whole_warp(c.qe);
            const bool stays = whole_warp((int)pw_stays(A, c)) != 0;
            PwCur nx = c;
            pw_next(A, nx);
            const bool keeps = whole_warp((int)pw_keeps(A, c, nx)) != 0;
            // few columns where the query tile has few rows
            const uint32_t idesc = (whole_warp((int)(c.q.rows * A.group <= 16)) ? at_idesc(128, 16, false)
                                                                               : at_idesc(128, kPwN, false)) |
                                   (BF || (mixed && stays) ? (1u << 7) | (1u << 10) : 0u);  // A, B: bf16, or f16
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ok && i < nt) {
                    if (stays) {
                        ok = pw_wait(&ctl.stay[i], sn[i]++);
                        if (pt_elect()) mbar_arrive(&ctl.k_empty[(kn + i) % S::kSlots]);
                    } else {
                        ok = pw_wait(&ctl.k_full[(kn + i) % S::kSlots], (kn + i) / S::kSlots);
                    }
                }
            for (int qt = q0; ok && qt <= qe; ++qt) {
                if (qt > q0 || !kept) {
                    ok = pw_wait(&ctl.q_full[qn % kPwQSlots], qn / kPwQSlots);
                    ++qn;
                }
                const int qs = (qn - 1) % kPwQSlots;
                const uint64_t qd = dq0 + (uint64_t)(qs * (S::kQItem >> 4));
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (ok && i < nt) {
                        const int buf = dn % kPwScores;
                        if (dn >= kPwScores && !(ok = pw_wait(&ctl.d_empty[buf], dn / kPwScores - 1))) break;
                        ++dn;
                        fence_proxy_async_smem();
                        at_fence_after();
                        const uint32_t d = tm + (uint32_t)(S::kColS + buf * kPwN);
                        const uint64_t kd = dk0 + (uint64_t)(((kn + i) % S::kSlots) * (S::kItem >> 4));
                        if (pt_elect()) {
                            if (stays) {
#pragma unroll
                                for (int j = 0; j < HD / 16; ++j)
                                    at_mma_ts(d, tm + (uint32_t)(S::kColK + i * (HD / 2) + 8 * j),
                                              qd + (uint64_t)(((j >> 2) * (kPwN * 128) + (j & 3) * 32) >> 4), idesc, j > 0 ? 1u : 0u);
                            } else {
#pragma unroll
                                for (int j = 0; j < HD / 16; ++j)
                                    pw_mma(d, kd + (uint64_t)(((j >> 2) * (kPaTile * 128) + (j & 3) * 32) >> 4),
                                           qd + (uint64_t)(((j >> 2) * (kPwN * 128) + (j & 3) * 32) >> 4), idesc, j > 0 ? 1u : 0u);
                            }
                            uint64_t* full = &ctl.d_full[i][hn[i] % kPwFull];
                            at_commit(full);
                            mbar_arrive(full);  // (an arrival of this thread's own, which orders the key masks)
                        }
                        ++hn[i];
                        __syncwarp();
                    }
                if (ok && nt == 1 && qt == qe) {
                    if (pt_elect()) {
                        uint64_t* full = &ctl.d_full[1][hn[1] % kPwFull];
                        at_commit(full);
                        mbar_arrive(full);
                    }
                    ++hn[1];
                    __syncwarp();
                }
                if ((qt < qe || !keeps) && pt_elect()) at_commit(&ctl.q_empty[qs]);
            }
            if (!stays && pt_elect())
                for (int i = 0; i < nt; ++i) at_commit(&ctl.k_empty[(kn + i) % S::kSlots]);
            __syncwarp();
            kn += nt;
            kept = keeps;
            c = nx;
        }
        // every MMA issued has completed before the CTA moves on
        if (pt_elect()) at_commit(&ctl.fin);
        __syncwarp();
        mbar_wait(&ctl.fin, 0, kPwWait);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ sums
        const int half = warp >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        bool ok = true, kept = false;
        int kn = 0, qn = 0;          // key tiles before this pair, query tiles so far
        int buf0 = 0, hn = 0;        // the next score buffer, this half's waits so far
        PwCur c = cur;
        while (c.left > 0) {
            bool keeps;
            {
                PwCur nx = c;
                pw_next(A, nx);
                keeps = pw_keeps(A, c, nx);
            }
            const bool mine = half < c.nt;
            const PaSeq& sq = c.q;
            const int kfirst = sq.lo + (c.kt + half) * kPaTile, r = (warp & 3) * 32 + lane, j = kfirst + r;
            float* w = A.W.p + (int64_t)c.s * A.W.ss + (int64_t)c.h * A.W.hs + j;
            const float old = mine && j < sq.hi && j < sq.p0 ? *w : 0.f;  // (a position that the call brings starts at 0)
            if (mine && pw_stays(A, c)) {
                // this lane's key to tensor memory (the products that read the one before are done: their sums were taken)
                const int slot = (kn + half) % S::kSlots;
                ok = ok && pw_wait(&ctl.k_full[slot], (kn + half) / S::kSlots);
                if (ok) {
                    at_fence_after();
                    const unsigned char* item = ring + slot * S::kItem;
#pragma unroll 1
                    for (int x = 0; x < HD / 8; x += 4) {
                        uint4 v[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            v[y] = *reinterpret_cast<const uint4*>(item + ((x + y) >> 3) * (kPaTile * 128) + at_swz(r, (x + y) & 7));
                        if (mixed) {
                            uint32_t (&u)[16] = *reinterpret_cast<uint32_t(*)[16]>(v);
#pragma unroll
                            for (int y = 0; y < 16; ++y) {
                                const float2 f = unpack2<false>(u[y]);
                                u[y] = pack2<true>(f.x, f.y);
                            }
                        }
                        at_st16(lane_addr + S::kColK + half * (HD / 2) + 4 * x, *reinterpret_cast<const float(*)[16]>(v));
                    }
                    at_wait_st();
                    at_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.stay[half]);
            }
            // query tiles from `clear` on are past this tile: every row sees all of it (but for the last tile's few rows, and
            // rows whose window has gone past)
            const int past = kfirst + kPaTile - 1 - sq.p0;  // rows from this one on
            const int clear = past <= 0 ? 0 : past <= sq.rows ? (past * A.group + kPwN - 1) / kPwN : INT_MAX;
            const int full = sq.rows * A.group / kPwN;  // tiles before this one have all their rows
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int qt = c.qt; qt <= c.qe; ++qt) {
                if (qt > c.qt || !kept) ++qn;
                const int qs = (qn - 1) % kPwQSlots;
                // (tiles of the other half too, one by one: a warp that ran ahead would release a tile twice)
                ok = ok && pw_wait(&ctl.q_full[qs], (qn - 1) / kPwQSlots);
                if (mine) {
                    const int buf = buf0 + half < kPwScores ? buf0 + half : buf0 + half - kPwScores;
                    ok = ok && pw_wait(&ctl.d_full[half][hn % kPwFull], hn / kPwFull);
                    ++hn;
                    const uint32_t from = lane_addr + S::kColS + buf * kPwN;
                    bool plain = qt >= clear && qt < full;
                    if (A.window > 0) plain = plain && kfirst > sq.p0 + div_by(A.by_group, qt * kPwN + kPwN - 1) - A.window;
                    at_fence_after();
                    if (ok && plain && (ctl.dead[qs][0] | ctl.dead[qs][1]) == 0) {
                        const uint64_t cs0 = pw_pair2(ctl.c[qs][0], ctl.c[qs][0]);
                        uint64_t part[2] = {0, 0};
                        // 32 columns at a time, the next ones on their way meanwhile
                        uint32_t v[2][32];
                        pt_ld32(from, v[0]);
#pragma unroll
                        for (int x = 0; x < kPwN / 32; ++x) {
                            at_wait_ld();
                            if (x + 1 < kPwN / 32) {
                                pt_ld32(from + 32 * (x + 1), v[(x + 1) & 1]);
                            } else {
                                at_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&ctl.d_empty[buf]);
                            }
                            const uint32_t(&w)[32] = v[x & 1];
#pragma unroll
                            for (int y = 0; y < 32; y += 4) {
                                const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(&ctl.nl[qs][32 * x + y]);
                                ulonglong2 cs = make_ulonglong2(cs0, cs0);  // (16-bit queries: one scale)
                                if constexpr (E8) cs = *reinterpret_cast<const ulonglong2*>(&ctl.c[qs][32 * x + y]);
                                pw_add2(part[0], pw_exp2(pw_fma2(pw_pair2(w[y], w[y + 1]), cs.x, nl.x)));
                                pw_add2(part[1], pw_exp2(pw_fma2(pw_pair2(w[y + 2], w[y + 3]), cs.y, nl.y)));
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            sum[2 * y] += __uint_as_float((uint32_t)part[y]);
                            sum[2 * y + 1] += __uint_as_float((uint32_t)(part[y] >> 32));
                        }
                    } else {
                        // the columns that see this lane's key: from `a` on, before `b`, not dead
                        const int nv = ok ? min(kPwN, sq.rows * A.group - qt * kPwN) : 0;
                        const int64_t shift = -(int64_t)qt * kPwN, row = j - sq.p0;
                        const int64_t a = max(row, (int64_t)0) * A.group + shift;
                        const int64_t b = A.window > 0 ? min((row + A.window) * A.group + shift, (int64_t)nv) : nv;
                        const auto below = [](int64_t n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
#pragma unroll 1
                        for (int x = 0; x < nv; x += 16) {
                            const int part = x & 64;
                            const uint64_t see = below(b - part) & ~below(a - part) & ~ctl.dead[qs][part >> 6];
                            const uint32_t bits = (uint32_t)(see >> (x & 63));
                            float v[16];
                            at_ld16(from + x, v);
                            at_wait_ld();
#pragma unroll
                            for (int y = 0; y < 16; ++y) {
                                const float e = fmaf(v[y], ctl.c[qs][x + y], ctl.nl[qs][x + y]);
                                sum[y & 3] += pa_exp2((bits >> y) & 1u ? e : -INFINITY);
                            }
                        }
                        at_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl.d_empty[buf]);
                    }
                }
                if (!mine && qt == c.qe) {
                    ok = ok && pw_wait(&ctl.d_full[half][hn % kPwFull], hn / kPwFull);
                    ++hn;
                }
                buf0 = buf0 + c.nt < kPwScores ? buf0 + c.nt : buf0 + c.nt - kPwScores;
                if ((qt < c.qe || !keeps) && lane == 0) mbar_arrive(&ctl.q_empty[qs]);
            }
            const uint32_t held = ctl.bits[(kn + half) % kPwBits][warp & 3];
            if (mine && j < sq.hi && (!ok || ((held >> lane) & 1u))) *w = ok ? old + ((sum[0] + sum[1]) + (sum[2] + sum[3])) : NAN;
            kn += c.nt;
            kept = keeps;
            pw_next(A, c);  // (again: it would not stay in registers)
        }
    }
    at_fence_before();
    __syncthreads();
    if (warp == kPwMma) {
        at_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <bool BF, int CB, int HD>
static int pw_launch(const PwArgs& A, int num_sms, cudaStream_t st) {
    using S = PwShape<CB, HD>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_weights_kernel<BF, CB, HD>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(kPwThreads), S::kSmem, st, A);
}
template <int HD>
static int pw_type(const PwArgs& A, int cd, int num_sms, cudaStream_t st) {
    return cd == kBF16   ? pw_launch<true, 16, HD>(A, num_sms, st)
           : cd == kF16  ? pw_launch<false, 16, HD>(A, num_sms, st)
           : cd == kE4M3 ? pw_launch<false, 8, HD>(A, num_sms, st)
                         : pw_launch<false, 4, HD>(A, num_sms, st);
}
int paged_key_weights(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                      const float* lse, float scale, int window, const KeyWeights& W, int num_sms, cudaStream_t st) {
    PwArgs A{};
    A.C = C, A.R = R, A.q = q, A.W = W, A.lse = lse, A.window = window;
    A.scale_log2 = scale * 1.4426950408889634f;
    A.group = q.heads / C.kv_heads;
    A.stay = (cache_dtype == kE4M3 || cache_dtype == kE2M1) && q.dtype == kBF16 ? kPwStayMixed : kPwStay;
    A.by_group = fast_div(A.group);
    if (R.cap == 0) return 0;
    // few rows a sequence's head, on average: the warp MMAs (over 32768 e2m1 keys of 8 heads, four query heads each:
    // 16 rows 22 us and 28 below, 20 rows 34 and 30; 32 sequences of 2048 bf16 keys: one row 28 and 39, 16 rows 45 and 42;
    // rows unlike each other: 31 single ones over 4096 keys and one sequence of 400 200 us there, of 600 103 here)
    const int64_t per = ((int64_t)R.n_rows + R.n_seqs - 1) / R.n_seqs * A.group;
    if (per <= 64) {
        PaArgs F{};
        F.C = C, F.R = R, F.q = q, F.window = window, F.scale_log2 = A.scale_log2, F.group = A.group;
        return paged_key_weights_few(F, W, lse, cache_dtype, hd, num_sms, st);
    }
    return hd == 64 ? pw_type<64>(A, cache_dtype, num_sms, st) : pw_type<128>(A, cache_dtype, num_sms, st);
}

}  // namespace dflash
