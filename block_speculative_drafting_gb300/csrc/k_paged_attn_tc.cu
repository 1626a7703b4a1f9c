// Attention of a pass's new rows over a paged cache for drafted blocks: units
// of up to 128 rows (rows x the query heads of a key/value head) on the
// fifth-generation tensor cores.  The line of work, its cut into equal parts
// and the joining of shared units are k_paged_attn.cu's.
//
// Tiles of 128 keys.  S = Q K^T (tcgen05.mma, M 128, N 128, Q in tensor
// memory, f32 scores in tensor memory), P = 2^(S c - m) by the thread that
// owns the row's tensor-memory lane, written over S as the A operand of
// O += P V (V as stored, the MN-major B operand; O in tensor memory).  Two S
// buffers: the next tile's scores are multiplied while this tile's softmax
// runs.  m moves only where a row's maximum passes it by some powers of two; O
// is then rescaled in place.  P is a hi + lo pair (the products then add no
// rounding of their own to the output's; with a 16-bit cache the tensor pipe has the
// time: a tile's MMAs take 0.8 us, its 64 KB 1.4 us of this SM's share of the
// memory).  Only bf16 outputs over 8 or 4 bits take P as one f16: off by 2^-11 of
// each key's part at most, an eighth of the output's own 2^-8 (32 blocks over 4 bits are
// 1.671e-3 of their norm from 64 bits, 1.659e-3 with the pair), where the pair costs
// 7 to 8 % (32 blocks over e4m3 64.2 -> 68.8 us, over 4 bits 65.0 -> 70.3: the softmax's
// registers and conversions).
//
// An MMA of M 128 costs what it costs with fewer rows, so a unit of up to 64
// rows holds every query twice: lanes r and r + 64 take the lower and the upper
// half of every tile's keys (zeros in P for the other half), each with its own
// m and sum, and are joined at the unit's end.  The softmax's exponentials,
// 4 lanes a clock and SM quarter, then spread over all four quarters (a tile's
// softmax on two quarters took 1.7 us).
//
// Warps: 0-3 softmax and epilogue, 4 the scores' MMAs, 5 the values', 6-9 load
// keys, 10-13 values, each into a ring of slots, one tile each, in the 128-byte
// swizzle.  16-bit loaders copy 16-byte chunks asynchronously (the slot's
// barrier counts them as they land); e4m3 loaders copy codes to places of their
// own and write their f16 values (exact) into the slots.  The MMA warps order
// those writes before their reads of them (a proxy fence after the barrier).
// A unit's queries are fetched by the softmax warps as the unit before ends, with
// an e4m3 cache by four more warps: 3 us less a unit (32 blocks 73.8 -> 66.6 us);
// a 16-bit cache's softmax needs the registers that those warps would take (71
// -> 75 us).
// The page of a key is looked up a tile before it is needed.
//
// Keys that no row sees are zeros behind a bit mask; keys that only some rows
// see are masked a row at a time, and where such a tile's values are not all
// finite (0 times an infinity would not be 0), those elements are taken out of
// the tile and added to the rows that see them.
//
// Per tile 1.36 us with a bf16 cache, the memory's rate (19 blocks over 16384 keys x
// 8 heads: 186 us, 6.8 TB/s), 1.26 us with an e4m3 one (173 us) and 1.25 with 4 bits (171 us), the
// softmax and the codes' way into the slots (an e2m1 lane's 16 bytes are 32 elements of a row and
// two block scales: paged_tile.cuh).  32 blocks over 1024 to 4096 keys: 65, 64 and 65 us; f16
// queries over e4m3 67, over 4 bits 69.  A unit's end and the next one's beginning take about
// 4 us, of which a tile that some rows see in part 2 and the outputs 2; start,
// epilogue and join of a call 13.
//
// Every wait is bounded (1 s of %globaltimer).  A role whose wait expires stops;
// the softmax then walks its remaining units without waiting and leaves NaN in
// their rows.
#include "kernels.cuh"
#include "paged_tile.cuh"

namespace dflash {

constexpr int kPtM = 128;
constexpr int kPtSoft = 128;  // softmax threads: warps 0-3
constexpr int kPtQk = kPtSoft / 32, kPtPv = kPtQk + 1, kPtLoad = kPtPv + 1;  // warps
constexpr uint64_t kPtWait = 1000000000ull;
constexpr int kPtBits = 16;  // tiles whose key masks are kept: more than the loaders can be ahead of the softmax

// BF: queries and outputs in bf16 (else f16), and a 16-bit cache with them; CB: bits of a cache's element, 16, 8
// (e4m3) or 4 (e2m1)
template <bool BF, int CB, int HD>
struct PtShape {
    static constexpr bool E8 = CB < 16;
    static constexpr int kLoadWarps = 4;  // of the keys, and as many of the values
    static constexpr int kLoaders = kLoadWarps * 32;
    static constexpr int kQueryWarps = E8 ? 4 : 0;
    static constexpr int kThreads = (kPtLoad + kQueryWarps) * 32 + 2 * kLoaders;
    static constexpr int KPW = kPaTile / kLoadWarps;  // keys of a loader warp: one a lane
    static constexpr int kItem = kPaTile * HD * 2;    // a slot: a tile's keys or values in 16 bits
    static constexpr int kSlots = (E8 ? 2 : 3) * (128 / HD);  // of the keys, and as many of the values
    // codes: half tiles on their way, 16 bytes a place, each place copied and read by one thread; beside a place of e2m1
    // codes the four bytes of the row's block scales that hold its two
    static constexpr int kRawCh = HD * CB / 128;  // places of a row
    static constexpr int kRaw = E8 ? 4 * (128 / HD) * 8 / CB : 0, kRawLd = KPW * kRawCh / 64;
    static constexpr int kRawCodes = kRaw * kRawLd * 16 * 2 * kLoaders;
    static constexpr int kRawBytes = kRawCodes + (CB == 4 ? kRawCodes / 4 : 0);
    static constexpr bool kSplitP = !E8 || !BF;
    static constexpr int kCtl = 15 * 1024;
    static constexpr size_t kSmem = 1024 /*alignment*/ + kCtl + 2 * (size_t)kSlots * kItem + kRawBytes;
    // tensor memory: two S / P buffers, O, Q
    static constexpr int kColS = 0, kColO = 256, kColQ = 384, kCols = 512;
};

struct PtCtl {
    // a slot's data written / its MMAs done; a tile's scores in S; its P in
    // place of them (a barrier a buffer: a thread may be a tile ahead of
    // another); its P V added; a unit's Q in place, its last scores multiplied
    uint64_t full[2][6], empty[2][6], s_full[2], p_full[2], o_done[2], q_full, q_free, fin[2];
    uint32_t tmem;
    uint32_t bits[kPtBits][4];  // a tile's valid keys
    uint32_t bad[4];            // keys whose values are not all finite
    float rf[4][kPtM];          // what the queries of a unit (and the three after it) were scaled down by
    float2 ml[kPtM];            // a unit's row references and sums, for the join of a row's two lanes
    alignas(16) float xo[2][64][20];        // sixteen columns of the upper lanes' outputs on their way to the lower ones
};

DF_DEV uint32_t pt_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return r;
}
DF_DEV void pt_st16(uint32_t taddr, const uint32_t (&w)[16]) {
    at_st16(taddr, *reinterpret_cast<const float(*)[16]>(w));
}
// named barrier 1: the softmax threads
DF_DEV void pt_soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPtSoft) : "memory"); }
DF_DEV bool pt_soft_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(kPtSoft)
        : "memory");
    return r != 0;
}
// the part of a unit that a share holds: from c on
DF_DEV int pt_tiles(const PaCur& c) { return min(c.q.ntiles - c.tile, c.left); }
template <int MT>
DF_DEV void pt_skip(const PaArgs& A, PaCur& c, int n) {
    c.left -= n - 1;
    c.tile += n - 1;
    pa_next(A, MT, c);
}

// A unit's queries to tensor memory at `to` (row t % MT of the unit), after `free` has waited for it.  An 8-bit cache's
// warps of queries: a bf16 row is brought into f16 by a power of two, left in ctl.rf, its halves read for their largest
// element and then again (registers).
template <bool BF, int CB, int HD, int MT, class F>
DF_DEV bool pt_queries(const PaArgs& A, PtCtl& ctl, const PaCur& c, int unit, int t, uint32_t to, F free) {
    constexpr bool E8 = CB < 16;
    constexpr int kHalves = E8 ? 2 : 1, NX = HD / 8 / kHalves;
    const int h = c.u % A.C.kv_heads, mm = (c.u / A.C.kv_heads) * MT + t % MT;
    const bool in = mm < c.q.rows * A.group;
    const int row = c.q.row0 + mm / A.group, hq = h * A.group + mm % A.group;
    const unsigned char* qp = A.q.p + (int64_t)row * A.q.rs + (int64_t)hq * A.q.hs;
    uint4 x[NX];
    uint32_t (&w)[4 * NX] = *reinterpret_cast<uint32_t(*)[4 * NX]>(x);
    auto load = [&](int half) {
#pragma unroll
        for (int j = 0; j < NX; ++j)
            x[j] = in ? *reinterpret_cast<const uint4*>(qp + 16 * (half * NX + j)) : make_uint4(0u, 0u, 0u, 0u);
    };
    float rf = 1.f, down = 1.f;
    if constexpr (!E8) {
        load(0);
    } else if constexpr (BF) {
        float mx = 0.f;
#pragma unroll 1
        for (int half = 0; half < kHalves; ++half) {
            load(half);
#pragma unroll
            for (int j = 0; j < 4 * NX; ++j) {
                const float2 f = unpack2<true>(w[j]);
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        // times 2^-x, the largest in [1, 2): what f16 cannot hold of the row then is under 2^-25 of that
        if (mx > 0.f && mx < INFINITY) {
            const int e = min(max(ilogbf(mx), -120), 120);
            down = ldexpf(1.f, -e);
            rf = ldexpf(1.f, e);
        }
    }
    if (!free()) return false;
    at_fence_after();
    if constexpr (E8) ctl.rf[unit & 3][t] = rf;
#pragma unroll 1
    for (int half = 0; half < kHalves; ++half) {
        if constexpr (E8) {
            load(half);
            if constexpr (BF) {
#pragma unroll
                for (int j = 0; j < 4 * NX; ++j) {
                    const float2 f = unpack2<true>(w[j]);
                    w[j] = pack2<false>(f.x * down, f.y * down);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * NX; i += 16)
            pt_st16(to + 4 * NX * half + i, *reinterpret_cast<const uint32_t(*)[16]>(w + i));
    }
    at_wait_st();
    at_fence_before();
    mbar_arrive(&ctl.q_full);
    return true;
}

// MT: rows of a unit's tile, 64 (each query on two lanes) or 128
template <bool BF, int CB, int HD, int MT>
__global__ void __launch_bounds__((PtShape<BF, CB, HD>::kThreads), 1)
    paged_attn_tc_kernel(const __grid_constant__ PaArgs A) {
    using S = PtShape<BF, CB, HD>;
    constexpr bool E8 = S::E8;
    constexpr bool PB = BF && !E8;  // the MMAs' type: bf16, or f16
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    unsigned char* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
    PtCtl& ctl = *reinterpret_cast<PtCtl*>(sm);
    static_assert(sizeof(PtCtl) <= S::kCtl, "control block");
    unsigned char* ring = sm + S::kCtl;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S::kSlots; ++i) {
            // (16-bit keys' copies arrive by themselves; their warps arrive beside them for the key masks)
            mbar_init(&ctl.full[i & 1][i >> 1], S::kLoaders + (!E8 && (i & 1) == 0 ? S::kLoadWarps : 0));
            mbar_init(&ctl.empty[i & 1][i >> 1], 1);
        }
        // (the commit, and an arrival of the MMA thread's own that orders the key masks)
        mbar_init(&ctl.s_full[0], 2);
        mbar_init(&ctl.s_full[1], 2);
        mbar_init(&ctl.p_full[0], kPtSoft);
        mbar_init(&ctl.p_full[1], kPtSoft);
        mbar_init(&ctl.o_done[0], 1);
        mbar_init(&ctl.o_done[1], 1);
        mbar_init(&ctl.q_full, kPtSoft);
        mbar_init(&ctl.q_free, 1);
        mbar_init(&ctl.fin[0], 1);
        mbar_init(&ctl.fin[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPtQk) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&ctl.tmem)),
                     "r"(S::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    at_fence_before();
    __syncthreads();
    at_fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_wait();
    pdl_trigger();
    // this CTA's share of the line
    int chunk;
    const PaCur cur = pa_share(A, MT, kPtOver, lane, chunk);
    if (threadIdx.x == 0) A.ws_join[blockIdx.x].last = -1, A.ws_odd[blockIdx.x] = 0;

    if (S::kQueryWarps > 0 && warp >= kPtLoad + 2 * S::kLoadWarps) {
        // ------------------------------------------------------------ queries (an e4m3 cache's)
        const int t = (warp & 3) * 32 + lane;
        int unit = 0;
        for (PaCur c = cur; c.left > 0; ++unit) {
            // (the unit before has multiplied its last scores)
            auto free = [&]() {
                return unit == 0 || __all_sync(0xffffffffu, mbar_wait(&ctl.q_free, (unit - 1) & 1, kPtWait));
            };
            if (!pt_queries<BF, CB, HD, MT>(A, ctl, c, unit, t, tmem + ((uint32_t)((warp & 3) * 32) << 16) + S::kColQ, free))
                break;
            pt_skip<MT>(A, c, pt_tiles(c));
        }
    } else if (warp >= kPtLoad) {
        // ------------------------------------------------------------ loads
        const int side = (warp - kPtLoad) / S::kLoadWarps, lw = (warp - kPtLoad) % S::kLoadWarps;  // 0 keys, 1 values
        unsigned char* slots = ring + side * S::kSlots * S::kItem;
        const unsigned char* tensor = side ? A.C.v : A.C.k;
        const int64_t sp = side ? A.C.vs[0] : A.C.ks[0], ss = side ? A.C.vs[1] : A.C.ks[1],
                      sh = side ? A.C.vs[2] : A.C.ks[2];
        int n = 0;  // the next tile
        // this lane's key of a tile: its page (-1: not held), looked up early, and its rows of the two tensors
        struct Look {
            int id, slot, h;
        };
        auto look = [&](const PaCur& c) -> Look {
            Look k;
            const int key = c.q.lo + c.tile * kPaTile + lw * S::KPW + lane;
            k.h = c.u % A.C.kv_heads;
            k.id = -1;
            k.slot = 0;
            if (key < c.q.hi) k.id = page_entry(A.R, c.s, key, k.slot);
            return k;
        };
        auto wait_empty = [&](int tile) -> bool {
            return tile < S::kSlots ||
                   __all_sync(0xffffffffu, mbar_wait(&ctl.empty[side][tile % S::kSlots], ((tile / S::kSlots) - 1) & 1, kPtWait));
        };
        // the tiles in order: emit(row, blocks) is called with a lane's key's row and its block scales (null: not held)
        auto walk = [&](auto emit) {
            PaCur c = cur;
            Look ahead{-1, 0, 0};
            if (c.left > 0) ahead = look(c);
            while (c.left > 0) {
                const unsigned char *row = nullptr, *blocks = nullptr;
                if (page_held(ahead.id, A.C.n_pages)) {
                    row = tensor + ahead.id * sp + ahead.slot * ss + ahead.h * sh;
                    if constexpr (CB == 4)
                        blocks = (side ? A.C.vb : A.C.kb) + ahead.id * (side ? A.C.vbs[0] : A.C.kbs[0]) +
                                 ahead.slot * (side ? A.C.vbs[1] : A.C.kbs[1]) + ahead.h * (side ? A.C.vbs[2] : A.C.kbs[2]);
                }
                if (side == 0) {
                    const uint32_t b = __ballot_sync(0xffffffffu, row != nullptr);
                    if (lane == 0) ctl.bits[n % kPtBits][lw] = b;
                }
                pa_next(A, MT, c);
                if (c.left > 0) ahead = look(c);
                if (!emit(row, blocks)) return;
            }
        };
        if constexpr (!E8) {
            constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows a copy instruction covers
            walk([&](const unsigned char* rows, const unsigned char*) -> bool {
                if (!wait_empty(n)) return false;
                const uint32_t dst = smem_addr(slots) + (n % S::kSlots) * S::kItem;
#pragma unroll
                for (int i = 0; i < S::KPW / RPI; ++i) {
                    const int r = i * RPI + lane / CH, ch = lane % CH;
                    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                    const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * ch : A.q.p;  // (nothing is read)
                    cp16(dst + (ch >> 3) * (kPaTile * 128) + at_swz(lw * S::KPW + r, ch & 7), src, p ? 16 : 0);
                }
                // arrives once this thread's copies have landed
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(&ctl.full[side][n % S::kSlots]))
                             : "memory");
                // (that follows the copies alone: the tile's key mask, written by this lane, takes an arrival of its own)
                if (side == 0 && lane == 0) mbar_arrive(&ctl.full[0][n % S::kSlots]);
                ++n;
                return true;
            });
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            using Lanes = TileLanes<CB, HD>;
            constexpr int RPI = Lanes::RPI, LD = S::kRawLd;  // copies of a lane a half tile
            const int ch = Lanes::place(lane), lane_row = Lanes::row(lane);
            const int self = threadIdx.x - kPtLoad * 32;
            unsigned char* raw = ring + 2 * S::kSlots * S::kItem + self * 16;
            unsigned char* raw_scale = ring + 2 * S::kSlots * S::kItem + S::kRawCodes + self * 4;
            constexpr int kPlace = 2 * S::kLoaders * 16;  // from one of a thread's places to the next
            // a half tile's codes as f16, 32 bytes a place (64 of e2m1 codes)
            auto write = [&](int half) -> bool {
                const int tile = half >> 1, slot = tile % S::kSlots;
                if ((half & 1) == 0 && !wait_empty(tile)) return false;
                unsigned char* dst = slots + slot * S::kItem;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int key = lw * S::KPW + ((half & 1) * LD + i) * RPI + lane_row;
                    const uint4 x = *reinterpret_cast<const uint4*>(raw + ((half % S::kRaw) * LD + i) * kPlace);
                    uint32_t scales = 0;
                    if constexpr (CB == 4)
                        scales = *reinterpret_cast<const uint32_t*>(raw_scale + ((half % S::kRaw) * LD + i) * (kPlace / 4)) >>
                                 ((2 * ch & 3) * 8);
                    tile_place<CB, HD>(dst, key, ch, x, scales);
                }
                if (half & 1) mbar_arrive(&ctl.full[side][slot]);
                return true;
            };
            walk([&](const unsigned char* rows, const unsigned char* blocks) -> bool {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int half = 2 * n + hf;
#pragma unroll
                    for (int i = 0; i < LD; ++i) {
                        const int r = (hf * LD + i) * RPI + lane_row;
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
    } else if (warp >= kPtQk) {
        // ------------------------------------------------------------ MMAs
        // Two warps, so that the waits of one fall into the other's MMAs: an issuing thread is held up to within
        // three or four MMAs of the pipe, and one warp's waits left the pipe idle for 0.6 us a tile.
        // (whole-warp values, said so to the compiler: see pt_elect in paged_tile.cuh)
        auto whole_warp = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t kType = PB ? (1u << 7) | (1u << 10) : 0u;  // A, B: bf16, or f16
        constexpr uint64_t kItemD = S::kItem >> 4;
        auto wait = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, kPtWait)); };
        bool ok = true;
        int tg = 0, unit = 0;  // tiles, units so far
        PaCur c = cur;
        while (ok && whole_warp((int)(c.left > 0)) != 0) {
            const int tiles = whole_warp(pt_tiles(c));
            if (warp == kPtQk) {
                constexpr uint32_t idS = at_idesc(kPtM, kPaTile, false) | kType;
                const uint64_t dk0 = at_desc(smem_addr(ring), 16);
                ok = wait(&ctl.q_full, unit);
                for (int i = 0; ok && i < tiles; ++i, ++tg) {
                    const int slot = tg % S::kSlots;
                    // the tile's keys are there, and its buffer's last P V (tile tg - 2) is added
                    if (!(ok = wait(&ctl.full[0][slot], tg / S::kSlots) &&
                               (tg < 2 || wait(&ctl.o_done[tg & 1], (tg >> 1) - 1))))
                        break;
                    fence_proxy_async_smem();
                    at_fence_after();
                    const uint64_t kd = dk0 + (uint64_t)slot * kItemD;
                    if (pt_elect()) {
#pragma unroll
                        for (int j = 0; j < HD / 16; ++j)
                            at_mma_ts(tm + S::kColS + (tg & 1) * 128, tm + (uint32_t)(S::kColQ + 8 * j),
                                      kd + (uint64_t)(((j >> 2) * (kPaTile * 128) + (j & 3) * 32) >> 4), idS, j > 0 ? 1u : 0u);
                        at_commit(&ctl.empty[0][slot]);
                        at_commit(&ctl.s_full[tg & 1]);
                        mbar_arrive(&ctl.s_full[tg & 1]);
                    }
                    __syncwarp();
                }
                if (S::kQueryWarps > 0 && pt_elect()) at_commit(&ctl.q_free);
                __syncwarp();
            } else {
                constexpr uint32_t idO = at_idesc(kPtM, HD, true) | kType;
                const uint64_t dv0 = at_desc(smem_addr(ring) + S::kSlots * S::kItem, kPaTile * 128);
                for (int i = 0; ok && i < tiles; ++i, ++tg) {
                    const int slot = tg % S::kSlots;
                    if (!(ok = wait(&ctl.full[1][slot], tg / S::kSlots) && wait(&ctl.p_full[tg & 1], tg >> 1))) break;
                    fence_proxy_async_smem();
                    at_fence_after();
                    const uint64_t vd = dv0 + (uint64_t)slot * kItemD;
                    if (pt_elect()) {
#pragma unroll
                        for (int j = 0; j < kPaTile / 16; ++j) {
                            // keys 16 j ..: eight columns of P, hi, and sixteen columns on its lo
                            const uint32_t p = tm + (uint32_t)(S::kColS + (tg & 1) * 128 + 32 * (j >> 1) + 8 * (j & 1));
                            const uint64_t v = vd + (uint64_t)((j * 2048) >> 4);
                            at_mma_ts(tm + S::kColO, p, v, idO, 1u);
                            if constexpr (S::kSplitP) at_mma_ts(tm + S::kColO, p + 16, v, idO, 1u);
                        }
                        at_commit(&ctl.empty[1][slot]);
                        at_commit(&ctl.o_done[tg & 1]);
                    }
                    __syncwarp();
                }
            }
            ++unit;
            pt_skip<MT>(A, c, tiles);
        }
        // every MMA issued has completed before the CTA moves on
        if (pt_elect()) at_commit(&ctl.fin[warp - kPtQk]);
        __syncwarp();
        mbar_wait(&ctl.fin[warp - kPtQk], 0, kPtWait);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ queries, softmax, epilogue
        constexpr int D = kPtM / MT;      // lanes of a row
        constexpr int NC = 4 / D;         // 32-key chunks of a lane
        const int t = threadIdx.x, r = t % MT, copy = t / MT;  // this lane's row of the unit, and its share of the keys
        const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        int tg = 0, unit = 0;  // tiles, units so far
        PaCur c = cur;
        auto queries = [&]() {  // (where no warps of their own bring them)
            if (S::kQueryWarps == 0 && c.left > 0)
                pt_queries<BF, CB, HD, MT>(A, ctl, c, unit, t, lane_addr + S::kColQ, []() { return true; });
        };
        queries();
        while (c.left > 0) {
            const PaSeq sq = c.q;
            const int u = c.u, tile0 = c.tile, tiles = pt_tiles(c);
            const int h = u % A.C.kv_heads, rt = u / A.C.kv_heads;
            const int mvalid = min(MT, sq.rows * A.group - rt * MT);
            const bool in = r < mvalid, warp_in = (warp * 32) % MT < mvalid;
            const int mm = rt * MT + r, row = sq.row0 + mm / A.group, hq = h * A.group + mm % A.group;
            const int pos = in ? sq.p0 + mm / A.group : -1;
            const int wlo = A.window > 0 ? pos - A.window + 1 : 0;
            const int pmin = sq.p0 + (rt * MT) / A.group, pmax = sq.p0 + (rt * MT + mvalid - 1) / A.group;
            const int wtop = A.window > 0 ? pmax - A.window + 1 : 0;
            {
                // O cleared (the unit before has read it)
                const uint32_t zero[16] = {};
#pragma unroll 1
                for (int i = 0; i < HD / 16; ++i) pt_st16(lane_addr + S::kColO + 16 * i, zero);
                at_wait_st();
            }
            const float ks = E8 && A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f;
            float cs = 0.f;

            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < tiles; ++i, ++tg) {
                const uint32_t sb = lane_addr + (uint32_t)(S::kColS + (tg & 1) * 128);
                const uint32_t mine = sb + 32 * NC * copy;  // this lane's chunks
                // (all threads or none: a warp that went on alone would leave the others at a barrier)
                ok = __all_sync(0xffffffffu, ok && mbar_wait(&ctl.s_full[tg & 1], (tg >> 1) & 1, kPtWait));
                const int kfirst = sq.lo + (tile0 + i) * kPaTile, klast = kfirst + kPaTile - 1;
                const bool edge = klast > pmin || kfirst < wtop;  // (the same for every thread)
                if (edge) {
                    if (t < 4) ctl.bad[t] = 0;
                    ok = !pt_soft_or(!ok);
                }
                if (!ok) continue;
                at_fence_after();
                if (i == 0) cs = fminf(fmaxf(A.scale_log2 * ks * (E8 ? ctl.rf[unit & 3][t] : 1.f), 1e-37f), 3e38f);
                const uint32_t* bits = ctl.bits[tg % kPtBits];
                const bool full = !edge && (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
                // this row's view of 32 keys
                auto view = [&](int q) -> uint32_t {
                    const int hi = pos - kfirst - 32 * q, lo = wlo - kfirst - 32 * q;
                    uint32_t v = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
                    if (lo > 0) v = lo > 31 ? 0u : v & (0xffffffffu << lo);
                    return v & bits[q];
                };
                // 32 scores, those out of view at -inf
                auto scores = [&](int q, float* v) {
                    pt_ld32(mine + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(v));
                };
                auto hide = [&](int q, float* v) {
                    if (full) return;
                    const uint32_t see = view(NC * copy + q);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((see >> j) & 1u)) v[j] = -INFINITY;
                };
                auto largest = [](const float* v) {
                    float a[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int j = 4; j < 32; ++j) a[j & 3] = fmaxf(a[j & 3], v[j]);
                    return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                };
                // (a lane's 64 or 128 scores are read twice, 32 at a time: more of them do not fit the registers)
                float v[32];
                float mx = -INFINITY;
                if (warp_in) {
#pragma unroll 1
                    for (int q = 0; q < NC; ++q) {
                        scores(q, v);
                        at_wait_ld();
                        hide(q, v);
                        mx = fmaxf(mx, largest(v));
                    }
                    mx *= cs;
                }
                constexpr float under = kPaUnder<PB>;
                if (__any_sync(0xffffffffu, mx > m + (kPaLazy + under))) {
                    const float to = mx > m + (kPaLazy + under) ? mx - under : m;
                    const float f = to == m ? 1.f : pa_exp2(m - to);
                    m = to;
                    l *= f;
                    if (i > 0) {
                        // P V of the tile before has been added
                        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.o_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, kPtWait));
                        at_fence_after();
#pragma unroll 1
                        for (int x = 0; x < HD; x += 16) {
                            float o[16];
                            at_ld16(lane_addr + S::kColO + x, o);
                            at_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= f;
                            at_st16(lane_addr + S::kColO + x, o);
                        }
                    }
                }
                const float mr = m == -INFINITY ? 0.f : m;
                if (edge) {
                    // keys that some rows see and others do not: are their values finite?  (thread t: key t)
                    unsigned char* vt = ring + (S::kSlots + tg % S::kSlots) * S::kItem;
                    bool bad = false;
                    const bool got = ok && mbar_wait(&ctl.full[1][tg % S::kSlots], (tg / S::kSlots) & 1, kPtWait);
#pragma unroll 4
                    for (int x = 0; x < (got ? HD / 8 : 0); ++x) {
                        const uint4 y = *reinterpret_cast<const uint4*>(vt + (x >> 3) * (kPaTile * 128) + at_swz(t, x & 7));
                        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) bad |= !finite16<PB>(w[j]) || !finite16<PB>(w[j] >> 16);
                    }
                    const uint32_t b = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0 && b != 0) ctl.bad[warp] = b;
                    if (pt_soft_or(!got)) {
                        ok = false;
                        continue;
                    }
                    if ((ctl.bad[0] | ctl.bad[1] | ctl.bad[2] | ctl.bad[3]) != 0) {
                        if (i > 0) ok = __all_sync(0xffffffffu, mbar_wait(&ctl.o_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, kPtWait));
                        at_fence_after();
#pragma unroll 1
                        for (int j = 0; j < kPaTile; ++j) {
                            if (!((ctl.bad[j >> 5] >> (j & 31)) & 1u)) continue;
                            const float s = __uint_as_float(pt_ld1(sb + j));
                            at_wait_ld();
                            // (a row's lanes each take their own keys)
                            const bool see = ((view(j >> 5) >> (j & 31)) & 1u) && (j >> 5) / NC == copy;
                            const float p = pa_exp2(fmaf(s, cs, -mr));
#pragma unroll 1
                            for (int x = 0; x < HD; x += 16) {
                                float o[16];
                                at_ld16(lane_addr + S::kColO + x, o);
                                at_wait_ld();
#pragma unroll
                                for (int y = 0; y < 16; ++y) {
                                    const int d = x + y;
                                    const uint16_t e = *reinterpret_cast<const uint16_t*>(
                                        vt + (d >> 6) * (kPaTile * 128) + at_swz(j, (d & 63) >> 3) + (d & 7) * 2);
                                    if (see && !finite16<PB>(e)) o[y] = fmaf(p, unpack2<PB>(e).x, o[y]);
                                }
                                at_st16(lane_addr + S::kColO + x, o);
                                at_wait_st();
                            }
                        }
                        pt_soft_sync();
                        if (bad) {
#pragma unroll 1
                            for (int d = 0; d < HD; ++d) {
                                uint16_t* e = reinterpret_cast<uint16_t*>(vt + (d >> 6) * (kPaTile * 128) +
                                                                          at_swz(t, (d & 63) >> 3) + (d & 7) * 2);
                                if (!finite16<PB>(*e)) *e = 0;
                            }
                        }
                        fence_proxy_async_smem();
                    }
                }
                // P over S, 32 keys at a time: sixteen columns of hi pairs, sixteen of lo
                if (warp_in) {
                    float ls[4] = {l, 0.f, 0.f, 0.f};
                    auto weights = [&](int q, const float* x) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float a = pa_exp2(fmaf(x[2 * j], cs, -mr)), b = pa_exp2(fmaf(x[2 * j + 1], cs, -mr));
                            ls[(2 * j) & 3] += a;
                            ls[(2 * j + 1) & 3] += b;
                            hi[j] = pack2<PB>(a, b);
                            if constexpr (S::kSplitP) {
                                const float2 y = unpack2<PB>(hi[j]);
                                lo[j] = pack2<PB>(a - y.x, b - y.y);
                            }
                        }
                        pt_st16(mine + 32 * q, hi);
                        if constexpr (S::kSplitP) pt_st16(mine + 32 * q + 16, lo);
                    };
#pragma unroll 1
                    for (int q = 0; q < NC; ++q) {
                        scores(q, v);
                        at_wait_ld();
                        hide(q, v);
                        weights(q, v);
                    }
                    l = (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    // the keys of the row's other lane
                    if constexpr (D > 1) {
                        const uint32_t zero[16] = {};
#pragma unroll
                        for (int q = 0; q < NC; ++q) {
                            pt_st16(sb + 32 * (NC * (copy ^ 1) + q), zero);
                            if constexpr (S::kSplitP) pt_st16(sb + 32 * (NC * (copy ^ 1) + q) + 16, zero);
                        }
                    }
                }
                at_wait_st();
                at_fence_before();
                mbar_arrive(&ctl.p_full[tg & 1]);
            }

            // ------------------------------------------------------------ the unit's end
            const bool whole = tile0 == 0 && tile0 + tiles == sq.ntiles;
            const int part = blockIdx.x * 2 + (tile0 == 0 ? 1 : 0);
            if (!whole && tile0 == 0 && t == 0)
                A.ws_join[blockIdx.x] = pa_join_entry(c, rt, MT, mvalid, h, sq.ntiles - tiles, chunk);
            // the next unit's queries, whose scores may then be multiplied while this one's outputs are written
            // (its last scores have been read: Q is free)
            pt_skip<MT>(A, c, tiles);
            ++unit;
            queries();
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&ctl.o_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, kPtWait));
            at_fence_after();
            if (!ok) l = NAN;
            float fo = 1.f;  // this lane's output to the row's reference
            if constexpr (D > 1) {
                ctl.ml[t] = make_float2(m, l);
                pt_soft_sync();
                const float2 y = ctl.ml[t ^ MT];
                const float to = fmaxf(m, y.x);
                fo = m == -INFINITY ? 1.f : pa_exp2(m - to);  // (without a maximum the sums are 0 or NaN)
                l = l * fo + y.y * (y.x == -INFINITY ? 1.f : pa_exp2(y.x - to));
                m = to;
            }
            const float vs = E8 && A.C.v_scale != nullptr ? A.C.v_scale[h] : 1.f;
            const float inv = l == 0.f ? 0.f : vs / l;
            unsigned char* op = A.out.p + (int64_t)row * A.out.rs + (int64_t)hq * A.out.hs;
            float* wp = A.ws_o + ((int64_t)part * MT + r) * HD;
            bool odd = false;
#pragma unroll 1
            for (int x = 0; x < HD; x += 16) {
                float o[16];
                at_ld16(lane_addr + S::kColO + x, o);
                at_wait_ld();
                if constexpr (D > 1) {
                    // the upper lane's columns to the lower lane
                    float* xo = ctl.xo[(x >> 4) & 1][r];
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] *= fo;
                    if (copy == 1) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<float4*>(xo + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                    pt_soft_sync();
                    if (copy == 0) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(xo + j);
                            o[j] += y.x, o[j + 1] += y.y, o[j + 2] += y.z, o[j + 3] += y.w;
                        }
                    }
                }
                if (!in || copy != 0) continue;
                if (whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = pack2<BF>(o[2 * j] * inv, o[2 * j + 1] * inv);
                    if constexpr (!E8) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) odd |= o[j] != o[j];
                    }
                    *reinterpret_cast<uint4*>(op + 2 * x) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(op + 2 * x + 16) = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(wp + x + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
            if (!E8 && odd && pa_weighs(l)) {
                pa_mark_odd<BF>(op, HD);
                A.ws_odd[blockIdx.x] = 1;
            }
            if (in && copy == 0) {
                if (!whole)
                    A.ws_ml[(int64_t)part * MT + r] = make_float2(m, l);
                else if (A.lse != nullptr)
                    A.lse[(int64_t)row * A.q.heads + hq] =
                        l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + log2f(l)) * 0.69314718056f);
            }
            at_fence_before();
        }
    }
    at_fence_before();
    __syncthreads();
    if (warp == kPtQk) {
        at_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
    }
}

template <bool BF, int CB, int HD, int MT>
static int pt_launch(const PaArgs& A, int num_sms, cudaStream_t st) {
    using S = PtShape<BF, CB, HD>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_attn_tc_kernel<BF, CB, HD, MT>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(S::kThreads), S::kSmem, st, A);
}
template <int HD, int MT>
static int pt_type(const PaArgs& A, int cache_dtype, int num_sms, cudaStream_t st) {
    if (cache_dtype == kE2M1)
        return A.q.dtype == kBF16 ? pt_launch<true, 4, HD, MT>(A, num_sms, st) : pt_launch<false, 4, HD, MT>(A, num_sms, st);
    return cache_dtype == kBF16  ? pt_launch<true, 16, HD, MT>(A, num_sms, st)
           : cache_dtype == kF16 ? pt_launch<false, 16, HD, MT>(A, num_sms, st)
           : A.q.dtype == kBF16 ? pt_launch<true, 8, HD, MT>(A, num_sms, st)
                                 : pt_launch<false, 8, HD, MT>(A, num_sms, st);
}

int paged_attention_tc(const PaArgs& A, int cache_dtype, int hd, int mt, int num_sms, cudaStream_t st) {
    if (mt == 64)
        return hd == 64 ? pt_type<64, 64>(A, cache_dtype, num_sms, st) : pt_type<128, 64>(A, cache_dtype, num_sms, st);
    return hd == 64 ? pt_type<64, 128>(A, cache_dtype, num_sms, st) : pt_type<128, 128>(A, cache_dtype, num_sms, st);
}

}  // namespace dflash
