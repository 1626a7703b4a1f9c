// Attention of a pass's new rows over a paged cache for drafted blocks: units
// of up to 128 rows (rows x the query heads of a key/value head) on the
// fifth-generation tensor cores.  The line of work, its cut into equal parts
// and the joining of shared units are k_paged_attn.cu's.
//
// Tiles of 128 keys.  S = Q K^T (tcgen05.mma, M 128, N 128, Q in tensor
// memory, f32 scores in tensor memory), P = 2^(S c - m) by one thread a row,
// written over S as the A operand of O += P V (V as stored, the MN-major B
// operand; O in tensor memory).  Two S buffers: the next tile's scores are
// multiplied while this tile's softmax runs.  m moves only where a row's
// maximum passes it by kPaLazy; O is then rescaled in place.  A 16-bit cache's
// P is a hi + lo pair (the products then add no rounding of their own to the
// output's; the tensor pipe has the time: a tile's MMAs take 0.8 us, its 64 KB
// 1.4 us of this SM's share of the memory); an e4m3 cache's, whose tile is
// half the bytes, is one f16 (2^-12 relative, under a bf16 output's 2^-9).
//
// Warps: 0-3 softmax and epilogue (thread = query row = tensor-memory lane),
// 4 the MMAs (one lane), the rest loaders.  Keys and values go through a ring
// of slots, one tile's keys or values each, in the 128-byte swizzle, in the
// order the MMAs take them: K0, K1, V0, K2, V1, ..., V(n-1) of a unit, then
// the next unit's.  16-bit loaders copy 16-byte chunks asynchronously and
// signal a slot kLag items later; e4m3 loaders hold four items in registers
// and write their codes' f16 values (exact).
//
// Keys that no row sees are zeros behind a bit mask; keys that only some rows
// see are masked a row at a time, and where such a tile's values are not all
// finite (0 times an infinity would not be 0), those elements are taken out of
// the tile and added to the rows that see them.
//
// Every wait is bounded (1 s of %globaltimer).  Where one expires the CTA
// gives up: it walks its remaining units without waiting and leaves NaN in
// their rows.
#include <type_traits>

#include "kernels.cuh"
#include "paged_attn.cuh"
#include "tc.cuh"

namespace dflash {

constexpr int kPtM = 128;
constexpr int kPtSoft = 128;  // softmax threads: warps 0-3
constexpr uint64_t kPtWait = 1000000000ull;
constexpr int kPtBits = 16;  // tiles whose key masks are kept: more than the loaders can be ahead of the softmax

template <bool BF, bool E8, int HD>
struct PtShape {
    static constexpr int kLoadWarps = E8 ? 8 : 4;
    static constexpr int kLoaders = kLoadWarps * 32;
    static constexpr int kThreads = kPtSoft + 32 + kLoaders;
    static constexpr int KPW = kPaTile / kLoadWarps;  // keys a loader warp handles
    static constexpr int kItem = kPaTile * HD * 2;    // a slot: a tile's keys or values in 16 bits
    static constexpr int kSlots = HD == 128 ? 6 : 12;
    static constexpr int kLag = HD == 128 ? 3 : 6;    // items copied and not yet signalled
    static constexpr bool kSplitP = !E8;
    static constexpr int kCtl = 1024;
    static constexpr size_t kSmem = 1024 /*alignment*/ + kCtl + (size_t)kSlots * kItem;
    // tensor memory: two S / P buffers, O, Q
    static constexpr int kColS = 0, kColO = 256, kColQ = 384, kCols = 512;
};

struct PtCtl {
    // a slot's data written / its MMAs done; a tile's scores in S; its P in
    // place of them (a barrier a buffer: a thread may be a tile ahead of
    // another); its P V added; a unit's Q in place and O cleared
    uint64_t full[12], empty[12], s_full[2], p_full[2], o_done, q_full, fin;
    uint32_t tmem;
    int abort;
    uint32_t bits[kPtBits][4];  // a tile's valid keys
    uint32_t bad[4];            // keys whose values are not all finite
};

DF_DEV void pt_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
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
template <bool BF>
DF_DEV bool finite16(uint32_t h) {
    return BF ? (h & 0x7f80u) != 0x7f80u : (h & 0x7c00u) != 0x7c00u;
}
// the part of a unit that a share holds: from c on
DF_DEV int pt_tiles(const PaCur& c) { return (int)min((int64_t)(c.q.ntiles - c.tile), c.left); }
DF_DEV void pt_skip(const PaArgs& A, PaCur& c, int n) {
    c.left -= n - 1;
    c.tile += n - 1;
    pa_next(A, kPtM, c);
}

template <bool BF, bool E8, int HD>
__global__ void __launch_bounds__((PtShape<BF, E8, HD>::kThreads), 1)
    paged_attn_tc_kernel(const __grid_constant__ PaArgs A) {
    using S = PtShape<BF, E8, HD>;
    constexpr bool PB = BF && !E8;  // the MMAs' type: bf16, or f16
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    unsigned char* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
    PtCtl& ctl = *reinterpret_cast<PtCtl*>(sm);
    static_assert(sizeof(PtCtl) <= S::kCtl, "control block");
    unsigned char* ring = sm + S::kCtl;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&ctl.full[i], S::kLoaders);
            mbar_init(&ctl.empty[i], 1);
        }
        // (the commit, and an arrival of the MMA thread's own that orders the key masks)
        mbar_init(&ctl.s_full[0], 2);
        mbar_init(&ctl.s_full[1], 2);
        mbar_init(&ctl.p_full[0], kPtSoft);
        mbar_init(&ctl.p_full[1], kPtSoft);
        mbar_init(&ctl.o_done, 1);
        mbar_init(&ctl.q_full, kPtSoft);
        mbar_init(&ctl.fin, 1);
        ctl.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
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
    auto give_up = [&]() { *reinterpret_cast<volatile int*>(&ctl.abort) = 1; };
    auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&ctl.abort) != 0; };

    // this CTA's share of the line
    const int64_t total = pa_total(A, kPtM, lane);
    const int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
    const int64_t t0 = (int64_t)blockIdx.x * chunk;
    PaCur cur{};
    if (t0 < total) {
        int64_t before;
        cur.s = pa_find(A, kPtM, lane, t0, before);
        cur.q = pa_seq(A, cur.s, kPtM);
        cur.u = (int)((t0 - before) / cur.q.ntiles);
        cur.tile = (int)((t0 - before) % cur.q.ntiles);
        cur.left = min(chunk, total - t0);
    }

    if (warp > 4) {
        // ------------------------------------------------------------ loads
        const int lw = warp - 5;
        int n = 0;  // the next item
        int tile_no = 0;
        // a key's rows of the two tensors, null where it is not held
        struct Place {
            const unsigned char *k, *v;
        };
        auto place = [&](const PaCur& c) -> Place {
            const int key = c.q.lo + c.tile * kPaTile + lw * S::KPW + lane % S::KPW;
            int slot = 0;
            const int64_t page = key < c.q.hi ? page_of(A.R, A.C.n_pages, c.s, key, slot) : -1;
            if (page < 0) return {nullptr, nullptr};
            const int h = c.u % A.C.kv_heads;
            return {A.C.k + page * A.C.ks[0] + slot * A.C.ks[1] + h * A.C.ks[2],
                    A.C.v + page * A.C.vs[0] + slot * A.C.vs[1] + h * A.C.vs[2]};
        };
        auto wait_empty = [&](int item) -> bool {
            if (item < S::kSlots) return true;
            if (!aborted() && mbar_wait(&ctl.empty[item % S::kSlots], ((item / S::kSlots) - 1) & 1, kPtWait)) return true;
            give_up();
            return false;
        };
        auto mask = [&](const Place& p) {
            const uint32_t b = __ballot_sync(0xffffffffu, p.k != nullptr);
            if (lane == 0) {
                if constexpr (E8)
                    reinterpret_cast<uint16_t*>(ctl.bits[tile_no % kPtBits])[lw] = (uint16_t)b;
                else
                    ctl.bits[tile_no % kPtBits][lw] = b;
            }
            ++tile_no;
        };
        // The items in order: `next` places the keys of the tile after the one
        // at hand, `held` the values of the tile at hand.  emit(rows) is called
        // with each item's row pointers.
        auto walk = [&](auto emit) {
            PaCur c = cur;
            Place ahead{nullptr, nullptr};
            if (c.left > 0) ahead = place(c);
            while (c.left > 0) {
                const int tiles = pt_tiles(c);
                Place held = ahead, next;
                mask(held);
                for (int i = -1; i < tiles; ++i) {
                    // K(i+1), then V(i)
                    if (i + 1 < tiles) {
                        next = ahead;
                        if (i >= 0) mask(next);
                        const unsigned char* kp = next.k;
                        pa_next(A, kPtM, c);
                        if (c.left > 0) ahead = place(c);
                        if (!emit(kp)) return;
                    }
                    if (i >= 0) {
                        if (!emit(held.v)) return;
                    }
                    if (i + 1 < tiles) held = next;
                }
            }
        };
        if constexpr (!E8) {
            constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows a copy instruction covers
            auto signal = [&](int item) {
                fence_proxy_async_smem();
                mbar_arrive(&ctl.full[item % S::kSlots]);
            };
            walk([&](const unsigned char* rows) -> bool {
                if (!wait_empty(n)) return false;
                const uint32_t dst = smem_addr(ring) + (n % S::kSlots) * S::kItem;
#pragma unroll
                for (int i = 0; i < S::KPW / RPI; ++i) {
                    const int r = i * RPI + lane / CH, ch = lane % CH;
                    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                    const void* src = p ? reinterpret_cast<const unsigned char*>(p) + 16 * ch : A.C.k;
                    cp16(dst + (ch >> 3) * (kPaTile * 128) + at_swz(lw * S::KPW + r, ch & 7), src, p ? 16 : 0);
                }
                cp_commit();
                cp_wait<S::kLag>();
                if (n >= S::kLag) signal(n - S::kLag);
                ++n;
                return true;
            });
            cp_wait<0>();
            for (int i = max(0, n - S::kLag); i < n; ++i) signal(i);
        } else {
            constexpr int CH = HD / 16, RPI = 32 / CH, LD = S::KPW / RPI, kHeld = 4;
            uint4 raw[kHeld][LD];
            const int ch = lane % CH;
            // item `item` out of raw[b]: a chunk's 16 codes as 32 bytes of f16
            auto write = [&](int item, const uint4 (&x)[LD]) -> bool {
                if (!wait_empty(item)) return false;
                unsigned char* dst = ring + (item % S::kSlots) * S::kItem;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int key = lw * S::KPW + i * RPI + lane / CH;
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t y[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[2 * j] = e4m3x2_f16x2(w[j]);
                        y[2 * j + 1] = e4m3x2_f16x2(w[j] >> 16);
                    }
                    // (lanes of the upper blocks write their halves in the other order: other banks)
                    const bool flip = ch >= CH / 2;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int half = flip ? 1 - j : j, chunk = 2 * ch + half;
                        const uint4 v = half ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4*>(dst + (chunk >> 3) * (kPaTile * 128) + at_swz(key, chunk & 7)) = v;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&ctl.full[item % S::kSlots]);
                return true;
            };
            // registers need fixed places: the b-th of every four items goes to raw[b]
            auto step = [&](auto B, const unsigned char* rows) -> bool {
                constexpr int b = decltype(B)::value;
                if (n >= kHeld && !write(n - kHeld, raw[b])) return false;
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const int r = i * RPI + lane / CH;
                    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rows), r);
                    raw[b][i] = p ? ldg_stream_v4(reinterpret_cast<const unsigned char*>(p) + 16 * ch)
                                  : make_uint4(0u, 0u, 0u, 0u);
                }
                ++n;
                return true;
            };
            walk([&](const unsigned char* rows) -> bool {
                switch (n & 3) {
                    case 0: return step(std::integral_constant<int, 0>{}, rows);
                    case 1: return step(std::integral_constant<int, 1>{}, rows);
                    case 2: return step(std::integral_constant<int, 2>{}, rows);
                    default: return step(std::integral_constant<int, 3>{}, rows);
                }
            });
            for (int i = max(0, n - kHeld); i < n; ++i) {
                bool ok = true;
                switch (i & 3) {
                    case 0: ok = write(i, raw[0]); break;
                    case 1: ok = write(i, raw[1]); break;
                    case 2: ok = write(i, raw[2]); break;
                    default: ok = write(i, raw[3]); break;
                }
                if (!ok) break;
            }
        }
    } else if (warp == 4) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0 && cur.left > 0) {
            constexpr uint32_t kType = PB ? (1u << 7) | (1u << 10) : 0u;  // A, B: bf16, or f16
            constexpr uint32_t idS = at_idesc(kPtM, kPaTile, false) | kType, idO = at_idesc(kPtM, HD, true) | kType;
            const uint64_t dk0 = at_desc(smem_addr(ring), 16), dv0 = at_desc(smem_addr(ring), kPaTile * 128);
            constexpr uint64_t kItemD = S::kItem >> 4;
            int n = 0, tg = 0, unit = 0;  // items, tiles, units so far
            bool ok = true;
            auto item_in = [&](int item) {
                return !aborted() && mbar_wait(&ctl.full[item % S::kSlots], (item / S::kSlots) & 1, kPtWait);
            };
            auto scores = [&](int tile) -> bool {
                const int item = n++;
                if (!item_in(item)) return false;
                at_fence_after();
                const uint64_t kd = dk0 + (uint64_t)(item % S::kSlots) * kItemD;
#pragma unroll
                for (int j = 0; j < HD / 16; ++j)
                    at_mma_ts(tmem + S::kColS + (tile & 1) * 128, tmem + (uint32_t)(S::kColQ + 8 * j),
                              kd + (uint64_t)(((j >> 2) * (kPaTile * 128) + (j & 3) * 32) >> 4), idS, j > 0 ? 1u : 0u);
                at_commit(&ctl.empty[item % S::kSlots]);
                at_commit(&ctl.s_full[tile & 1]);
                mbar_arrive(&ctl.s_full[tile & 1]);
                return true;
            };
            PaCur c = cur;
            while (ok && c.left > 0) {
                const int tiles = pt_tiles(c);
                if (!(ok = !aborted() && mbar_wait(&ctl.q_full, unit & 1, kPtWait))) break;
                at_fence_after();
                if (!(ok = scores(tg))) break;
                for (int i = 0; ok && i < tiles; ++i, ++tg) {
                    // the next tile's scores: their buffer held P of tile tg - 1, whose P V is issued before
                    if (i + 1 < tiles && !(ok = scores(tg + 1))) break;
                    if (!(ok = !aborted() && mbar_wait(&ctl.p_full[tg & 1], (tg >> 1) & 1, kPtWait))) break;
                    const int item = n++;
                    if (!(ok = item_in(item))) break;
                    at_fence_after();
                    const uint64_t vd = dv0 + (uint64_t)(item % S::kSlots) * kItemD;
#pragma unroll
                    for (int j = 0; j < kPaTile / 16; ++j) {
                        // keys 16 j ..: eight columns of P, hi, and sixteen columns on its lo
                        const uint32_t p = tmem + (uint32_t)(S::kColS + (tg & 1) * 128 + 32 * (j >> 1) + 8 * (j & 1));
                        const uint64_t v = vd + (uint64_t)((j * 2048) >> 4);
                        at_mma_ts(tmem + S::kColO, p, v, idO, 1u);
                        if constexpr (S::kSplitP) at_mma_ts(tmem + S::kColO, p + 16, v, idO, 1u);
                    }
                    at_commit(&ctl.empty[item % S::kSlots]);
                    at_commit(&ctl.o_done);
                }
                ++unit;
                pt_skip(A, c, tiles);
            }
            if (!ok) give_up();
            // every MMA issued has completed before the CTA moves on
            at_commit(&ctl.fin);
            mbar_wait(&ctl.fin, 0, kPtWait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ queries, softmax, epilogue
        const int r = threadIdx.x;  // this thread's row of the unit
        const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        int n = 0, tg = 0;
        PaCur c = cur;
        while (c.left > 0) {
            const PaSeq sq = c.q;
            const int u = c.u, tile0 = c.tile, tiles = pt_tiles(c);
            const int h = u % A.C.kv_heads, rt = u / A.C.kv_heads;
            const int mvalid = min(kPtM, sq.rows * A.group - rt * kPtM);
            const bool in = r < mvalid, warp_in = warp * 32 < mvalid;
            const int mm = rt * kPtM + r, row = sq.row0 + mm / A.group, hq = h * A.group + mm % A.group;
            const int pos = in ? sq.p0 + mm / A.group : -1;
            const int wlo = A.window > 0 ? pos - A.window + 1 : 0;
            const int pmin = sq.p0 + (rt * kPtM) / A.group, pmax = sq.p0 + (rt * kPtM + mvalid - 1) / A.group;
            const int wtop = A.window > 0 ? pmax - A.window + 1 : 0;
            // the row's query to tensor memory, O cleared (the unit before has read it)
            float rf = 1.f;
            const unsigned char* qp = A.q.p + (int64_t)row * A.q.rs + (int64_t)hq * A.q.hs;
            float down = 1.f;
            const bool conv = E8 && A.q.dtype == kBF16;
            if (conv) {
                float mx = 0.f;
                if (in)
#pragma unroll 4
                    for (int i = 0; i < HD / 8; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(qp + 16 * i);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = unpack2<true>(w[j]);
                            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                // times 2^-x, the largest in [1, 2): what f16 cannot hold of the row then is under 2^-25 of that
                if (mx > 0.f && mx < INFINITY) {
                    const int x = min(max(ilogbf(mx), -120), 120);
                    down = ldexpf(1.f, -x);
                    rf = ldexpf(1.f, x);
                }
            }
#pragma unroll 1
            for (int i = 0; i < HD / 32; ++i) {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 x = in ? *reinterpret_cast<const uint4*>(qp + 64 * i + 16 * j) : make_uint4(0u, 0u, 0u, 0u);
                    w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
                }
                if (conv) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 f = unpack2<true>(w[j]);
                        w[j] = pack2<false>(f.x * down, f.y * down);
                    }
                }
                pt_st16(lane_addr + S::kColQ + 16 * i, w);
            }
            const uint32_t zero[16] = {};
#pragma unroll 1
            for (int i = 0; i < HD / 16; ++i) pt_st16(lane_addr + S::kColO + 16 * i, zero);
            at_wait_st();
            at_fence_before();
            mbar_arrive(&ctl.q_full);
            const float ks = E8 && A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f;
            const float cs = fminf(fmaxf(A.scale_log2 * ks * rf, 1e-37f), 3e38f);

            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < tiles; ++i, ++tg) {
                const uint32_t sb = lane_addr + (uint32_t)(S::kColS + (tg & 1) * 128);
                // (all threads or none: a warp that went on alone would leave the others at a barrier)
                ok = ok && !aborted() && mbar_wait(&ctl.s_full[tg & 1], (tg >> 1) & 1, kPtWait);
                const int kfirst = sq.lo + (tile0 + i) * kPaTile, klast = kfirst + kPaTile - 1;
                const bool edge = klast > pmin || kfirst < wtop;  // (the same for every thread)
                if (edge) ok = !pt_soft_or(!ok);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    give_up();
                    continue;
                }
                at_fence_after();
                const uint32_t* bits = ctl.bits[tg % kPtBits];
                const bool full = !edge && (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
                // this row's view of 32 keys
                auto view = [&](int q) -> uint32_t {
                    const int hi = pos - kfirst - 32 * q, lo = wlo - kfirst - 32 * q;
                    uint32_t v = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
                    if (lo > 0) v = lo > 31 ? 0u : v & (0xffffffffu << lo);
                    return v & bits[q];
                };
                float mx = -INFINITY;
                if (warp_in) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t s[32];
                        pt_ld32(sb + 32 * q, s);
                        at_wait_ld();
                        if (full) {
                            float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
                            for (int j = 2; j < 32; j += 2) {
                                a = fmaxf(a, __uint_as_float(s[j]));
                                b = fmaxf(b, __uint_as_float(s[j + 1]));
                            }
                            mx = fmaxf(mx, fmaxf(a, b));
                        } else {
                            const uint32_t v = view(q);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if ((v >> j) & 1u) mx = fmaxf(mx, __uint_as_float(s[j]));
                        }
                    }
                    mx *= cs;
                }
                if (__any_sync(0xffffffffu, mx > m + kPaLazy)) {
                    const float to = mx > m + kPaLazy ? mx : m;
                    const float f = to == m ? 1.f : pa_exp2(m - to);
                    m = to;
                    l *= f;
                    if (i > 0) {
                        // P V of the tile before has been added
                        if (!__all_sync(0xffffffffu, mbar_wait(&ctl.o_done, (tg - 1) & 1, kPtWait))) {
                            ok = false;
                            give_up();
                        }
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
                    // keys that some rows see and others do not: are their values finite?  (thread r: key r)
                    const int item = n + (i + 1 == tiles ? 2 * tiles - 1 : 2 + 2 * i);
                    unsigned char* vt = ring + (item % S::kSlots) * S::kItem;
                    bool bad = false;
                    const bool got = ok && mbar_wait(&ctl.full[item % S::kSlots], (item / S::kSlots) & 1, kPtWait);
#pragma unroll 1
                    for (int x = 0; got && x < HD / 8; ++x) {
                        const uint4 v = *reinterpret_cast<const uint4*>(vt + (x >> 3) * (kPaTile * 128) + at_swz(r, x & 7));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) bad |= !finite16<PB>(w[j]) || !finite16<PB>(w[j] >> 16);
                    }
                    const uint32_t b = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) ctl.bad[warp] = b;
                    if (pt_soft_or(!got)) {
                        ok = false;
                        give_up();
                        continue;
                    }
                    if ((ctl.bad[0] | ctl.bad[1] | ctl.bad[2] | ctl.bad[3]) != 0) {
                        if (i > 0 && !mbar_wait(&ctl.o_done, (tg - 1) & 1, kPtWait)) give_up();
                        __syncwarp();
                        at_fence_after();
#pragma unroll 1
                        for (int j = 0; j < kPaTile; ++j) {
                            if (!((ctl.bad[j >> 5] >> (j & 31)) & 1u)) continue;
                            const float s = __uint_as_float(pt_ld1(sb + j));
                            at_wait_ld();
                            const bool see = (view(j >> 5) >> (j & 31)) & 1u;
                            const float p = pa_exp2(fmaf(s, cs, -mr));
#pragma unroll 1
                            for (int x = 0; x < HD; x += 16) {
                                float o[16];
                                at_ld16(lane_addr + S::kColO + x, o);
                                at_wait_ld();
#pragma unroll
                                for (int y = 0; y < 16; ++y) {
                                    const int d = x + y;
                                    const uint16_t v = *reinterpret_cast<const uint16_t*>(
                                        vt + (d >> 6) * (kPaTile * 128) + at_swz(j, (d & 63) >> 3) + (d & 7) * 2);
                                    if (see && !finite16<PB>(v)) o[y] = fmaf(p, unpack2<PB>(v).x, o[y]);
                                }
                                at_st16(lane_addr + S::kColO + x, o);
                                at_wait_st();
                            }
                        }
                        pt_soft_sync();
                        if (bad) {
#pragma unroll 1
                            for (int d = 0; d < HD; ++d) {
                                uint16_t* v = reinterpret_cast<uint16_t*>(vt + (d >> 6) * (kPaTile * 128) +
                                                                          at_swz(r, (d & 63) >> 3) + (d & 7) * 2);
                                if (!finite16<PB>(*v)) *v = 0;
                            }
                        }
                        fence_proxy_async_smem();
                    }
                }
                // P over S, 32 keys at a time: sixteen columns of hi pairs, sixteen of lo
                if (warp_in) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t s[32];
                        pt_ld32(sb + 32 * q, s);
                        at_wait_ld();
                        uint32_t hi[16], lo[16];
                        float l2 = 0.f;
                        const uint32_t v = full ? 0xffffffffu : view(q);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float a = pa_exp2(fmaf(__uint_as_float(s[2 * j]), cs, -mr));
                            float b = pa_exp2(fmaf(__uint_as_float(s[2 * j + 1]), cs, -mr));
                            if (!full) {
                                if (!((v >> (2 * j)) & 1u)) a = 0.f;
                                if (!((v >> (2 * j + 1)) & 1u)) b = 0.f;
                            }
                            l += a;
                            l2 += b;
                            hi[j] = pack2<PB>(a, b);
                            if constexpr (S::kSplitP) {
                                const float2 x = unpack2<PB>(hi[j]);
                                lo[j] = pack2<PB>(a - x.x, b - x.y);
                            }
                        }
                        l += l2;
                        pt_st16(sb + 32 * q, hi);
                        if constexpr (S::kSplitP) pt_st16(sb + 32 * q + 16, lo);
                    }
                }
                at_wait_st();
                at_fence_before();
                mbar_arrive(&ctl.p_full[tg & 1]);
            }
            n += 2 * tiles;

            // ------------------------------------------------------------ the unit's end
            const bool whole = tile0 == 0 && tile0 + tiles == sq.ntiles;
            const int part = blockIdx.x * 2 + (tile0 == 0 ? 1 : 0);
            if (ok && !mbar_wait(&ctl.o_done, (tg - 1) & 1, kPtWait)) {
                ok = false;
                give_up();
            }
            ok = __all_sync(0xffffffffu, ok);
            at_fence_after();
            const float vs = E8 && A.C.v_scale != nullptr ? A.C.v_scale[h] : 1.f;
            const float inv = !ok ? NAN : l == 0.f ? 0.f : vs / l;
            unsigned char* op = A.out.p + (int64_t)row * A.out.rs + (int64_t)hq * A.out.hs;
            float* wp = A.ws_o + ((int64_t)part * kPtM + r) * HD;
            const bool ob = A.out.dtype == kBF16;
#pragma unroll 1
            for (int x = 0; x < HD; x += 16) {
                float o[16];
                at_ld16(lane_addr + S::kColO + x, o);
                at_wait_ld();
                if (!in) continue;
                if (whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = ob ? pack2<true>(o[2 * j] * inv, o[2 * j + 1] * inv)
                                  : pack2<false>(o[2 * j] * inv, o[2 * j + 1] * inv);
                    *reinterpret_cast<uint4*>(op + 2 * x) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(op + 2 * x + 16) = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(wp + x + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
            if (in) {
                if (!ok) l = NAN;
                if (!whole)
                    A.ws_ml[(int64_t)part * kPtM + r] = make_float2(m, l);
                else if (A.lse != nullptr)
                    A.lse[(int64_t)row * A.q.heads + hq] =
                        l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + log2f(l)) * 0.69314718056f);
            }
            at_fence_before();
            pt_skip(A, c, tiles);
        }
    }
    at_fence_before();
    __syncthreads();
    if (warp == 4) {
        at_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
    }
}

template <bool BF, bool E8, int HD>
static int pt_launch(const PaArgs& A, int num_sms, cudaStream_t st) {
    using S = PtShape<BF, E8, HD>;
    static size_t limit[kMaxDevices] = {};
    auto kern = paged_attn_tc_kernel<BF, E8, HD>;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return (int)e;
    if (cudaError_t e = raise_smem_limit(kern, S::kSmem, &limit[dev])) return (int)e;
    return (int)launch(kern, dim3(num_sms), dim3(S::kThreads), S::kSmem, st, A);
}

int paged_attention_tc(const PaArgs& A, int cache_dtype, int hd, int num_sms, cudaStream_t st) {
    if (hd == 64)
        return cache_dtype == kBF16  ? pt_launch<true, false, 64>(A, num_sms, st)
               : cache_dtype == kF16 ? pt_launch<false, false, 64>(A, num_sms, st)
                                     : pt_launch<false, true, 64>(A, num_sms, st);
    return cache_dtype == kBF16  ? pt_launch<true, false, 128>(A, num_sms, st)
           : cache_dtype == kF16 ? pt_launch<false, false, 128>(A, num_sms, st)
                                 : pt_launch<false, true, 128>(A, num_sms, st);
}

}  // namespace dflash
