// Eviction from a paged cache by accumulated attention weight: per sequence and
// key/value head, of L > keep tokens the first `first`, the last `recent` and the
// heaviest others stay, and move, in order, to the first `keep` slots.
//
// Two kernels.  The first finds, a CTA a (sequence, head), the weight that the last
// kept token has, digit by digit of an order-preserving integer key (11, 11 and 10
// bits, a histogram each: the counts are whole numbers, so the order of the
// additions says nothing), and writes the slots that stay in ascending order:
// tokens over that weight and, of those at it, the lowest slots.
//
// The second moves.  Token i of the kept ones comes from a slot of at least i, so
// in ascending order nothing is overwritten before it is read: a CTA takes all kept
// tokens of one head and a slice of a row's bytes (slices share nothing, so they
// are other CTAs' and need not wait), in rounds of some thousand vectors, each read whole
// before it is written; the next round's reads are on their way meanwhile, whose
// slots lie past everything this round writes.
//
// One sequence of 32768 tokens, 8 heads of 128 in bf16, cut to 16384: 65 us, 25 of them the choice
// (eight CTAs, four times over their weights: latency) and 38 the move (3.5 TB/s: its threads find the
// place of every 16 bytes, some 130 instructions a warp's).  32 sequences of 1024 to 4096 tokens in e4m3
// cut to 2048: 52 us, 11 and 41.
#include "kernels.cuh"
#include "paged.cuh"

namespace dflash {

constexpr int kEvThreads = 1024, kEvWarps = kEvThreads / 32, kEvBins = 2048;

// larger keys for larger weights; NaN counts as -inf, the zeros as one
DF_DEV uint32_t ev_key(float w) { return float_order_key(w != w ? -INFINITY : w == 0.f ? 0.f : w); }

constexpr int kEvRound = 4 * kEvThreads;  // tokens of a round: a warp 128 in a row, four a lane

__global__ void __launch_bounds__(kEvThreads) paged_evict_select_kernel(const __grid_constant__ EvictArgs A) {
    __shared__ uint32_t hist[kEvBins];
    __shared__ uint32_t sums[kEvWarps];
    __shared__ uint2 found;
    __shared__ uint2 totals[2][kEvWarps];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int s = blockIdx.x / A.C.kv_heads, h = blockIdx.x - s * A.C.kv_heads;
    pdl_wait();
    pdl_trigger();
    const int L = min(max(A.R.kv_len[s], 0), A.R.cap);
    if (h == 0 && t == 0) A.lens[s] = make_int2(L, min(L, A.keep));
    int32_t* kept = A.kept + (int64_t)blockIdx.x * A.keep;
    if (L <= A.keep) {
        for (int i = t; i < A.keep; i += kEvThreads) kept[i] = i < L ? i : -1;
        return;
    }
    const float* w = A.in.p + (int64_t)s * A.in.ss + (int64_t)h * A.in.hs;
    const int lo = A.first, hi = L - A.recent;
    uint32_t need = (uint32_t)(A.keep - A.first - A.recent);  // (of hi - lo, which are more)
    uint32_t border = 0xffffffffu, ties = 0;                  // keys over `border` stay, and `ties` at it
    if (need > 0) {
        uint32_t prefix = 0, mask = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 0x3ffu : 0x7ffu;
            for (int i = t; i < kEvBins; i += kEvThreads) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = lo + t; i < hi; i += kEvThreads) {
                const uint32_t k = ev_key(w[i]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1u);
            }
            __syncthreads();
            // the digit at which, counted from the largest, `need` is reached: two bins a thread, from the top
            const int b1 = kEvBins - 1 - 2 * t, b0 = b1 - 1;
            const uint32_t h1 = hist[b1], h0 = hist[b0];
            uint32_t in = h1 + h0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += y;
            }
            if (lane == 31) sums[warp] = in;
            __syncthreads();
            uint32_t before = lane < warp ? sums[lane] : 0u;
            before = __reduce_add_sync(0xffffffffu, before);
            in += before;
            const uint32_t out = in - h1 - h0;  // larger ones than both bins'
            if (out < need && need <= out + h1) found = make_uint2((uint32_t)b1, out);
            if (out + h1 < need && need <= in) found = make_uint2((uint32_t)b0, out + h1);
            __syncthreads();
            prefix |= found.x << shift;
            mask |= digits << shift;
            need -= found.y;
            __syncthreads();  // (`found` is read before the next pass writes it)
        }
        border = prefix;
        ties = need;
    }
    // the slots that stay, in order
    uint32_t over = 0, at = 0;  // tokens before this round over the border (or kept in any case), and at it
    int buf = 0;
    auto round = [&](int base, const uint32_t (&key)[4]) {
        const int i0 = base + warp * 128 + lane;
        uint32_t go[4], ge[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k;
            const bool mid = i >= lo && i < hi;
            go[k] = __ballot_sync(0xffffffffu, i < L && (!mid || key[k] > border));
            ge[k] = __ballot_sync(0xffffffffu, mid && key[k] == border && ties > 0);
        }
        const uint32_t no = __popc(go[0]) + __popc(go[1]) + __popc(go[2]) + __popc(go[3]);
        const uint32_t ne = __popc(ge[0]) + __popc(ge[1]) + __popc(ge[2]) + __popc(ge[3]);
        if (lane == 0) totals[buf][warp] = make_uint2(no, ne);
        __syncthreads();
        const uint2 x = totals[buf][lane];
        uint32_t o = over + __reduce_add_sync(0xffffffffu, lane < warp ? x.x : 0u);
        uint32_t e = at + __reduce_add_sync(0xffffffffu, lane < warp ? x.y : 0u);
        over += __reduce_add_sync(0xffffffffu, x.x);
        at += __reduce_add_sync(0xffffffffu, x.y);
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t mo = o + __popc(go[k] & below), me = e + __popc(ge[k] & below);
            const bool stays = (go[k] >> lane) & 1u, tie = ((ge[k] >> lane) & 1u) && me < ties;
            const uint32_t place = mo + min(me, ties);
            if ((stays || tie) && place < (uint32_t)A.keep) kept[place] = i0 + 32 * k;
            o += __popc(go[k]);
            e += __popc(ge[k]);
        }
        buf ^= 1;
    };
#pragma unroll 1
    for (int base = 0; base < L; base += kEvRound) {
        uint32_t key[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = base + warp * 128 + lane + 32 * k;
            key[k] = i >= lo && i < hi ? ev_key(w[i]) : 0u;
        }
        round(base, key);
    }
}

constexpr int kMvRound = 4;  // vectors a thread and round

// One head's kept rows of one tensor, `VR` vectors of type V a row from column `col` on: round by round, by T threads.
template <class V, int VR, int T, class From, class To>
DF_DEV void ev_move(const int32_t* kept, int count, From from, To to) {
    constexpr int RR = T * kMvRound / VR;  // rows of a round
    const int t = threadIdx.x, c = t % VR;
    V x[2][kMvRound];
    bool on[2][kMvRound];
    int src[kMvRound];  // the next round's slots, read a round ahead
    auto slots = [&](int round) {
#pragma unroll
        for (int k = 0; k < kMvRound; ++k) {
            const int i = round * RR + k * (T / VR) + t / VR;
            src[k] = i < count ? kept[i] : -1;
        }
    };
    auto load = [&](int round, int b) {
#pragma unroll
        for (int k = 0; k < kMvRound; ++k) {
            const int i = round * RR + k * (T / VR) + t / VR;
            const V* p = src[k] > i ? from(src[k], c) : nullptr;
            on[b][k] = p != nullptr;
            if (p != nullptr) x[b][k] = *p;
        }
        slots(round + 1);
    };
    auto store = [&](int round, int b) {
#pragma unroll
        for (int k = 0; k < kMvRound; ++k) {
            const int i = round * RR + k * (T / VR) + t / VR;
            if (!on[b][k]) continue;
            V* p = to(i, c);
            if (p != nullptr) *p = x[b][k];
        }
    };
    const int rounds = (count + RR - 1) / RR;
    slots(0);
    load(0, 0);
#pragma unroll 1
    for (int r = 0; r < rounds; r += 2) {
        if (r + 1 < rounds) load(r + 1, 1);
        __syncthreads();  // every thread has read round r
        store(r, 0);
        if (r + 2 < rounds) load(r + 2, 0);
        __syncthreads();
        if (r + 1 < rounds) store(r + 1, 1);
    }
}

// RB: bytes of a row; SB: of a slice of it; T: threads
template <int RB, int SB, int T>
__global__ void __launch_bounds__(T) paged_evict_move_kernel(const __grid_constant__ EvictArgs A, int block_bytes) {
    constexpr int SL = RB / SB, JOBS = 2 * SL + 1;
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x / JOBS, job = blockIdx.x - unit * JOBS;
    const int s = unit / A.C.kv_heads, h = unit - s * A.C.kv_heads;
    const int2 len = A.lens[s];
    if (job == 2 * SL && h == 0 && threadIdx.x == 0) {
        A.new_len[s] = len.y;
        if (A.evicted != nullptr) A.evicted[s] += len.x - len.y;
    }
    const bool aside = A.in.p != A.out.p;  // weights that go elsewhere go whole
    if (len.x == len.y && !(aside && job == 2 * SL)) return;
    const int count = len.y;
    const int32_t* kept = A.kept + (int64_t)unit * A.keep;
    auto place = [&](unsigned char* base, const int64_t* st, int slot_of, int64_t col) -> unsigned char* {
        int slot;
        const int64_t page = page_of(A.R, A.C.n_pages, s, slot_of, slot);
        return page < 0 ? nullptr : base + page * st[0] + slot * st[1] + h * st[2] + col;
    };
    if (job < 2 * SL) {
        unsigned char* base = job < SL ? A.C.k : A.C.v;
        const int64_t* st = job < SL ? A.C.ks : A.C.vs;
        const int64_t col = (int64_t)(job % SL) * SB;
        auto at = [&](int i, int c) { return reinterpret_cast<uint4*>(place(base, st, i, col + 16 * c)); };
        ev_move<uint4, SB / 16, T>(kept, count, at, at);
        return;
    }
    const float* in = A.in.p + (int64_t)s * A.in.ss + (int64_t)h * A.in.hs;
    float* out = A.out.p + (int64_t)s * A.out.ss + (int64_t)h * A.out.hs;
    if (aside) {
#pragma unroll 1
        for (int i0 = threadIdx.x; i0 < count; i0 += 8 * T) {
            int j[8];
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) j[k] = i0 + k * T < count ? kept[i0 + k * T] : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = in[j[k]];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + k * T < count) out[i0 + k * T] = x[k];
        }
        if (len.x == len.y) return;
    } else {
        auto at = [&](int i, int) { return out + i; };
        ev_move<float, 1, T>(kept, count, at, at);
    }
    for (int side = 0; side < 2 && block_bytes > 0; ++side) {
        unsigned char* base = side == 0 ? A.C.kb : A.C.vb;
        const int64_t* st = side == 0 ? A.C.kbs : A.C.vbs;
        __syncthreads();
        if (block_bytes == 8) {
            auto at = [&](int i, int) { return reinterpret_cast<uint2*>(place(base, st, i, 0)); };
            ev_move<uint2, 1, T>(kept, count, at, at);
        } else {
            auto at = [&](int i, int) { return reinterpret_cast<uint32_t*>(place(base, st, i, 0)); };
            ev_move<uint32_t, 1, T>(kept, count, at, at);
        }
    }
}

int64_t paged_evict_workspace(int n_seqs, int kv_heads, int keep, bool own_kept) {
    const int64_t lens = ((int64_t)n_seqs * (int64_t)sizeof(int2) + 15) & ~15ll;
    return lens + (own_kept ? (int64_t)n_seqs * kv_heads * keep * 4 : 0);
}

// Few heads: each one's rows over as many CTAs as have a sector of 32 bytes each, of 1024 threads (eight heads of 32768
// tokens, 256 bytes a row, cut to half: 175 us with slices of 64 bytes and 256 threads, 38 so); many: a CTA a tensor.
template <int RB>
static int ev_launch(const EvictArgs& A, int block_bytes, int num_sms, cudaStream_t st) {
    const int64_t units = (int64_t)A.R.n_seqs * A.C.kv_heads;
    if (units * 3 < num_sms) {
        constexpr int T = 1024;
        return (int)launch(paged_evict_move_kernel<RB, 32, T>, dim3((unsigned)(units * (2 * (RB / 32) + 1))), dim3(T), 0, st,
                           A, block_bytes);
    }
    constexpr int T = 512;
    return (int)launch(paged_evict_move_kernel<RB, RB, T>, dim3((unsigned)(units * 3)), dim3(T), 0, st, A, block_bytes);
}

int paged_evict(const EvictArgs& A, int cache_dtype, int hd, int num_sms, cudaStream_t st) {
    const int64_t units = (int64_t)A.R.n_seqs * A.C.kv_heads;
    const int e = (int)launch(paged_evict_select_kernel, dim3((unsigned)units), dim3(kEvThreads), 0, st, A);
    if (e != 0) return e;
    const int rb = cache_dtype == kE2M1 ? hd / 2 : cache_dtype == kE4M3 ? hd : 2 * hd;
    const int bb = cache_dtype == kE2M1 ? hd / 16 : 0;
    return rb == 256   ? ev_launch<256>(A, bb, num_sms, st)
           : rb == 128 ? ev_launch<128>(A, bb, num_sms, st)
           : rb == 64  ? ev_launch<64>(A, bb, num_sms, st)
                       : ev_launch<32>(A, bb, num_sms, st);
}

}  // namespace dflash
