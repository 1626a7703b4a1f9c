// Keys and values appended to a paged cache, with the head norm and the
// rotation applied on the way, and the queries of the same rows rotated: q, k
// and v are read once and written once.
//
// Warps hold rows: one warp a row where there are many, up to eight where
// there are few (they then share the row's heads).  An angle p f turns many
// times at far positions, so it is formed in 64 bits, in turns (p f / 2 pi),
// reduced there to [-1/2, 1/2] and only then taken to 32 bits: the error is
// that of one f32 rounding of the reduced turn at any position.  The row's
// sines and cosines are computed once and passed through shared memory to the
// lanes that use them: head_dim / 8 lanes hold a head, eight columns (16 bytes
// of a 16-bit type) a lane, the same columns of every head, so that a lane
// keeps its eight sines and cosines in registers over all heads.
//
// Memory bound where rows are many: 8192 rows of 32 query and 8 key/value heads
// of 128, bf16, half of each rotated: 39.7 us, 5.1 TB/s (75 % of a copy).  512
// rows with head norms into an e4m3 cache: 9.0 us, the chain of a row's norms
// and rotations; one row: 4.5 us, launch and lookups.
//
// Into a 4-bit cache, where two elements are a byte, two neighbouring lanes hold a block of sixteen columns with
// its scale.  Keys and values as they come have a kernel of their own (paged_append4_kernel): 8192 rows of 8 heads
// 18 us, bound by issue (66 %: the block's maximum, its scale, the quotients); the read of them as bf16 another 9.
// 32 blocks of 16 rows: 6.7 us together.  With 32 query heads, head norms, a rotation and counts of evicted
// tokens, the general kernel: 8192 rows 60 us (55 without norms), 32 blocks 11.3, one row 6.4.
#include "kernels.cuh"
#include "paged_attn.cuh"

namespace dflash {

constexpr int kApWarps = 8;

// Eight elements as loaded, and their values.
template <int DT>
struct Raw8 {
    uint4 w[DT == kF32 ? 2 : 1];
    DF_DEV void load(const unsigned char* p) {
        w[0] = *reinterpret_cast<const uint4*>(p);
        if constexpr (DT == kF32) w[1] = *reinterpret_cast<const uint4*>(p + 16);
    }
    DF_DEV void values(float (&x)[8]) const {
        if constexpr (DT == kF32) {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == kBF16) {
                    x[2 * i] = __uint_as_float(u[i] << 16);
                    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                    x[2 * i] = f.x, x[2 * i + 1] = f.y;
                }
            }
        }
    }
};

// Two e2m1 codes a byte of eight values, the first in the lower bits: nearest, ties to even, clamped to +-6.
DF_DEV uint32_t e2m1x8(const float (&u)[8]) {
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(w)
        : "f"(u[0]), "f"(u[1]), "f"(u[2]), "f"(u[3]), "f"(u[4]), "f"(u[5]), "f"(u[6]), "f"(u[7]));
    return w;
}
DF_DEV float rcp_near(float d) {  // within 2^-22 of it
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
    return y;
}
// x / d rounded as the division rounds it, y near 1 / d: with a quotient within a unit in the last place, q + y (x - q d)
// rounds to the correct one (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990); the first such step brings x y within that unit.  For 2^-60 <= d <= 2^60 and |x| <= 2^60 (what underflows is far
// below a block's smallest code).
DF_DEV float quotient(float x, float d, float y) {
    y = fmaf(fmaf(-d, y, 1.f), y, y);
    float q = x * y;
    q = fmaf(fmaf(-d, q, x), y, q);
    return fmaf(fmaf(-d, q, x), y, q);
}
DF_DEV float max_nan(float a, float b) {  // NaN where one is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// The codes by the definition: t = x / scale and t / s, each rounded as the division rounds.
__device__ __noinline__ uint32_t e2m1_defined(const float* x, float scale, float s) {
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = s > 0.f ? __fdiv_rn(__fdiv_rn(x[i], scale), s) : 0.f;
    return e2m1x8(u);
}
// Eight values of a 4-bit cache's row; with the eight of the neighbouring lane they are a block of 16.  In units of the
// head's scale, t = x / scale: s = e4m3(min(max |t| / 6, 448)) and codes e2m1(t / s), all rounded to nearest, ties to even.
// A NaN makes its block's scale NaN, and so all that the block stands for; a block whose scale rounds to 0 is 0.  The
// even lane writes the scale.  (All lanes take part.)
//
// The scale needs the quotient of the largest value alone (rounding keeps the order).  The codes come from one product with
// the reciprocals of both scales, which is within 2^-21 of t / s, a little lower and a little higher: where the two agree
// they are t / s's code; where some differ (one element of 10^5 lies that near to a border), the warp divides.  (8192 rows
// of 8 + 8 heads: two divisions an element 30.7 us.)
DF_DEV void store8_e2m1(unsigned char* p, unsigned char* block, const float (&x)[8], float scale, bool in, int c) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const bool plain = m <= 0x1p60f && scale >= 0x1p-60f && scale <= 0x1p60f;  // (false for NaN)
    const float rs = rcp_near(scale);
    float sixth = quotient(quotient(m, scale, rs), 6.f, 0x1.555556p-3f);
    if (__any_sync(0xffffffffu, !plain)) sixth = __fdiv_rn(__fdiv_rn(m, scale), 6.f);
    uint16_t s8;  // (clamped to 448; NaN stays)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(sixth));
    const float s = unpack2<false>(e4m3x2_f16x2(s8)).x;
    const float ry = rcp_near(s), near = s > 0.f ? rs * ry : 0.f;
    const float low = near * (1.f - 0x1p-20f), high = near * (1.f + 0x1p-20f);
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = x[i] * low, b[i] = x[i] * high;
    uint32_t w = e2m1x8(a);
    if (__any_sync(0xffffffffu, w != e2m1x8(b))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = s > 0.f ? quotient(quotient(x[i], scale, rs), s, ry) : 0.f;
        w = e2m1x8(a);
    }
    // (numbers near the ends of f32, where the products are not that near, and what is not a number)
    if (__any_sync(0xffffffffu, !plain)) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
        w = e2m1_defined(v, scale, s);
    }
    if (!in) return;
    *reinterpret_cast<uint32_t*>(p) = w;
    if ((c & 1) == 0) *block = (unsigned char)s8;
}

// Eight values as type DT, rounded to nearest even.
template <int DT>
DF_DEV void store8(unsigned char* p, const float (&x)[8]) {
    if constexpr (DT == kF32) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (DT == kE4M3) {
        // clamped to the largest finite value by the conversion; NaN stays NaN
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t b =
                __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = a | (b << 16);
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == kBF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// One tensor's heads of a row, for the lanes that hold columns 8 c ..: heads
// first, first + step, .. (`count` rounds, the same for the whole warp).
struct HeadLoop {
    const unsigned char* from;  // the first head's columns
    unsigned char* to;
    int64_t from_step, to_step;  // bytes to the next round's head
    int first, step, heads, rounds;
    const float *gain, *scale;  // the norm's gain (columns 8 c ..), the cache's scales by head; null: none
    unsigned char* block;       // a 4-bit cache: where the first head's scale of the lane's block goes
    int64_t block_step;         // bytes to the next round's
    float eps;
    bool rotates, turned, interleaved;
    int other;  // the lane with the other columns of the pairs
};
template <int HD, int IN, int OUT>
DF_DEV void head_loop(const HeadLoop& H, const float (&co)[8], const float (&si)[8]) {
    constexpr int L = HD / 8, AHEAD = IN == kF32 ? 1 : 2;
    Raw8<IN> next[AHEAD];
    const unsigned char* from = H.from;
    unsigned char* to = H.to;
    [[maybe_unused]] unsigned char* block = H.block;
    int h = H.first;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (h + i * H.step < H.heads) next[i].load(from + i * H.from_step);
#pragma unroll 1
    for (int n = 0; n < H.rounds; n += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            float x[8];
            next[i].values(x);
            if (OUT == kE2M1 && h >= H.heads) {  // (nothing was loaded)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.f;
            }
            if (h + AHEAD * H.step < H.heads) next[i].load(from + AHEAD * H.from_step);
            if (H.gain != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(ss / HD + H.eps);  // (within 2^-22)
                const float4 g0 = *reinterpret_cast<const float4*>(H.gain),
                             g1 = *reinterpret_cast<const float4*>(H.gain + 4);
                x[0] *= r * g0.x, x[1] *= r * g0.y, x[2] *= r * g0.z, x[3] *= r * g0.w;
                x[4] *= r * g1.x, x[5] *= r * g1.y, x[6] *= r * g1.z, x[7] *= r * g1.w;
            }
            if (H.rotates) {
                if (H.interleaved) {
                    if (H.turned) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const float y = x[j];
                            x[j] = fmaf(y, co[j], x[j + 1] * si[j]);
                            x[j + 1] = fmaf(x[j + 1], co[j + 1], y * si[j + 1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float y = __shfl_sync(0xffffffffu, x[j], H.other, L);
                        if (H.turned) x[j] = fmaf(x[j], co[j], y * si[j]);
                    }
                }
            }
            if (OUT == kE2M1 || h < H.heads) {
                const float sc = H.scale != nullptr ? H.scale[min(h, H.heads - 1)] : 1.f;
                if constexpr (OUT == kE2M1) {  // (all lanes: pairs of them share a block)
                    store8_e2m1(to, block, x, sc, h < H.heads, threadIdx.x & (L - 1));
                } else {
                    if (H.scale != nullptr) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], sc);
                    }
                    store8<OUT>(to, x);
                }
            }
            h += H.step;
            if constexpr (OUT == kE2M1) block += H.block_step;
            from += H.from_step;
            to += H.to_step;
        }
    }
}
// IN: the type of q, k and v; QO, OUT: of the queries' destination and of the cache
template <int HD, int IN, int QO, int OUT>
__global__ void __launch_bounds__(kApWarps * 32, OUT == kE2M1 ? 3 : 4)
    paged_append_kernel(const __grid_constant__ PagedCache C, const __grid_constant__ PagedRows R,
                        const __grid_constant__ HeadRows k, const __grid_constant__ HeadRows v,
                        const __grid_constant__ HeadRows q, const __grid_constant__ HeadRows qo,
                        const float* __restrict__ q_norm, const float* __restrict__ k_norm, float eps,
                        const __grid_constant__ Rotation rot, const int32_t* __restrict__ evicted, int warps_log2) {
    constexpr int L = HD / 8;     // lanes of a head
    constexpr int HPW = 32 / L;   // heads a warp holds at once
    __shared__ float2 turns_of[kApWarps][HD / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % L;
    const int64_t id = (int64_t)blockIdx.x * kApWarps + warp;
    const int row = (int)(id >> warps_log2), share = (int)(id & ((1 << warps_log2) - 1));
    pdl_wait();
    pdl_trigger();
    const int s = row < R.n_rows ? seq_of(R, row) : -1;
    if (s < 0) return;
    int a, b;
    rows_of(R, s, a, b);
    const int64_t pos64 = (int64_t)R.kv_len[s] - (b - a) + (row - a);
    int slot = 0;
    const int64_t page = page_of(R, C.n_pages, s, (int)max(pos64, (int64_t)-1), slot);
    const int64_t turn64 = evicted != nullptr ? pos64 + evicted[s] : pos64;  // the token's place in its sequence
    // column 8 c + i becomes x co[i] + y si[i], y the other column of its pair
    const bool turned = 8 * c < rot.rotary;
    const int half = rot.rotary / 16;  // lanes between the columns of a pair (pairs (i, i + rotary / 2))
    const int other = !turned || rot.interleaved ? c : c < half ? c + half : c - half;
    float co[8], si[8];
    if (rot.rotary > 0) {
        for (int i = lane; i < rot.rotary / 2; i += 32) {
            const double t = (double)turn64 * rot.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
            float sn, cn;
            sincospif(2.f * (float)(t - rint(t)), &sn, &cn);
            turns_of[warp][i] = make_float2(cn * rot.scale, sn * rot.scale);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = rot.interleaved ? 4 * c + i / 2 : 8 * (c < half ? c : c - half) + i;
            const bool low = rot.interleaved ? (i & 1) == 0 : c < half;
            const float2 t = turned ? turns_of[warp][pair] : make_float2(1.f, 0.f);
            co[i] = t.x;
            si[i] = low ? -t.y : t.y;
        }
    }
    HeadLoop H;
    H.eps = eps;
    H.turned = turned;
    H.interleaved = rot.interleaved;
    H.other = other;
    H.step = HPW << warps_log2;
    H.first = share * HPW + lane / L;
    // bytes of this lane's columns before its own (8 c of them)
    const auto before = [c](int dtype) { return dtype == kE2M1 ? 4 * c : 8 * c * (dtype == kF32 ? 4 : dtype == kE4M3 ? 1 : 2); };
    auto set = [&](const HeadRows& src, unsigned char* to, int64_t hs, int out) {
        H.heads = src.heads;
        H.rounds = (src.heads - share * HPW + H.step - 1) / H.step;
        H.from = src.p + (int64_t)row * src.rs + H.first * src.hs + before(IN);
        H.from_step = H.step * src.hs;
        H.to = to + H.first * hs + before(out);
        H.to_step = H.step * hs;
    };
    if (q.heads > 0) {
        set(q, qo.p + (int64_t)row * qo.rs, qo.hs, QO);
        H.gain = q_norm != nullptr ? q_norm + 8 * c : nullptr;
        H.scale = nullptr;
        H.rotates = rot.rotary > 0;
        head_loop<HD, IN, QO>(H, co, si);
    }
    if (page < 0) return;  // not held: neither keys nor values are written
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int64_t* st = side == 0 ? C.ks : C.vs;
        set(side == 0 ? k : v, (side == 0 ? C.k : C.v) + page * st[0] + slot * st[1], st[2], OUT);
        H.gain = side == 0 && k_norm != nullptr ? k_norm + 8 * c : nullptr;
        H.scale = side == 0 ? C.k_scale : C.v_scale;
        if constexpr (OUT == kE2M1) {
            const int64_t* bt = side == 0 ? C.kbs : C.vbs;
            H.block = (side == 0 ? C.kb : C.vb) + page * bt[0] + slot * bt[1] + H.first * bt[2] + c / 2;
            H.block_step = H.step * bt[2];
        }
        H.rotates = side == 0 && rot.rotary > 0;
        head_loop<HD, IN, OUT>(H, co, si);
    }
}

// ---------------------------------------------------------------- rows read back
// A cache's rows as values: eight columns a lane (so that a warp's stores are contiguous), warps over the call's rows as
// in the append.  Code times block scale is exact, the head's scale rounds in 32 bits, and the output's type once.
// Positions that are not held read as zeros.
template <int HD, int CD, int OUT>
__global__ void __launch_bounds__(kApWarps * 32)
    paged_read_kernel(const __grid_constant__ PagedCache C, const __grid_constant__ PagedRows R,
                      const __grid_constant__ HeadRows ko, const __grid_constant__ HeadRows vo, int warps_log2) {
    constexpr int L = HD / 8;    // lanes of a head
    constexpr int HPW = 32 / L;  // heads a warp holds at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % L;
    const int64_t id = (int64_t)blockIdx.x * kApWarps + warp;
    const int row = (int)(id >> warps_log2), share = (int)(id & ((1 << warps_log2) - 1));
    pdl_wait();
    pdl_trigger();
    const int s = row < R.n_rows ? seq_of(R, row) : -1;
    if (s < 0) return;
    int a, b;
    rows_of(R, s, a, b);
    const int64_t pos64 = (int64_t)R.kv_len[s] - (b - a) + (row - a);
    int slot = 0;
    const int64_t page = page_of(R, C.n_pages, s, (int)max(pos64, (int64_t)-1), slot);
    const int64_t pg = max(page, (int64_t)0);
    const unsigned char *k = C.k + pg * C.ks[0] + slot * C.ks[1], *v = C.v + pg * C.vs[0] + slot * C.vs[1];
    const unsigned char *kb = C.kb + pg * C.kbs[0] + slot * C.kbs[1] + c / 2, *vb = C.vb + pg * C.vbs[0] + slot * C.vbs[1] + c / 2;
    unsigned char *kt = ko.p + (int64_t)row * ko.rs + 8 * c * (OUT == kF32 ? 4 : 2), *vt = vo.p + (int64_t)row * vo.rs + 8 * c * (OUT == kF32 ? 4 : 2);
    constexpr int E = CD == kE2M1 ? 4 : CD == kE4M3 ? 8 : 16;  // bytes of eight columns
    struct Codes {
        Raw8<CD == kF16 ? kF16 : kBF16> raw;
        uint2 w;
        uint32_t s;
        float sc;
    };
    auto load = [&](const unsigned char* from, const unsigned char* blocks, const float* scale, int h) {
        Codes x{};
        if (page < 0) return x;
        if constexpr (E == 16) x.raw.load(from + E * c);
        if constexpr (E == 8) x.w = *reinterpret_cast<const uint2*>(from + E * c);
        if constexpr (E == 4) x.w.x = *reinterpret_cast<const uint32_t*>(from + E * c), x.s = *blocks;
        if constexpr (E < 16) x.sc = scale != nullptr ? scale[h] : 1.f;
        return x;
    };
    auto store = [&](unsigned char* to, const Codes& x) {
        float y[8];
        if constexpr (E == 16) {
            x.raw.values(y);
        } else {
            uint32_t z[4];
            if constexpr (E == 8) {
                e4m3x4_f16x4(x.w.x, z[0], z[1]);
                e4m3x4_f16x4(x.w.y, z[2], z[3]);
            } else {
                e2m1x8_f16x8(x.w.x, z);
                const uint32_t s2 = __byte_perm(e4m3x2_f16x2(x.s), 0, 0x1010);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = mul_f16x2(z[i], s2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<false>(z[i]);
                y[2 * i] = f.x * x.sc;
                y[2 * i + 1] = f.y * x.sc;
            }
        }
        store8<OUT>(to, y);
    };
#pragma unroll 2
    for (int h = share * HPW + lane / L; h < C.kv_heads; h += HPW << warps_log2) {
        Codes x{}, y{};
        if (ko.p != nullptr) x = load(k + h * C.ks[2], kb + h * C.kbs[2], C.k_scale, h);
        if (vo.p != nullptr) y = load(v + h * C.vs[2], vb + h * C.vbs[2], C.v_scale, h);
        if (ko.p != nullptr) store(kt + h * ko.hs, x);
        if (vo.p != nullptr) store(vt + h * vo.hs, y);
    }
}
template <int HD, int CD>
static auto read_kernel(int out) {
    return out == kBF16  ? paged_read_kernel<HD, CD, kBF16>
           : out == kF16 ? paged_read_kernel<HD, CD, kF16>
                         : paged_read_kernel<HD, CD, kF32>;
}
template <int HD>
static auto read_kernel(int cd, int out) {
    return cd == kBF16   ? read_kernel<HD, kBF16>(out)
           : cd == kF16  ? read_kernel<HD, kF16>(out)
           : cd == kE4M3 ? read_kernel<HD, kE4M3>(out)
                         : read_kernel<HD, kE2M1>(out);
}
int paged_read(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& ko, const HeadRows& vo,
               int num_sms, cudaStream_t st) {
    const int out = ko.p != nullptr ? ko.dtype : vo.dtype;
    auto kern = hd == 64 ? read_kernel<64>(cache_dtype, out) : read_kernel<128>(cache_dtype, out);
    int wl = 0;
    while (wl < 3 && ((int64_t)R.n_rows << (wl + 1)) <= (int64_t)num_sms * 20) ++wl;
    const int64_t warps = (int64_t)R.n_rows << wl;
    return (int)launch(kern, dim3((unsigned)((warps + kApWarps - 1) / kApWarps)), dim3(kApWarps * 32), 0, st, C, R, ko,
                       vo, wl);
}

// Keys and values into a 4-bit cache as they come, no queries beside them: a warp a row and tensor (more where rows are
// few), four rounds of heads on their way at once.  In registers enough for half as many warps the general kernel took
// 25.5 us (8192 rows of 8 + 8 heads of 128), this one 17.9 us.
template <int HD, int IN>
__global__ void __launch_bounds__(kApWarps * 32, 4)
    paged_append4_kernel(const __grid_constant__ PagedCache C, const __grid_constant__ PagedRows R,
                         const __grid_constant__ HeadRows k, const __grid_constant__ HeadRows v, int warps_log2) {
    constexpr int L = HD / 8, HPW = 32 / L, AHEAD = IN == kF32 ? 2 : 4, E = IN == kF32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % L;
    const int64_t id = (int64_t)blockIdx.x * kApWarps + warp;
    const int row = (int)(id >> (warps_log2 + 1)), side = (int)(id & 1), share = (int)(id >> 1) & ((1 << warps_log2) - 1);
    pdl_wait();
    pdl_trigger();
    if (row >= R.n_rows) return;
    const HeadRows& src = side == 0 ? k : v;
    const int h0 = share * HPW + lane / L, step = HPW << warps_log2;
    const unsigned char* from = src.p + (int64_t)row * src.rs + h0 * src.hs + 8 * c * E;
    const int64_t from_step = step * src.hs;
    Raw8<IN> raw[AHEAD];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (h + i * step < C.kv_heads) raw[i].load(from + i * from_step);
    };
    load(h0);
    const int s = seq_of(R, row);
    if (s < 0) return;
    int a, b;
    rows_of(R, s, a, b);
    int slot = 0;
    const int64_t page =
        page_of(R, C.n_pages, s, (int)max((int64_t)R.kv_len[s] - (b - a) + (row - a), (int64_t)-1), slot);
    if (page < 0) return;
    const int64_t *st = side == 0 ? C.ks : C.vs, *bt = side == 0 ? C.kbs : C.vbs;
    const float* scale = side == 0 ? C.k_scale : C.v_scale;
    unsigned char* to = (side == 0 ? C.k : C.v) + page * st[0] + slot * st[1] + h0 * st[2] + 4 * c;
    unsigned char* block = (side == 0 ? C.kb : C.vb) + page * bt[0] + slot * bt[1] + h0 * bt[2] + c / 2;
#pragma unroll 1
    for (int h = h0; h - lane / L < C.kv_heads; h += AHEAD * step) {
        float sc[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) sc[i] = scale != nullptr ? scale[min(h + i * step, C.kv_heads - 1)] : 1.f;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = h + i * step < C.kv_heads;
            if (h - lane / L + i * step >= C.kv_heads) break;  // (none of the warp's)
            float x[8];
            raw[i].values(x);
            if (!in) {  // (nothing was loaded)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.f;
            }
            store8_e2m1(to + i * step * st[2], block + i * step * bt[2], x, sc[i], in, c);
        }
        from += AHEAD * from_step;
        load(h + AHEAD * step);
        to += AHEAD * step * st[2];
        block += AHEAD * step * bt[2];
    }
}

template <int HD, int IN, int QO>
static auto append_kernel(int out) {
    return out == kBF16  ? paged_append_kernel<HD, IN, QO, kBF16>
           : out == kF16 ? paged_append_kernel<HD, IN, QO, kF16>
           : out == kE4M3 ? paged_append_kernel<HD, IN, QO, kE4M3>
                         : paged_append_kernel<HD, IN, QO, kE2M1>;
}
template <int HD, int IN>
static auto append_kernel(int qo, int out) {
    return qo == kBF16  ? append_kernel<HD, IN, kBF16>(out)
           : qo == kF16 ? append_kernel<HD, IN, kF16>(out)
                        : append_kernel<HD, IN, kF32>(out);
}
template <int HD>
static auto append_kernel(int in, int qo, int out) {
    return in == kBF16  ? append_kernel<HD, kBF16>(qo, out)
           : in == kF16 ? append_kernel<HD, kF16>(qo, out)
                        : append_kernel<HD, kF32>(qo, out);
}

int paged_append(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& k, const HeadRows& v,
                 const HeadRows& q, const HeadRows& qo, const float* q_norm, const float* k_norm, float eps,
                 const Rotation& rot, const int32_t* evicted, int num_sms, cudaStream_t st) {
    // (keys and values into one memory are the general kernel's: its lanes write values after keys, here warps do both at once)
    const bool apart = C.k != C.v && C.kb != C.vb;
    if (cache_dtype == kE2M1 && q.heads == 0 && k_norm == nullptr && rot.rotary == 0 && apart) {
        auto kern = hd == 64 ? (k.dtype == kBF16  ? paged_append4_kernel<64, kBF16>
                                : k.dtype == kF16 ? paged_append4_kernel<64, kF16>
                                                  : paged_append4_kernel<64, kF32>)
                             : (k.dtype == kBF16  ? paged_append4_kernel<128, kBF16>
                                : k.dtype == kF16 ? paged_append4_kernel<128, kF16>
                                                  : paged_append4_kernel<128, kF32>);
        int wl = 0;
        while (wl < 3 && ((int64_t)R.n_rows << (wl + 2)) <= (int64_t)num_sms * 20) ++wl;
        const int64_t warps = (int64_t)R.n_rows << (wl + 1);
        return (int)launch(kern, dim3((unsigned)((warps + kApWarps - 1) / kApWarps)), dim3(kApWarps * 32), 0, st, C, R, k, v, wl);
    }
    const int qd = q.heads > 0 ? qo.dtype : k.dtype;
    auto kern = hd == 64 ? append_kernel<64>(k.dtype, qd, cache_dtype) : append_kernel<128>(k.dtype, qd, cache_dtype);
    // more warps a row while that leaves the SMs under a third of their warps (512 rows: one warp a row 12.7 us, four
    // 8.5, eight 10.2; one row: one warp 6.7 us, eight 4.5)
    int wl = 0;
    while (wl < 3 && ((int64_t)R.n_rows << (wl + 1)) <= (int64_t)num_sms * 20) ++wl;
    const int64_t warps = (int64_t)R.n_rows << wl;
    return (int)launch(kern, dim3((unsigned)((warps + kApWarps - 1) / kApWarps)), dim3(kApWarps * 32), 0, st, C,
                       R, k, v, q, qo, q_norm, k_norm, eps, rot, evicted, wl);
}

}  // namespace dflash
