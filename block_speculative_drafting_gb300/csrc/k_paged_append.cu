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

// Eight values of a 4-bit cache's row, in units of the head's scale: with the eight of the neighbouring lane they are a
// block of 16.  s = e4m3(min(max |x| / 6, 448)), codes e2m1(x / s) (nearest, ties to even, clamped to +-6; the
// conversions and the division round as IEEE's do).  A NaN makes its block's scale NaN, and so all that the block stands for; a
// block whose scale rounds to 0 is 0.  The even lane writes the scale.
DF_DEV void store8_e2m1(unsigned char* p, unsigned char* block, const float (&x)[8], bool in, int c) {
    float m = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(x[i]));
        nan |= x[i] != x[i];
    }
    if (nan) m = NAN;
    const float o = __shfl_xor_sync(0xffffffffu, m, 1);
    m = m != m || o != o ? NAN : fmaxf(m, o);
    const float q = __fdiv_rn(m, 6.f);
    const uint32_t s8 = m != m ? 0x7fu : __nv_cvt_float_to_fp8(fminf(q, 448.f), __NV_SATFINITE, __NV_E4M3);
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3)));
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = s > 0.f ? __fdiv_rn(x[i], s) : 0.f;
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(w)
        : "f"(u[0]), "f"(u[1]), "f"(u[2]), "f"(u[3]), "f"(u[4]), "f"(u[5]), "f"(u[6]), "f"(u[7]));
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
                if (H.scale != nullptr) {
                    const float sc = H.scale[min(h, H.heads - 1)];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], sc);
                }
                if constexpr (OUT == kE2M1)  // (all lanes: pairs of them share a block)
                    store8_e2m1(to, block, x, h < H.heads, threadIdx.x & (L - 1));
                else
                    store8<OUT>(to, x);
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
__global__ void __launch_bounds__(kApWarps * 32, 4)
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
// A cache's rows as values: 16 columns a lane and round (16 bytes of codes at most from an 8-bit cache, 8 from a 4-bit
// one), warps over the call's rows as in the append.  Code times block scale is exact, the head's scale rounds in 32
// bits, and the output's type once.  Positions that are not held read as zeros.
template <int HD, int CD, int OUT>
__global__ void __launch_bounds__(kApWarps * 32)
    paged_read_kernel(const __grid_constant__ PagedCache C, const __grid_constant__ PagedRows R,
                      const __grid_constant__ HeadRows ko, const __grid_constant__ HeadRows vo, int warps_log2) {
    constexpr int L = HD / 16;   // lanes of a head
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
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const HeadRows& O = side == 0 ? ko : vo;
        if (O.p == nullptr) continue;
        const unsigned char* from = (side == 0 ? C.k : C.v) + max(page, (int64_t)0) * (side == 0 ? C.ks[0] : C.vs[0]) +
                                    slot * (side == 0 ? C.ks[1] : C.vs[1]);
        const int64_t hs = side == 0 ? C.ks[2] : C.vs[2];
        const float* scale = side == 0 ? C.k_scale : C.v_scale;
#pragma unroll 2
        for (int h = share * HPW + lane / L; h < C.kv_heads; h += HPW << warps_log2) {
            float x[2][8] = {};
            if (page >= 0) {
                const unsigned char* p = from + h * hs;
                const float sc = scale != nullptr ? scale[h] : 1.f;
                if constexpr (CD == kBF16 || CD == kF16) {
                    Raw8<CD> r[2];
                    r[0].load(p + 32 * c);
                    r[1].load(p + 32 * c + 16);
                    r[0].values(x[0]);
                    r[1].values(x[1]);
                } else {
                    uint32_t y[8];
                    float f = sc;
                    if constexpr (CD == kE4M3) {
                        const uint4 w = *reinterpret_cast<const uint4*>(p + 16 * c);
                        e4m3x4_f16x4(w.x, y[0], y[1]);
                        e4m3x4_f16x4(w.y, y[2], y[3]);
                        e4m3x4_f16x4(w.z, y[4], y[5]);
                        e4m3x4_f16x4(w.w, y[6], y[7]);
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(p + 8 * c);
                        const unsigned char* bl = side == 0 ? C.kb + page * C.kbs[0] + slot * C.kbs[1] + h * C.kbs[2]
                                                            : C.vb + page * C.vbs[0] + slot * C.vbs[1] + h * C.vbs[2];
                        const uint32_t s2 = __byte_perm(e4m3x2_f16x2(bl[c]), 0, 0x1010);
                        uint32_t z[4];
                        e2m1x8_f16x8(w.x, z);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = mul_f16x2(z[i], s2);
                        e2m1x8_f16x8(w.y, z);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[4 + i] = mul_f16x2(z[i], s2);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 v = unpack2<false>(y[i]);
                        x[i >> 2][2 * (i & 3)] = v.x * f;
                        x[i >> 2][2 * (i & 3) + 1] = v.y * f;
                    }
                }
            }
            constexpr int E = OUT == kF32 ? 4 : 2;
            unsigned char* to = O.p + (int64_t)row * O.rs + h * O.hs + 16 * c * E;
            store8<OUT>(to, x[0]);
            store8<OUT>(to + 8 * E, x[1]);
        }
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
