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
#include "paged.cuh"

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
            if (h < H.heads) {
                if (H.scale != nullptr) {
                    const float sc = H.scale[h];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], sc);
                }
                store8<OUT>(to, x);
            }
            h += H.step;
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
                        const __grid_constant__ Rotation rot, int warps_log2) {
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
    // column 8 c + i becomes x co[i] + y si[i], y the other column of its pair
    const bool turned = 8 * c < rot.rotary;
    const int half = rot.rotary / 16;  // lanes between the columns of a pair (pairs (i, i + rotary / 2))
    const int other = !turned || rot.interleaved ? c : c < half ? c + half : c - half;
    float co[8], si[8];
    if (rot.rotary > 0) {
        for (int i = lane; i < rot.rotary / 2; i += 32) {
            const double t = (double)pos64 * rot.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
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
    const auto bytes = [](int dtype) { return dtype == kF32 ? 4 : dtype == kE4M3 ? 1 : 2; };
    auto set = [&](const HeadRows& src, unsigned char* to, int64_t hs, int out) {
        H.heads = src.heads;
        H.rounds = (src.heads - share * HPW + H.step - 1) / H.step;
        H.from = src.p + (int64_t)row * src.rs + H.first * src.hs + 8 * c * bytes(IN);
        H.from_step = H.step * src.hs;
        H.to = to + H.first * hs + 8 * c * bytes(out);
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
        H.rotates = side == 0 && rot.rotary > 0;
        head_loop<HD, IN, OUT>(H, co, si);
    }
}

template <int HD, int IN, int QO>
static auto append_kernel(int out) {
    return out == kBF16  ? paged_append_kernel<HD, IN, QO, kBF16>
           : out == kF16 ? paged_append_kernel<HD, IN, QO, kF16>
                         : paged_append_kernel<HD, IN, QO, kE4M3>;
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
                 const Rotation& rot, int num_sms, cudaStream_t st) {
    const int qd = q.heads > 0 ? qo.dtype : k.dtype;
    auto kern = hd == 64 ? append_kernel<64>(k.dtype, qd, cache_dtype) : append_kernel<128>(k.dtype, qd, cache_dtype);
    // more warps a row while that leaves the SMs under a third of their warps (512 rows: one warp a row 12.7 us, four
    // 8.5, eight 10.2; one row: one warp 6.7 us, eight 4.5)
    int wl = 0;
    while (wl < 3 && ((int64_t)R.n_rows << (wl + 1)) <= (int64_t)num_sms * 20) ++wl;
    const int64_t warps = (int64_t)R.n_rows << wl;
    return (int)launch(kern, dim3((unsigned)((warps + kApWarps - 1) / kApWarps)), dim3(kApWarps * 32), 0, st, C,
                       R, k, v, q, qo, q_norm, k_norm, eps, rot, wl);
}

}  // namespace dflash
