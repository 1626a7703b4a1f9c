// Keys and values appended to a paged cache, with the head norm and the
// rotation applied on the way, and the queries of the same rows rotated: q, k
// and v are read once and written once.
//
// One CTA per row.  The row's angles are the same for all its heads: thread i
// computes pair i's sine and cosine once, into shared memory.  An angle p f
// turns many times at far positions, so it is formed in 64 bits, in turns (p f
// / 2 pi), reduced there to [-1/2, 1/2] and only then taken to 32 bits: the
// error is that of one f32 rounding of the reduced turn at any position.
// Then 16-byte vectors: head_dim / 8 lanes hold a head, eight columns a lane.
#include "kernels.cuh"
#include "paged.cuh"

namespace dflash {

constexpr int kApThreads = 256;

DF_DEV void load8(const unsigned char* p, int dtype, float (&x)[8]) {
    if (dtype == kF32) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 16);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        return;
    }
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if (dtype == kBF16)
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
        else
            f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Eight values in `dtype`, rounded to nearest even.
DF_DEV void store8(unsigned char* p, int dtype, const float (&x)[8]) {
    if (dtype == kF32) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
    } else if (dtype == kE4M3) {
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
            if (dtype == kBF16) {
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

DF_DEV int bytes_of(int dtype) { return dtype == kF32 ? 4 : dtype == kE4M3 ? 1 : 2; }

template <int HD>
__global__ void __launch_bounds__(kApThreads)
    paged_append_kernel(const __grid_constant__ PagedCache C, int cache_dtype, const __grid_constant__ PagedRows R,
                        const __grid_constant__ HeadRows k, const __grid_constant__ HeadRows v,
                        const __grid_constant__ HeadRows q, const __grid_constant__ HeadRows qo,
                        const float* __restrict__ q_norm, const float* __restrict__ k_norm, float eps,
                        const __grid_constant__ Rotation rot) {
    constexpr int L = HD / 8;             // lanes of a head
    constexpr int HPB = kApThreads / L;   // heads a CTA handles at once
    __shared__ float2 cs[HD / 2];
    const int row = blockIdx.x, c = threadIdx.x % L;
    pdl_wait();
    pdl_trigger();
    const int s = seq_of(R, row);
    if (s < 0) return;
    int a, b;
    rows_of(R, s, a, b);
    const int64_t pos64 = (int64_t)R.kv_len[s] - (b - a) + (row - a);
    const int pos = (int)max(pos64, (int64_t)-1);
    int slot = 0;
    const int64_t page = page_of(R, C.n_pages, s, pos, slot);
    if (rot.rotary > 0) {
        for (int i = threadIdx.x; i < rot.rotary / 2; i += kApThreads) {
            const double turns = (double)pos64 * rot.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
            float sn, cn;
            sincospif(2.f * (float)(turns - rint(turns)), &sn, &cn);
            cs[i] = make_float2(cn * rot.scale, sn * rot.scale);
        }
        __syncthreads();
    }
    // heads in order: queries, keys, values
    const int nh = q.heads + 2 * C.kv_heads;
    for (int h0 = 0; h0 < nh; h0 += HPB) {
        const int h = h0 + threadIdx.x / L;
        const bool in = h < nh;
        const int kind = !in ? 3 : h < q.heads ? 0 : h < q.heads + C.kv_heads ? 1 : 2;
        const int hh = kind == 0 ? h : (h - q.heads) - (kind == 2 ? C.kv_heads : 0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (in) {
            const HeadRows& src = kind == 0 ? q : kind == 1 ? k : v;
            load8(src.p + (int64_t)row * src.rs + (int64_t)hh * src.hs + 8 * c * bytes_of(src.dtype), src.dtype, x);
        }
        const float* gain = kind == 0 ? q_norm : kind == 1 ? k_norm : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (gain != nullptr) {
            const float r = 1.f / sqrtf(ss / HD + eps);
            const float4 g0 = *reinterpret_cast<const float4*>(gain + 8 * c),
                         g1 = *reinterpret_cast<const float4*>(gain + 8 * c + 4);
            x[0] *= r * g0.x, x[1] *= r * g0.y, x[2] *= r * g0.z, x[3] *= r * g0.w;
            x[4] *= r * g1.x, x[5] *= r * g1.y, x[6] *= r * g1.z, x[7] *= r * g1.w;
        }
        if (rot.rotary > 0) {
            const bool turned = kind < 2 && 8 * c < rot.rotary;
            if (rot.interleaved) {
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = cs[4 * c + i];
                        const float p0 = x[2 * i], p1 = x[2 * i + 1];
                        x[2 * i] = p0 * t.x - p1 * t.y;
                        x[2 * i + 1] = p0 * t.y + p1 * t.x;
                    }
                }
            } else {
                // columns i and i + rotary / 2: lanes rotary / 16 apart
                const int half = rot.rotary / 16;
                const bool low = c < half;
                const int other = turned ? (low ? c + half : c - half) : c;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = __shfl_sync(0xffffffffu, x[i], other, L);
                    if (turned) {
                        const float2 t = cs[8 * (low ? c : c - half) + i];
                        x[i] = low ? x[i] * t.x - y * t.y : y * t.y + x[i] * t.x;
                    }
                }
            }
        }
        if (kind == 0) {
            store8(qo.p + (int64_t)row * qo.rs + (int64_t)hh * qo.hs + 8 * c * bytes_of(qo.dtype), qo.dtype, x);
        } else if (in && page >= 0) {
            const float* scale = kind == 1 ? C.k_scale : C.v_scale;
            if (scale != nullptr) {
                const float sc = scale[hh];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], sc);
            }
            unsigned char* dst = kind == 1 ? C.k + page * C.ks[0] + slot * C.ks[1] + hh * C.ks[2]
                                           : C.v + page * C.vs[0] + slot * C.vs[1] + hh * C.vs[2];
            store8(dst + 8 * c * bytes_of(cache_dtype), cache_dtype, x);
        }
    }
}

int paged_append(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& k, const HeadRows& v,
                 const HeadRows& q, const HeadRows& qo, const float* q_norm, const float* k_norm, float eps,
                 const Rotation& rot, cudaStream_t st) {
    auto kern = hd == 64 ? paged_append_kernel<64> : paged_append_kernel<128>;
    return (int)launch(kern, dim3(R.n_rows), dim3(kApThreads), 0, st, C, cache_dtype, R, k, v, q, qo, q_norm, k_norm,
                       eps, rot);
}

}  // namespace dflash
