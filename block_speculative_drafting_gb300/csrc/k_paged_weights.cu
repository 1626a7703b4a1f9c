// The attention weight that each cached key receives: for every (sequence,
// key/value head) and key j the sum of exp(scale q . k_j - lse) over the rows that see j and
// the query heads that share the head, added to what is there.
#include "kernels.cuh"
#include "paged_attn.cuh"

namespace dflash {

constexpr int kPwKeys = 128;

struct PwArgs {
    PagedCache C;
    PagedRows R;
    HeadRows q;
    KeyWeights W;
    const float* lse;
    float scale;
    int window, group, tiles;
};

template <int CD, int HD>
__global__ void __launch_bounds__(kPwKeys) paged_weights_kernel(const __grid_constant__ PwArgs A) {
    __shared__ float qs[HD];
    const int t = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = blockIdx.x / A.tiles;
    const int tile = (int)(blockIdx.x - unit * A.tiles), s = (int)(unit / A.C.kv_heads), h = (int)(unit - (int64_t)s * A.C.kv_heads);
    int a, b;
    rows_of(A.R, s, a, b);
    const int rows = b - a, len = max(A.R.kv_len[s], -1), p0 = len - rows, L = min(max(len, 0), A.R.cap);
    if (rows == 0 || tile * kPwKeys >= L) return;
    const int j = tile * kPwKeys + t;
    int slot = 0;
    const int64_t page = j < L ? page_of(A.R, A.C.n_pages, s, j, slot) : -1;
    float k[HD];
    const float ks = A.C.k_scale != nullptr ? A.C.k_scale[h] : 1.f;
    const unsigned char* p = A.C.k + max(page, (int64_t)0) * A.C.ks[0] + slot * A.C.ks[1] + h * A.C.ks[2];
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {
        uint32_t y[8] = {};
        if (page >= 0) {
            if constexpr (CD == kE4M3) {
                const uint4 w = *reinterpret_cast<const uint4*>(p + 16 * i);
                e4m3x4_f16x4(w.x, y[0], y[1]);
                e4m3x4_f16x4(w.y, y[2], y[3]);
                e4m3x4_f16x4(w.z, y[4], y[5]);
                e4m3x4_f16x4(w.w, y[6], y[7]);
            } else if constexpr (CD == kE2M1) {
                const uint2 w = *reinterpret_cast<const uint2*>(p + 8 * i);
                const uint32_t s2 = __byte_perm(
                    e4m3x2_f16x2(A.C.kb[page * A.C.kbs[0] + slot * A.C.kbs[1] + h * A.C.kbs[2] + i]), 0, 0x1010);
                uint32_t z[4];
                e2m1x8_f16x8(w.x, z);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = mul_f16x2(z[e], s2);
                e2m1x8_f16x8(w.y, z);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 + e] = mul_f16x2(z[e], s2);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = *reinterpret_cast<const uint32_t*>(p + 32 * i + 4 * e);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = unpack2<CD == kBF16>(y[e]);
            k[16 * i + 2 * e] = f.x;
            k[16 * i + 2 * e + 1] = f.y;
        }
    }
    float sum = 0.f;
    for (int m = 0; m < rows * A.group; ++m) {
        const int row = a + m / A.group, hq = h * A.group + m % A.group, pos = p0 + m / A.group;
        __syncthreads();
        const unsigned char* qp = A.q.p + (int64_t)row * A.q.rs + (int64_t)hq * A.q.hs;
        for (int i = t; i < HD / 2; i += kPwKeys) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(qp + 4 * i);
            const float2 f = A.q.dtype == kBF16 ? unpack2<true>(w) : unpack2<false>(w);
            qs[2 * i] = f.x;
            qs[2 * i + 1] = f.y;
        }
        __syncthreads();
        const float lse = A.lse[(int64_t)row * A.q.heads + hq];
        if (j > pos || (A.window > 0 && j <= pos - A.window) || lse == -INFINITY) continue;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < HD; ++i) dot = fmaf(qs[i], k[i], dot);
        sum += expf(dot * (A.scale * ks) - lse);
    }
    if (page >= 0) {
        float* w = A.W.p + (int64_t)s * A.W.ss + (int64_t)h * A.W.hs + j;
        *w = j >= p0 ? sum : *w + sum;
    }
}

template <int HD>
static auto weights_kernel(int cd) {
    return cd == kBF16   ? paged_weights_kernel<kBF16, HD>
           : cd == kF16  ? paged_weights_kernel<kF16, HD>
           : cd == kE4M3 ? paged_weights_kernel<kE4M3, HD>
                         : paged_weights_kernel<kE2M1, HD>;
}
int paged_key_weights(const PagedCache& C, int cache_dtype, int hd, const PagedRows& R, const HeadRows& q,
                      const float* lse, float scale, int window, const KeyWeights& W, int num_sms, cudaStream_t st) {
    PwArgs A{};
    A.C = C, A.R = R, A.q = q, A.W = W, A.lse = lse, A.scale = scale, A.window = window;
    A.group = q.heads / C.kv_heads;
    A.tiles = (R.cap + kPwKeys - 1) / kPwKeys;
    if (A.tiles == 0) return 0;
    auto kern = hd == 64 ? weights_kernel<64>(cache_dtype) : weights_kernel<128>(cache_dtype);
    return (int)launch(kern, dim3((unsigned)((int64_t)R.n_seqs * C.kv_heads * A.tiles)), dim3(kPwKeys), 0, st, A);
}

}  // namespace dflash
