// Attention over the 4-bit cache (decode): first form, one CTA per query row.
#include <cmath>

#include "kv4_common.cuh"

namespace fa {

namespace {

constexpr int kAttnThreads = 128;

template <int D>
__global__ void __launch_bounds__(kAttnThreads) fa_kv4_attn_kernel(const Kv4AttnParams p)
{
    constexpr int G = D / 16;
    __shared__ float qs[D], ps[kAttnThreads], red[kAttnThreads / 32];
    const int tid = threadIdx.x;
    const long long row = blockIdx.x;  // (b * Hq + hq) * Lq + i
    const int i = (int)(row % p.Lq), hq = (int)(row / p.Lq % p.Hq), b = (int)(row / p.Lq / p.Hq);
    const int h = hq / p.group;
    int slot;
    const int len = kv4_sequence(p.c, b, slot);
    const float gk = p.c.k_scale ? p.c.k_scale[h] : 1.f, gv = p.c.v_scale ? p.c.v_scale[h] : 1.f;
    for (int d = tid; d < D; d += kAttnThreads) qs[d] = __uint_as_float((uint32_t)p.q[row * D + d] << 16);
    const int lim = p.causal ? min(len, i + len - p.Lq + 1) : len;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int j0 = 0; j0 < lim; j0 += kAttnThreads) {
        __syncthreads();
        const int j = j0 + tid;
        float s = -INFINITY;
        if (j < lim) {
            const uint8_t* u = p.c.pool + kv4_unit(p.c, D, kv4_page(p.c, slot, j), h, j);
            s = 0.f;
            for (int g = 0; g < G; ++g) {
                const float sc = f16x2_to_f32(e4m3x2_to_f16x2(u[16 * D + (j & 15) * G + g])).x;
                float x = 0.f;
                for (int e = 0; e < 8; ++e) {
                    const float2 c = f16x2_to_f32(e2m1x2_to_f16x2<0>(u[(j & 15) * (D / 2) + g * 8 + e]));
                    x += c.x * qs[g * 16 + 2 * e] + c.y * qs[g * 16 + 2 * e + 1];
                }
                s += x * sc;
            }
            s *= p.scale * gk;
        }
        float t = s;
        for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o));
        if ((tid & 31) == 0) red[tid >> 5] = t;
        __syncthreads();
        for (int w = 0; w < kAttnThreads / 32; ++w) t = fmaxf(t, red[w]);
        const float mn = fmaxf(m, t), use = mn == -INFINITY ? 0.f : mn;
        const float a = expf(m - use);
        ps[tid] = j < lim ? expf(s - use) : 0.f;
        m = mn;
        l *= a;
        acc *= a;
        __syncthreads();
        const int n = min(kAttnThreads, lim - j0);
        for (int k = 0; k < n; ++k) {
            l += ps[k];
            if (tid < D) {
                const int jj = j0 + k, kk = jj & 15;
                const uint8_t* u = p.c.pool + kv4_unit(p.c, D, kv4_page(p.c, slot, jj), h, jj);
                const float sc = f16x2_to_f32(e4m3x2_to_f16x2(u[17 * D + (tid >> 4) * 16 + kk])).x;
                const float2 c = f16x2_to_f32(e2m1x2_to_f16x2<0>(
                    u[8 * D + (kk >> 3) * 4 * D + (tid >> 4) * 64 + ((kk & 7) >> 1) * 16 + (tid & 15)]));
                acc += ps[k] * ((kk & 1) ? c.y : c.x) * sc;
            }
        }
    }
    if (tid < D) p.o[row * D + tid] = lim > 0 ? acc / l * gv : 0.f;
    if (tid == 0) p.lse[row] = lim > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t kv4_attn_workspace(int, int, int, int, size_t* bytes)
{
    *bytes = 0;
    return cudaSuccess;
}

cudaError_t launch_kv4_attn(int D, const Kv4AttnParams& p, int, cudaStream_t stream, int* launches)
{
    const unsigned grid = (unsigned)(p.B * p.Hq * p.Lq);
    if (D == 128)
        fa_kv4_attn_kernel<128><<<grid, kAttnThreads, 0, stream>>>(p);
    else
        fa_kv4_attn_kernel<64><<<grid, kAttnThreads, 0, stream>>>(p);
    *launches = 1;
    return cudaGetLastError();
}

}  // namespace fa
