// Rotary positions: q and k rows turned by their positions' angles (and the
// gradients, turned back), and the same on the way into the paged 16-bit
// cache.
//
//   (y1, y2) = m (cos t x1 - sin t x2, sin t x1 + cos t x2),  t = p w_c
//
// for pair c of a row at position p.  The gradient is the same with -t.  The
// frequency is held as turns per position times 2^64, so that the product
// with a 32-bit position modulo 2^64 is the angle's part of a turn with no
// rounding at all; its top 32 bits go to sincospif.  Products and sums are in
// fp32, rounded once to the output's type.
//
// Bound: HBM, each element read and written once.  A thread holds the cosines
// and sines of 8 pairs (16 dimensions) of one token and takes its rows of
// several heads, so that the angles' work (about 200 instructions) is shared,
// with four rows' loads in flight.  Dimensions that do not turn are copied by
// threads of the same kind.
#include <cuda_bf16.h>

#include <algorithm>

#include "kv16_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct Eight {  // 8 elements of a row
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p)
{
    Eight<T> x;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    return x;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Eight<T>& x, float (&f)[8])
{
    const uint32_t* w = &x.w[0].x;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
}

__device__ __forceinline__ void store8(float* p, const float (&f)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// m cos and m sin of the angles of 8 pairs from pair c0 on.
__device__ __forceinline__ void angles(const RotaryParams& p, int pos, int c0, float (&c)[8], float (&s)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const unsigned long long turn = (unsigned long long)(long long)pos * __ldg(p.freqs + c0 + i);
        const float x = (float)(int)(turn >> 32) * 4.656612873077393e-10f;  // half turns, -1 .. 1
        float sn, cs;
        sincospif(x, &sn, &cs);
        c[i] = p.mscale * cs;
        s[i] = p.mscale * (p.backward ? -sn : sn);
    }
}

template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float& x1 = INTER ? (i < 4 ? a[2 * i & 7] : b[2 * i & 7]) : a[i];
        float& x2 = INTER ? (i < 4 ? a[(2 * i + 1) & 7] : b[(2 * i + 1) & 7]) : b[i];
        const float u = x1, v = x2;
        x1 = c[i] * u - s[i] * v;
        x2 = s[i] * u + c[i] * v;
    }
}

// A block takes `tokens` tokens (blockIdx.x) and, with gridDim.y > 1, a share
// of their heads.  Of a token's threads, neighbours take the D / 16 units of a
// row: the first R / 16 turn, the others copy.
template <typename In, typename Out, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads) fa_rope_kernel(const RotaryParams p, const int tokens)
{
    constexpr int U = sizeof(In) == 2 ? 4 : 2;  // rows in flight
    if constexpr (APPEND) {
        if (p.c.ids && blockIdx.x == gridDim.x - 1) {  // the last blocks: only this check
            if (blockIdx.y == 0) kv16_check_slots<kThreads>(p.c, p.cu, p.num_seqs);
            return;
        }
    }
    __shared__ long long s_row[8];  // append: the token's K of head 0 in the pool, or -1
    __shared__ int s_pos[8];
    const int per = kThreads / tokens, units = p.D >> 4, slots = per / units;
    const int tok = threadIdx.x / per, rest = threadIdx.x % per, slot = rest / units, unit = rest % units;
    const long long t = (long long)blockIdx.x * tokens + tok;
    const bool on = slot < slots && t < (long long)p.B * p.T;
    const int b = on ? (int)(t / p.T) : 0, l = on ? (int)(t % p.T) : 0;

    const int nturn = p.R >> 4;
    const bool turns = unit < nturn;
    int o1, o2;  // the unit's two runs of 8 dimensions
    if (turns) {
        o1 = p.start + (INTER ? 16 : 8) * unit;
        o2 = o1 + (INTER ? 8 : p.R / 2);
    } else {
        o1 = 16 * (unit - nturn);
        if (o1 >= p.start) o1 += p.R;
        o2 = o1 + 8;
    }
    const int h1 = p.r[0].heads, h2 = h1 + p.r[1].heads, heads = h2 + p.r[2].heads;
    const int step = slots * gridDim.y;

    Eight<In> x1[U], x2[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) break;
            const int kind = (h >= h1) + (h >= h2);
            const RotaryRows& r = p.r[kind];
            if (!turns && r.in_place) continue;
            const In* x = static_cast<const In*>(r.x) + b * r.xb + l * r.xt +
                          (h - (kind == 0 ? 0 : kind == 1 ? h1 : h2)) * r.xh;
            x1[i] = load8(x + o1);
            x2[i] = load8(x + o2);
        }
    };
    int h0 = slot + slots * blockIdx.y;
    if (on) load(h0);

    int pos = 0;
    long long row = 0;
    if constexpr (APPEND) {
        if (threadIdx.x < tokens) {
            const long long mine = (long long)blockIdx.x * tokens + threadIdx.x;
            long long at = -1;
            int ps = 0;
            if (mine < p.T) {
                int s = 0, end = p.num_seqs - 1;  // the last sequence that begins at the token or before
                while (s < end) {
                    const int mid = (s + end + 1) >> 1;
                    if (p.cu[mid] <= (int)mine)
                        s = mid;
                    else
                        end = mid - 1;
                }
                const Kv16Seq q = kv16_sequence(p.c, p.cu, p.T, s);
                const int i = (int)mine - q.row0;
                if (i >= 0 && i < q.n) {  // else a row behind the last sequence
                    ps = q.len - q.n + i;
                    at = kv16_row(p.c, p.D, q.pages, ps);
                }
            }
            s_row[threadIdx.x] = at;
            s_pos[threadIdx.x] = ps;
        }
        __syncthreads();
        row = s_row[tok];
        pos = s_pos[tok];
        if (row < 0) return;
        if (p.pos && on) pos = __ldg(p.pos + l);
    } else {
        pos = !on ? 0 : p.pos ? __ldg(p.pos + b * p.pos_b + l) : l;
    }
    if (!on) return;
    float c[8], s[8];
    if (turns) angles(p, pos, 8 * unit, c, s);

    while (h0 < heads) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) break;
            const int kind = (h >= h1) + (h >= h2), hh = h - (kind == 0 ? 0 : kind == 1 ? h1 : h2);
            const RotaryRows& r = p.r[kind];
            if (!turns && r.in_place) continue;
            Out* y;
            if (APPEND && kind > 0)
                y = reinterpret_cast<Out*>(p.c.pool) + row + (hh + (kind == 2 ? p.c.Hkv : 0)) * kv16_head_stride(p.c, p.D);
            else
                y = static_cast<Out*>(r.y) + b * r.yb + l * r.yt + hh * r.yh;
            float a[8], d[8];
            unpack8<In>(x1[i], a);
            unpack8<In>(x2[i], d);
            if (turns && kind < 2) turn<INTER>(a, d, c, s);
            store8(y + o1, a);
            store8(y + o2, d);
        }
        h0 += U * step;
        load(h0);
    }
}

// Tokens of a block, and blocks per token: with few tokens a block takes one
// token, and its heads are spread over blocks so that no thread has a second
// row; with many, eight tokens, and a thread takes all heads of its slot.
struct RopeGrid {
    dim3 grid;
    int tokens;
};

RopeGrid rope_grid(const RotaryParams& p, int num_sms, bool extra)
{
    const long long n = (long long)p.B * p.T;
    const int units = p.D / 16, heads = p.r[0].heads + p.r[1].heads + p.r[2].heads;
    RopeGrid g;
    g.tokens = 1;
    while (g.tokens < 8 && kThreads / (2 * g.tokens) >= units && n >= (long long)16 * num_sms * g.tokens) g.tokens *= 2;
    const int slots = kThreads / g.tokens / units;
    const int parts = n * heads / slots < 8ll * num_sms ? (heads + slots - 1) / slots : 1;
    g.grid = dim3((unsigned)((n + g.tokens - 1) / g.tokens + (extra ? 1 : 0)), (unsigned)parts);
    return g;
}

template <typename In, typename Out, bool INTER, bool APPEND>
cudaError_t launch(const RotaryParams& p, int num_sms, cudaStream_t stream)
{
    const RopeGrid g = rope_grid(p, num_sms, APPEND && p.c.ids);
    fa_rope_kernel<In, Out, INTER, APPEND><<<g.grid, kThreads, 0, stream>>>(p, g.tokens);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(bool in_f32, bool out_f32, bool interleaved, const RotaryParams& p, int num_sms,
                        cudaStream_t stream)
{
    if (!in_f32)
        return interleaved ? launch<uint16_t, uint16_t, true, false>(p, num_sms, stream)
                           : launch<uint16_t, uint16_t, false, false>(p, num_sms, stream);
    if (out_f32)
        return interleaved ? launch<float, float, true, false>(p, num_sms, stream)
                           : launch<float, float, false, false>(p, num_sms, stream);
    return interleaved ? launch<float, uint16_t, true, false>(p, num_sms, stream)
                       : launch<float, uint16_t, false, false>(p, num_sms, stream);
}

cudaError_t launch_kv16_append(bool interleaved, const RotaryParams& p, int num_sms, cudaStream_t stream)
{
    return interleaved ? launch<uint16_t, uint16_t, true, true>(p, num_sms, stream)
                       : launch<uint16_t, uint16_t, false, true>(p, num_sms, stream);
}

}  // namespace fa
