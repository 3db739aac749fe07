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
// Bound: HBM, each element read and written once.  A block computes the cosines
// and sines of its tokens once, into shared memory (a thread that computes its
// own takes 145 us where this takes 126); a thread holds those of 8 pairs (16
// dimensions) of one token and takes its rows of several heads, with four rows'
// loads in flight.  Dimensions that do not turn are copied by threads of the same
// kind.  Measured: 39235 tokens, 40 heads, D = 128, bf16 (804 MB) 126 us, 6380
// GB/s; their gradients, fp32 to bf16, 183 us, 6600 GB/s; 26600 tokens' K and V
// (8 heads each) into the cache, 32 heads of q turned alike (653 MB), 107 us, 6100.
#include <cuda_bf16.h>

#include <algorithm>

#include "kv16_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128, kMaxTokens = 8;

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
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// m cos and m sin of pair c of a row at position pos.
__device__ __forceinline__ float2 angle(const RotaryParams& p, int pos, int c)
{
    const unsigned long long turn = (unsigned long long)(long long)pos * __ldg(p.freqs + c);
    const float x = (float)(int)(turn >> 32) * 4.656612873077393e-10f;  // half turns, -1 .. 1
    float sn, cs;
    sincospif(x, &sn, &cs);
    return make_float2(p.mscale * cs, p.mscale * (p.backward ? -sn : sn));
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
// of their heads.  It computes the tokens' cosines and sines once, into shared
// memory.  Of a token's threads, neighbours take the D / 16 units of a row: the
// first R / 16 turn, the others copy.  Append: the last `checks` blocks look at
// the sequences, each for itself, as tokens lead only to those that have some.
template <typename In, typename Out, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads, 4)
    fa_rope_kernel(const RotaryParams p, const int tokens, const int slots, const int checks)
{
    constexpr int U = sizeof(In) == 2 ? 4 : 2;  // rows in flight
    if constexpr (APPEND) {
        const int check = (int)(blockIdx.x - (gridDim.x - checks));
        if (check >= 0) {
            if (blockIdx.y != 0) return;
            for (long long s = (long long)check * blockDim.x + threadIdx.x; s < p.num_seqs; s += (long long)checks * blockDim.x)
                kv16_sequence(p.c, p.cu, p.T, (int)s);  // latches one that is not sound
            if (p.c.ids && check == 0) kv16_check_slots(p.c, p.cu, p.num_seqs);
            return;
        }
    }
    extern __shared__ __align__(16) float s_angle[];  // [tokens][R / 16][cosines 8, sines 8]
    __shared__ long long s_row[kMaxTokens];  // append: the token's K of head 0 in the pool, or -1
    __shared__ int s_pos[kMaxTokens];
    const int units = p.D >> 4, slot = (int)threadIdx.x / units % slots, unit = (int)threadIdx.x % units;
    const int tok = (int)threadIdx.x / (units * slots);
    const long long t0 = (long long)blockIdx.x * tokens, t = t0 + tok;
    const bool on = tok < tokens && t < (long long)p.B * p.T;  // threads behind the tokens' fill a warp
    const int b = on ? (int)(t / p.T) : 0, l = on ? (int)(t - (long long)b * p.T) : 0;

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

    // with few tokens (gridDim.y > 1) a thread has one row at most: it is on its
    // way while the position is looked up
    const int step = slots * gridDim.y;
    int h = slot + slots * blockIdx.y;  // of the rows of all kinds
    const int h1 = p.r[0].heads, h2 = h1 + p.r[1].heads, heads_all = h2 + p.r[2].heads;
    Eight<In> e1, e2;
    const bool early = gridDim.y > 1 && on && h < heads_all;
    if (early) {
        const int kind = (h >= h1) + (h >= h2);
        const RotaryRows& r = p.r[kind];
        const In* x = static_cast<const In*>(r.x) + b * r.xb + l * r.xt + (h - (kind == 0 ? 0 : kind == 1 ? h1 : h2)) * r.xh;
        e1 = load8(x + o1);
        e2 = load8(x + o2);
    }

    if constexpr (APPEND) {
        // the tokens' sequences, a warp a token: lanes look at 32 offsets at once
        const int lane = threadIdx.x & 31;
        for (int k = threadIdx.x >> 5; k < tokens; k += (int)blockDim.x >> 5) {
            const long long mine = t0 + k;
            long long at = -1;
            int pos = 0;
            if (mine < p.T) {
                int s = 0, n = p.num_seqs;  // the last sequence that begins at the token or before is in [s, s + n)
                while (n > 1) {
                    const int run = (n + 31) >> 5, i = s + lane * run;
                    const int before = __popc(__ballot_sync(~0u, i < s + n && p.cu[min(i, s + n - 1)] <= (int)mine));
                    const int skip = max(before - 1, 0) * run;
                    s += skip;
                    n = min(run, n - skip);
                }
                const Kv16Seq q = kv16_sequence(p.c, p.cu, p.T, s);
                const int i = (int)mine - q.row0;
                if (i >= 0 && i < q.n) {  // else a row behind the last sequence
                    pos = q.len - q.n + i;
                    at = kv16_row(p.c, p.D, q.pages, pos);
                }
                if (p.pos) pos = __ldg(p.pos + mine);
            }
            if (lane == 0) {
                s_row[k] = at;
                s_pos[k] = pos;
            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < tokens * nturn * 8; i += blockDim.x) {
        const int k = i / (nturn * 8), c = i - k * (nturn * 8);
        int pos = 0;
        if constexpr (APPEND) {
            pos = s_pos[k];
        } else {
            const long long mine = min(t0 + k, (long long)p.B * p.T - 1);
            const int mb = (int)(mine / p.T), ml = (int)(mine - (long long)mb * p.T);
            pos = p.pos ? __ldg(p.pos + mb * p.pos_b + ml) : ml;
        }
        const float2 cs = angle(p, pos, c);
        float* at = s_angle + (i & ~7) * 2 + (c & 7);
        at[0] = cs.x;
        at[8] = cs.y;
    }
    __syncthreads();
    if (!on) return;
    long long row = 0;
    if constexpr (APPEND) {
        row = s_row[tok];
        if (row < 0) return;
    }
    float c[8], s[8];
    if (turns) {
        const float4* at = reinterpret_cast<const float4*>(s_angle + (tok * nturn + unit) * 16);
        const float4 v[4] = {at[0], at[1], at[2], at[3]};
        const float* f = &v[0].x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = f[i];
            s[i] = f[8 + i];
        }
    }

#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
        const RotaryRows& r = p.r[kind];
        const int heads = r.heads;
        const int mine = h;  // the slot's rows of this kind: every `step`-th from here
        h = (mine - heads) % step;
        if (h < 0) h += step;  // and the next kind's
        if (mine >= heads || (!turns && r.in_place)) continue;
        const In* x = static_cast<const In*>(r.x) + b * r.xb + l * r.xt + mine * r.xh;
        Out* y;
        long long ys;
        if (APPEND && kind > 0) {
            ys = kv16_head_stride(p.c, p.D);
            y = reinterpret_cast<Out*>(p.c.pool) + row + (mine + (kind == 2 ? p.c.Hkv : 0)) * ys;
        } else {
            ys = r.yh;
            y = static_cast<Out*>(r.y) + b * r.yb + l * r.yt + mine * ys;
        }
        const long long dx = r.xh * step, dy = ys * step;
        const bool turning = turns && kind < 2;
#pragma unroll 1
        for (int k = mine; k < heads; k += U * step, x += U * dx, y += U * dy) {
            Eight<In> x1[U], x2[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (i == 0 && early) {
                    x1[0] = e1;
                    x2[0] = e2;
                } else if (k + i * step < heads) {
                    x1[i] = load8(x + i * dx + o1);
                    x2[i] = load8(x + i * dx + o2);
                }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k + i * step < heads) {
                    float a[8], d[8];
                    unpack8<In>(x1[i], a);
                    unpack8<In>(x2[i], d);
                    if (turning) turn<INTER>(a, d, c, s);
                    store8(y + i * dy + o1, a);
                    store8(y + i * dy + o2, d);
                }
        }
    }
}

// Tokens of a block, and blocks per token: with few tokens a block takes one
// token, and its heads are spread over blocks so that no thread has a second
// row; with many, eight tokens, and a thread takes all heads of its slot.
struct RopeGrid {
    dim3 grid;
    int threads, tokens, slots, checks;
};

RopeGrid rope_grid(const RotaryParams& p, int num_sms, bool append)
{
    const long long n = (long long)p.B * p.T;
    const int units = p.D / 16, heads = p.r[0].heads + p.r[1].heads + p.r[2].heads;
    RopeGrid g;
    g.tokens = 1;
    while (g.tokens < kMaxTokens && kThreads / (2 * g.tokens) >= units && n >= (long long)16 * num_sms * g.tokens) g.tokens *= 2;
    g.slots = std::min(heads, kThreads / g.tokens / units);
    g.threads = (g.tokens * g.slots * units + 31) / 32 * 32;  // whole warps: they look for sequences together
    const int parts = n * heads / g.slots < 8ll * num_sms ? (heads + g.slots - 1) / g.slots : 1;
    g.checks = append ? std::min((p.num_seqs - 1) / g.threads + 1, num_sms) : 0;  // a sequence a thread
    g.grid = dim3((unsigned)((n + g.tokens - 1) / g.tokens + g.checks), (unsigned)parts);
    return g;
}

template <typename In, typename Out, bool INTER, bool APPEND>
cudaError_t launch(const RotaryParams& p, int num_sms, cudaStream_t stream)
{
    const RopeGrid g = rope_grid(p, num_sms, APPEND);
    fa_rope_kernel<In, Out, INTER, APPEND>
        <<<g.grid, g.threads, g.tokens * p.R * 4, stream>>>(p, g.tokens, g.slots, g.checks);
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
