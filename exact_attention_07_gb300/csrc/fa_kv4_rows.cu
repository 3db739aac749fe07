// Rows into and out of the 4-bit cache: append (quantise) and read
// (dequantise) of packed bf16 rows.  Both move a few bytes per operation and
// are bound by HBM: 4 D bytes of bf16 and 18 D / 16 bytes of cache per
// (position, KV head).
//
// One thread handles one group of 16 dimensions of one KV head at the two
// positions 2 i and 2 i + 1, which share the bytes of V (one nibble each): K
// and V of both are eight independent 16-byte loads (or stores) of bf16, and
// the cache's side is 16 bytes of V codes and 8 + 8 bytes of K codes.
#include "kv4_common.cuh"

namespace fa {

namespace {

constexpr int kRowsThreads = 256;

// Slots of position pairs: sequence s of the call starts at pair slot
// cu[s] / 2 + s, which leaves it at least the n / 2 + 1 pairs that n positions
// may touch, so a grid of total / 2 + num_seqs slots needs no prefix sums.
__device__ __forceinline__ int pair_slot(const int* cu, int s) { return (cu[s] >> 1) + s; }

struct PairTask {
    int slot;        // slot of the sequence
    int pos;         // even position of the pair
    long long row;   // packed row of `pos` (of pos + 1: row + 1)
    bool even, odd;  // which of the two are the call's
};

// False when the pair slot holds nothing to do.
__device__ __forceinline__ bool find_pair(const Kv4RowsParams& p, int u, PairTask& t)
{
    int lo = 0, hi = p.num_seqs - 1;  // the last sequence whose first slot is <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pair_slot(p.cu, mid) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int c0 = p.cu[lo], c1 = p.cu[lo + 1];
    if (c0 < 0 || c1 < c0 || c1 > p.total || (lo == 0 && c0 != 0)) {
        atomicOr(p.c.err, 2);
        return false;
    }
    const int len = kv4_sequence(p.c, lo, t.slot), n = c1 - c0;
    if (n > len) {
        if (n > 0) atomicOr(p.c.err, 2);
        return false;
    }
    const int first = len - n;
    const long long pos = 2ll * ((first >> 1) + (u - pair_slot(p.cu, lo)));
    if (pos < 0 || pos >= len) return false;
    t.pos = (int)pos;
    t.even = t.pos >= first;
    t.odd = t.pos + 1 < len && t.pos + 1 >= first;
    t.row = (long long)c0 + t.pos - first;
    return t.even || t.odd;
}

// ------------------------------------------------------------------ append

struct Group {
    uint32_t w[8];  // 16 bf16
};

__device__ __forceinline__ Group load_group(const uint16_t* src, bool on)
{
    Group x;
    if (on) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src)), b = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
        x = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    } else {
        x = {{0, 0, 0, 0, 0, 0, 0, 0}};
    }
    return x;
}

// Scale byte of a group and the 16 quotients x / (head scale * scale).  The
// maximum is taken on the magnitudes' bits, where infinities and NaN come out
// above every number; such a group gets a NaN scale and zero codes.
__device__ __forceinline__ uint32_t quantise_group(const Group& x, float head, float (&y)[16])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x.w[i] & 0x7fff7fffu);
    const uint32_t top = max(m & 0xffffu, m >> 16);
    const float amax = __fdiv_rn(__uint_as_float(top << 16), head);
    uint16_t pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.f), "f"(__fdiv_rn(amax, 6.f)));
    const bool none = top >= 0x7f80u || (pair & 0x7f) == 0;
    const float s = none ? 0.f : f16x2_to_f32(e4m3x2_to_f16x2(pair)).x * head;
    // Quotients with Markstein's correction (x r, then the remainder's share):
    // the rounded quotient, so that a value exactly between two codes is seen
    // as such; x r alone is off by an ulp there.
    const float r = none ? 0.f : __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float v = none ? 0.f : __uint_as_float((i & 1) ? x.w[i >> 1] & 0xffff0000u : x.w[i >> 1] << 16);
        const float q = v * r;
        y[i] = __fmaf_rn(__fmaf_rn(-q, s, v), r, q);
    }
    return top >= 0x7f80u ? 0x7fu : (pair & 0xffu);
}

// e2m1 codes of eight values, two a byte, the first in the low nibble: ties
// to even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_word(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                              float x7)
{
    uint32_t r;
    asm("{.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) fa_kv4_append_kernel(const Kv4RowsParams p)
{
    constexpr int G = D / 16;
    // the last block looks for slots that the call names twice
    if (p.c.ids && blockIdx.x == gridDim.x - 1) {
        __shared__ uint32_t seen[kKv4MaxSlots / 32];
        for (int i = threadIdx.x; i < kKv4MaxSlots / 32; i += kRowsThreads) seen[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.num_seqs; i += kRowsThreads) {
            const int s = p.c.ids[i];
            if (s < 0 || s >= p.c.num_slots) continue;
            const uint32_t bit = 1u << (s & 31);
            if (atomicOr(&seen[s >> 5], bit) & bit) atomicOr(p.c.err, 2);
        }
        return;
    }
    const long long flat = (long long)blockIdx.x * kRowsThreads + threadIdx.x;
    const int per = p.c.Hkv * G;
    const long long u = flat / per;
    if (u >= (long long)(p.total >> 1) + p.num_seqs) return;
    PairTask t;
    if (!find_pair(p, (int)u, t)) return;
    const int hg = (int)(flat - u * per), h = hg / G, g = hg % G;
    const int page = p.c.table[(long long)t.slot * p.c.table_width + (t.pos >> p.c.page_shift)];
    if ((unsigned)page >= (unsigned)p.c.num_pages) {
        atomicOr(p.c.err, 2);
        return;
    }
    const long long src = (t.row * p.c.Hkv + h) * D + g * 16, row = (long long)p.c.Hkv * D;
    const Group ka = load_group(p.k_in + src, t.even), kb = load_group(p.k_in + src + row, t.odd);
    const Group va = load_group(p.v_in + src, t.even), vb = load_group(p.v_in + src + row, t.odd);
    uint8_t* unit = p.c.pool + kv4_unit(p.c, D, page, h, t.pos);
    const int key = t.pos & 15;
    const float gk = p.c.k_scale ? p.c.k_scale[h] : 1.f, gv = p.c.v_scale ? p.c.v_scale[h] : 1.f;

#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i ? t.odd : t.even) {
            float y[16];
            const uint32_t s = quantise_group(i ? kb : ka, gk, y);
            *reinterpret_cast<uint2*>(unit + (key + i) * (D / 2) + g * 8) =
                make_uint2(e2m1_word(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]),
                           e2m1_word(y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]));
            unit[16 * D + (key + i) * G + g] = (uint8_t)s;
        }
    }
    {
        float ya[16], yb[16];
        const uint32_t sa = quantise_group(va, gv, ya), sb = quantise_group(vb, gv, yb);
        uint4* codes = reinterpret_cast<uint4*>(unit + 8 * D + (key >> 3) * (4 * D) + g * 64 + ((key & 7) >> 1) * 16);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = e2m1_word(ya[4 * e], yb[4 * e], ya[4 * e + 1], yb[4 * e + 1], ya[4 * e + 2], yb[4 * e + 2],
                             ya[4 * e + 3], yb[4 * e + 3]);
        uint8_t* scales = unit + 17 * D + g * 16 + key;
        if (t.even && t.odd) {
            *codes = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint16_t*>(scales) = (uint16_t)(sa | sb << 8);
        } else {  // the pair's other position keeps its nibbles
            const uint32_t mine = t.even ? 0x0f0f0f0fu : 0xf0f0f0f0u;
            const uint4 old = *codes;
            *codes = make_uint4((old.x & ~mine) | (w[0] & mine), (old.y & ~mine) | (w[1] & mine),
                                (old.z & ~mine) | (w[2] & mine), (old.w & ~mine) | (w[3] & mine));
            scales[t.even ? 0 : 1] = (uint8_t)(t.even ? sa : sb);
        }
    }
}

// ------------------------------------------------------------------ read

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void store_group(uint16_t* dst, const uint32_t (&w)[8])
{
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) fa_kv4_read_kernel(const Kv4RowsParams p)
{
    constexpr int G = D / 16;
    const long long flat = (long long)blockIdx.x * kRowsThreads + threadIdx.x;
    const int per = p.c.Hkv * G;
    const long long u = flat / per;
    if (u >= (long long)(p.total >> 1) + p.num_seqs) return;
    PairTask t;
    if (!find_pair(p, (int)u, t)) return;
    const int hg = (int)(flat - u * per), h = hg / G, g = hg % G;
    const int page = kv4_page(p.c, t.slot, t.pos);
    const uint8_t* unit = p.c.pool + kv4_unit(p.c, D, page, h, t.pos);
    const int key = t.pos & 15;
    const uint4 vc =
        *reinterpret_cast<const uint4*>(unit + 8 * D + (key >> 3) * (4 * D) + g * 64 + ((key & 7) >> 1) * 16);
    const uint32_t vs = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(unit + 17 * D + g * 16 + key));
    const float gk = p.c.k_scale ? p.c.k_scale[h] : 1.f, gv = p.c.v_scale ? p.c.v_scale[h] : 1.f;
    const long long dst = (t.row * p.c.Hkv + h) * D + g * 16, row = (long long)p.c.Hkv * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i ? t.odd : t.even) {
            const uint2 kc = *reinterpret_cast<const uint2*>(unit + (key + i) * (D / 2) + g * 8);
            const uint32_t s1 = unit[16 * D + (key + i) * G + g];
            const uint32_t s = e4m3x2_to_f16x2((uint16_t)(s1 | s1 << 8));
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t c = e ? kc.y : kc.x;
                const uint32_t f[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c), e2m1x2_to_f16x2<2>(c),
                                       e2m1x2_to_f16x2<3>(c)};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float2 x = f16x2_to_f32(hmul2(f[b], s));
                    w[4 * e + b] = bf16x2(x.x * gk, x.y * gk);
                }
            }
            store_group(p.k_out + dst + i * row, w);
        }
    }
    uint32_t wa[8], wb[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t c = e == 0 ? vc.x : e == 1 ? vc.y : e == 2 ? vc.z : vc.w;
        const uint32_t f[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c), e2m1x2_to_f16x2<2>(c),
                               e2m1x2_to_f16x2<3>(c)};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float2 x = f16x2_to_f32(hmul2(f[2 * b], vs)), y = f16x2_to_f32(hmul2(f[2 * b + 1], vs));
            wa[2 * e + b] = bf16x2(x.x * gv, y.x * gv);
            wb[2 * e + b] = bf16x2(x.y * gv, y.y * gv);
        }
    }
    if (t.even) store_group(p.v_out + dst, wa);
    if (t.odd) store_group(p.v_out + dst + row, wb);
}

long long rows_blocks(int D, const Kv4RowsParams& p)
{
    const long long threads = ((long long)(p.total >> 1) + p.num_seqs) * p.c.Hkv * (D / 16);
    return (threads + kRowsThreads - 1) / kRowsThreads;
}

}  // namespace

cudaError_t launch_kv4_append(int D, const Kv4RowsParams& p, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(rows_blocks(D, p) + (p.c.ids ? 1 : 0));
    if (D == 128)
        fa_kv4_append_kernel<128><<<grid, kRowsThreads, 0, stream>>>(p);
    else
        fa_kv4_append_kernel<64><<<grid, kRowsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(int D, const Kv4RowsParams& p, cudaStream_t stream)
{
    const unsigned grid = (unsigned)rows_blocks(D, p);
    if (D == 128)
        fa_kv4_read_kernel<128><<<grid, kRowsThreads, 0, stream>>>(p);
    else
        fa_kv4_read_kernel<64><<<grid, kRowsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
