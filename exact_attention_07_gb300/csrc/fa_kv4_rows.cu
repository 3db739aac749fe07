// Rows into and out of the 4-bit cache: append (quantise) and read
// (dequantise) of packed bf16 rows.  Both move a few bytes per operation and
// are bound by HBM: 4 D bytes of bf16 and 18 D / 16 bytes of cache per
// (position, KV head).
//
// One warp handles one unit: 16 positions of one KV head, 18 D contiguous
// bytes of the cache (append: one warp for its K and one for its V).  A lane's
// piece is a group of 16 dimensions: of one position for K, of two
// neighbouring ones for V, whose codes share bytes.  The order of the pieces
// is that of the cache's bytes, so that a warp reads or writes them in
// contiguous runs, and the bf16 side goes in whole 32-byte sectors (one
// 32-byte access per lane where the caller's rows are so aligned).  All loads
// of a warp's piece are issued before the first is used.  Read: 67 us for
// 80757 positions of 8 heads, D = 128, 93 % of the copy bandwidth (91 us with
// a thread per group of two positions and 16-byte accesses).
#include <algorithm>

#include "kv4_common.cuh"

namespace fa {

namespace {

constexpr int kRowsThreads = 256;

// Slots of units: sequence s of the call starts at unit slot cu[s] / 16 + 2 s,
// which leaves it at least the (n + 14) / 16 + 1 units that n positions may
// touch, so a grid of total / 16 + 2 num_seqs slots needs no prefix sums.
__device__ __forceinline__ int unit_slot(const int* cu, int s) { return (cu[s] >> 4) + 2 * s; }

struct UnitTask {
    uint8_t* unit;      // its bytes in the cache; null for a bad page
    int lo, hi;         // rows lo .. hi - 1 of the unit are the call's
    long long row;      // packed row of the unit's row 0
    int h;
};

// The w-th (unit slot, group of `heads` KV heads); false when there is nothing
// to do.  The task's unit is that of the group's first head; the other heads'
// follow one page_size / 16 units apart.
template <int D>
__device__ __forceinline__ bool find_unit(const Kv4RowsParams& p, unsigned w, int heads, UnitTask& t)
{
    const unsigned groups = (unsigned)((p.c.Hkv + heads - 1) / heads), u = w / groups;
    t.h = (int)(w - u * groups) * heads;
    if (u >= (unsigned)(p.total >> 4) + 2u * (unsigned)p.num_seqs) return false;
    int s = 0, end = p.num_seqs - 1;  // the last sequence whose first slot is <= u
    while (s < end) {
        const int mid = (s + end + 1) >> 1;
        if (unit_slot(p.cu, mid) <= (int)u)
            s = mid;
        else
            end = mid - 1;
    }
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    if (c0 < 0 || c1 < c0 || c1 > p.total || (s == 0 && c0 != 0)) {
        atomicOr(p.c.err, 2);
        return false;
    }
    int slot;
    const int len = kv4_sequence(p.c, s, slot), n = c1 - c0, first = len - n;
    if (first < 0) {
        atomicOr(p.c.err, 2);
        return false;
    }
    const long long pos = 16ll * ((first >> 4) + ((int)u - unit_slot(p.cu, s)));
    if (pos < 0 || pos >= len) return false;
    t.lo = max(0, first - (int)pos);
    t.hi = min(16, len - (int)pos);
    if (t.lo >= t.hi) return false;
    t.row = c0 + (pos - first);
    const int page = p.c.table[(long long)slot * p.c.table_width + (pos >> p.c.page_shift)];
    if ((unsigned)page >= (unsigned)p.c.num_pages) {
        atomicOr(p.c.err, 2);
        return false;
    }
    t.unit = p.c.pool + kv4_unit(p.c, D, page, t.h, (int)pos);
    return true;
}

// ------------------------------------------------------------------ append

struct Group {
    uint32_t w[8];  // 16 bf16
};

__device__ __forceinline__ Group load_group(const uint16_t* src, bool on, bool wide)
{
    Group x = {{0, 0, 0, 0, 0, 0, 0, 0}};
    if (on && wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]),
                       "=r"(x.w[6]), "=r"(x.w[7])
                     : "l"(src));
    } else if (on) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src)), b = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
        x = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return x;
}

// e2m1 codes of eight values in four packed pairs, two a byte, the first in
// the low nibble: ties to even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_word(const uint64_t (&y)[4])
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(y[i], x[2 * i], x[2 * i + 1]);
    uint32_t r;
    asm("{.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A quotient x / y from r, 1 / y to an ulp, with Markstein's correction: the
// product x r, then the remainder's share of it.  A quotient that is a number
// comes out as that number, so a value exactly between two codes is seen as
// such; x r alone is off by an ulp there.
__device__ __forceinline__ float quotient(float x, float y, float r)
{
    const float q = x * r;
    return __fmaf_rn(__fmaf_rn(-q, y, x), r, q);
}

// max(a, |x|) of two bf16 each; a NaN stays one.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t x)
{
    uint32_t r;
    asm("{.reg .b32 t; abs.bf16x2 t, %2; max.NaN.bf16x2 %0, %1, t;}" : "=r"(r) : "r"(a), "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two bf16 each, brought into -bound .. bound.
__device__ __forceinline__ uint32_t clamp_pair(uint32_t x, uint32_t bound)
{
    uint32_t r;
    asm("{.reg .b32 t; min.bf16x2 t, %1, %2; max.bf16x2 %0, t, %3;}"
        : "=r"(r)
        : "r"(x), "r"(bound), "r"(bound ^ 0x80008000u));
    return r;
}

struct Codes {
    uint32_t w[2];  // dimensions 0 .. 7, 8 .. 15
    uint32_t scale;
};

// Quantises a group.  head6 = 6 * head scale, r6 its reciprocal.  The maximum
// is taken on the magnitudes' bits, where infinities and NaN come out above
// every number; such a group gets a NaN scale and zero codes.  Quotients that
// could overflow are brought to 512 (the scale) and 8 (values of a group that
// the largest scale does not reach), which round as anything above them.
__device__ __forceinline__ Codes quantise_group(Group& x, float head, float head6, float r6)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_magnitude(m, x.w[i]);
    const uint32_t top = max(m & 0xffffu, m >> 16);
    const bool bad = top >= 0x7f80u;
    uint16_t pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(pair)
        : "f"(0.f), "f"(bad ? 0.f : quotient(fminf(__uint_as_float(top << 16), 512.f * head6), head6, r6)));
    Codes c;
    c.scale = bad ? 0x7fu : (uint32_t)pair;
    const float s = f16x2_to_f32(e4m3x2_to_f16x2(pair)).x * head;
    const float r = pair == 0 ? 0.f : rcp_approx(s);
    const uint64_t r2 = f2_pack(r, r), s2 = f2_pack(-s, -s);
    if (pair == 0x7e) {
        const uint32_t bound = bf16x2(8.f * s, 8.f * s);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.w[i] = clamp_pair(x.w[i], bound);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint64_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // quotient(), two values at a time
            const uint32_t w = x.w[4 * e + i];
            const uint64_t v = f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            const uint64_t q = f2_mul(v, r2);
            y[i] = f2_fma(f2_fma(q, s2, v), r2, q);
        }
        c.w[e] = pair == 0 ? 0u : e2m1_word(y);
    }
    return c;
}

// Codes of two positions, eight dimensions a word, to one byte a dimension
// (position a in the low nibble): dimensions 0 .. 3 and 4 .. 7.
__device__ __forceinline__ uint2 pair_codes(uint32_t a, uint32_t b)
{
    const uint32_t even = (a & 0x0f0f0f0fu) | (b & 0x0f0f0f0fu) << 4;
    const uint32_t odd = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
    return make_uint2(__byte_perm(even, odd, 0x5140), __byte_perm(even, odd, 0x7362));
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 4) fa_kv4_append_kernel(const Kv4RowsParams p)
{
    constexpr int G = D / 16, KI = D / 32, VI = D / 64;
    // the last block looks for slots that the call names twice
    if (p.c.ids && blockIdx.x == gridDim.x - 1) {
        __shared__ uint32_t seen[kKv4MaxSlots / 32];
        for (int i = threadIdx.x; i < kKv4MaxSlots / 32; i += kRowsThreads) seen[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.num_seqs; i += kRowsThreads) {
            const int s = p.c.ids[i];
            if (s < 0 || s >= p.c.num_slots || p.cu[i + 1] <= p.cu[i]) continue;  // no rows: a padded batch
            const uint32_t bit = 1u << (s & 31);
            if (atomicOr(&seen[s >> 5], bit) & bit) atomicOr(p.c.err, 2);
        }
        return;
    }
    // One warp for K and one for V of a unit: with both in one the loaded rows
    // took 88 registers and left 16 warps an SM (46 us for 8 prompts of 32916
    // tokens in all, 8 heads, D = 128; so 36 us, 4.8 TB/s).
    const unsigned w = blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
    UnitTask t;
    if (!find_unit<D>(p, w >> 1, p.heads, t)) return;
    const int lane = threadIdx.x & 31;
    const long long pitch = (long long)p.c.Hkv * D;
    const auto mine = [&](int r) { return r >= t.lo && r < t.hi; };
    const float* scales = w & 1 ? p.c.v_scale : p.c.k_scale;
    const int end = min(t.h + p.heads, p.c.Hkv);
#pragma unroll 1
    for (int h = t.h; h < end; ++h, t.unit += (18 * D) << (p.c.page_shift - 4)) {
        const long long base = t.row * pitch + h * D;
        const float head = scales ? scales[h] : 1.f, head6 = 6.f * head, r6 = rcp_approx(head6);
        if (!(w & 1)) {
            Group k[KI];
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int x = 32 * i + lane, r = x / G, g = x % G;
                k[i] = load_group(p.k_in + base + r * pitch + g * 16, mine(r), p.wide);
            }
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const int x = 32 * i + lane;
                const Codes c = quantise_group(k[i], head, head6, r6);
                if (!mine(x / G)) continue;
                *reinterpret_cast<uint2*>(t.unit + x * 8) = make_uint2(c.w[0], c.w[1]);
                t.unit[16 * D + x] = (uint8_t)c.scale;
            }
            continue;
        }
        Group v[VI][2];
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int x = 32 * i + lane, g = x / 4 % G, r = x / (4 * G) * 8 + x % 4 * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                v[i][e] = load_group(p.v_in + base + (r + e) * pitch + g * 16, mine(r + e), p.wide);
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int x = 32 * i + lane, g = x / 4 % G, r = x / (4 * G) * 8 + x % 4 * 2;
            const bool even = mine(r), odd = mine(r + 1);
            const Codes a = quantise_group(v[i][0], head, head6, r6), b = quantise_group(v[i][1], head, head6, r6);
            if (!even && !odd) continue;
            const uint2 lo = pair_codes(a.w[0], b.w[0]), hi = pair_codes(a.w[1], b.w[1]);
            uint4* codes = reinterpret_cast<uint4*>(t.unit + 8 * D + x * 16);
            uint8_t* to = t.unit + 17 * D + g * 16 + r;
            if (even && odd) {
                *codes = make_uint4(lo.x, lo.y, hi.x, hi.y);
                *reinterpret_cast<uint16_t*>(to) = (uint16_t)(a.scale | b.scale << 8);
            } else {  // the pair's other position keeps its nibbles
                const uint32_t own = even ? 0x0f0f0f0fu : 0xf0f0f0f0u;
                const uint4 old = *codes;
                *codes = make_uint4((old.x & ~own) | (lo.x & own), (old.y & ~own) | (lo.y & own),
                                    (old.z & ~own) | (hi.x & own), (old.w & ~own) | (hi.y & own));
                to[even ? 0 : 1] = (uint8_t)(even ? a.scale : b.scale);
            }
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

__device__ __forceinline__ void store_group(uint16_t* dst, const uint32_t (&w)[8], bool on, bool wide)
{
    if (on && wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else if (on) {
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(reinterpret_cast<uint4*>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) fa_kv4_read_kernel(const Kv4RowsParams p)
{
    constexpr int G = D / 16, KI = D / 32, VI = D / 64;
    UnitTask t;
    if (!find_unit<D>(p, blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5), 1, t)) return;
    const int lane = threadIdx.x & 31;
    uint2 kc[KI];
    uint4 vc[VI];
    uint32_t ks[KI], vs[VI];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int x = 32 * i + lane;
        kc[i] = __ldcs(reinterpret_cast<const uint2*>(t.unit + x * 8));
        ks[i] = t.unit[16 * D + x];
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
        const int x = 32 * i + lane, g = x / 4 % G, r = x / (4 * G) * 8 + x % 4 * 2;
        vc[i] = __ldcs(reinterpret_cast<const uint4*>(t.unit + 8 * D + x * 16));
        vs[i] = *reinterpret_cast<const uint16_t*>(t.unit + 17 * D + g * 16 + r);
    }
    const long long pitch = (long long)p.c.Hkv * D, base = t.row * pitch + t.h * D;
    const auto mine = [&](int r) { return r >= t.lo && r < t.hi; };
    const float gk = p.c.k_scale ? p.c.k_scale[t.h] : 1.f, gv = p.c.v_scale ? p.c.v_scale[t.h] : 1.f;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int x = 32 * i + lane, r = x / G, g = x % G;
        const uint32_t s = e4m3x2_to_f16x2((uint16_t)(ks[i] | ks[i] << 8));
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t c = e ? kc[i].y : kc[i].x;
            const uint32_t f[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c), e2m1x2_to_f16x2<2>(c),
                                   e2m1x2_to_f16x2<3>(c)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float2 y = f16x2_to_f32(hmul2(f[b], s));
                w[4 * e + b] = bf16x2(y.x * gk, y.y * gk);
            }
        }
        store_group(p.k_out + base + r * pitch + g * 16, w, mine(r), p.wide);
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
        const int x = 32 * i + lane, g = x / 4 % G, r = x / (4 * G) * 8 + x % 4 * 2;
        const uint32_t s = e4m3x2_to_f16x2((uint16_t)vs[i]);
        uint32_t wa[8], wb[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t c = e == 0 ? vc[i].x : e == 1 ? vc[i].y : e == 2 ? vc[i].z : vc[i].w;
            const uint32_t f[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c), e2m1x2_to_f16x2<2>(c),
                                   e2m1x2_to_f16x2<3>(c)};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float2 y = f16x2_to_f32(hmul2(f[2 * b], s)), z = f16x2_to_f32(hmul2(f[2 * b + 1], s));
                wa[2 * e + b] = bf16x2(y.x * gv, z.x * gv);
                wb[2 * e + b] = bf16x2(y.y * gv, z.y * gv);
            }
        }
        store_group(p.v_out + base + r * pitch + g * 16, wa, mine(r), p.wide);
        store_group(p.v_out + base + (r + 1) * pitch + g * 16, wb, mine(r + 1), p.wide);
    }
}

long long unit_slots(const Kv4RowsParams& p) { return (long long)(p.total >> 4) + 2ll * p.num_seqs; }

unsigned rows_blocks(long long warps) { return (unsigned)((warps + kRowsThreads / 32 - 1) / (kRowsThreads / 32)); }

}  // namespace

cudaError_t launch_kv4_append(int D, const Kv4RowsParams& params, int num_sms, cudaStream_t stream)
{
    // A warp finds its unit through five dependent loads and some 150
    // instructions.  Where there are more warps than run at once (32 an SM), one
    // takes several heads of the unit and pays for them once (8 prompts appended
    // and read back 64 -> 62 us), while a decode step's few tokens want a warp
    // per head.
    Kv4RowsParams p = params;
    const long long warps = 2 * unit_slots(p) * p.c.Hkv;
    p.heads = (int)std::max(1ll, std::min({4ll, (long long)p.c.Hkv, warps / (32ll * num_sms)}));
    const unsigned grid = rows_blocks(2 * unit_slots(p) * ((p.c.Hkv + p.heads - 1) / p.heads)) + (p.c.ids ? 1 : 0);
    if (D == 128)
        fa_kv4_append_kernel<128><<<grid, kRowsThreads, 0, stream>>>(p);
    else
        fa_kv4_append_kernel<64><<<grid, kRowsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(int D, const Kv4RowsParams& p, cudaStream_t stream)
{
    const unsigned grid = rows_blocks(unit_slots(p) * p.c.Hkv);
    if (D == 128)
        fa_kv4_read_kernel<128><<<grid, kRowsThreads, 0, stream>>>(p);
    else
        fa_kv4_read_kernel<64><<<grid, kRowsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
