// Attention over the 4-bit cache (decode): few query rows per KV head, a long
// key range, keys and values as e2m1 codes with e4m3 scales.
//
//   s_ij = scale * sum_d q_id K_jd,  p_ij = 2^(s_ij log2 e - m_i),
//   O_i = sum_j p_ij V_j / sum_j p_ij
//
// Bound: the cache's bytes are read once, 18 D / 16 per (key, KV head).  At
// 6.8 TB/s that is 23 bytes, 41 values, per clock and SM, so the arithmetic
// between HBM and the tensor cores decides: a value costs half a conversion
// (e2m1x2 -> f16x2, measured 64 lanes a clock and SM), half a product with its
// scale (64 a clock) and its share of an MMA.  Staging dequantised tiles in
// shared memory for tcgen05 would write and read 2 bytes per value more, 164
// bytes a clock and SM where shared memory gives 128; so the codes go from
// shared memory straight into the registers that are the operand fragments
// of mma.sync (measured 1024 multiply-adds a clock and SM; 330 needed with up
// to 4 rows, 490 with up to 8), and the cache's layout is the one in which
// each lane's fragments are contiguous:
//
//   S^T [16 keys x 8 rows] = K (A, from codes) Q^T (B, registers)
//   O^T [16 dims x 8 rows] += V^T (A, from codes) P^T (B: S^T after the
//   exponential, turned by movmatrix)
//
// Codes times scales are exact in fp16 (2 + 4 significant bits, 2^-10 to
// 2688).  q becomes fp16 after a power of two per row, which brings the row's
// largest magnitude to the top of fp16's range, [2^15, 2^16): exact down to
// 2^-32 of that.  P is the sum of two fp16 numbers, hi and 2^-11 lo (kHead,
// below): with up to 4 rows the two fill the 8 columns of one MMA, with up to
// 8 they take two.
//
// Each warp streams tiles of 4608 bytes through a ring of its own with
// cp.async.bulk (no block-wide step in the loop), keeps its own maximum, sum
// and O^T, and raises the maximum only when a score exceeds it by 2^3, so
// that the rescaling and its shuffles are rare.  The work of all sequences is
// one list, cut evenly over the blocks (two an SM, 128 registers a thread)
// from the lengths on the device; an item that lies in several blocks is
// joined by a second kernel.
//
// Measured (device time): 8 sequences of 32768 keys, 32 x 8 heads, D = 128, 4
// rows, 59 us, 75 % of the copy bandwidth; of 131072 keys 196 us, 91 %: about
// 14 us go into finding the share, the first copies, the last warps and the
// join.  8 rows take 68 us, 16 rows 118, more go in chunks of 16.  What the
// tile loop has in registers decides (spilled at D = 128: 38 bytes with up to
// 4 rows, 70 with up to 8, 376 with more; at D = 64: 0, 18, 18): 90 bytes in
// place of 38 took 10 % more at 131072 keys, 12 warps of 168 registers in
// place of 16 took 66 us in place of 62 at 32768.
#include <cfloat>
#include <climits>
#include <cmath>
#include <utility>

#include "kv4_common.cuh"

namespace fa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// What beginning and joining an item costs a block, in tiles (the lists of
// short sequences took 107 us where items counted only by their tiles), and
// what beginning a group of items of one warp each does.  From a sweep with up
// to 4 rows and D = 128; with more rows a tile costs up to twice as much and
// the same weights serve.
constexpr int kItemCost = 24, kSoloCost = 16;
// P is held as two fp16 numbers, hi = fp16(p) and lo = fp16(2^11 (p - hi)): to
// 22 bits, or to 2^-36.  p is 2^kHead where a score equals the maximum, which
// is raised when a score exceeds it by 2^kRaise.  A key so has its 22 bits
// where it weighs 2^-19 of the heaviest that its warp has seen, and is lost
// below 2^-41 of that.  p stays below 2^8 where fp16 ends at 2^16: the rest is
// for scores so large that their own ulp is up to 8.
constexpr float kHead = 5.f, kRaise = 3.f;
constexpr float kLoUp = 2048.f, kLoDown = 1.f / kLoUp;

// Keys of a warp's tile: 4608 bytes.
__host__ __device__ constexpr int tile_keys(int D) { return D == 128 ? 32 : 64; }

// MODE 0: up to 4 rows; 1: up to 8; 2: up to 16 (more rows: several items).
template <int D, int MODE>
struct Cfg {
    static constexpr int UNIT = 18 * D;
    static constexpr int NU = tile_keys(D) / 16;  // units of a tile
    static constexpr int UG = MODE == 2 ? NU / 2 : NU;  // units worked on at once (registers)
    static constexpr int STAGE = NU * UNIT;
    static constexpr int STAGES = 2;  // per warp
    static constexpr int ROWS = 4 << MODE;
    static constexpr int NT = MODE == 2 ? 2 : 1;  // column tiles of 8
    static constexpr int KS = D / 16;             // MMA steps over D, and 16-row tiles of O^T
    static constexpr int OSTRIDE = D + (D == 128 ? 4 : 2);  // floats per column in the joining buffer
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int OBUF = kWarps * 8 * OSTRIDE * 4;
    static constexpr int ML = kWarps * ROWS * 8;
    static constexpr int DESC = kWarps * 32 * NU * 8;  // the copies to come
    static constexpr int BARS = RING + OBUF + ML + DESC;
    // MODE 2 keeps a warp's fragments of Q in its part of the joining buffer
    static_assert(MODE != 2 || 32 * KS * NT * 8 <= 8 * OSTRIDE * 4, "Q fragments");
    static constexpr int SMEM = BARS + kWarps * STAGES * 8 + 64;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t low_twice(uint32_t a)
{
    uint32_t r;
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %1; mov.b32 %0, {x, x};}" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t high_twice(uint32_t a)
{
    uint32_t r;
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %1; mov.b32 %0, {y, y};}" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint16_t lds_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ void prefetch_l2(const char* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Codes 2 i, 2 i + 1 (in bytes) of a lane's run as fp16 pairs.
template <int I>
__device__ __forceinline__ uint32_t code_pair(const uint32_t* w)
{
    return e2m1x2_to_f16x2<(I & 3)>(w[I >> 2]);
}

// step(0), step(1), ... with the index as a constant.
template <typename F, int... I>
__device__ __forceinline__ void for_steps(F& step, std::integer_sequence<int, I...>)
{
    (step(std::integral_constant<int, I>{}), ...);
}

// NaN halves of a pair of scales (bit 0: low, bit 1: high).
__device__ __forceinline__ uint32_t nan_halves(uint32_t s)
{
    return ((s & 0x7fffu) > 0x7c00u ? 1u : 0u) | ((s >> 16 & 0x7fffu) > 0x7c00u ? 2u : 0u);
}

template <int D>
__device__ __forceinline__ int tiles_of(int len)
{
    return len > 0 ? (len + tile_keys(D) - 1) / tile_keys(D) : 1;
}

// The item that begins in a block and ends in a later one: its end in the
// list of work and the blocks' share of that; item -1: none.
struct Cut {
    int b, item;
    long long end, share;
};

__device__ __forceinline__ uint32_t without_nan(uint32_t s)
{
    const uint32_t n = nan_halves(s);
    return (n & 1 ? 0u : s & 0xffffu) | (n & 2 ? 0u : s & 0xffff0000u);
}

struct List {
    long long last, share;  // end of the block's share, and its length
};

// Where the kernels keep what they share in the workspace.
struct Parts {
    float* o;   // [blocks][2][ROWS][D]
    float2* ml; // [blocks][2][ROWS]: maximum (log2 units) and sum
    Cut* join;  // [blocks]
};

template <int D, int MODE>
__host__ __device__ inline Parts parts_of(float* ws, int blocks)
{
    constexpr int ROWS = Cfg<D, MODE>::ROWS;
    Parts p;
    p.join = reinterpret_cast<Cut*>(ws);
    p.ml = reinterpret_cast<float2*>(p.join + blocks);
    p.o = reinterpret_cast<float*>(p.ml + (size_t)blocks * 2 * ROWS);
    return p;
}

// The list of work.  Every sequence has `items` (KV head and chunk of rows).
// Those of a long sequence are entries of the list one by one, kItemCost +
// tiles long, and may be cut between blocks; the block's warps share an
// entry's tiles.  Those of a short sequence come in groups of one item per
// warp, which need no joining: 8 x tiles + kSoloCost long and never cut (they
// are the block's in which their last unit lies).  A sequence is short when a
// group of it has at most 5/4 of the tiles that a block has on average (more
// would leave other blocks waiting), or two tiles an item.
struct Seg {  // a block's part of an entry
    int b, e;         // sequence, entry
    int t, n;         // tiles t .. t + n - 1 (of each item, in a group)
    int left;         // of the block's share, from tile t on
    int len, nt, entries;
    bool solo;        // a group
    const int* row;   // of the table
};

struct Split {
    int items, limit;  // limit: most tiles of a group

    __device__ __forceinline__ bool solo(int nt) const { return items >= kWarps / 2 && kWarps * nt <= limit; }
    __device__ __forceinline__ int entries(bool solo) const { return solo ? (items + kWarps - 1) / kWarps : items; }
    // units in front of the part that may be cut
    __device__ __forceinline__ int ahead(bool solo, int nt) const { return solo ? kWarps * nt + kSoloCost - 1 : kItemCost; }
    __device__ __forceinline__ int body(bool solo, int nt) const { return solo ? 1 : nt; }
    __device__ __forceinline__ long long cost(int nt) const
    {
        const bool one = solo(nt);
        return (long long)(ahead(one, nt) + body(one, nt)) * entries(one);
    }
};

template <int D>
__device__ __forceinline__ void seg_open(const Kv4AttnParams& p, const Split& sp, Seg& s)
{
    int slot;
    s.len = kv4_sequence(p.c, s.b, slot);
    s.row = p.c.table + (long long)slot * p.c.table_width;
    s.nt = tiles_of<D>(s.len);
    s.solo = sp.solo(s.nt);
    s.entries = sp.entries(s.solo);
}

// The block's part of the next entry; false at the end of its share.
template <int D>
__device__ __forceinline__ bool seg_next(const Kv4AttnParams& p, const Split& sp, Seg& s)
{
    s.left -= s.solo ? 1 : s.n;
    if (s.left <= 0) return false;
    if (++s.e == s.entries) {
        s.e = 0;
        ++s.b;
        seg_open<D>(p, sp, s);
    }
    s.left -= sp.ahead(s.solo, s.nt);
    s.t = 0;
    s.n = s.solo ? s.nt : min(s.left, s.nt);
    return s.left > 0;
}

// KV head and chunk of rows of an item (chunk * Hkv + head; few chunks).
__device__ __forceinline__ int2 head_and_chunk(int item, int Hkv)
{
    int chunk = 0;
#pragma unroll 1
    for (; item >= Hkv; item -= Hkv) ++chunk;
    return make_int2(item, chunk);
}

// Tiles of warp w in it, and its item.
__device__ __forceinline__ int seg_item(const Seg& s, int w) { return s.solo ? kWarps * s.e + w : s.e; }
__device__ __forceinline__ int seg_tiles(const Split& sp, const Seg& s, int w)
{
    if (s.len == 0) return 0;
    return s.solo ? (seg_item(s, w) < sp.items ? s.n : 0) : max(0, (s.n - w + kWarps - 1) / kWarps);
}
__device__ __forceinline__ int seg_tile(const Seg& s, int w, int k) { return s.solo ? k : s.t + w + kWarps * k; }

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 2) fa_kv4_attn_kernel(const Kv4AttnParams p, const int chunks)
{
    using C = Cfg<D, MODE>;
    constexpr int NT = C::NT, KS = C::KS, NU = C::NU, UG = C::UG, TILE = tile_keys(D);
    extern __shared__ __align__(128) uint8_t smem[];
    // a warp's part in hand and the part of its next copies: looked at once in
    // a while, and not to take registers from the tiles
    __shared__ Seg s_now[kWarps], s_ld[kWarps];
    __shared__ int s_ld_k[kWarps];
    __shared__ List s_list;
    __shared__ long long s_sum[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t base = smem_u32(smem);
    const uint32_t ring = base + warp * (C::STAGES * C::STAGE);
    const uint32_t bars = base + C::BARS + warp * (C::STAGES * 8);
    float* obuf = reinterpret_cast<float*>(smem + C::RING);
    float2* mlbuf = reinterpret_cast<float2*>(smem + C::RING + C::OBUF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::BARS + kWarps * C::STAGES * 8);
    const WaitFailure wf{p.c.err, p.c.diag};
    Split sp{p.c.Hkv * chunks, 0};

    let_dependents_launch();
    if (lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) mbar_init(bars + 8 * s, 1);
        mbar_init_fence();
    }
    if (tid == 0) *abort_flag = 0;
    {
        // Q and (where the call names no slots) the table into L2 while the
        // lengths are on their way, a line per thread of the grid
        const long long line = ((long long)blockIdx.x * kThreads + tid) * 128;
        const long long q_bytes = (long long)p.B * p.Hq * p.Lq * D * 2;
        const long long t_bytes = p.c.ids ? 0 : (long long)p.B * p.c.table_width * 4;
        if (line < t_bytes)
            prefetch_l2(reinterpret_cast<const char*>(p.c.table) + line);
        else if (line - t_bytes < q_bytes)
            prefetch_l2(reinterpret_cast<const char*>(p.q) + (line - t_bytes));
    }

    // This block's share of the list, from the lengths: thread i (lane i where
    // there are no more than 32 sequences: then every warp finds the share for
    // itself) sums a run of sequences.  First the tiles alone, only for the
    // limit of a group, then the list's units, whose prefix sums say in which
    // run the share begins.
    const bool few = p.B <= 32;
    const int run = (p.B + kThreads - 1) / kThreads, me = few ? lane : tid;
    const int run0 = min(p.B, me * run), run1 = min(p.B, run0 + run);
    auto tiles = [&](int b) {
        int slot;
        return tiles_of<D>(kv4_sequence(p.c, b, slot));
    };
    const int nt0 = run0 < run1 ? tiles(run0) : 0;  // of the run's first; most have no other
    float all = (float)nt0;
#pragma unroll 1
    for (int b = run0 + 1; b < run1; ++b) all += (float)tiles(b);
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
    if (!few) {
        if (lane == 0) s_sum[warp] = __float_as_int(all);
        __syncthreads();
        all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += __int_as_float((int)s_sum[w]);
        __syncthreads();
    }
    const float per_block = 1.f / gridDim.x;
    sp.limit = (int)fminf(fmaxf(1.25f * per_block * all * (float)sp.items, 2.f * kWarps), 1e9f);
    long long mine = run0 < run1 ? sp.cost(nt0) : 0;
#pragma unroll 1
    for (int b = run0 + 1; b < run1; ++b) mine += sp.cost(tiles(b));
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += y;
    }
    long long total = __shfl_sync(~0u, upto, 31);
    if (!few) {
        if (lane == 0) s_sum[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) upto += total;
            total += s_sum[w];
        }
    }
    // ceil(total / blocks), or a little above
    long long share = (long long)((float)total * per_block * 1.000002f + 0.999f);
    share += share * gridDim.x < total;
    share = max(share, (long long)kWarps);
    const long long first = share * blockIdx.x, last = min(total, first + share);
    if (tid == 0) parts_of<D, MODE>(p.part, gridDim.x).join[blockIdx.x].item = -1;
    if (first >= last) return;
    if (first < upto && first >= upto - mine) {
        long long at = upto - mine;
        Seg s;
        s.b = run0;
#pragma unroll 1
        for (long long x; at + (x = sp.cost(s.b == run0 ? nt0 : tiles(s.b))) <= first; ++s.b) at += x;
        seg_open<D>(p, sp, s);
        const int ahead = sp.ahead(s.solo, s.nt), one = ahead + sp.body(s.solo, s.nt);
#pragma unroll 1
        for (s.e = 0; at + one <= first; at += one) ++s.e;
        s.left = (int)(last - first);
        s.t = (int)(first - at) - ahead;
        if (s.t < 0) {
            s.left += s.t;
            s.t = 0;
        }
        s.n = s.solo ? s.nt : min(s.left, s.nt - s.t);
        for (int w = 0; w < kWarps; ++w)
            if (!few || w == warp) {
                s_now[w] = s_ld[w] = s;
                s_ld_k[w] = 0;
            }
        if (!few || warp == 0) s_list = List{last, share};
    }
    __syncthreads();  // and the abort flag's initial value
    if (s_now[warp].left <= 0) return;

    // Raw Q of a part: lane (g, t4) holds dimensions t4 D/4 ... of rows g, 8 + g
    // of the warp's item.  Those of the block's first part are asked for before
    // its tiles, whose loads fill the memory's queues for microseconds.
    uint32_t qraw[NT][KS * 2];
    auto load_q = [&](const Seg& x) {
        const int item = min(seg_item(x, warp), sp.items - 1);  // a group's last warps may have none
        const int2 hc = head_and_chunk(item, p.c.Hkv);
        const int r0 = hc.y * C::ROWS;
        const long long row0 = ((long long)x.b * p.Hq + (long long)hc.x * p.group) * p.Lq + r0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = 8 * nt + g, r = MODE == 0 ? (col & 3) : col;
            const bool on = r0 + r < p.R;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (row0 + r) * D + t4 * (D / 4));
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                const uint4 v = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                qraw[nt][4 * i] = v.x, qraw[nt][4 * i + 1] = v.y, qraw[nt][4 * i + 2] = v.z, qraw[nt][4 * i + 3] = v.w;
            }
        }
    };
    load_q(s_now[warp]);

    // ---- the warp's loads, running ahead of its tiles: lane i holds where the
    // warp's i-th tile from (s_ld, s_ld_k) on; -1: none lies and copies it when its turn comes
    // sources of the lane's tile, one per page it lies in; the first with the
    // number of its units in the low bits
    uint64_t* desc = reinterpret_cast<uint64_t*>(smem + C::RING + C::OBUF + C::ML) + (warp * 32 + lane) * NU;
    uint32_t turn = 0;  // lanes that have a tile to copy
    auto refill = [&]() {
        Seg w = s_ld[warp];
        int k = s_ld_k[warp] + lane;
        bool ok = true;
#pragma unroll 1
        for (int c; ok && k >= (c = seg_tiles(sp, w, warp));) {
            k -= c;
            ok = seg_next<D>(p, sp, w);
        }
        if (ok) {
            const int shift = p.c.page_shift, units = 1 << (shift - 4);
            const int key0 = seg_tile(w, warp, k) * TILE, n = min(NU, (w.len - key0 + 15) >> 4);
            const uint32_t head_bytes = (uint32_t)units * C::UNIT;
            const uint8_t* src = p.c.pool + (long long)head_and_chunk(seg_item(w, warp), p.c.Hkv).x * head_bytes +
                                 ((key0 >> 4) & (units - 1)) * C::UNIT;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (i * units >= n) break;
                int page = w.row[(key0 >> shift) + i];
                if ((unsigned)page >= (unsigned)p.c.num_pages) {
                    atomicOr(p.c.err, 2);
                    page = 0;
                }
                const uint64_t from = reinterpret_cast<uint64_t>(src + page * ((long long)p.c.Hkv * head_bytes));
                desc[i] = i == 0 ? from + n : from;
            }
        }
        turn = __ballot_sync(~0u, ok);
        __syncwarp();
        if (lane == 31) {  // the next batch begins behind this tile, if there is one
            s_ld[warp] = w;
            s_ld_k[warp] = ok ? k + 1 : -1;
        }
        __syncwarp();
    };
    int issued = 0;
    auto issue = [&]() {
        if (turn == 0) {
            if (s_ld_k[warp] < 0) return false;
            refill();
            if (turn == 0) return false;
        }
        if (lane == __ffs(turn) - 1 && !(p.fault == 1 && issued == 0)) {
            const int st = issued % C::STAGES;
            const uint32_t dst = ring + st * C::STAGE, bar = bars + 8 * st;
            const uint64_t from = desc[0];
            const int n = (int)(from & 15), per = 1 << (p.c.page_shift - 4);
            mbar_arrive_expect_tx(bar, n * C::UNIT);
            bulk_load(dst, from & ~15ull, min(per, n) * C::UNIT, bar);
#pragma unroll
            for (int i = 1; i < NU; ++i)  // pages shorter than the tile
                if (i * per < n) bulk_load(dst + i * per * C::UNIT, desc[i], min(per, n - i * per) * C::UNIT, bar);
        }
        turn &= turn - 1;
        ++issued;
        return true;
    };
    int used = 0;      // stages consumed
    auto leave = [&]() {  // waits ran out: let the copies in flight land
        for (; used < issued; ++used)
            if (!(p.fault == 1 && used == 0))
                mbar_settle(bars + 8 * (used % C::STAGES), (used / C::STAGES) & 1, wf, 51);
    };
    uint32_t qf[MODE == 2 ? 1 : NT * KS * 2];  // fragments of Q
    float sc[NT][2];
    float m[NT][2], l[NT][2], acc[NT][KS][4];
    const uint32_t qbuf = base + C::RING + warp * (8 * C::OSTRIDE * 4);
    bool failed = false;
    // One loop over the beginning of each part, the warp's tiles in it and its
    // end, so that the code of the copies, which is long, exists once.
    int len = 0;
    int key = 0, key_step = 0;  // first key of the warp's next tile, and from one to the next
    for (int count = -1;;) {    // count: tiles left
        while (issued < used + C::STAGES && issue()) {}
        if (count < 0) {
            const Seg& seg = s_now[warp];
            len = seg.len;
            key = seg_tile(seg, warp, 0) * TILE;
            key_step = seg.solo ? TILE : kWarps * TILE;
            count = failed ? 0 : seg_tiles(sp, seg, warp);
            const int2 hc = head_and_chunk(min(seg_item(seg, warp), sp.items - 1), p.c.Hkv);
            const int h = hc.x, r0 = hc.y * C::ROWS;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t(&x)[KS * 2] = qraw[nt];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < KS * 2; ++i) top = __vmaxu2(top, x[i] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                // power of two of the row: its largest magnitude comes to [2^15, 2^16),
                // or as near as a normal power of two brings it
                const int e = top >= 0x7f80u || top == 0 ? 0 : max((int)(top >> 7) - (127 + 15), -126);
                const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < KS * 2; ++i) {
                    const uint32_t f = f16x2(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xffff0000u) * down);
                    if constexpr (MODE == 2)
                        x[i] = f;
                    else
                        qf[nt * KS * 2 + i] = f;
                }
                if constexpr (MODE == 2) {  // each lane reads back what it wrote
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qbuf + ((nt * KS + i) * 32 + lane) * 8),
                                     "r"(x[2 * i]), "r"(x[2 * i + 1])
                                     : "memory");
                }
                const float s = p.scale * 1.4426950408889634f * (p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // kept off 0 and infinity, whose product with a masked score
                    // (-infinity) or a score of 0 would be NaN
                    sc[nt][c] = fminf(fmaxf(s * __shfl_sync(~0u, up, (2 * t4 + c) * 4), FLT_MIN), FLT_MAX);
                    m[nt][c] = -FLT_MAX;
                    l[nt][c] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[nt][i][c] = 0.f;
            }
        }
        if (count > 0) {
            const uint32_t st = used % C::STAGES, stage = ring + st * C::STAGE;
            // each lane polls for itself: the warp goes one way, together, whatever its lanes saw
            const bool ok = mbar_wait(bars + 8 * st, (used / C::STAGES) & 1, abort_flag, wf, 50, used);
            if (!__all_sync(~0u, ok)) {
                failed = true;
                count = 0;
                continue;
            }
#pragma unroll 1
            for (int v0 = 0; v0 < NU; v0 += UG) {
                if (UG < NU && v0 > 0 && key + 16 * v0 >= len) break;
                const int key0 = key + 16 * v0;
                const uint32_t tile = stage + v0 * C::UNIT;
                const int all_see = p.causal ? len - p.Lq + 1 : len;  // keys every row may see
                const bool border = key0 + 16 * UG > all_see;          // behind them scores are masked one by one

                // ---- S^T = K Q^T.  Units behind the sequence's end hold old
                // bytes: their scores are masked, their V scales zeroed.
                float s[UG][NT][4];
#pragma unroll
                for (int u = 0; u < UG; ++u) {
                    const uint32_t unit = tile + u * C::UNIT;
                    uint32_t ka[KS / 2], kb[KS / 2], sa[KS / 4], sb[KS / 4];
                    if constexpr (D == 128) {
                        const uint4 a = lds16(unit + g * 64 + t4 * 16), b = lds16(unit + (g + 8) * 64 + t4 * 16);
                        ka[0] = a.x, ka[1] = a.y, ka[2] = a.z, ka[3] = a.w;
                        kb[0] = b.x, kb[1] = b.y, kb[2] = b.z, kb[3] = b.w;
                        const uint32_t x = e4m3x2_to_f16x2(lds_u16(unit + 16 * D + g * 8 + t4 * 2));
                        const uint32_t y = e4m3x2_to_f16x2(lds_u16(unit + 16 * D + (g + 8) * 8 + t4 * 2));
                        sa[0] = low_twice(x), sa[1] = high_twice(x);
                        sb[0] = low_twice(y), sb[1] = high_twice(y);
                    } else {
                        const uint2 a = lds8(unit + g * 32 + t4 * 8), b = lds8(unit + (g + 8) * 32 + t4 * 8);
                        ka[0] = a.x, ka[1] = a.y;
                        kb[0] = b.x, kb[1] = b.y;
                        const uint32_t x = lds_u8(unit + 16 * D + g * 4 + t4), y = lds_u8(unit + 16 * D + (g + 8) * 4 + t4);
                        sa[0] = low_twice(e4m3x2_to_f16x2((uint16_t)x));
                        sb[0] = low_twice(e4m3x2_to_f16x2((uint16_t)y));
                    }
                    auto step = [&](auto jj) {
                        constexpr int j = decltype(jj)::value;
                        const uint32_t a0 = hmul2(code_pair<2 * j>(ka), sa[j / 4]);
                        const uint32_t a1 = hmul2(code_pair<2 * j>(kb), sb[j / 4]);
                        const uint32_t a2 = hmul2(code_pair<2 * j + 1>(ka), sa[j / 4]);
                        const uint32_t a3 = hmul2(code_pair<2 * j + 1>(kb), sb[j / 4]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint2 b;
                            if constexpr (MODE == 2)
                                b = lds8(qbuf + ((nt * KS + j) * 32 + lane) * 8);
                            else
                                b = make_uint2(qf[2 * j], qf[2 * j + 1]);
                            if constexpr (j == 0)
                                mma_f16_first(s[u][nt], a0, a1, a2, a3, b.x, b.y);
                            else
                                mma_f16(s[u][nt], a0, a1, a2, a3, b.x, b.y);
                        }
                    };
                    for_steps(step, std::make_integer_sequence<int, KS>{});
                }
                // V's scales, with what a border tile must not use taken out
                const int grp = D == 128 ? g : g >> 1;
                uint32_t va_s[UG], vb_s[UG];
#pragma unroll
                for (int u = 0; u < UG; ++u) {
                    const uint32_t at = tile + u * C::UNIT + 17 * D + grp * 16 + 2 * t4;
                    va_s[u] = e4m3x2_to_f16x2(lds_u16(at));
                    vb_s[u] = e4m3x2_to_f16x2(lds_u16(at + 8));
                }
                // ---- masks, the running maximum less kHead, in log2 units
                if (border) {
                    int lim[NT][2];  // keys that the columns' rows see
                    const int r0 = head_and_chunk(min(seg_item(s_now[warp], warp), sp.items - 1), p.c.Hkv).y * C::ROWS;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int col = 8 * nt + 2 * t4 + c, r = r0 + (MODE == 0 ? (col & 3) : col);
                            lim[nt][c] = p.causal && p.Lq > 1 ? r % p.Lq + all_see : len;
                        }
#pragma unroll
                    for (int u = 0; u < UG; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (key0 + 16 * u + g + 8 * (c >> 1) >= lim[nt][c & 1]) s[u][nt][c] = -INFINITY;
#pragma unroll
                    for (int u = 0; u < UG; ++u) {
                        // positions behind the end: whatever their scales hold becomes 0
                        const int k = key0 + 16 * u + 2 * t4;
                        uint32_t &x = va_s[u], &y = vb_s[u];
                        if (k >= len) x = 0;
                        if (k + 1 >= len) x &= 0xffffu;
                        if (k + 8 >= len) y = 0;
                        if (k + 9 >= len) y &= 0xffffu;
                    }
                    // A NaN scale reaches only the rows that see its key: it is
                    // taken out of the product and put into their sums.
                    uint32_t nans = 0;
#pragma unroll
                    for (int u = 0; u < UG; ++u) nans |= nan_halves(va_s[u]) | nan_halves(vb_s[u]);
                    if (__any_sync(~0u, nans)) {
                        bool hit[NT][2] = {};
#pragma unroll
                        for (int u = 0; u < UG; ++u) {
                            va_s[u] = without_nan(va_s[u]);
                            vb_s[u] = without_nan(vb_s[u]);
#pragma unroll 1
                            for (int j = 0; j < 16; ++j) {
                                if ((lds_u8(tile + u * C::UNIT + 17 * D + grp * 16 + j) & 0x7f) != 0x7f) continue;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int c = 0; c < 2; ++c) hit[nt][c] |= key0 + 16 * u + j < min(lim[nt][c], len);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < KS; ++i)
                                    if (hit[nt][c]) acc[nt][i][c] = acc[nt][i][c + 2] = NAN;
                    }
                }
                bool raise = false;
                float mx[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
                        for (int u = 1; u < UG; ++u) x = fmaxf(x, fmaxf(s[u][nt][c], s[u][nt][c + 2]));
                        mx[nt][c] = x * sc[nt][c];
                        raise |= mx[nt][c] > m[nt][c] + (kHead + kRaise);
                    }
                if (__any_sync(~0u, raise)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = mx[nt][c];
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                            x = fmaxf(x - kHead, m[nt][c]);
                            const float a = x == m[nt][c] ? 1.f : ex2_approx(m[nt][c] - x);
                            m[nt][c] = x;
                            l[nt][c] *= a;
#pragma unroll
                            for (int i = 0; i < KS; ++i) {
                                acc[nt][i][c] *= a;
                                acc[nt][i][c + 2] *= a;
                            }
                        }
                }
                // ---- P^T as two fp16 numbers, turned into B fragments
                uint32_t pb[UG][NT][MODE == 0 ? 1 : 2][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint64_t sc2 = f2_pack(sc[nt][0], sc[nt][1]), m2 = f2_pack(-m[nt][0], -m[nt][1]);
                    uint64_t l2 = f2_pack(l[nt][0], l[nt][1]);
#pragma unroll
                    for (int u = 0; u < UG; ++u)
#pragma unroll
                        for (int k8 = 0; k8 < 2; ++k8) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(s[u][nt][2 * k8], s[u][nt][2 * k8 + 1]), sc2, m2), x0, x1);
                            const uint64_t p2 = f2_pack(x0 = ex2_approx(x0), x1 = ex2_approx(x1));
                            l2 = f2_add(l2, p2);
                            const uint32_t hi = f16x2(x0, x1);
                            const float2 f = f16x2_to_f32(hi);
                            if constexpr (MODE == 0) {
                                // lanes of columns 0 .. 3 keep p, which rounds to hi; those of 4 .. 7 take lo
                                const float take = t4 < 2 ? 0.f : -1.f, up = t4 < 2 ? 1.f : kLoUp;
                                const uint64_t y2 = f2_fma(f2_pack(f.x, f.y), f2_pack(take, take), p2);
                                f2_unpack(f2_mul(y2, f2_pack(up, up)), x0, x1);
                                pb[u][nt][0][k8] = transpose8x8(f16x2(x0, x1));
                            } else {
                                const uint64_t y2 = f2_fma(f2_pack(f.x, f.y), f2_pack(-1.f, -1.f), p2);
                                f2_unpack(f2_mul(y2, f2_pack(kLoUp, kLoUp)), x0, x1);
                                pb[u][nt][0][k8] = transpose8x8(hi);
                                pb[u][nt][1][k8] = transpose8x8(f16x2(x0, x1));
                            }
                        }
                    f2_unpack(l2, l[nt][0], l[nt][1]);
                }
                // ---- O^T += V^T P^T.  The MMA adds to its accumulator without
                // rounding to nearest, a bias that grows with the number of
                // additions (9e-7 of O after 54 of them, 3e-7 so), so each
                // group starts from 0 and is added here.
                uint32_t va[UG][KS / 2], vb[UG][KS / 2];
#pragma unroll
                for (int u = 0; u < UG; ++u) {
                    const uint32_t unit = tile + u * C::UNIT;
                    if constexpr (D == 128) {
                        const uint4 a = lds16(unit + 8 * D + g * 64 + t4 * 16), b = lds16(unit + 12 * D + g * 64 + t4 * 16);
                        va[u][0] = a.x, va[u][1] = a.y, va[u][2] = a.z, va[u][3] = a.w;
                        vb[u][0] = b.x, vb[u][1] = b.y, vb[u][2] = b.z, vb[u][3] = b.w;
                    } else {
                        const uint32_t at = unit + 8 * D + grp * 64 + t4 * 16 + (g & 1) * 8;
                        const uint2 a = lds8(at), b = lds8(at + 4 * D);
                        va[u][0] = a.x, va[u][1] = a.y;
                        vb[u][0] = b.x, vb[u][1] = b.y;
                    }
                }
                auto step = [&](auto ii) {
                    constexpr int i = decltype(ii)::value;
                    // lo's share comes down by 2^-11: with up to 8 rows from an
                    // accumulator of its own, with more, where registers are
                    // short, before hi's is added to the same one (8 rows at 8 x
                    // 32768 keys, D = 128: 66.3 us against 70.7; 16 rows of 6
                    // sequences of 900 .. 9001, D = 64: 15.1 against 14.8)
                    float part[NT][4], low[4];
                    if constexpr (MODE == 2) {
                        const uint64_t down = f2_pack(kLoDown, kLoDown);
                        uint32_t a[UG][4];
#pragma unroll
                        for (int u = 0; u < UG; ++u) {
                            a[u][0] = hmul2(code_pair<2 * i>(va[u]), va_s[u]);
                            a[u][1] = hmul2(code_pair<2 * i + 1>(va[u]), va_s[u]);
                            a[u][2] = hmul2(code_pair<2 * i>(vb[u]), vb_s[u]);
                            a[u][3] = hmul2(code_pair<2 * i + 1>(vb[u]), vb_s[u]);
                        }
#pragma unroll
                        for (int half = 1; half >= 0; --half)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                                for (int u = 0; u < UG; ++u) {
                                    const uint32_t(&b)[2] = pb[u][nt][half];
                                    if (half == 1 && u == 0)
                                        mma_f16_first(part[nt], a[u][0], a[u][1], a[u][2], a[u][3], b[0], b[1]);
                                    else
                                        mma_f16(part[nt], a[u][0], a[u][1], a[u][2], a[u][3], b[0], b[1]);
                                }
                                if (half == 0) continue;
                                f2_unpack(f2_mul(f2_pack(part[nt][0], part[nt][1]), down), part[nt][0], part[nt][1]);
                                f2_unpack(f2_mul(f2_pack(part[nt][2], part[nt][3]), down), part[nt][2], part[nt][3]);
                            }
                    } else {
#pragma unroll
                        for (int u = 0; u < UG; ++u) {
                            const uint32_t sa = va_s[u], sb = vb_s[u];
                            const uint32_t a0 = hmul2(code_pair<2 * i>(va[u]), sa), a1 = hmul2(code_pair<2 * i + 1>(va[u]), sa);
                            const uint32_t a2 = hmul2(code_pair<2 * i>(vb[u]), sb), a3 = hmul2(code_pair<2 * i + 1>(vb[u]), sb);
                            if (u == 0)
                                mma_f16_first(part[0], a0, a1, a2, a3, pb[u][0][0][0], pb[u][0][0][1]);
                            else
                                mma_f16(part[0], a0, a1, a2, a3, pb[u][0][0][0], pb[u][0][0][1]);
                            if constexpr (MODE == 1) {
                                if (u == 0)
                                    mma_f16_first(low, a0, a1, a2, a3, pb[u][0][1][0], pb[u][0][1][1]);
                                else
                                    mma_f16(low, a0, a1, a2, a3, pb[u][0][1][0], pb[u][0][1][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float(&o)[4] = acc[nt][i];
                        if constexpr (MODE == 1) {
                            const uint64_t down = f2_pack(kLoDown, kLoDown);
                            f2_unpack(f2_fma(f2_pack(low[0], low[1]), down, f2_pack(o[0], o[1])), o[0], o[1]);
                            f2_unpack(f2_fma(f2_pack(low[2], low[3]), down, f2_pack(o[2], o[3])), o[2], o[3]);
                        }
                        f2_unpack(f2_add(f2_pack(o[0], o[1]), f2_pack(part[nt][0], part[nt][1])), o[0], o[1]);
                        f2_unpack(f2_add(f2_pack(o[2], o[3]), f2_pack(part[nt][2], part[nt][3])), o[2], o[3]);
                    }
                };
                for_steps(step, std::make_integer_sequence<int, KS>{});
            }
            __syncwarp();  // the stage has been read
            ++used;
            --count;
            key += key_step;
            continue;
        }
        Seg seg = s_now[warp];
        const int item = min(seg_item(seg, warp), sp.items - 1);  // a group's last warps may have none
        const int2 hc = head_and_chunk(item, p.c.Hkv);
        const int h = hc.x, r0 = hc.y * C::ROWS, nrows = min(C::ROWS, p.R - r0);
        const long long row0 = ((long long)seg.b * p.Hq + (long long)h * p.group) * p.Lq + r0;
        const float gv = p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.f;
        if (seg.solo) {  // ---- the warp's own item: straight to the output
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = l[nt][c];
                    x += __shfl_xor_sync(~0u, x, 4);
                    x += __shfl_xor_sync(~0u, x, 8);
                    x += __shfl_xor_sync(~0u, x, 16);
                    const int r = 8 * nt + 2 * t4 + c;
                    const bool on = r < nrows && seg_item(seg, warp) < sp.items;
                    const float inv = x == 0.f ? 0.f : __fdividef(gv, x);
                    float* dst = p.o + (row0 + r) * D + (D / 8) * g;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        float y = acc[nt][i][c], z = acc[nt][i][c + 2];
                        if constexpr (MODE == 0) {  // hi's share and lo's
                            y = fmaf(__shfl_xor_sync(~0u, y, 2), kLoDown, y);
                            z = fmaf(__shfl_xor_sync(~0u, z, 2), kLoDown, z);
                        }
                        if (on) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(y * inv, z * inv);
                    }
                    if (on && g == 0)
                        p.lse[row0 + r] = x == 0.f ? -INFINITY : (m[nt][c] + __log2f(x)) * 0.6931471805599453f;
                }
        } else {  // ---- join the warps
            const bool whole = seg.t == 0 && seg.n == seg.nt;
            const int part = (int)blockIdx.x * 2 + (seg.t == 0 ? 1 : 0);
            const Parts parts = parts_of<D, MODE>(p.part, gridDim.x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = l[nt][c];
                    x += __shfl_xor_sync(~0u, x, 4);
                    x += __shfl_xor_sync(~0u, x, 8);
                    x += __shfl_xor_sync(~0u, x, 16);
                    const int col = 8 * nt + 2 * t4 + c;
                    if (g == 0 && col < C::ROWS) mlbuf[warp * C::ROWS + col] = make_float2(m[nt][c], x);
                    // the buffer holds column `col`, dimension d at a place that
                    // spreads a store's lanes over the banks
                    float* dst = obuf + (warp * 8 + 2 * t4 + c) * C::OSTRIDE;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        const int at = D == 128 ? 16 * g + ((2 * i + 2 * g) & 15) : 8 * g + 2 * i;
                        *reinterpret_cast<float2*>(dst + at) = make_float2(acc[nt][i][c], acc[nt][i][c + 2]);
                    }
                }
                if (__syncthreads_or(failed)) {
                    leave();
                    return;
                }
                const int cols = MODE == 0 ? 4 : 8;
#pragma unroll 1
                for (int x = tid; x < cols * D; x += kThreads) {
                    const int col = x / D, d = x % D, r = 8 * nt + col;
                    if (r >= nrows) break;
                    const int at = D == 128 ? (d & ~15) | ((d + 2 * (d >> 4)) & 15) : d;
                    float mm = -FLT_MAX;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, mlbuf[w * C::ROWS + r].x);
                    float o = 0.f, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = mlbuf[w * C::ROWS + r];
                        const float a = ml.x == mm ? 1.f : ex2_approx(ml.x - mm);
                        float v = obuf[(w * 8 + col) * C::OSTRIDE + at];
                        if constexpr (MODE == 0) v = fmaf(obuf[(w * 8 + col + 4) * C::OSTRIDE + at], kLoDown, v);
                        o = fmaf(a, v, o);
                        sum = fmaf(a, ml.y, sum);
                    }
                    if (whole) {
                        p.o[(row0 + r) * D + d] = sum == 0.f ? 0.f : o * __fdividef(gv, sum);
                        if (d == 0) p.lse[row0 + r] = sum == 0.f ? -INFINITY : (mm + __log2f(sum)) * 0.6931471805599453f;
                    } else {
                        parts.o[((long long)part * C::ROWS + r) * D + d] = o;
                        if (d == 0) parts.ml[(long long)part * C::ROWS + r] = make_float2(mm, sum);
                    }
                }
                __syncthreads();
            }
            if (tid == 0 && seg.t == 0 && !whole) {
                parts.join[blockIdx.x] = Cut{seg.b, item, s_list.last - seg.left + seg.nt, s_list.share};
            }
        }
        if (!seg_next<D>(p, sp, seg)) break;
        load_q(seg);
        __syncwarp();
        if (lane == 0) s_now[warp] = seg;
        __syncwarp();
        count = -1;
    }
    if (failed) leave();
}

// Joins the parts of the item that begins in block blockIdx.x and ends in a
// later one: four rows a block, four warps a row.  A warp takes every fourth
// part, four at a time, all loads before the first use; the warps' sums are
// added in order.
constexpr int kJoinRows = 4, kJoinWarps = 4, kJoinThreads = 32 * kJoinRows * kJoinWarps;

template <int D, int MODE>
__global__ void __launch_bounds__(kJoinThreads) fa_kv4_join_kernel(const Kv4AttnParams p)
{
    constexpr int ROWS = Cfg<D, MODE>::ROWS, V = D / 32, U = 4;
    __shared__ float s_o[kJoinRows][kJoinWarps][D];
    __shared__ float2 s_ml[kJoinRows][kJoinWarps];
    const Parts parts = parts_of<D, MODE>(p.part, gridDim.x);
    wait_for_primary();
    const Cut j = parts.join[blockIdx.x];
    if (j.item < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int2 hc = head_and_chunk(j.item, p.c.Hkv);
    const int h = hc.x, first = blockIdx.y * kJoinRows;  // of the item's rows
    const int r0 = hc.y * ROWS + first, nrows = min(kJoinRows, min(ROWS - first, p.R - r0));
    if (nrows <= 0) return;
    const long long row0 = ((long long)j.b * p.Hq + (long long)h * p.group) * p.Lq + r0;
    const int n = (int)((j.end - 1) / j.share) - (int)blockIdx.x + 1;
    const int r = warp / kJoinWarps, w = warp % kJoinWarps;
    float acc[V] = {}, sum = 0.f, mm = -FLT_MAX;
    if (r < nrows) {
        for (int k0 = w; k0 < n; k0 += U * kJoinWarps) {
            float2 ml[U];
            float x[U][V];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = k0 + i * kJoinWarps;
                ml[i] = make_float2(-FLT_MAX, 0.f);
#pragma unroll
                for (int e = 0; e < V; ++e) x[i][e] = 0.f;
                if (k < n) {
                    const long long at = ((long long)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + first + r;
                    ml[i] = parts.ml[at];
#pragma unroll
                    for (int e = 0; e < V; ++e) x[i][e] = parts.o[at * D + lane + 32 * e];
                }
            }
            float top = mm;
#pragma unroll
            for (int i = 0; i < U; ++i) top = fmaxf(top, ml[i].x);
            const float down = mm == top ? 1.f : ex2_approx(mm - top);
            mm = top;
            sum *= down;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] *= down;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float a = ml[i].x == top ? 1.f : ex2_approx(ml[i].x - top);
                sum = fmaf(a, ml[i].y, sum);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(a, x[i][e], acc[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) s_o[r][w][lane + 32 * e] = acc[e];
        if (lane == 0) s_ml[r][w] = make_float2(mm, sum);
    }
    __syncthreads();
    const float gv = p.c.v_scale ? p.c.v_scale[h] : 1.f;
    for (int x = threadIdx.x; x < nrows * D; x += kJoinThreads) {
        const int rr = x / D, d = x % D;
        float top = -FLT_MAX, o = 0.f, l = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, s_ml[rr][i].x);
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
            const float2 ml = s_ml[rr][i];
            const float a = ml.x == top ? 1.f : ex2_approx(ml.x - top);
            o = fmaf(a, s_o[rr][i][d], o);
            l = fmaf(a, ml.y, l);
        }
        p.o[(row0 + rr) * D + d] = l == 0.f ? 0.f : o * __fdividef(gv, l);
        if (d == 0) p.lse[row0 + rr] = l == 0.f ? -INFINITY : (top + __log2f(l)) * 0.6931471805599453f;
    }
}

int mode_of(int R) { return R <= 4 ? 0 : R <= 8 ? 1 : 2; }

template <int D, int MODE>
cudaError_t launch(const Kv4AttnParams& p, int blocks, cudaStream_t stream)
{
    using C = Cfg<D, MODE>;
    static_assert(2 * (C::SMEM + 1024 + 1024) <= 233472, "two blocks per SM");
    const cudaError_t e = smem_limit_once<fa_kv4_attn_kernel<D, MODE>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const int chunks = (p.R + C::ROWS - 1) / C::ROWS;
    fa_kv4_attn_kernel<D, MODE><<<blocks, kThreads, C::SMEM, stream>>>(p, chunks);
    const cudaError_t f = cudaGetLastError();
    if (f != cudaSuccess) return f;
    return launch_dependent(fa_kv4_join_kernel<D, MODE>, dim3(blocks, C::ROWS / kJoinRows), kJoinThreads, stream, p);
}

int blocks_of(int num_sms) { return 2 * num_sms; }

}  // namespace

size_t kv4_attn_workspace(int D, int R, int num_sms)
{
    const size_t blocks = (size_t)blocks_of(num_sms), rows = blocks * 2 * (4u << mode_of(R));
    return blocks * sizeof(Cut) + rows * sizeof(float2) + rows * D * sizeof(float);
}

cudaError_t launch_kv4_attn(int D, const Kv4AttnParams& p, int num_sms, cudaStream_t stream, int* launches)
{
    *launches = 2;
    const int blocks = blocks_of(num_sms), mode = mode_of(p.R);
    if (D == 128)
        return mode == 0   ? launch<128, 0>(p, blocks, stream)
               : mode == 1 ? launch<128, 1>(p, blocks, stream)
                           : launch<128, 2>(p, blocks, stream);
    return mode == 0 ? launch<64, 0>(p, blocks, stream)
           : mode == 1 ? launch<64, 1>(p, blocks, stream)
                       : launch<64, 2>(p, blocks, stream);
}

}  // namespace fa
