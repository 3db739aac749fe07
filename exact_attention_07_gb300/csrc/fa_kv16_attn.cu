// Attention over the paged 16-bit cache: packed queries that are the last
// positions of their sequences, each seeing the prefix and, of the call's own
// positions, those that its bits name (drafted trees) or that do not follow it.
//
//   s_ij = scale q_i . k_j,  p_ij = 2^(s_ij log2 e - r_i),
//   O_i = sum_j p_ij v_j / sum_j p_ij,  LSE_i = ln sum_j exp(s_ij)
//
// The `group` query heads of a KV head and the call's positions make its rows,
// 128 to a tile of tcgen05.mma (M = 128).  A key costs 4 D bytes and a row
// 4 D operations on it, so up to some 280 rows per KV head HBM bounds the call,
// more (chunks of prompts) the tensor core.
//
// One persistent block per SM.  Two softmax warpgroups, "streams", each with
// its own scores (128 columns of tensor memory, P over them) and its own
// accumulator, take turns on the tensor core, so that one's exponentials
// overlap the other's products.  With up to 128 rows the streams take
// alternate tiles of 128 keys and are added at the end; with more they take
// two tiles of rows over the same keys, which are then read once for 256 rows.
//
// K and V come by TMA, one box per page and 64 dimensions, into a ring of
// tiles.  Positions behind the sequence's end, and what no row may see, can
// hold anything: scores are replaced where a key is masked, and in tiles with
// masked keys V is looked over in shared memory first: rows behind the end
// become zeros, and so do elements that are not finite, which are added to the
// rows that may see them at the end (0 * inf would be NaN in the others).
//
// The work of all sequences is one list of (sequence, KV head, tile of rows)
// items, cut evenly over the blocks from the lengths on the device; an item
// that lies in several blocks is joined by a second kernel.
#include <cuda_bf16.h>

#include <cfloat>

#include "kv16_common.cuh"

namespace fa {

namespace {

constexpr int kWarps = 12, kThreads = 32 * kWarps;  // 8 softmax warps, producer, MMA, 2 without work
constexpr int kTile = 128;     // keys of a tile, rows of a stream
constexpr int kBox = 128 * 128;  // bytes of 64 dimensions of 128 rows
constexpr float kTau = 8.f;      // the reference moves when a maximum exceeds it by 2^8
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kItemCost = 2;     // what an item costs a block beside its tiles, in tiles

constexpr int kItemBytes = 80;  // struct Item

template <int D>
struct Smem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 12;
    static constexpr int kQ = 0;  // [2] tiles
    static constexpr int kKV = 2 * kTileBytes;
    static constexpr int kStats = kKV + kStages * kTileBytes;  // float [3][128]: stream 1's r, l, l_rnd
    static constexpr int kBars = kStats + 3 * 128 * 4;
    static constexpr int bQFull = 0, bQEmpty = 1, bSFull = 2, bPFull = 4, bOFull = 6, bOEmpty = 8, bStFull = 10,
                         bStEmpty = 11, bDrain = 12, bKVFull = 13, bKVEmpty = bKVFull + kStages,
                         kNumBars = bKVEmpty + kStages;
    static constexpr int kMisc = kBars + kNumBars * 8;  // tensor memory base, abort flag, poison flag
    static constexpr int kSums = kMisc + 16;            // long long [kWarps], and the block's share
    static constexpr int kItems = kSums + (kWarps + 2) * 8;  // Item [kWarps]
    static constexpr int kBytes = kItems + kWarps * kItemBytes;
    static_assert(kBytes <= 232448, "shared memory of one block");
    static constexpr uint32_t kColS = 0, kColO = 256;  // [2] of 128 columns, [2] of D
};

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Three barrier phases tested by one thread back to back; true when all have completed.
__device__ __forceinline__ bool mbar_try_wait3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred q0, q1, q2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q0, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q1, [%3], %4;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q2, [%5], %6;\n\t"
        "and.pred q0, q0, q1;\n\t"
        "and.pred q0, q0, q2;\n\t"
        "selp.u32 %0, 1, 0, q0;\n\t}\n"
        : "=r"(ok)
        : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const WaitFailure& wf,
                                          int site, int item)
{
    const bool ok = mbar_wait(bar, parity, abort_flag, wf, site, item);
    return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ the list of work

// A sequence's items: for every KV head, blocks of up to 2 npt of its query
// tokens.  An item costs kItemCost and its tiles of keys.
struct Item {
    int s, e;        // sequence, item of it
    int t, n;        // the block's part: tiles t .. t + n - 1
    int nt;          // tiles of the item
    int blocks;      // of the sequence's query tokens
    long long left;  // of the block's share, from tile t on
    Kv16Seq q;
    int h, tok0, ntok;  // KV head, first query token, and how many
    int clear;          // keys in front of this are seen by every row
    bool pair;          // two tiles of rows
};
static_assert(sizeof(Item) == kItemBytes, "shared memory layout");

__device__ __forceinline__ Kv16Seq open_sequence(const Kv16AttnParams& p, int s)
{
    Kv16Seq q = kv16_sequence(p.c, p.cu, p.T, s);
    if (p.mask && q.n > 32 * p.mask_words) {
        atomicOr(p.c.err, 2);
        q.n = 0;
    }
    return q;
}

__device__ __forceinline__ int row_blocks(const Kv16AttnParams& p, int n) { return (n + 2 * p.npt - 1) / (2 * p.npt); }

// Tiles of keys that block rb of a sequence's query tokens reads.
__device__ __forceinline__ int tiles_of(const Kv16AttnParams& p, const Kv16Seq& q, int rb)
{
    const int keys = p.causal ? q.len - q.n + min(q.n, (rb + 1) * 2 * p.npt) : q.len;
    return (keys + kTile - 1) / kTile;
}

// Cost of one KV head of a sequence.
__device__ __forceinline__ long long head_cost(const Kv16AttnParams& p, const Kv16Seq& q)
{
    const int nb = row_blocks(p, q.n);
    if (!p.causal) return (long long)nb * (kItemCost + tiles_of(p, q, 0));
    long long sum = 0;
    for (int rb = 0; rb < nb; ++rb) sum += kItemCost + tiles_of(p, q, rb);
    return sum;
}

// Fills in what follows from the item: its KV head, query tokens and keys.
__device__ __forceinline__ void open_item(const Kv16AttnParams& p, Item& x)
{
    x.h = x.e / x.blocks;
    const int rb = x.e - x.h * x.blocks;
    x.nt = tiles_of(p, x.q, rb);
    x.tok0 = rb * 2 * p.npt;
    x.ntok = min(x.q.n - x.tok0, 2 * p.npt);
    x.pair = x.ntok > p.npt;
    const int prefix = x.q.len - x.q.n;
    x.clear = p.mask ? prefix : p.causal ? prefix + x.tok0 + 1 : x.q.len;
}

// The block's part of the next item; left <= 0 at the end of its share.  One
// copy of this code serves all warps: a short call's time is largely that of
// fetching code for the first time.
__device__ __forceinline__ void next_item(const Kv16AttnParams& p, Item& x)
{
    x.left -= x.n;
    if (x.left <= 0) return;
    if (++x.e == x.blocks * p.c.Hkv) {
        x.e = 0;
        do {
            if (++x.s >= p.B) {
                x.left = 0;
                return;
            }
            x.q = open_sequence(p, x.s);
            x.blocks = row_blocks(p, x.q.n);
        } while (x.blocks == 0);
    }
    open_item(p, x);
    x.left -= kItemCost;
    x.t = 0;
    x.n = (int)min(x.left, (long long)x.nt);
}

// The item that begins in a block and ends in a later one: its end in the
// list and the blocks' share of that; e -1: none.
struct Cut {
    int s, e;
    long long end, share;
};

// Where the kernels keep what they share in the workspace.
struct Parts {
    Cut* join;    // [blocks]
    float4* stat; // [blocks][2][rows]: r, l, l_rnd
    float4* o;    // [blocks][2][D / 4][rows]
};

__host__ __device__ inline Parts parts_of(float* ws, int blocks, int rows)
{
    Parts p;
    p.join = reinterpret_cast<Cut*>(ws);
    p.stat = reinterpret_cast<float4*>(p.join + ((blocks + 1) & ~1));
    p.o = p.stat + (size_t)blocks * 2 * rows;
    return p;
}

// Bits of the keys k0 .. k0 + 31 that query token i of the sequence may see.
__device__ __forceinline__ uint32_t seen_word(const Kv16AttnParams& p, const Kv16Seq& q, int i, int k0)
{
    const int prefix = q.len - q.n;
    const auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
    if (!p.mask) return below((p.causal ? prefix + min(i, q.n - 1) + 1 : q.len) - k0);
    uint32_t bits = below(prefix - k0);
    const int j0 = k0 - prefix;  // of the call's positions
    if (j0 > -32 && j0 < q.n) {
        const int* row = p.mask + (long long)(q.row0 + min(i, q.n - 1)) * p.mask_words;
        const int w = j0 >> 5;
        const uint32_t lo = w >= 0 ? (uint32_t)__ldg(row + w) : 0u;
        const uint32_t hi = w + 1 < p.mask_words ? (uint32_t)__ldg(row + w + 1) : 0u;
        bits |= __funnelshift_r(lo, hi, (uint32_t)j0 & 31u) & below(q.n - j0);
    }
    return bits;
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }

// 16 bytes of V with the elements that are not finite made 0; true if there were any.
__device__ __forceinline__ bool make_finite(uint4& x)
{
    uint32_t* w = &x.x;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = not_finite(w[i]), hi = not_finite(w[i] >> 16);
        any |= lo | hi;
        w[i] = (lo ? 0u : w[i] & 0xffffu) | (hi ? 0u : w[i] & 0xffff0000u);
    }
    return any;
}

// Adds to 32 columns of a row's sum what make_finite took out of the keys that
// the row sees, of the part's tiles with masked keys.
__device__ __noinline__ void add_poison(const Kv16AttnParams& p, const Item& x, int tok, int D, int c0,
                                        float (&o)[32])
{
    const int end = min(x.q.len, (x.t + x.n) * kTile);
    const int from = max(x.t, x.clear / kTile) * kTile;  // the tile of the first masked key
    for (int k0 = from; k0 < end; k0 += 32) {
        uint32_t bits = seen_word(p, x.q, tok, k0);
        while (bits) {
            const int k = k0 + __ffs(bits) - 1;
            bits &= bits - 1;
            if (k >= end) break;
            const long long at = kv16_row(p.c, D, x.q.pages, k);
            if (at < 0) continue;
            const uint16_t* val = p.c.pool + at + (long long)(p.c.Hkv + x.h) * kv16_head_stride(p.c, D) + c0;
            for (int i = 0; i < 32; ++i) {
                const uint32_t e = val[i];
                if (not_finite(e)) o[i] += __uint_as_float(e << 16);
            }
        }
    }
}

// ------------------------------------------------------------------ the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fa_kv16_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKV,
                        const Kv16AttnParams p)
{
    using L = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    if (sb & 1023u) {  // the operands' swizzle needs it; the window begins so where a kernel has no other shared memory
        if (threadIdx.x == 0) atomicOr(p.c.err, 4);
        return;
    }
    long long* s_sum = reinterpret_cast<long long*>(smem + L::kSums);
    long long* s_share = s_sum + kWarps;  // end of the block's share, and its length
    Item* s_item = reinterpret_cast<Item*>(smem + L::kItems);  // each warp's part in hand: not in registers
    auto bar = [&](int i) -> uint32_t { return sb + L::kBars + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    volatile int* poison = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);
    float* stats = reinterpret_cast<float*>(smem + L::kStats);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitFailure wf{p.c.err, p.c.diag};
    const Parts parts = parts_of(p.part, gridDim.x, p.rows);

    let_dependents_launch();
    if (threadIdx.x == 0) {
        mbar_init(bar(L::bQFull), 1);
        mbar_init(bar(L::bQEmpty), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::bSFull + t), 1);
            mbar_init(bar(L::bPFull + t), 128);
            mbar_init(bar(L::bOFull + t), 1);
            mbar_init(bar(L::bOEmpty + t), 128);
        }
        mbar_init(bar(L::bStFull), 128);
        mbar_init(bar(L::bStEmpty), 128);
        mbar_init(bar(L::bDrain), 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar(L::bKVFull + s), 1);
            mbar_init(bar(L::bKVEmpty + s), 1);
        }
        *abort_flag = 0;
        *poison = 0;
        mbar_init_fence();
        parts.join[blockIdx.x].e = -1;
        for (int w = 0; w < kWarps; ++w) s_item[w].left = 0;
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmKV);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }

    // This block's share of the list: every thread sums a run of sequences.
    {
        const int run = (p.B + kThreads - 1) / kThreads, run0 = min(p.B, (int)threadIdx.x * run), run1 = min(p.B, run0 + run);
        long long mine = 0;
        for (int s = run0; s < run1; ++s) mine += p.c.Hkv * head_cost(p, open_sequence(p, s));
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) upto += total;
            total += s_sum[w];
        }
        const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)kItemCost + 1);
        const long long first = share * blockIdx.x, last = min(total, first + share);
        if (first < last && first < upto && first >= upto - mine) {
            long long at = upto - mine, cost;
            Item x;
            x.s = run0;
            for (;; ++x.s) {
                x.q = open_sequence(p, x.s);
                cost = head_cost(p, x.q);
                if (at + cost * p.c.Hkv > first) break;
                at += cost * p.c.Hkv;
            }
            x.blocks = row_blocks(p, x.q.n);
            const int h = (int)((first - at) / cost);
            at += h * cost;
            int rb = 0;
            for (;; ++rb) {
                const int one = kItemCost + tiles_of(p, x.q, rb);
                if (at + one > first) break;
                at += one;
            }
            x.e = h * x.blocks + rb;
            open_item(p, x);
            x.left = last - first;
            const long long t = first - at - kItemCost;
            if (t < 0) x.left += t;
            x.t = t < 0 ? 0 : (int)t;
            x.n = (int)min(x.left, (long long)(x.nt - x.t));
            for (int w = 0; w < kWarps; ++w) s_item[w] = x;
            s_share[0] = last;
            s_share[1] = share;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Item& x = s_item[warp];
    auto next = [&]() {
        __syncwarp();
        if (lane == 0) next_item(p, x);
        __syncwarp();
    };

    // K and V tiles of a part in the ring: K(0), then for each tile j K(j + 1)
    // and V(j), as the tensor core needs them.
    auto k_load = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_load = [](int j, int n) { return j == n - 1 ? 2 * j + 1 : 2 * j + 2; };

    if (warp < 8) {
        // ============================================================ softmax
        regs_increase<208>();
        const int t = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = lane_base + L::kColS + (uint32_t)(128 * t);
        uint32_t s_ph = 0, st_ph = 0, o_ph[2] = {0, 0};
        uint32_t ring = 0;  // loads of the parts before
        const int tok_row = row / p.group, head_row = row - tok_row * p.group;
        for (; x.left > 0; next()) {
            const int n = x.n, clear = x.clear;
            const bool pair = x.pair;
            const int key_first = x.t * kTile;
            const int rows_t = min(p.npt, x.ntok - (pair && t ? p.npt : 0)) * p.group;  // rows of this stream
            const int tok = x.tok0 + (pair && t ? p.npt : 0) + tok_row;                 // of the sequence
            const bool valid = row < rows_t;
            const bool work = (row & ~31) < rows_t;  // the warp has a row
            const int step = pair ? 1 : 2;
            float r = -INFINITY, l = 0.f, l_rnd = 0.f;
            for (int j = pair ? 0 : t; j < n; j += step) {
                const int key0 = key_first + j * kTile;
                const bool edge = key0 + kTile > clear;
                if (!warp_wait(bar(L::bSFull + t), s_ph, abort_flag, wf, 80 + t, x.e)) goto done;
                s_ph ^= 1;
                // S1(j) is complete, and so is all that was issued before it: K(j)
                // and V(j - 1) are no longer read
                if (pair && t == 1 && row == 0) {
                    mbar_arrive(bar(L::bKVEmpty + (ring + (uint32_t)k_load(j)) % L::kStages));
                    if (j > 0) mbar_arrive(bar(L::bKVEmpty + (ring + (uint32_t)v_load(j - 1, n)) % L::kStages));
                }
                tc_fence_after_sync();
                if (work) {
                    uint32_t sv[4][32];
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32u * c, sv[c], mx[c]);
                    tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t bits = seen_word(p, x.q, tok, key0 + 32 * c);
                            mx[c] = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (!(bits >> i & 1u)) sv[c][i] = __float_as_uint(-INFINITY);
                                mx[c] = fmaxf(mx[c], __uint_as_float(sv[c][i]));
                            }
                        }
                    }
                    const float mraw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float mrow = mraw * p.scale_log2;
                    const float r_new = mrow - r > kTau ? mrow : r;
                    const float alpha = r_new == r ? 1.f : ex2_approx(r - r_new);
                    const float r_use = r_new == -INFINITY ? 0.f : r_new;
                    // P in bf16 for the product with V.  LSE takes the sum of the
                    // fp32 p.  O is divided by that sum plus the rounding error of
                    // each tile's largest p, so that a row which one key dominates
                    // (some tile's largest) weighs it alike above and below; the
                    // other errors, at most 2^-9 of a key's weight, average out
                    // against O's own rounding to bf16.
                    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nr2 = f2_pack(-r_use, -r_use);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int e = 64 * c + 2 * i;
                            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(sv[e >> 5][e & 31]),
                                                               __uint_as_float(sv[e >> 5][(e + 1) & 31])),
                                                       c2, nr2);
                            float x0, x1;
                            f2_unpack(x2, x0, x1);
                            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
                            sum[i & 1] = f2_add(sum[i & 1], f2_pack(e0, e1));
                            pk[i] = pack_bf16x2(e0, e1);
                        }
                        tmem_st32(tS + 32u * c, pk);
                    }
                    float a0, a1;
                    f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
                    l = fmaf(l, alpha, a0 + a1);
                    const float pm = ex2_approx(fmaf(mraw, p.scale_log2, -r_use));
                    l_rnd = fmaf(l_rnd, alpha, __uint_as_float(pack_bf16x2(pm, 0.f) << 16) - pm);
                    // the stream's last P.V was complete before this S was: O is idle
                    if (j >= step && __any_sync(0xffffffffu, alpha != 1.f)) {
                        const uint32_t tO = lane_base + L::kColO + (uint32_t)(D * t);
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t ov[32];
                            tmem_ld32(tO + 32u * c, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            tmem_st32(tO + 32u * c, ov);
                        }
                    }
                    r = r_new;
                    tmem_wait_st();
                }
                // V of a tile with masked keys (one stream: its reader, or the first of a pair)
                if (edge && !(pair && t)) {
                    const uint32_t vl = ring + (uint32_t)v_load(j, n), stage = vl % L::kStages;
                    if (!warp_wait(bar(L::bKVFull + stage), (vl / L::kStages) & 1u, abort_flag, wf, 82 + t, x.e)) goto done;
                    uint8_t* vrow = smem + L::kKV + stage * L::kTileBytes + row * 128;
                    const bool past = key0 + row >= x.q.len;
                    bool any = false;
#pragma unroll 4
                    for (int i = 0; i < D / 8; ++i) {
                        uint4* at = reinterpret_cast<uint4*>(vrow + (i >> 3) * kBox + (((i & 7) ^ (lane & 7)) << 4));
                        if (past) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            uint4 e = *at;
                            if (make_finite(e)) {
                                *at = e;
                                any = true;
                            }
                        }
                    }
                    if (any) *poison = 1;
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                mbar_arrive(bar(L::bPFull + t));
            }
            ring += 2u * (uint32_t)n;

            // ---- the part's end.  Each stream of a pair ends its own rows; else
            // stream 0 adds stream 1's, whose state it gets through shared memory.
            const bool two = !pair && n > 1;
            if (!pair && t == 1) {
                if (two) {
                    if (!warp_wait(bar(L::bStEmpty), st_ph ^ 1u, abort_flag, wf, 84, x.e)) goto done;
                    stats[row] = r;
                    stats[128 + row] = l;
                    stats[256 + row] = l_rnd;
                    mbar_arrive(bar(L::bStFull));
                    st_ph ^= 1;
                    o_ph[1] ^= 1;
                }
                continue;
            }
            if (!warp_wait(bar(L::bOFull + t), o_ph[t], abort_flag, wf, 85 + t, x.e)) goto done;
            o_ph[t] ^= 1;
            if (pair && t == 0) o_ph[1] ^= 1;  // stream 1 waits for its own
            float w0 = 1.f, w1 = 0.f;
            if (two) {
                if (!warp_wait(bar(L::bOFull + 1), o_ph[1], abort_flag, wf, 87, x.e)) goto done;
                o_ph[1] ^= 1;
                if (!warp_wait(bar(L::bStFull), st_ph, abort_flag, wf, 88, x.e)) goto done;
                st_ph ^= 1;
                const float r1 = stats[row], top = fmaxf(r, r1), m = top == -INFINITY ? 0.f : top;
                w0 = ex2_approx(r - m);
                w1 = ex2_approx(r1 - m);
                l = fmaf(w0, l, w1 * stats[128 + row]);
                l_rnd = fmaf(w0, l_rnd, w1 * stats[256 + row]);
                r = top;
                mbar_arrive(bar(L::bStEmpty));
            }
            tc_fence_after_sync();
            const bool whole = x.t == 0 && n == x.nt;
            const long long part = (long long)blockIdx.x * 2 + (x.t == 0 ? 1 : 0);
            const long long prow = part * p.rows + (pair ? 128 * t : 0) + row;
            const float inv = l > 0.f || l != l ? 1.f / (l + l_rnd) : 0.f;  // NaN stays
            const bool poisoned = *poison != 0;
            if (work) {
                const uint32_t tO = lane_base + L::kColO;
                const long long token = (long long)x.q.row0 + tok;
                const int head = x.h * p.group + head_row;
                uint4* dst = reinterpret_cast<uint4*>(p.o + (token * p.Hq + head) * D);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t ov[32], o1[32];
                    float o[32];
                    tmem_ld32(tO + (uint32_t)(D * t + 32 * c), ov);
                    if (two) tmem_ld32(tO + (uint32_t)(D + 32 * c), o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = two ? fmaf(w0, __uint_as_float(ov[i]), w1 * __uint_as_float(o1[i])) : __uint_as_float(ov[i]);
                    if (!valid) continue;
                    if (poisoned) {
                        float fix[32];  // o itself stays in registers
#pragma unroll
                        for (int i = 0; i < 32; ++i) fix[i] = o[i];
                        add_poison(p, x, tok, D, 32 * c, fix);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fix[i];
                    }
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[4 * c + i] = make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                        pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                        pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                                        pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    } else {
                        float4* to = parts.o + (part * (D / 4) + 8 * c) * p.rows + (pair ? 128 * t : 0) + row;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            to[(long long)i * p.rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (valid) {
                    if (whole)
                        p.lse[(long long)head * p.T + token] = l == 0.f ? -INFINITY : (r + __log2f(l)) * kLn2;
                    else
                        parts.stat[prow] = make_float4(r, l, l_rnd, 0.f);
                }
            }
            tc_fence_before_sync();
            mbar_arrive(bar(L::bOEmpty + t));
            if (two) mbar_arrive(bar(L::bOEmpty + 1));
            if (!whole && x.t == 0 && t == 0 && row == 0)
                parts.join[blockIdx.x] = Cut{x.s, x.e, s_share[0] - x.left + x.nt, s_share[1]};
        }
    } else {
        regs_decrease<88>();
        if (warp == 8) {
            // ============================================================ TMA producer
            const int shift = p.c.page_shift, page_rows = 1 << min(shift, 7), boxes = D / 64;
            const int per_tile = kTile / page_rows;  // boxes of pages in a tile
            uint32_t ring = 0;
            int q_armed = -1;
            uint32_t qe_ph = 1;
            bool drop = p.fault == 1;
            bool ok = true;
            uint32_t armed = 0;  // loads whose stage was armed
            for (; ok && x.left > 0; next()) {
                const bool pair = x.pair;
                const int row0 = x.q.row0 + x.tok0, h = x.h, n = x.n, t0 = x.t;
                const int* pages = x.q.pages;
                if (!(ok = warp_wait(bar(L::bQEmpty), qe_ph, abort_flag, wf, 89, x.e))) break;
                qe_ph ^= 1;
                const int q_tiles = pair ? 2 : 1;
                if (lane == 0) mbar_arrive_expect_tx(bar(L::bQFull), q_tiles * boxes * p.npt * p.group * 128);
                __syncwarp();
                if (lane < q_tiles * boxes) {
                    const int tile = lane / boxes, half = lane % boxes;
                    tma_load_3d(sb + L::kQ + tile * L::kTileBytes + half * kBox, &tmQ, bar(L::bQFull), 64 * half,
                                h * p.group, row0 + tile * p.npt);
                }
                q_armed = (int)(qe_ph & 1u);
                // lane i has the page of box i of a tile: those of K(j) are V(j)'s
                const int pages_end = (x.q.len + page_rows - 1) / page_rows;  // boxes of the sequence
                auto page_of = [&](int tile) {
                    const int i = (t0 + tile) * per_tile + lane;  // box of the sequence
                    int page = 0;
                    if (lane < per_tile && i < pages_end) {
                        page = pages[(long long)i * page_rows >> shift];
                        if ((unsigned)page >= (unsigned)p.c.num_pages) {
                            atomicOr(p.c.err, 2);
                            page = 0;
                        }
                    }
                    return page;
                };
                auto load = [&](int tile, int page, int which) -> bool {
                    const uint32_t stage = ring % L::kStages;
                    if (!warp_wait(bar(L::bKVEmpty + stage), ((ring / L::kStages) & 1u) ^ 1u, abort_flag, wf, 90, x.e))
                        return false;
                    const int i0 = (t0 + tile) * per_tile, boxes_in = min(per_tile, pages_end - i0);
                    if (!drop) {
                        if (lane == 0) mbar_arrive_expect_tx(bar(L::bKVFull + stage), boxes_in * boxes * page_rows * 128);
                        __syncwarp();
                        const int i = lane % per_tile, half = lane / per_tile;
                        const int pg = __shfl_sync(~0u, page, i);
                        if (i < boxes_in && half < boxes)
                            tma_load_3d(sb + L::kKV + stage * L::kTileBytes + half * kBox + i * page_rows * 128, &tmKV,
                                        bar(L::bKVFull + stage), 64 * half, (i0 + i) * page_rows & ((1 << shift) - 1),
                                        (pg * 2 + which) * p.c.Hkv + h);
                        armed |= 1u << stage;
                    }
                    drop = false;
                    ++ring;
                    return true;
                };
                int page = page_of(0), page_k = page;
                ok = load(0, page, 0);
                for (int j = 0; j < n && ok; ++j) {
                    if (j + 1 < n) {
                        page_k = page_of(j + 1);
                        ok = load(j + 1, page_k, 0);
                    }
                    if (ok) ok = load(j, page, 1);
                    page = page_k;
                }
            }
            // every copy that this warp started has landed before the block retires
            if (q_armed >= 0) mbar_settle(bar(L::bQFull), (uint32_t)q_armed, wf, 91);
            for (uint32_t s = 0; s < (uint32_t)L::kStages; ++s)
                if (armed >> s & 1u) {
                    const uint32_t last = (ring - 1 - s) / L::kStages;  // the stage's last load
                    mbar_settle(bar(L::bKVFull + s), last & 1u, wf, 92);
                }
        } else if (warp == 9) {
            // ============================================================ MMA issuer
            // The whole warp runs this loop; lane 0 issues every MMA and commit (a
            // commit tracks the MMAs of the thread that executes it).
            constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false), kIdescPV = idesc_bf16_f32(128, D, true);
            const bool leader = lane == 0;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto commit = [&](int b) {
                if (leader) tc_commit(bar(b));
                __syncwarp();
            };
            // S_t = Q_q K^T of the tile in a ring stage, and O_t (+)= P_t V
            auto mma_s = [&](int t, int q, uint32_t stage) {
                const uint64_t qd = smem_desc_sw128(sb + L::kQ + q * L::kTileBytes, 16, 1024);
                const uint64_t kd = smem_desc_sw128(sb + L::kKV + stage * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kBox + (kk & 3) * 32) >> 4);
                        mma_ss(tm + L::kColS + (uint32_t)(128 * t), qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);
                    }
                }
                __syncwarp();
            };
            auto mma_pv = [&](int t, uint32_t stage, bool acc) {
                const uint64_t vd = smem_desc_sw128(sb + L::kKV + stage * L::kTileBytes, kBox, 1024);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_ts(tm + L::kColO + (uint32_t)(D * t), tm + L::kColS + (uint32_t)(128 * t + 8 * kk),
                               vd + (uint64_t)((kk * 16 * 128) >> 4), kIdescPV, (acc || kk > 0) ? 1u : 0u);
                }
                __syncwarp();
            };
            uint32_t stage = 0, ph = 0;  // of the next load in the ring
            auto take = [&](uint32_t& st, uint32_t& p_) {
                st = stage;
                p_ = ph;
                if (++stage == (uint32_t)L::kStages) {
                    stage = 0;
                    ph ^= 1u;
                }
            };
            uint32_t q_ph = 0, p_ph[2] = {0, 0}, oe_ph[2] = {1, 1};
            bool ok = true, issued = false;
            auto full = [&](uint32_t st, uint32_t p_, int site) {
                return warp_wait(bar(L::bKVFull + st), p_, abort_flag, wf, site, x.e);
            };
            auto o_empty = [&](int t) {
                const bool got = warp_wait(bar(L::bOEmpty + t), oe_ph[t], abort_flag, wf, 97, x.e);
                oe_ph[t] ^= 1;
                return got;
            };
            auto p_full = [&](int t) { return warp_wait(bar(L::bPFull + t), p_ph[t], abort_flag, wf, 96, x.e); };
            for (; ok && x.left > 0; next()) {
                const int n = x.n;
                const bool pair = x.pair;
                if (!(ok = warp_wait(bar(L::bQFull), q_ph, abort_flag, wf, 93, x.e))) break;
                q_ph ^= 1;
                uint32_t ks, kp, vs, vp;
                take(ks, kp);
                if (!(ok = full(ks, kp, 94))) break;
                tc_fence_after_sync();
                mma_s(0, 0, ks);
                issued = true;
                commit(L::bSFull);
                if (pair) {
                    // Both streams read every tile.  A wait or a commit of this warp
                    // idles the tensor core for some 100 cycles, so a tile takes two of
                    // each: V(j), K(j + 1) and P0(j) are tested at once, and the second
                    // softmax group frees the stages when it sees S1.
                    mma_s(1, 1, ks);
                    commit(L::bSFull + 1);
                    if (n == 1) commit(L::bQEmpty);
                    for (int j = 0; j < n; ++j) {
                        const bool last = j + 1 == n;
                        if (!last) take(ks, kp);
                        take(vs, vp);
                        if (j == 0 || !__all_sync(0xffffffffu,
                                                  mbar_try_wait3(bar(L::bKVFull + vs), vp, bar(L::bKVFull + (last ? vs : ks)),
                                                                 last ? vp : kp, bar(L::bPFull), p_ph[0]))) {
                            if (!last && !(ok = full(ks, kp, 94))) break;
                            if (!(ok = full(vs, vp, 95))) break;
                            if (!(ok = p_full(0))) break;
                        }
                        p_ph[0] ^= 1;
                        if (j == 0 && !(ok = o_empty(0))) break;
                        tc_fence_after_sync();
                        mma_pv(0, vs, j > 0);
                        if (last) {
                            commit(L::bOFull);
                        } else {
                            mma_s(0, 0, ks);
                            commit(L::bSFull);
                        }
                        if (!(ok = p_full(1))) break;
                        p_ph[1] ^= 1;
                        if (j == 0 && !(ok = o_empty(1))) break;
                        tc_fence_after_sync();
                        mma_pv(1, vs, j > 0);
                        if (last) {
                            commit(L::bOFull + 1);
                            commit(L::bKVEmpty + vs);
                        } else {
                            mma_s(1, 1, ks);
                            commit(L::bSFull + 1);
                            if (j + 2 == n) commit(L::bQEmpty);
                        }
                    }
                } else {
                    commit(L::bKVEmpty + ks);
                    if (n > 1) {
                        take(ks, kp);
                        if (!(ok = full(ks, kp, 94))) break;
                        tc_fence_after_sync();
                        mma_s(1, 0, ks);
                        commit(L::bSFull + 1);
                        commit(L::bKVEmpty + ks);
                    }
                    if (n <= 2) commit(L::bQEmpty);
                    for (int j = 0; j < n; ++j) {
                        const int t = j & 1;
                        take(vs, vp);
                        if (!(ok = full(vs, vp, 95))) break;
                        if (!(ok = p_full(t))) break;
                        p_ph[t] ^= 1;
                        if (j < 2 && !(ok = o_empty(t))) break;
                        tc_fence_after_sync();
                        mma_pv(t, vs, j >= 2);
                        commit(L::bKVEmpty + vs);
                        if (j >= n - 2) commit(L::bOFull + t);
                        if (j + 2 < n) {
                            take(ks, kp);
                            if (!(ok = full(ks, kp, 94))) break;
                            tc_fence_after_sync();
                            mma_s(t, 0, ks);
                            commit(L::bSFull + t);
                            commit(L::bKVEmpty + ks);
                            if (j + 3 == n) commit(L::bQEmpty);
                        }
                    }
                }
            }
            if (issued) {
                commit(L::bDrain);
                mbar_settle(bar(L::bDrain), 0, wf, 98);
            }
            __syncwarp();
        }
    }
done:
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the item that begins in block blockIdx.x and ends in a
// later one: 32 rows a block (blockIdx.y), a lane a row, a warp every eighth
// run of four columns.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) fa_kv16_join_kernel(const Kv16AttnParams p)
{
    __shared__ __align__(16) uint16_t s_o[32][D + 8];
    const Parts parts = parts_of(p.part, gridDim.x, p.rows);
    wait_for_primary();
    const Cut cut = parts.join[blockIdx.x];
    if (cut.e < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Item x;
    x.s = cut.s;
    x.e = cut.e;
    x.q = open_sequence(p, x.s);
    x.blocks = row_blocks(p, x.q.n);
    open_item(p, x);
    const bool pair = x.pair;
    const int t = pair ? blockIdx.y >> 2 : 0;  // tile of rows
    const int row = 32 * blockIdx.y + lane - 128 * t;
    const int rows_t = min(p.npt, x.ntok - t * p.npt) * p.group;
    if (row - lane >= rows_t) return;
    const bool valid = row < rows_t;
    const int n = (int)((cut.end - 1) / cut.share) - (int)blockIdx.x + 1;
    auto part = [&](int k) { return (long long)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0); };
    const int prow = 32 * blockIdx.y + lane;
    float top = -INFINITY;
    if (valid)
        for (int k = 0; k < n; ++k) top = fmaxf(top, parts.stat[part(k) * p.rows + prow].x);
    const float m = top == -INFINITY ? 0.f : top;
    constexpr int V = D / 32;
    float4 acc[V];
    float l = 0.f, l_o = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (valid)
        for (int k = 0; k < n; ++k) {
            const float4 st = parts.stat[part(k) * p.rows + prow];
            const float w = ex2_approx(st.x - m);
            l = fmaf(w, st.y, l);
            l_o = fmaf(w, st.y + st.z, l_o);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 o = parts.o[(part(k) * (D / 4) + warp + 8 * i) * p.rows + prow];
                acc[i].x = fmaf(w, o.x, acc[i].x);
                acc[i].y = fmaf(w, o.y, acc[i].y);
                acc[i].z = fmaf(w, o.z, acc[i].z);
                acc[i].w = fmaf(w, o.w, acc[i].w);
            }
        }
    const float inv = l > 0.f || l != l ? 1.f / l_o : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        *reinterpret_cast<uint2*>(&s_o[lane][4 * (warp + 8 * i)]) =
            make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (valid && warp == 0) {
        const int head = x.h * p.group + row % p.group;
        const long long token = (long long)x.q.row0 + x.tok0 + t * p.npt + row / p.group;
        p.lse[(long long)head * p.T + token] = l == 0.f ? -INFINITY : (top + __log2f(l)) * kLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (D / 8); i += kJoinThreads) {
        const int rr = i / (D / 8), c = i % (D / 8), at = row - lane + rr;
        if (at >= rows_t) break;
        const int head = x.h * p.group + at % p.group;
        const long long token = (long long)x.q.row0 + x.tok0 + t * p.npt + at / p.group;
        reinterpret_cast<uint4*>(p.o + (token * p.Hq + head) * D)[c] = *reinterpret_cast<const uint4*>(&s_o[rr][8 * c]);
    }
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& kv, const Kv16AttnParams& p, int blocks, cudaStream_t stream)
{
    const cudaError_t e = smem_limit_once<fa_kv16_attn_kernel<D>>(Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    fa_kv16_attn_kernel<D><<<blocks, kThreads, Smem<D>::kBytes, stream>>>(q, kv, p);
    const cudaError_t f = cudaGetLastError();
    if (f != cudaSuccess) return f;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)(p.rows / 32));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_kv16_join_kernel<D>, p);
}

}  // namespace

int kv16_attn_rows(long long T, int group)
{
    const long long rows = T * group;  // of one sequence, at most
    if (rows > 128 / group * group) return 256;
    return (int)((rows + 31) / 32 * 32);
}

size_t kv16_attn_workspace(int D, int rows, int num_sms)
{
    return (size_t)((num_sms + 1) & ~1) * sizeof(Cut) + (size_t)num_sms * 2 * rows * (sizeof(float4) + 4u * D);
}

cudaError_t launch_kv16_attn(int D, const CUtensorMap& q, const CUtensorMap& kv, const Kv16AttnParams& p, int num_sms,
                             cudaStream_t stream)
{
    return D == 128 ? launch<128>(q, kv, p, num_sms, stream) : launch<64>(q, kv, p, num_sms, stream);
}

}  // namespace fa
