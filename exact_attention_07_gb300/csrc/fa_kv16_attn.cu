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
// One persistent block per SM.  Its work is one sequence of steps, a tile of
// rows against a tile of 128 keys each, that two softmax warpgroups take in
// turn, each with its own scores (128 columns of tensor memory) and its own
// accumulator: one's exponentials overlap the other's products.  With up to 128
// rows the steps of an item are its tiles of keys, and what the two accumulators
// hold is added at its end; with more they are two tiles of rows for each tile of
// keys, which are then read once for 256 rows.  The scores of a step are issued
// two steps ahead, over the ends of items too, so that short sequences follow one
// another without a gap.  At D = 128 P lies over the scores.  At D = 64 it has 64
// columns of its own, and within an item the scores run three steps ahead: chunks
// of 1024 tokens over 8192 keys take 246 us (1050 TFLOP/s), 280 with P over S.
//
// The warp that issues the MMAs paces the kernel where there are many rows: a
// step is its wait, P.V, S and a commit (at D = 64 one behind P.V too), 1560 cycles
// at D = 128 for 1024 of products.  So it branches on an elected lane, which keeps its operands in
// uniform registers (a rolled loop of MMAs is 15 % slower), and a step tests all
// its barriers at once.
//
// K and V come by TMA, one box per page and 64 dimensions, each into a ring of
// its own with a producer warp of its own.  Positions behind the sequence's end,
// and what no row may see, can hold anything: scores are replaced where a key is
// masked, and in tiles with masked keys V is looked over in shared memory first:
// rows behind the end become zeros, and so do elements that are not finite, which
// are added to the rows that may see them at the end (0 * inf would be NaN in the
// others).
//
// The work of all sequences is one list of (sequence, KV head, tile of rows)
// items, cut evenly over the blocks from the lengths on the device; an item
// that lies in several blocks is joined by a second kernel.
#include <cuda_bf16.h>

#include <climits>

#include "kv16_common.cuh"

namespace fa {

namespace {

constexpr int kWarps = 12, kThreads = 32 * kWarps;  // 8 softmax warps, K, MMA, V, list of work
constexpr int kTile = 128;     // keys of a tile, rows of a tile
constexpr int kBox = 128 * 128;  // bytes of 64 dimensions of 128 rows
constexpr float kTau = 8.f;      // the reference moves when a maximum exceeds it by 2^8
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kAhead = 4;        // items that the list runs ahead
// What an item costs a block beside its tiles, in tiles, and the least that a
// block takes.  With one tile of rows and D = 128, 64 sequences of 1 .. 4096 keys
// (8 heads) take 43.5, 36.3, 37.4 us with a cost of 0, 1, 2; with D = 64, 32 of
// 1 .. 8192 keys (4 heads) 23.5, 22.5, 22.1 and 64 of 1 .. 4096 (8 heads) 31.8,
// 29.7, 30.2 with 2, 3, 4; with two tiles of rows, 8 sequences of up to 9000 30.9,
// 30.9, 30.3 and 8 of 32768 202.8, 202.9, 204.5 with 4, 5, 7.  One sequence of 777
// keys takes 11.0, 11.7, 12.7 us with a least share of 1, 2, 3, one of 100 keys
// 9.7 and 9.0 with 1 and 2.
template <int D>
__host__ __device__ constexpr int item_cost(bool pair)
{
    return pair ? 5 : D == 64 ? 3 : 1;
}
constexpr int kLeastShare = 1;

// A block's part of an item.  A sequence has, for every KV head, blocks of up
// to 2 npt of its query tokens: the items of the list of work.
struct Item {
    Kv16Seq q;
    long long left;  // of the block's share, from tile t on
    int s, h, rb;       // sequence, KV head, block of query tokens
    int blocks;         // of the sequence's query tokens
    int t, n;           // the block's part: tiles t .. t + n - 1; n 0: no more
    int nt;             // tiles of the item
    int tok0, ntok;     // first query token, and how many
    int clear;          // keys in front of this are seen by every row
    int pair;           // two tiles of rows
    uint32_t step, tile, qtile;  // of the block's parts before: steps, tiles of keys, tiles of rows
};

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The descriptors of smem_desc_sw128 with a stride of 1024 bytes differ in their
// low word only (start address and leading dimension), and MMAs that take it
// alone are a third of the code.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }

// One lane of the warp, always the same.  A branch on it costs its body some ten
// percent less code than one on a lane number: operands stay warp-uniform.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
    return e != 0;
}

// D[tmem] (+)= A[smem] * B[smem] and A[tmem] * B[smem] (kind::f16, bf16)
__device__ __forceinline__ void mma_ss_low(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
        : "memory");
}

__device__ __forceinline__ void mma_ts_low(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
        : "memory");
}

// Four and three barrier phases tested by one thread back to back; true when all have completed.
__device__ __forceinline__ bool mbar_try_wait4(const uint32_t (&b)[4], const uint32_t (&p)[4])
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred q0, q1, q2, q3;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q0, [%1], %5;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q1, [%2], %6;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q2, [%3], %7;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q3, [%4], %8;\n\t"
        "and.pred q0, q0, q1;\n\t"
        "and.pred q2, q2, q3;\n\t"
        "and.pred q0, q0, q2;\n\t"
        "selp.u32 %0, 1, 0, q0;\n\t}\n"
        : "=r"(ok)
        : "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3]), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
        : "memory");
    return ok != 0;
}

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

__device__ __forceinline__ uint32_t timer_low_ns()
{
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}

// A bounded wait for test() whose code is short (there are some twenty): false
// when the block's abort flag is raised or the time limit passes, which raises
// it to `site`; the block reports it at its end.
template <typename Test>
__device__ __forceinline__ bool wait_for(Test test, volatile int* abort_flag, int site)
{
    if (test()) return true;
    const uint32_t t0 = timer_low_ns();
#pragma unroll 1
    while (!test()) {
        if (*abort_flag) return false;
        if (timer_low_ns() - t0 > (uint32_t)kWaitLimitNs) {
            *abort_flag = site;
            return false;
        }
    }
    return true;
}

// ------------------------------------------------------------------ the list of work

__device__ __forceinline__ Kv16Seq open_sequence(const Kv16AttnParams& p, int s, const Kv16Raw& raw)
{
    Kv16Seq q = kv16_checked(p.c, p.T, s, raw);
    if (p.mask && q.n > 32 * p.mask_words) {
        atomicOr(p.c.err, 2);
        q.n = 0;
    }
    return q;
}

__device__ __forceinline__ Kv16Seq open_sequence(const Kv16AttnParams& p, int s)
{
    return open_sequence(p, s, kv16_raw(p.c, p.cu, s));
}

// The sequences to come, a lane each, so that one of them is at hand when the
// warp of the list gets there.
struct Window {
    int base;
    Kv16Raw raw;

    __device__ __forceinline__ void fill(const Kv16AttnParams& p, int s, int lane)
    {
        base = s;
        raw = Kv16Raw{0, 0, 0, 0};
        if (s + lane < p.B) raw = kv16_raw(p.c, p.cu, s + lane);
    }
    __device__ __forceinline__ Kv16Seq open(const Kv16AttnParams& p, int s, int lane)
    {
        if (s >= base + 32) fill(p, s, lane);
        const int i = s - base;
        return open_sequence(p, s, Kv16Raw{__shfl_sync(~0u, raw.c0, i), __shfl_sync(~0u, raw.c1, i),
                                           __shfl_sync(~0u, raw.slot, i), __shfl_sync(~0u, raw.len, i)});
    }
};

template <int D>
struct Smem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 3 : 8;  // tiles of the rings
    static constexpr int kQ = 0;  // [2] tiles
    static constexpr int kKRing = 2 * kTileBytes, kVRing = kKRing + kK * kTileBytes;
    static constexpr int kStats = kVRing + kV * kTileBytes;  // float [3][128]: r, l, l_rnd of the group that does not end an item
    static constexpr int kBars = kStats + 3 * 128 * 4;
    static constexpr int bQFull = 0, bQEmpty = 2, bSFull = 4, bPFull = 6, bOFull = 8, bOEmpty = 10, bStFull = 12,
                         bStEmpty = 13, bDrain = 14, bItemFull = 15, bItemEmpty = bItemFull + kAhead, bKFull = bItemEmpty + kAhead,
                         bKEmpty = bKFull + kK, bVFull = bKEmpty + kK, bVEmpty = bVFull + kV,
                         bSRead = bVEmpty + kV, bPvDone = bSRead + 2, kNumBars = bPvDone + 2;  // the last two: kOwnP
    static constexpr int kMisc = kBars + kNumBars * 8;  // tensor memory base, abort flag, poison flag
    static constexpr int kSums = kMisc + 16;            // long long [kWarps], and the blocks' share
    static constexpr int kItems = kSums + (kWarps + 1) * 8;  // Item [kAhead]
    static constexpr int kBytes = kItems + kAhead * (int)sizeof(Item);
    static_assert(kBytes <= 232448 && kBars % 8 == 0, "shared memory of one block");
    // [2] of 128 columns, [2] of D.  P of D = 64 has [2] of 64 columns of its own, so
    // that a group's next scores need not wait for its P.V; else it lies over the scores.
    static constexpr bool kOwnP = D == 64;
    static constexpr uint32_t kColS = 0, kColO = 256, kColP = kOwnP ? kColO + 2 * D : kColS;
    static constexpr uint32_t kPitchP = kOwnP ? 64 : 128;
    static constexpr int kLead = kOwnP ? 3 : 2;  // steps that the scores run ahead of P.V within an item
};

__device__ __forceinline__ int row_blocks(const Kv16AttnParams& p, int n)
{
    return n <= 2 * p.npt ? n > 0 : (n + 2 * p.npt - 1) / (2 * p.npt);
}

// Tiles of keys that block rb of a sequence's query tokens reads.
__device__ __forceinline__ int tiles_of(const Kv16AttnParams& p, const Kv16Seq& q, int rb)
{
    const int keys = p.causal ? q.len - q.n + min(q.n, (rb + 1) * 2 * p.npt) : q.len;
    return (keys + kTile - 1) / kTile;
}

template <int D>
__device__ __forceinline__ int item_cost(const Kv16AttnParams& p, const Kv16Seq& q, int rb)
{
    return item_cost<D>(q.n - rb * 2 * p.npt > p.npt);
}

// Length in the list of one KV head of a sequence: its items' tiles, and what
// each item costs in front of them.
template <int D>
__device__ __forceinline__ long long head_cost(const Kv16AttnParams& p, const Kv16Seq& q)
{
    const int nb = row_blocks(p, q.n);
    long long sum = 0;
    if (!p.causal && nb > 1) sum = (long long)(nb - 1) * (item_cost<D>(true) + tiles_of(p, q, 0));
#pragma unroll 1
    for (int rb = p.causal || nb == 0 ? 0 : nb - 1; rb < nb; ++rb) sum += item_cost<D>(p, q, rb) + tiles_of(p, q, rb);
    return sum;
}

// Fills in what follows from the sequence, the head and the block of tokens.
__device__ __forceinline__ void open_item(const Kv16AttnParams& p, Item& x)
{
    x.nt = tiles_of(p, x.q, x.rb);
    x.tok0 = x.rb * 2 * p.npt;
    x.ntok = min(x.q.n - x.tok0, 2 * p.npt);
    x.pair = x.ntok > p.npt;
    const int prefix = x.q.len - x.q.n;
    x.clear = p.mask ? prefix : p.causal ? prefix + x.tok0 + 1 : x.q.len;
}

// The block's part of the next item; n = 0 at the end of its share.  All lanes
// of a warp compute it alike.
template <int D>
__device__ __forceinline__ void next_item(const Kv16AttnParams& p, Item& x, Window& w, int lane)
{
    x.step += x.pair ? 2 * x.n : x.n;
    x.tile += x.n;
    x.qtile += x.pair ? 2 : 1;
    x.left -= x.n;
    x.n = 0;
    if (x.left <= 0) return;
    if (++x.rb == x.blocks) {
        x.rb = 0;
        if (++x.h == p.c.Hkv) {
            x.h = 0;
            do {
                if (++x.s >= p.B) return;
                x.q = w.open(p, x.s, lane);
                x.blocks = row_blocks(p, x.q.n);
            } while (x.blocks == 0);
        }
    }
    open_item(p, x);
    x.left -= item_cost<D>(x.pair);
    x.t = 0;
    x.n = (int)max(0ll, min(x.left, (long long)x.nt));
}

// The item that begins in a block and ends in a later one, for the kernel that
// joins its parts; parts 0: none.
struct Cut {
    int parts, token, ntok, h;  // blocks that hold a part; first row of q, how many, KV head
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
    p.stat = reinterpret_cast<float4*>(p.join + blocks);
    p.o = p.stat + (size_t)blocks * 2 * rows;
    return p;
}

// A word whose low n bits are set (n any).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    uint32_t r;
    asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(max(32 - n, 0)));  // 32 and more shift everything out
    return r;
}

// Bits of the keys k0 .. k0 + 32 N - 1 that query token i of the sequence may see.
template <int N>
__device__ __forceinline__ void seen_words(const Kv16AttnParams& p, const Kv16Seq& q, int i, int k0, uint32_t (&w)[N])
{
    const int prefix = q.len - q.n, j0 = k0 - prefix;  // the first key among the call's positions
    i = min(i, q.n - 1);
    const int all = (p.mask ? prefix : p.causal ? prefix + i + 1 : q.len) - k0;
    uint32_t m[N + 1];
#pragma unroll
    for (int c = 0; c <= N; ++c) m[c] = 0u;
    if (p.mask) {
        const int* row = p.mask + (long long)(q.row0 + i) * p.mask_words;
#pragma unroll
        for (int c = 0; c <= N; ++c) {
            const int at = (j0 >> 5) + c;
            if (at >= 0 && 32 * at < q.n) m[c] = (uint32_t)__ldg(row + at) & low_bits(q.n - 32 * at);
        }
    }
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = low_bits(all - 32 * c) | __funnelshift_r(m[c], m[c + 1], (uint32_t)j0 & 31u);
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }

// Not 0 where one of two bf16 elements is not finite: an exponent of all ones
// carries into the sign's place.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// 16 bytes of V with the elements that are not finite made 0.
__device__ __forceinline__ uint4 make_finite(uint4 x)
{
    uint32_t* w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (not_finite(w[i]) ? 0u : w[i] & 0xffffu) | (not_finite(w[i] >> 16) ? 0u : w[i] & 0xffff0000u);
    return x;
}

// Adds to a row's D sums what make_finite took out of the part's keys that the
// row sees: an infinity or a NaN swallows what it is added to, whether that is
// normalised and rounded (o16) or not (o32, four sums in every `step` float4).
__device__ __noinline__ void add_poison(const Kv16AttnParams& p, const Item& x, int tok, int D, uint16_t* o16, float* o32,
                                        int step)
{
    const int end = min(x.q.len, (x.t + x.n) * kTile);
#pragma unroll 1
    for (int k = max(x.t * kTile, x.clear); k < end; ++k) {
        uint32_t word[1];
        seen_words(p, x.q, tok, k, word);
        const long long at = word[0] & 1u ? kv16_row(p.c, D, x.q.pages, k) : -1;
        if (at < 0) continue;
        const uint16_t* val = p.c.pool + at + (p.c.Hkv + x.h) * kv16_head_stride(p.c, D);
#pragma unroll 1
        for (int d = 0; d < D; ++d) {
            const uint32_t v = val[d];
            if (!not_finite(v)) continue;
            float* sum = o32 + (long long)(d >> 2) * step * 4 + (d & 3);
            const float old = o16 ? __uint_as_float((uint32_t)o16[d] << 16) : *sum, now = old + __uint_as_float(v << 16);
            if (o16)
                o16[d] = (uint16_t)pack_bf16x2(now, 0.f);
            else
                *sum = now;
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
    constexpr uint32_t kK = L::kK, kV = L::kV;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    // The operands' swizzle needs an aligned base; the window begins so where a
    // kernel has no other shared memory.  The second kernel runs all the same, and
    // the workspace can hold anything: nothing to join.
    if (sb & 1023u) {
        if (threadIdx.x == 0) {
            parts_of(p.part, gridDim.x, p.rows).join[blockIdx.x].parts = 0;
            atomicOr(p.c.err, 4);
        }
        return;
    }
    long long* s_sum = reinterpret_cast<long long*>(smem + L::kSums);
    Item* s_item = reinterpret_cast<Item*>(smem + L::kItems);  // the items in hand: not in registers
    auto bar = [&](int i) -> uint32_t { return sb + L::kBars + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    volatile int* poison = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);
    float* stats = reinterpret_cast<float*>(smem + L::kStats);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitFailure wf{p.c.err, p.c.diag};
    const Parts parts = parts_of(p.part, gridDim.x, p.rows);

    let_dependents_launch();

    if (threadIdx.x == kThreads - 32) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::bQFull + t), 1);
            mbar_init(bar(L::bQEmpty + t), 1);
            mbar_init(bar(L::bSFull + t), 1);
            mbar_init(bar(L::bPFull + t), 128);
            mbar_init(bar(L::bOFull + t), 1);
            mbar_init(bar(L::bOEmpty + t), 128);
            mbar_init(bar(L::bSRead + t), 4);
            mbar_init(bar(L::bPvDone + t), 1);
        }
        mbar_init(bar(L::bStFull), 128);
        mbar_init(bar(L::bStEmpty), 128);
        mbar_init(bar(L::bDrain), 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(bar(L::bItemFull + i), 1);
            mbar_init(bar(L::bItemEmpty + i), 11);  // every warp but the list's
        }
        for (uint32_t s = 0; s < 2 * (kK + kV); ++s) mbar_init(bar(L::bKFull + s), 1);
        *abort_flag = 0;
        *poison = 0;
        mbar_init_fence();
        parts.join[blockIdx.x].parts = 0;
        s_item[0].n = 0;
    }
    if (warp == 8 && lane == 0) tma_prefetch_map(&tmQ);
    if (warp == 10 && lane == 0) tma_prefetch_map(&tmKV);
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // This block's share of the list: every thread sums a run of sequences.
    const int run = (p.B + kThreads - 1) / kThreads;
    const int run0 = min(p.B, (int)threadIdx.x * run), run1 = min(p.B, run0 + run);
    Kv16Seq own{};  // the run's first
    long long mine = 0, own_cost = 0;
    if (run0 < run1) {
        own = open_sequence(p, run0);
        own_cost = head_cost<D>(p, own);
        mine = p.c.Hkv * own_cost;
    }
#pragma unroll 1
    for (int s = run0 + 1; s < run1; ++s) mine += p.c.Hkv * head_cost<D>(p, open_sequence(p, s));

    {
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) upto += total;
            total += s_sum[w];
        }
        // ceil(total / blocks), or a little above
        long long share = (long long)((float)total * (1.f / gridDim.x) * 1.000002f + 0.999f);
        share += share * gridDim.x < total;
        share = max(share, (long long)kLeastShare);
        const long long first = share * blockIdx.x, last = min(total, first + share);
        if (first < last && first < upto && first >= upto - mine) {
            long long at = upto - mine, cost = own_cost;
            Item x;
            x.s = run0;
            x.q = own;
#pragma unroll 1
            while (at + cost * p.c.Hkv <= first) {
                at += cost * p.c.Hkv;
                x.q = open_sequence(p, ++x.s);
                cost = head_cost<D>(p, x.q);
            }
            x.blocks = row_blocks(p, x.q.n);
#pragma unroll 1
            for (x.h = 0; at + cost <= first; ++x.h) at += cost;
            int one;
#pragma unroll 1
            for (x.rb = 0; at + (one = item_cost<D>(p, x.q, x.rb) + tiles_of(p, x.q, x.rb)) <= first; ++x.rb) at += one;
            open_item(p, x);
            x.left = last - first;
            const long long t = first - at - item_cost<D>(x.pair);
            if (t < 0) x.left += t;
            x.t = t < 0 ? 0 : (int)t;
            x.n = (int)min(x.left, (long long)(x.nt - x.t));
            x.step = x.tile = x.qtile = 0;
            if (x.left > 0) s_item[0] = x;
            s_sum[kWarps] = share;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    {
    auto wait = [&](int b, uint32_t parity, int site) -> bool {
        const uint32_t at = bar(b);
        return __all_sync(0xffffffffu, wait_for([&]() { return mbar_try_wait(at, parity & 1u); }, abort_flag, site));
    };
    // The k-th item; n = 0: no more, or a wait ran out.
    auto item = [&](uint32_t k) -> const Item* { return s_item + k % kAhead; };
    auto item_here = [&](uint32_t k) -> bool {
        return (k == 0 || wait(L::bItemFull + k % kAhead, k / kAhead, 79)) && item(k)->n > 0;  // the first: from the start
    };
    auto item_done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bItemEmpty + k % kAhead));
    };

    if (warp < 8) {
        // ============================================================ softmax
        regs_increase<208>();
        const int t = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = lane_base + L::kColS + (uint32_t)(128 * t), tP = lane_base + L::kColP + L::kPitchP * (uint32_t)t;
        uint32_t st_ph = 0, o_ph = 0;  // o_ph: a bit per stream
        const int tok_row = row / p.group, head_row = row - tok_row * p.group;
#pragma unroll 1
        for (uint32_t k = 0; item_here(k); ++k) {
            const Item& x = *item(k);
            const int n = x.n, clear = x.clear, key_first = x.t * kTile;
            const bool pair = x.pair;
            const int u0 = (t ^ (int)x.step) & 1;  // the group's first step of the item; of a pair: its tile of rows
            const int rt = pair ? u0 : 0;
            const int rows_t = min(p.npt, x.ntok - rt * p.npt) * p.group;  // rows of the tile
            const int tok = x.tok0 + rt * p.npt + tok_row;                 // of the sequence
            const bool valid = row < rows_t;
            const bool work = (row & ~31) < rows_t;  // the warp has a row
            const int j0 = pair ? 0 : u0, dj = pair ? 1 : 2;
            uint32_t s_ph = (x.step + u0) >> 1;  // the group's steps so far
            const uint32_t tile0 = x.tile;
            float r = -INFINITY, l = 0.f, l_rnd = 0.f;
#pragma unroll 1
            for (int j = j0; j < n; j += dj, ++s_ph) {
                const int key0 = key_first + j * kTile;
                const bool edge = key0 + kTile > clear;
                // V of a tile with masked keys, before its first product: rows behind
                // the sequence's end become zeros, and so do elements of masked rows
                // that are not finite.  A wait by parity needs the phase before to be
                // over: the tile three before (kV at D = 128) has landed only when these
                // scores are complete, which come after its P.V; the one eight before (D =
                // 64) when the group's last ones were.
                const auto look_over_v = [&]() -> bool {
                    if (!edge || rt != 0) return true;
                    const uint32_t T = tile0 + (uint32_t)j, stage = T % kV;
                    if (!wait(L::bVFull + stage, T / kV, 82 + t)) return false;
                    uint8_t* vrow = smem + L::kVRing + stage * L::kTileBytes + row * 128;
                    const auto at = [&](int i) {  // the row's 16-byte pieces, lanes on different banks
                        return reinterpret_cast<uint4*>(vrow + (i >> 3) * kBox + (((i & 7) ^ (lane & 7)) << 4));
                    };
                    if (key0 + row >= x.q.len) {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) *at(i) = make_uint4(0, 0, 0, 0);
                    } else if (key0 + row >= clear) {
                        uint32_t odd = 0;
#pragma unroll 8
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 e = *at(i);
                            odd |= odd_halves(e.x) | odd_halves(e.y) | odd_halves(e.z) | odd_halves(e.w);
                        }
                        if (odd) {
                            *poison = 1;
#pragma unroll 1
                            for (int i = 0; i < D / 8; ++i) *at(i) = make_finite(*at(i));
                        }
                    }
                    fence_proxy_async_smem();
                    return true;
                };
                if (kV == 8 && !look_over_v()) goto done;
                if (!wait(L::bSFull + t, s_ph, 80 + t)) goto done;
                // These scores are complete, and so is all that was issued before
                // them: K(j) is no longer read (of a pair: when they are the second
                // of the tile), V of the step two before neither (unless kOwnP), and
                // the tile of rows when they are its last.
                if (row == 0) {
                    const uint32_t T = tile0 + (uint32_t)j;
                    if (!pair || rt == 1) {
                        mbar_arrive(bar(L::bKEmpty + T % kK));
                        if (!L::kOwnP && j >= dj) mbar_arrive(bar(L::bVEmpty + (T - dj) % kV));
                    }
                    if (j == n - 1) mbar_arrive(bar(L::bQEmpty + (int)((x.qtile + rt) & 1u)));
                }
                if (kV != 8 && !look_over_v()) goto done;
                tc_fence_after_sync();
                if (work) {
                    bool upper = true;  // some row sees some of the tile's upper 64 keys
                    if (edge) {
                        // masked scores become -inf where they lie, 32 keys at a time
                        // (rolled: a tile's code is long, and few tiles have masked keys)
                        uint32_t seen[4];
                        seen_words(p, x.q, tok, key0, seen);
                        upper = __any_sync(0xffffffffu, (seen[2] | seen[3]) != 0u);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t v[32];
                            tmem_ld32(tS + 32u * c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(seen[0] >> i & 1u)) v[i] = __float_as_uint(-INFINITY);
                            tmem_st32(tS + 32u * c, v);
                            seen[0] = seen[1];
                            seen[1] = seen[2];
                            seen[2] = seen[3];
                        }
                        tmem_wait_st();
                    }
                    uint32_t sv[4][32];
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32u * c, sv[c], mx[c]);
                    tmem_wait_ld();
                    if (L::kOwnP) {  // the next scores may come
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(L::bSRead + t));
                    }
                    const float mraw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float mrow = mraw * p.scale_log2;
                    const float r_new = mrow - r > kTau ? mrow : r;
                    const float alpha = r_new == r ? 1.f : ex2_approx(r - r_new);
                    const float r_use = r_new == -INFINITY ? 0.f : r_new;
                    // P in bf16 for the product with V, as the operands of an MMA
                    // have one type and V is in bf16.  On long caches that is an
                    // error of 1.2e-3 to 1.5e-3 of O, whose own rounding to bf16
                    // is 1.7e-3.  LSE takes the sum of the fp32 p.  O is divided by that sum plus the rounding error of
                    // each tile's largest p, so that a row which one key dominates
                    // (some tile's largest) weighs it alike above and below; the
                    // other errors, at most 2^-8 of a key's weight, average out
                    // against O's own rounding to bf16.
                    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nr2 = f2_pack(-r_use, -r_use);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[32];
                        if (c == 1 && !upper) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) pk[i] = 0u;
                            tmem_st32(tP + 32u * c, pk);
                            break;
                        }
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
                        if (L::kOwnP && c == 0) {
                            // the group's P.V before this one has read P and left O
                            if (!wait(L::bPvDone + t, s_ph ^ 1u, 83)) goto done;
                            tc_fence_after_sync();
                            if (row == 0 && j >= dj && (!pair || rt == 1))
                                mbar_arrive(bar(L::bVEmpty + (tile0 + (uint32_t)(j - dj)) % kV));
                        }
                        tmem_st32(tP + 32u * c, pk);
                    }
                    float a0, a1;
                    f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
                    l = fmaf(l, alpha, a0 + a1);
                    const float pm = ex2_approx(fmaf(mraw, p.scale_log2, -r_use));
                    l_rnd = fmaf(l_rnd, alpha, __uint_as_float(pack_bf16x2(pm, 0.f) << 16) - pm);
                    // the group's last P.V is complete: O is idle
                    if (j != j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
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
                } else if (L::kOwnP) {
                    // a warp without rows keeps step: it must not arrive for two steps at once
                    if (lane == 0) mbar_arrive(bar(L::bSRead + t));
                    if (!wait(L::bPvDone + t, s_ph ^ 1u, 83)) goto done;
                }
                tc_fence_before_sync();
                mbar_arrive(bar(L::bPFull + t));
            }

            // ---- the item's end.  Each group of a pair ends its own rows; else one
            // group, in turn, adds the other's, whose state it gets through shared
            // memory, and the other goes on.
            const bool two = !pair && n > 1;
            const int g = pair ? t : (int)(two ? k : x.step) & 1;
            const uint32_t o_now = o_ph;
            o_ph ^= pair || two ? 3u : 1u << g;
            if (g != t) {
                if (two) {
                    if (!wait(L::bStEmpty, st_ph ^ 1u, 84)) goto done;
                    stats[row] = r;
                    stats[128 + row] = l;
                    stats[256 + row] = l_rnd;
                    mbar_arrive(bar(L::bStFull));
                    st_ph ^= 1;
                }
                item_done(k);
                continue;
            }
            if (!wait(L::bOFull + t, o_now >> t, 85 + t)) goto done;
            float w0 = 1.f, w1 = 0.f;
            if (two) {
                if (!wait(L::bOFull + (t ^ 1), o_now >> (t ^ 1), 87)) goto done;
                if (!wait(L::bStFull, st_ph, 88)) goto done;
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
            if (row == 0 && (!pair || rt == 1)) {  // V of the last steps
                const uint32_t T = tile0 + (uint32_t)n - 1u;
                mbar_arrive(bar(L::bVEmpty + T % kV));
                if (two) mbar_arrive(bar(L::bVEmpty + (T - 1u) % kV));
            }
            const bool whole = x.t == 0 && n == x.nt;
            const long long part = (long long)blockIdx.x * 2 + (x.t == 0 ? 1 : 0);
            const int prow = 128 * rt + row;
            const float inv = l > 0.f || l != l ? 1.f / (l + l_rnd) : 0.f;  // NaN stays
            if (work) {
                // Half of the columns at a time: each half is a trip to tensor memory,
                // but a short sequence runs this code once, from a cold instruction
                // cache.  128 sequences of 200 keys take 39.5 us, 41.2 unrolled; at D = 64
                // (8 heads, 64 of 1 .. 4096) 28.1 and 29.7.
                constexpr int C = D / 64;
                const uint32_t tO = lane_base + L::kColO;
                const long long token = (long long)x.q.row0 + tok;
                const int head = x.h * p.group + head_row;
                uint4* dst = reinterpret_cast<uint4*>(p.o + (token * p.Hq + head) * D);
                float4* to = parts.o + part * (D / 4) * p.rows + prow;
#pragma unroll 1
                for (int c = 0; c < D / 32; c += C) {
                    uint32_t ov[C][32];
#pragma unroll
                    for (int b = 0; b < C; ++b) tmem_ld32(tO + (uint32_t)(D * t + 32 * (c + b)), ov[b]);
                    if (two) {
#pragma unroll
                        for (int b = 0; b < C; ++b) {
                            uint32_t o1[32];
                            tmem_ld32(tO + (uint32_t)(D * (t ^ 1) + 32 * (c + b)), o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                ov[b][i] = __float_as_uint(fmaf(w0, __uint_as_float(ov[b][i]), w1 * __uint_as_float(o1[i])));
                        }
                    } else {
                        tmem_wait_ld();
                    }
                    if (c == D / 32 - C) {
                        tc_fence_before_sync();
                        mbar_arrive(bar(L::bOEmpty + t));
                        if (two) mbar_arrive(bar(L::bOEmpty + (t ^ 1)));
                    }
                    if (valid) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 4 * C; ++i) {
                                const float* f = reinterpret_cast<const float*>(&ov[i >> 2][8 * (i & 3)]);
                                dst[4 * c + i] = make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                                                            pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
                            }
                        } else {
                            float4* at = to + (long long)(8 * c) * p.rows;
#pragma unroll
                            for (int i = 0; i < 8 * C; ++i, at += p.rows) {
                                const float* f = reinterpret_cast<const float*>(&ov[i >> 3][4 * (i & 7)]);
                                *at = make_float4(f[0], f[1], f[2], f[3]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (valid) {
                    if (whole)
                        p.lse[(long long)head * p.T + token] = l == 0.f ? -INFINITY : (r + __log2f(l)) * kLn2;
                    else
                        parts.stat[part * p.rows + prow] = make_float4(r, l, l_rnd, 0.f);
                    if (*poison)
                        add_poison(p, x, tok, D, whole ? reinterpret_cast<uint16_t*>(dst) : nullptr, reinterpret_cast<float*>(to),
                                   p.rows);
                }
            } else {
                mbar_arrive(bar(L::bOEmpty + t));
                if (two) mbar_arrive(bar(L::bOEmpty + (t ^ 1)));
            }
            if (!whole && x.t == 0 && rt == 0 && row == 0) {
                const int rest = x.nt - n, share = (int)min(s_sum[kWarps], 1ll << 30);
                parts.join[blockIdx.x] = Cut{1 + (rest + share - 1) / share, x.q.row0 + x.tok0, x.ntok, x.h};
            }
            item_done(k);
        }
    } else {
        regs_decrease<88>();
        if (warp != 9 && warp < 11) {
            // ============================================================ TMA producers: Q and K, V
            const bool keys = warp == 8;
            const uint32_t stages = keys ? kK : kV;
            const int full = keys ? L::bKFull : L::bVFull, empty = keys ? L::bKEmpty : L::bVEmpty;
            const uint32_t ring = sb + (keys ? L::kKRing : L::kVRing);
            const int shift = p.c.page_shift, page_rows = 1 << min(shift, 7);
            constexpr int boxes = D / 64;
            const int per_tile = kTile / page_rows;  // boxes of pages in a tile
            const int sub = lane & (per_tile - 1), half = lane / per_tile;  // this lane's box
            uint32_t stage = 0, ph = 1;  // of the next tile in the ring, and the parity of its stage's release
            uint32_t q_armed = 0, armed = 0;  // stages with a copy, and the parity of the last one
            uint32_t q_par = 0, par = 0;
            bool drop = keys && p.fault == 1, ok = true;
            // the page of this lane's box in tile j of an item, as it lies in the table
            auto page_of = [&](const Item& y, int j) {
                const int i = (y.t + j) * per_tile + sub;
                return half < boxes && (long long)i * page_rows < y.q.len ? y.q.pages[(long long)i * page_rows >> shift] : 0;
            };
            uint32_t k = 0;
            ok = item_here(0);
            int page = ok ? page_of(*item(0), 0) : 0;
#pragma unroll 1
            while (ok) {
                const Item& y = *item(k);
                const int n = y.n, h = y.h, t0 = y.t;
                const int pages_end = (y.q.len + page_rows - 1) / page_rows;  // boxes of the sequence
                if (keys) {
                    const int tiles = y.pair ? 2 : 1, row0 = y.q.row0 + y.tok0;
#pragma unroll 1
                    for (int i = 0; i < tiles && ok; ++i) {
                        const uint32_t qt = y.qtile + i, b = qt & 1u;
                        if (!(ok = wait(L::bQEmpty + b, (qt >> 1) ^ 1u, 89))) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar(L::bQFull + b), boxes * p.npt * p.group * 128);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_3d(sb + L::kQ + b * L::kTileBytes + lane * kBox, &tmQ, bar(L::bQFull + b), 64 * lane,
                                        h * p.group, row0 + i * p.npt);
                        q_armed |= 1u << b;
                        q_par = (q_par & ~(1u << b)) | (qt >> 1 & 1u) << b;
                    }
                    if (!ok) break;
                }
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    int pg = page;
                    if (j + 1 < n) page = page_of(y, j + 1);  // on its way while this tile's stage is awaited
                    if (!(ok = wait(empty + stage, ph, 90))) break;
                    const int i0 = (t0 + j) * per_tile, count = min(per_tile, pages_end - i0);
                    if ((unsigned)pg >= (unsigned)p.c.num_pages) {
                        atomicOr(p.c.err, 2);
                        pg = 0;
                    }
                    if (!drop) {
                        if (lane == 0) mbar_arrive_expect_tx(bar(full + stage), count * boxes * page_rows * 128);
                        __syncwarp();
                        if (sub < count && half < boxes)
                            tma_load_3d(ring + stage * L::kTileBytes + half * kBox + sub * page_rows * 128, &tmKV,
                                        bar(full + stage), 64 * half, (i0 + sub) * page_rows & ((1 << shift) - 1),
                                        (pg * 2 + (keys ? 0 : 1)) * p.c.Hkv + h);
                        armed |= 1u << stage;
                        par = (par & ~(1u << stage)) | (ph ^ 1u) << stage;
                    }
                    drop = false;
                    if (++stage == stages) {
                        stage = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                item_done(k);
                if (!item_here(++k)) break;
                page = page_of(*item(k), 0);
            }
            // every copy that this warp started has landed before the block retires
#pragma unroll 1
            for (uint32_t b = 0; b < 2; ++b)
                if (q_armed >> b & 1u) mbar_settle(bar(L::bQFull + b), q_par >> b & 1u, wf, 91);
#pragma unroll 1
            for (uint32_t s = 0; s < stages; ++s)
                if (armed >> s & 1u) mbar_settle(bar(full + s), par >> s & 1u, wf, 92);
        } else if (warp == 9) {
            // ============================================================ MMA issuer
            // The whole warp runs this loop; one lane issues every MMA and commit (a
            // commit tracks the MMAs of the thread that executes it).
            constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false), kIdescPV = idesc_bf16_f32(128, D, true);
            const bool leader = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto commit = [&](int b) {
                if (leader) tc_commit(bar(b));
                __syncwarp();
            };
            auto uniform = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
            // S of stream t = rows in buffer q times K in a stage; O of stream t (+)= P V
            auto mma_s = [&](int t, uint32_t q, uint32_t stage) {
                const uint32_t qd = uniform(desc_low(sb + L::kQ + q * L::kTileBytes, 16));
                const uint32_t kd = uniform(desc_low(sb + L::kKRing + stage * L::kTileBytes, 16));
                const uint32_t d = uniform(tm + L::kColS + (uint32_t)(128 * t));
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (uint32_t)(((kk >> 2) * kBox + (kk & 3) * 32) >> 4);
                        mma_ss_low(d, qd + off, kd + off, kIdescS, kk > 0);
                    }
                }
                __syncwarp();
            };
            auto mma_pv = [&](int t, uint32_t stage, bool acc) {
                const uint32_t vd = uniform(desc_low(sb + L::kVRing + stage * L::kTileBytes, kBox));
                const uint32_t d = uniform(tm + L::kColO + (uint32_t)(D * t)), pa = uniform(tm + L::kColP + L::kPitchP * (uint32_t)t);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_ts_low(d, pa + (uint32_t)(8 * kk), vd + (uint32_t)((kk * 16 * 128) >> 4), kIdescPV, acc || kk > 0);
                }
                __syncwarp();
            };
            struct Slot {
                uint32_t stage, ph;
            } kt{0, 0}, vt{0, 0};  // tiles of the rings that the next scores and the next P.V read
            auto advance = [](Slot& s, uint32_t stages) {
                if (++s.stage == stages) {
                    s.stage = 0;
                    s.ph ^= 1u;
                }
            };
            // The next scores are step su of item kx, up to kLead steps ahead of the next
            // P.V: two over the ends of items.  v_step and s_step count the steps, whose
            // streams alternate.
            uint32_t kx = 0, ky = 0, s_step = 0, v_step = 0, oe_ph = 3;
            int su = 0, u = 0;
            bool issued = false, ok = true;
            const Item *x = item_here(0) ? item(0) : nullptr, *y = x;
#pragma unroll 1
            while (y && ok) {
                const bool pr = x && x->pair;
                const bool new_q = x && su < (pr ? 2 : 1), same = x == y && !new_q;
                const uint32_t ahead = s_step - v_step;
                const bool pv = !x || ahead >= (same ? L::kLead : 2u);
                const bool sc = x && (same || ahead <= 2u);
                const bool pair = y->pair;
                const int steps = pair ? 2 * y->n : y->n;
                if (pv && same && u >= 2 && steps - u > L::kLead + 2) {
                    // In the middle of an item.  A wait or a commit of this warp idles the
                    // tensor core for some 100 cycles, so a step tests V, P and what the
                    // scores kLead steps ahead need at once, and the softmax groups free
                    // the stages.
                    auto step = [&](int g, uint32_t q, bool k_done, bool v_done) -> bool {
                        const int gs = L::kOwnP ? g ^ 1 : g;
                        uint32_t wb[4], wp[4];
                        wb[0] = bar(L::bVFull + vt.stage), wp[0] = vt.ph;
                        wb[1] = bar(L::bKFull + kt.stage), wp[1] = kt.ph;
                        wb[2] = bar(L::bPFull + g), wp[2] = v_step >> 1 & 1u;
                        wb[3] = bar(L::bSRead + gs), wp[3] = (v_step + 1u) >> 1 & 1u;
                        if (!__all_sync(0xffffffffu, wait_for([&]() {
                                            return L::kOwnP ? mbar_try_wait4(wb, wp)
                                                            : mbar_try_wait3(wb[0], wp[0], wb[1], wp[1], wb[2], wp[2]);
                                        },
                                                              abort_flag, 94)))
                            return false;
                        tc_fence_after_sync();
                        mma_pv(g, vt.stage, true);
                        if (L::kOwnP) commit(L::bPvDone + g);
                        mma_s(gs, q, kt.stage);
                        commit(L::bSFull + gs);
                        ++v_step;
                        ++u;
                        if (k_done) advance(kt, kK);
                        if (v_done) advance(vt, kV);
                        return true;
                    };
                    const uint32_t q0 = y->qtile & 1u, q1 = pair ? q0 ^ 1u : q0;
                    const int g = (int)v_step & 1, u0 = u;  // of a pair: u is even
#pragma unroll 1
                    while (steps - u > L::kLead + 2) {
                        if (!(ok = step(g, L::kOwnP ? q1 : q0, !pair || L::kOwnP, !pair))) break;
                        if (!(ok = step(g ^ 1, L::kOwnP ? q0 : q1, !pair || !L::kOwnP, true))) break;
                    }
                    s_step += (uint32_t)(u - u0);
                    su += u - u0;
                    continue;
                }
                // V, P and the accumulator's place for P.V, K and Q for the scores.  They are
                // tested together only within an item: the next item's K and Q can wait for
                // places that the softmax groups free after this P.V (the end of an item
                // needs it, and a pair's two Q tiles need both buffers), so P.V never waits
                // for them.
                const int tv = (int)v_step & 1, ts = (int)s_step & 1;
                const int all = !x ? 0 : pr ? 2 * x->n : x->n;
                const uint32_t qt = !x ? 0u : x->qtile + (pr ? su & 1 : 0), qb = qt & 1u;
                const bool together = !L::kOwnP && pv && same;
                const uint32_t bk = bar(L::bKFull + kt.stage);
                uint32_t wb[4], wp[4];  // what a step does not need is replaced by what it does
                if (pv) {
                    wb[0] = bar(L::bVFull + vt.stage), wp[0] = vt.ph;
                    wb[1] = bar(L::bPFull + tv), wp[1] = v_step >> 1 & 1u;
                    wb[2] = u < 2 ? bar(L::bOEmpty + tv) : wb[0], wp[2] = u < 2 ? oe_ph >> tv & 1u : wp[0];
                    wb[3] = together ? bk : wb[0], wp[3] = together ? kt.ph : wp[0];
                    if (!(ok = __all_sync(0xffffffffu, wait_for([&]() { return mbar_try_wait4(wb, wp); }, abort_flag, 95)))) break;
                    tc_fence_after_sync();
                    mma_pv(tv, vt.stage, u >= 2);
                    issued = true;
                    if (L::kOwnP) commit(L::bPvDone + tv);
                    if (u >= steps - 2) commit(L::bOFull + tv);
                    if (u < 2) oe_ph ^= 1u << tv;
                    if (!pair || (u & 1)) advance(vt, kV);
                    ++v_step;
                    if (++u == steps) {
                        item_done(ky);
                        u = 0;
                    }
                }
                if (sc && !together) {
                    wb[0] = wb[1] = wb[2] = wb[3] = bk, wp[0] = wp[1] = wp[2] = wp[3] = kt.ph;
                    if (new_q) wb[1] = bar(L::bQFull + qb), wp[1] = qt >> 1 & 1u;
                    if (L::kOwnP) wb[2] = bar(L::bSRead + ts), wp[2] = (s_step >> 1 & 1u) ^ 1u;
                    if (!(ok = __all_sync(0xffffffffu, wait_for([&]() { return mbar_try_wait4(wb, wp); }, abort_flag, 96)))) break;
                    tc_fence_after_sync();
                }
                if (sc) {
                    mma_s(ts, qb, kt.stage);
                    issued = true;
                    commit(L::bSFull + ts);
                    if (!pr || (su & 1)) advance(kt, kK);
                    ++s_step;
                    if (++su == all) {
                        su = 0;
                        x = item_here(++kx) ? item(kx) : nullptr;
                    }
                }
                if (pv && u == 0) y = item_here(++ky) ? item(ky) : nullptr;
            }
            if (issued) {
                commit(L::bDrain);
                mbar_settle(bar(L::bDrain), 0, wf, 98);
            }
            __syncwarp();
        } else {
            // ============================================================ the list of work
            Item y = s_item[0];
            if (lane == 0) mbar_arrive(bar(L::bItemFull));
            Window window;
            window.base = INT_MIN;  // filled when the first sequence ends
#pragma unroll 1
            for (uint32_t k = 1; y.n > 0; ++k) {
                next_item<D>(p, y, window, lane);
                if (!wait(L::bItemEmpty + k % kAhead, (k / kAhead) ^ 1u, 78)) break;
                if (lane == 0) {
                    s_item[k % kAhead] = y;
                    mbar_arrive(bar(L::bItemFull + k % kAhead));
                }
                __syncwarp();
            }
        }
    }
    }
done:
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        atomicOr(p.c.err, 1);
        if (atomicCAS(p.c.diag, 0, 1 + *abort_flag) == 0) p.c.diag[1] = (int)blockIdx.x;
    }
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the item that begins in block blockIdx.x and ends in a
// later one: 32 rows a block (blockIdx.y), a warp every eighth run of four
// columns.  A lane takes a row, or, where there are at most 4, 8 or 16 rows, every
// eighth, fourth or second of its parts; the lanes of a row are added at the end.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) fa_kv16_join_kernel(const Kv16AttnParams p)
{
    __shared__ __align__(16) uint16_t s_o[32][D + 8];
    constexpr int V = D / 32, U = 4;  // runs of a warp; parts whose loads are in flight together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Parts parts = parts_of(p.part, gridDim.x, p.rows);
    wait_for_primary();
    const Cut cut = parts.join[blockIdx.x];
    const int rt = cut.ntok > p.npt ? (int)blockIdx.y >> 2 : 0;  // tile of rows
    const int row0 = 32 * (int)blockIdx.y - 128 * rt;
    const int nrows = min(32, min(p.npt, cut.ntok - rt * p.npt) * p.group - row0);
    if (cut.parts == 0 || nrows <= 0) return;
    const int shift = nrows <= 4 ? 2 : nrows <= 8 ? 3 : nrows <= 16 ? 4 : 5, lanes = 32 >> shift;
    const int sub = lane & ((1 << shift) - 1), mine = lane >> shift;
    float r = -INFINITY, l = 0.f, l_o = 0.f;
    float4 acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto times = [](float w, float4 a) { return make_float4(w * a.x, w * a.y, w * a.z, w * a.w); };
    const auto plus = [](float w, float4 a, float4 b) {
        return make_float4(fmaf(w, a.x, b.x), fmaf(w, a.y, b.y), fmaf(w, a.z, b.z), fmaf(w, a.w, b.w));
    };
    if (sub < nrows) {
        const int prow = 32 * blockIdx.y + sub;
#pragma unroll 1
        for (int k0 = mine; k0 < cut.parts; k0 += U * lanes) {
            float4 st[U], o[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * lanes;
                if (k < cut.parts) {
                    const long long part = (long long)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0);
                    st[u] = parts.stat[part * p.rows + prow];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[u][i] = parts.o[(part * (D / 4) + warp + 8 * i) * p.rows + prow];
                }
            }
            float top = r;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * lanes < cut.parts) top = fmaxf(top, st[u].x);
            const float m = top == -INFINITY ? 0.f : top, down = ex2_approx(r - m);
            r = top;
            l *= down;
            l_o *= down;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = times(down, acc[i]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * lanes < cut.parts) {
                    const float w = ex2_approx(st[u].x - m);
                    l = fmaf(w, st[u].y, l);
                    l_o = fmaf(w, st[u].y + st[u].z, l_o);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = plus(w, o[u][i], acc[i]);
                }
        }
    }
#pragma unroll 1
    for (int off = 1 << shift; off < 32; off <<= 1) {
        const auto other = [&](float x) { return __shfl_xor_sync(~0u, x, off); };
        const float r1 = other(r), top = fmaxf(r, r1), m = top == -INFINITY ? 0.f : top;
        const float w0 = ex2_approx(r - m), w1 = ex2_approx(r1 - m);
        r = top;
        l = fmaf(w1, other(l), w0 * l);
        l_o = fmaf(w1, other(l_o), w0 * l_o);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = plus(w1, make_float4(other(acc[i].x), other(acc[i].y), other(acc[i].z), other(acc[i].w)), times(w0, acc[i]));
    }
    const int token0 = cut.token + rt * p.npt, head0 = cut.h * p.group;
    if (mine == 0) {
        const float inv = l > 0.f || l != l ? 1.f / l_o : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            *reinterpret_cast<uint2*>(&s_o[sub][4 * (warp + 8 * i)]) =
                make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
        const int row = row0 + sub;
        if (warp == 0 && sub < nrows)
            p.lse[(long long)(head0 + row % p.group) * p.T + token0 + row / p.group] =
                l == 0.f ? -INFINITY : (r + __log2f(l)) * kLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nrows * (D / 8); i += kJoinThreads) {
        const int rr = i / (D / 8), c = i % (D / 8), row = row0 + rr;
        const long long to = (long long)(token0 + row / p.group) * p.Hq + head0 + row % p.group;
        reinterpret_cast<uint4*>(p.o + to * D)[c] = *reinterpret_cast<const uint4*>(&s_o[rr][8 * c]);
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
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)((p.rows + 31) / 32));
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
    return (int)((rows + 3) / 4 * 4);
}

size_t kv16_attn_workspace(int D, int rows, int num_sms)
{
    return (size_t)num_sms * sizeof(Cut) + (size_t)num_sms * 2 * rows * (sizeof(float4) + 4u * D);
}

cudaError_t launch_kv16_attn(int D, const CUtensorMap& q, const CUtensorMap& kv, const Kv16AttnParams& p, int num_sms,
                             cudaStream_t stream)
{
    return D == 128 ? launch<128>(q, kv, p, num_sms, stream) : launch<64>(q, kv, p, num_sms, stream);
}

}  // namespace fa
