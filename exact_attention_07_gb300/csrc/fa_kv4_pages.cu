// Page operations of the 4-bit cache: reserve, fork, release, compact.
//
// The bookkeeping (validation, prefix sums, the search for free pages) is a
// few thousand integers: one block of 1024 threads does it, bound by the
// latency of a handful of dependent passes over L2.  Copies of pages run in a
// second kernel over the whole GPU, bound by HBM (each byte read and written
// once).
#include <algorithm>
#include <climits>

#include "kv4_common.cuh"

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// workspace of compact, in int32: header | map | sources | targets; of
// reserve and fork, where it has any: prefix sums
constexpr int kWsCount = 0;  // page moves
constexpr int kWsLive = 1;   // pages in use
constexpr int kWsBase = 16;  // first entry behind the header

__device__ __forceinline__ int pages_of(int len, int shift) { return (int)(((long long)len + (1 << shift) - 1) >> shift); }

// Exclusive prefix of x over the block, and its total.
template <typename T>
__device__ __forceinline__ T block_prefix(T x, T (&part)[kPlanWarps], T& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();  // `part` of the previous call has been read
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        T w = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(~0u, w, o);
            if (lane >= o) w += y;
        }
        part[lane] = w;
    }
    __syncthreads();
    total = part[kPlanWarps - 1];
    return v - x + (warp ? part[warp - 1] : 0);
}

// The pages are cut into one segment of whole int4 steps per warp.
__device__ __forceinline__ int segment(int n) { return ((n + kPlanWarps - 1) / kPlanWarps + 127) & ~127; }

// refs[i .. i + 3], -1 behind the end.
__device__ __forceinline__ int4 load_refs(const int* refs, int i, int n)
{
    if (i + 3 < n) return *reinterpret_cast<const int4*>(refs + i);
    int4 r = make_int4(-1, -1, -1, -1);
    if (i < n) r.x = refs[i];
    if (i + 1 < n) r.y = refs[i + 1];
    if (i + 2 < n) r.z = refs[i + 2];
    return r;
}

// Pages of the warp's segment that `pick` takes.
template <typename Pick>
__device__ __forceinline__ int count_pages(const int* refs, int n, Pick pick)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = segment(n);
    int count = 0;
    for (int i = warp * seg + 4 * lane; i < min(n, (warp + 1) * seg); i += 128) {
        const int4 r = load_refs(refs, i, n);
        count += (i < n && pick(i, r.x)) + (i + 1 < n && pick(i + 1, r.y)) + (i + 2 < n && pick(i + 2, r.z)) +
                 (i + 3 < n && pick(i + 3, r.w));
    }
    return __reduce_add_sync(~0u, count);
}

// Calls use(rank, page) for the pages that `pick` takes, ranked in order over
// the block, while the rank is below `most`; `rank` is the first of this warp.
template <typename Pick, typename Use>
__device__ __forceinline__ void for_pages(const int* refs, int n, int rank, int most, Pick pick, Use use)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = segment(n);
    const unsigned below = (1u << lane) - 1;
    for (int base = warp * seg; base < min(n, (warp + 1) * seg) && rank < most; base += 128) {
        const int i = base + 4 * lane;
        const int4 r = load_refs(refs, i, n);
        const bool t[4] = {i < n && pick(i, r.x), i + 1 < n && pick(i + 1, r.y), i + 2 < n && pick(i + 2, r.z),
                           i + 3 < n && pick(i + 3, r.w)};
        int mine = rank;
        rank = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned b = __ballot_sync(~0u, t[e]);
            mine += __popc(b & below);
            rank += __popc(b);
        }
        rank += __shfl_sync(~0u, mine, 0);  // lane 0 has nothing below it: its `mine` is the old rank
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t[e]) {
                if (mine < most) use(mine, i + e);
                ++mine;
            }
    }
}

// First rank of this warp's segment, and the block's total, of a per-warp count.
__device__ __forceinline__ int warp_rank(int count, int (&part)[kPlanWarps], int& total)
{
    const int before = block_prefix((threadIdx.x & 31) == 0 ? count : 0, part, total);
    return __shfl_sync(~0u, before, 0);
}

// The entry whose range of ranks [prefix[i], prefix[i + 1]) holds k.
__device__ __forceinline__ int find_entry(const int* prefix, int n, int k)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

struct PlanSmem {
    uint32_t seen[kKv4MaxSlots / 32];
    int part[kPlanWarps];
    long long part64[kPlanWarps];
    int bad;
};

__device__ __forceinline__ void plan_begin(PlanSmem& sm)
{
    for (int i = threadIdx.x; i < kKv4MaxSlots / 32; i += kPlanThreads) sm.seen[i] = 0;
    if (threadIdx.x == 0) sm.bad = 0;
    __syncthreads();
}

// True when the slot exists and its length fits its table row.
__device__ __forceinline__ bool slot_ok(const Kv4PageParams& p, int s)
{
    if (s < 0 || s >= p.num_slots) return false;
    const int len = p.lens[s];
    return len >= 0 && (long long)len <= ((long long)p.table_width << p.page_shift);
}

// Marks a slot; true if it was marked already.
__device__ __forceinline__ bool mark(PlanSmem& sm, int s)
{
    const uint32_t bit = 1u << (s & 31);
    return (atomicOr(&sm.seen[s >> 5], bit) & bit) != 0;
}

// Refusal: info, which also tells a second kernel, and the latch for bad
// arguments.
__device__ __forceinline__ bool refused(const Kv4PageParams& p, bool bad, int free_pages, long long need)
{
    if (!bad && need <= free_pages) return false;
    if (threadIdx.x == 0) {
        p.info[0] = free_pages;
        p.info[1] = bad ? -1 : (int)min(need - free_pages, (long long)INT_MAX);
        if (bad) atomicOr(p.err, 2);
    }
    return true;
}

// Takes a reference from a page; 1 when that was the last.
__device__ __forceinline__ int drop_page(const Kv4PageParams& p, int page)
{
    if ((unsigned)page >= (unsigned)p.num_pages) {
        atomicOr(p.err, 2);
        return 0;
    }
    const int held = atomicSub(p.refs + page, 1);
    if (held <= 0) {  // no one held it
        atomicAdd(p.refs + page, 1);
        atomicOr(p.err, 2);
    }
    return held == 1;
}

// ------------------------------------------------------------------ reserve

__global__ void __launch_bounds__(kPlanThreads) fa_kv4_reserve_kernel(const Kv4PageParams p)
{
    __shared__ PlanSmem sm;
    __shared__ int s_prefix[kKv4SharedSeqs];
    const int tid = threadIdx.x;
    int* prefix = p.n <= kKv4SharedSeqs ? s_prefix : p.ws;
    plan_begin(sm);
    long long need = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int want = 0;
        if (i < p.n) {
            const int s = p.ids ? p.ids[i] : i;
            const int add = p.other[i];
            if (!slot_ok(p, s) || (add != 0 && mark(sm, s))) {
                sm.bad = 1;
            } else {
                const int len = p.lens[s];
                const long long to = (long long)len + add;
                if (to < 0 || to > ((long long)p.table_width << p.page_shift))
                    sm.bad = 1;
                else if (add >= 0)
                    want = pages_of((int)to, p.page_shift) - pages_of(len, p.page_shift);
                else if (to & ((1 << p.page_shift) - 1)) {  // what becomes the partly filled page must be its own
                    const int page = p.table[(long long)s * p.table_width + (to >> p.page_shift)];
                    if ((unsigned)page >= (unsigned)p.num_pages || p.refs[page] != 1) sm.bad = 1;
                }
            }
        }
        long long total;  // far more pages may be asked for than there are
        const long long before = block_prefix<long long>(want, sm.part64, total);
        if (i < p.n) prefix[i] = (int)min(need + before, (long long)INT_MAX);
        need += total;
    }
    const int count = count_pages(p.refs, p.num_pages, [](int, int r) { return r == 0; });
    int free_pages;
    const int rank = warp_rank(count, sm.part, free_pages);
    if (refused(p, sm.bad != 0, free_pages, need)) return;
    for_pages(p.refs, p.num_pages, rank, (int)need, [](int, int r) { return r == 0; }, [&](int k, int page) {
        const int i = find_entry(prefix, p.n, k);
        const int s = p.ids ? p.ids[i] : i;
        p.table[(long long)s * p.table_width + pages_of(p.lens[s], p.page_shift) + (k - prefix[i])] = page;
        p.refs[page] = 1;
    });
    __syncthreads();
    int freed = 0;  // by the warp's sequences that give tokens back
    for (int i = tid >> 5; i < p.n; i += kPlanWarps) {
        if (p.other[i] >= 0) continue;
        const int s = p.ids ? p.ids[i] : i;
        const int from = pages_of(p.lens[s] + p.other[i], p.page_shift), to = pages_of(p.lens[s], p.page_shift);
        int* row = p.table + (long long)s * p.table_width;
        for (int j = from + (tid & 31); j < to; j += 32) {
            freed += drop_page(p, row[j]);
            row[j] = -1;
        }
    }
    freed = __reduce_add_sync(~0u, freed);
    if ((tid & 31) == 0) sm.part[tid >> 5] = freed;
    __syncthreads();
    for (int i = tid; i < p.n; i += kPlanThreads)
        if (p.other[i]) p.lens[p.ids ? p.ids[i] : i] += p.other[i];  // a slot named again adds nothing
    if (tid == 0) {
        freed = 0;
        for (int w = 0; w < kPlanWarps; ++w) freed += sm.part[w];
        p.info[0] = free_pages - (int)need + freed;
        p.info[1] = 0;
    }
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kPlanThreads) fa_kv4_fork_plan_kernel(const Kv4PageParams p)
{
    let_dependents_launch();
    __shared__ PlanSmem sm;
    __shared__ int s_prefix[kKv4SharedSeqs];
    const int tid = threadIdx.x, page_size = 1 << p.page_shift;
    int* prefix = p.n <= kKv4SharedSeqs ? s_prefix : p.ws;
    plan_begin(sm);
    for (int i = tid; i < p.n; i += kPlanThreads) {
        const int c = p.other[i];
        if (!slot_ok(p, c) || p.lens[c] != 0 || mark(sm, c)) sm.bad = 1;
    }
    __syncthreads();
    int need = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int want = 0;
        if (i < p.n) {
            const int s = p.ids[i];
            if (!slot_ok(p, s) || (sm.seen[s >> 5] >> (s & 31) & 1)) {
                sm.bad = 1;
            } else if (const int rest = p.lens[s] & (page_size - 1)) {
                const int page = p.table[(long long)s * p.table_width + (p.lens[s] >> p.page_shift)];
                if ((unsigned)page >= (unsigned)p.num_pages) sm.bad = 1;
                want = 1;
            }
        }
        int total;
        const int before = block_prefix(want, sm.part, total);
        if (i < p.n) prefix[i] = need + before;
        need += total;
    }
    const int count = count_pages(p.refs, p.num_pages, [](int, int r) { return r == 0; });
    int free_pages;
    const int rank = warp_rank(count, sm.part, free_pages);
    if (refused(p, sm.bad != 0, free_pages, need)) return;
    for_pages(p.refs, p.num_pages, rank, need, [](int, int r) { return r == 0; }, [&](int k, int page) {
        const int i = find_entry(prefix, p.n, k);
        p.table[(long long)p.other[i] * p.table_width + (p.lens[p.ids[i]] >> p.page_shift)] = page;
        p.refs[page] = 1;
    });
    __syncthreads();
    for (int i = tid; i < p.n; i += kPlanThreads) p.lens[p.other[i]] = p.lens[p.ids[i]];
    if (tid == 0) {
        p.info[0] = free_pages - need;
        p.info[1] = 0;
    }
}

// One warp copies the first units of one KV head's block of a page in one layer.
__device__ __forceinline__ void copy_block(const Kv4PageParams& p, int layer, int h, int src, int dst, int units)
{
    constexpr int U = 6;  // 16-byte loads in flight per lane
    const long long block = (long long)(18 * p.D) << (p.page_shift - 4);  // bytes of a head's block
    uint8_t* base = p.pool + (layer * (long long)p.num_pages * p.Hkv + h) * block;
    const uint4* from = reinterpret_cast<const uint4*>(base + src * (block * p.Hkv));
    uint4* to = reinterpret_cast<uint4*>(base + dst * (block * p.Hkv));
    const int n = units * (18 * p.D / 16);
    for (int v = threadIdx.x & 31; v < n; v += 32 * U) {
        uint4 x[U];
#pragma unroll
        for (int e = 0; e < U; ++e)
            if (v + 32 * e < n) x[e] = __ldcs(from + v + 32 * e);
#pragma unroll
        for (int e = 0; e < U; ++e)
            if (v + 32 * e < n) __stcs(to + v + 32 * e, x[e]);
    }
}

// Calls use(layer, k, head) for the warp's part of layers x count x heads.
template <typename Use>
__device__ __forceinline__ void for_blocks(const Kv4PageParams& p, int count, Use use)
{
    const long long tasks = (long long)count * p.layers * p.Hkv;
    const long long stride = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < tasks; t += stride) {
        const int h = (int)(t % p.Hkv);
        const long long r = t / p.Hkv;
        use((int)(r / count), (int)(r % count), h);
    }
}

__global__ void __launch_bounds__(256) fa_kv4_fork_kernel(const Kv4PageParams p)
{
    wait_for_primary();
    if (p.info[1] != 0) return;  // refused
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int s = p.ids[i], len = p.lens[s], full = len >> p.page_shift;
        const int own = (len & ((1 << p.page_shift) - 1)) ? full : -1;  // written by the plan
        const int* from = p.table + (long long)s * p.table_width;
        int* to = p.table + (long long)p.other[i] * p.table_width;
        for (int j = threadIdx.x; j < p.table_width; j += blockDim.x) {
            if (j == own) continue;
            int page = -1;
            if (j < full) {
                page = from[j];
                if ((unsigned)page < (unsigned)p.num_pages)
                    atomicAdd(p.refs + page, 1);
                else
                    atomicOr(p.err, 2);
            }
            to[j] = page;
        }
    }
    for_blocks(p, p.n, [&](int layer, int i, int h) {  // the partly filled pages; the plan has checked both
        const int s = p.ids[i], len = p.lens[s], at = len >> p.page_shift, rest = len & ((1 << p.page_shift) - 1);
        if (rest)
            copy_block(p, layer, h, p.table[(long long)s * p.table_width + at],
                       p.table[(long long)p.other[i] * p.table_width + at], (rest + 15) >> 4);
    });
}

// ------------------------------------------------------------------ release

__global__ void __launch_bounds__(128) fa_kv4_release_kernel(const Kv4PageParams p)
{
    const int i = blockIdx.x, s = p.ids[i];
    if (s < 0 || s >= p.num_slots) {
        if (threadIdx.x == 0) atomicOr(p.err, 2);
        return;
    }
    bool again = false;  // a slot named before is that entry's
    for (int j = threadIdx.x; j < i; j += blockDim.x) again |= p.ids[j] == s;
    if (__syncthreads_or(again)) return;
    const int len = p.lens[s];
    if (len < 0 || (long long)len > ((long long)p.table_width << p.page_shift)) {
        if (threadIdx.x == 0) atomicOr(p.err, 2);
        return;
    }
    __syncthreads();  // everyone has read the length
    const int n = pages_of(len, p.page_shift);
    int* row = p.table + (long long)s * p.table_width;
    for (int j = threadIdx.x; j < n; j += blockDim.x) drop_page(p, row[j]);
    __syncthreads();
    for (int j = threadIdx.x; j < p.table_width; j += blockDim.x) row[j] = -1;
    if (threadIdx.x == 0) p.lens[s] = 0;
}

// ------------------------------------------------------------------ compact

// workspace: header | map [num_pages] | sources | targets
__global__ void __launch_bounds__(kPlanThreads) fa_kv4_compact_plan_kernel(const Kv4PageParams p)
{
    let_dependents_launch();
    __shared__ PlanSmem sm;
    const int tid = threadIdx.x, n = p.num_pages;
    int* map = p.ws + kWsBase;
    int* src = map + n;
    int* dst = src + (n + 1) / 2;
    if (tid == 0) sm.bad = 0;
    __syncthreads();
    for (int s = tid; s < p.num_slots; s += kPlanThreads)
        if (!slot_ok(p, s)) sm.bad = 1;
    int live;
    warp_rank(count_pages(p.refs, n, [](int, int r) { return r != 0; }), sm.part, live);
    if (refused(p, sm.bad != 0, n - live, 0)) return;
    const auto hole = [live](int i, int r) { return i < live && r == 0; };
    const auto mover = [live](int i, int r) { return i >= live && r != 0; };
    int holes, movers;
    const int hole_rank = warp_rank(count_pages(p.refs, n, hole), sm.part, holes);
    const int mover_rank = warp_rank(count_pages(p.refs, n, mover), sm.part, movers);  // as many as holes
    for (int i = live + tid; i < n; i += kPlanThreads) map[i] = -1;
    for_pages(p.refs, n, hole_rank, holes, hole, [&](int k, int page) { dst[k] = page; });
    for_pages(p.refs, n, mover_rank, movers, mover, [&](int k, int page) { src[k] = page; });
    __syncthreads();
    for (int k = tid; k < movers; k += kPlanThreads) {
        const int a = src[k], b = dst[k];
        map[a] = b;
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
    if (tid == 0) {
        p.ws[kWsCount] = movers;
        p.ws[kWsLive] = live;
        p.info[0] = n - live;
        p.info[1] = 0;
    }
}

__global__ void __launch_bounds__(256) fa_kv4_compact_kernel(const Kv4PageParams p)
{
    wait_for_primary();
    if (p.info[1] != 0) return;  // refused
    const int count = p.ws[kWsCount], live = p.ws[kWsLive];
    if (count == 0) return;
    const int* map = p.ws + kWsBase;
    const int* src = map + p.num_pages;
    for (int s = blockIdx.x; s < p.num_slots; s += gridDim.x) {
        const int pages = pages_of(p.lens[s], p.page_shift);
        int* row = p.table + (long long)s * p.table_width;
        for (int j = threadIdx.x; j < pages; j += blockDim.x) {
            const int page = row[j];
            if (page >= 0 && page < live) continue;
            const int to = page >= 0 && page < p.num_pages ? map[page] : -1;
            if (to >= 0)
                row[j] = to;
            else
                atomicOr(p.err, 2);  // not a page in use
        }
    }
    const int* dst = src + (p.num_pages + 1) / 2;
    for_blocks(p, count, [&](int layer, int k, int h) {
        copy_block(p, layer, h, src[k], dst[k], 1 << (p.page_shift - 4));
    });
}

}  // namespace

size_t kv4_pages_workspace(int num_pages, int n)
{
    return 4 * ((size_t)kWsBase + 2 * (size_t)num_pages + 2 + (size_t)n);
}

cudaError_t launch_kv4_reserve(const Kv4PageParams& p, cudaStream_t stream)
{
    fa_kv4_reserve_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_fork(const Kv4PageParams& p, int num_sms, cudaStream_t stream)
{
    fa_kv4_fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long warps = (long long)p.n * p.layers * p.Hkv;
    const int grid = (int)std::min(8ll * num_sms, std::max((long long)p.n, (warps + 7) / 8));
    return launch_dependent(fa_kv4_fork_kernel, dim3(grid), 256, stream, p);
}

cudaError_t launch_kv4_release(const Kv4PageParams& p, cudaStream_t stream)
{
    fa_kv4_release_kernel<<<p.n, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_compact(const Kv4PageParams& p, int num_sms, cudaStream_t stream)
{
    fa_kv4_compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long warps = (long long)(p.num_pages + 1) / 2 * p.layers * p.Hkv;
    const int grid = (int)std::min(8ll * num_sms, std::max((long long)p.num_slots, (warps + 7) / 8));
    return launch_dependent(fa_kv4_compact_kernel, dim3(grid), 256, stream, p);
}

}  // namespace fa
