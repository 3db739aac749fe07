// Device helpers of the 16-bit cache: checked lookups of sequences and pages.
#pragma once

#include "fa_kv16.h"
#include "ptx_sm103.cuh"

namespace fa {

// A sequence of a call with packed rows: its rows [row0, row0 + n) are the
// last n of the `len` positions of its slot.
struct Kv16Seq {
    int n, len, row0;
    const int* pages;  // its row of the table
};

// What describes sequence s, as it lies in memory.
struct Kv16Raw {
    int c0, c1, slot, len;
};

__device__ __forceinline__ Kv16Raw kv16_raw(const Kv16Cache& c, const int* cu, int s)
{
    Kv16Raw r;
    r.c0 = cu[s];
    r.c1 = cu[s + 1];
    r.slot = c.ids ? c.ids[s] : s;
    r.len = r.slot >= 0 && r.slot < c.num_slots ? c.lens[r.slot] : -1;
    return r;
}

// Sequence s; one that is not sound is latched and counts as having no rows.
__device__ __forceinline__ Kv16Seq kv16_checked(const Kv16Cache& c, int total, int s, const Kv16Raw& r)
{
    Kv16Seq q{};
    if (r.c0 < 0 || r.c1 < r.c0 || r.c1 > total || (s == 0 && r.c0 != 0) || r.len < r.c1 - r.c0 ||
        (long long)r.len > ((long long)c.table_width << c.page_shift)) {
        atomicOr(c.err, 2);
        q.pages = c.table;
        return q;
    }
    q.n = r.c1 - r.c0;
    q.len = r.len;
    q.row0 = r.c0;
    q.pages = c.table + (long long)r.slot * c.table_width;
    return q;
}

__device__ __forceinline__ Kv16Seq kv16_sequence(const Kv16Cache& c, const int* cu, int total, int s)
{
    return kv16_checked(c, total, s, kv16_raw(c, cu, s));
}

// Element offset in the pool of K of head 0 at a position; -1 for a bad page.
__device__ __forceinline__ long long kv16_row(const Kv16Cache& c, int D, const int* pages, int pos)
{
    const int page = pages[pos >> c.page_shift];
    if ((unsigned)page >= (unsigned)c.num_pages) {
        atomicOr(c.err, 2);
        return -1;
    }
    return ((((long long)page * 2 * c.Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1))) * D;
}

// Elements from K of a head to K of the next (from K to V: Hkv of them).
__device__ __forceinline__ long long kv16_head_stride(const Kv16Cache& c, int D) { return (long long)D << c.page_shift; }

// One block looks for slots that a call names twice with rows.
__device__ __forceinline__ void kv16_check_slots(const Kv16Cache& c, const int* cu, int num_seqs)
{
    constexpr int kWords = 65536 / 32;  // FA_KV4_MAX_SLOTS
    __shared__ uint32_t seen[kWords];
    for (int i = threadIdx.x; i < kWords; i += blockDim.x) seen[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < num_seqs; i += blockDim.x) {
        const int s = c.ids[i];
        if (s < 0 || s >= c.num_slots || cu[i + 1] <= cu[i]) continue;  // no rows: a padded batch
        const uint32_t bit = 1u << (s & 31);
        if (atomicOr(&seen[s >> 5], bit) & bit) atomicOr(c.err, 2);
    }
}

}  // namespace fa
