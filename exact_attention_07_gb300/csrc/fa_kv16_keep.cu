// Keeping the accepted nodes of a drafted tree: rows of the 16-bit cache move
// to the front of their sequence's last positions, in every layer.
//
//   row (len - n + j) <- row (len - n + keep[j]),  j < count
//
// Bound: a few rows per sequence are read and written once, after a chain of
// dependent loads (offsets, slot, length, table, row) in each block.  So that
// most blocks run at once (32 registers, 8 an SM) a thread has four rows in
// flight and takes two columns: 64 sequences of 32 layers, 8 heads, D = 128, 34
// MB moved, 8.2 us (11.2 with eight rows and one column, 9.0 with four columns;
// 11.0 where three such caches take turns).  The accepted nodes ascend,
// keep[j] >= j, so a thread that takes one 16-byte column of all the moves, in
// order, needs no buffer: what it writes lies in front of all that it has yet to
// read.
#include "kv16_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256, kAtOnce = 4, kCols = 2;

__global__ void __launch_bounds__(kThreads, 8) fa_kv16_keep_kernel(const Kv16KeepParams p)
{
    __shared__ long long s_src[kThreads], s_dst[kThreads];
    const int s = blockIdx.x;
    if (s == p.num_seqs) {  // only this check
        if (blockIdx.y == 0) kv16_check_slots(p.c, p.cu, p.num_seqs);
        return;
    }
    const Kv16Seq q = kv16_sequence(p.c, p.cu, p.total, s);
    const int count = p.counts[s];
    const int* keep = p.keep + q.row0;
    bool bad = count < 0 || count > q.n;
    if (!bad)
        for (int j = threadIdx.x; j < count; j += kThreads)
            bad |= keep[j] >= q.n || keep[j] <= (j ? keep[j - 1] : -1);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        if (bad) atomicOr(p.c.err, 2);
        p.back[s] = bad ? 0 : count - q.n;
    }
    if (bad) return;

    const int chunks = p.D >> 3;  // 16-byte columns of a row
    const int rows = p.layers * 2 * p.c.Hkv;  // (layer, K or V, head)
    const int first = q.len - q.n;
    for (int j0 = 0; j0 < count; j0 += kThreads) {
        const int n = min(kThreads, count - j0), j = j0 + threadIdx.x;
        if (threadIdx.x < n) {
            const int k = keep[j];
            long long a = -1, b = -1;
            if (k != j) {
                a = kv16_row(p.c, p.D, q.pages, first + k);
                b = kv16_row(p.c, p.D, q.pages, first + j);
                if (b < 0) a = -1;
            }
            s_src[threadIdx.x] = a;
            s_dst[threadIdx.x] = b;
        }
        __syncthreads();
#pragma unroll 1
        for (int col = blockIdx.y * kThreads + threadIdx.x; col < rows * chunks; col += gridDim.y * kThreads) {
            const int row = col / chunks, layer = row / (2 * p.c.Hkv);
            uint16_t* base = p.c.pool + layer * p.layer_stride +
                             (row - layer * 2 * p.c.Hkv) * kv16_head_stride(p.c, p.D) + 8 * (col - row * chunks);
            for (int i0 = 0; i0 < n; i0 += kAtOnce) {
                uint4 x[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i < n && s_src[i0 + i] >= 0) x[i] = *reinterpret_cast<const uint4*>(base + s_src[i0 + i]);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i < n && s_src[i0 + i] >= 0) *reinterpret_cast<uint4*>(base + s_dst[i0 + i]) = x[i];
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv16_keep(const Kv16KeepParams& p, cudaStream_t stream)
{
    const long long cols = (long long)p.layers * 2 * p.c.Hkv * (p.D / 8);
    const dim3 grid((unsigned)p.num_seqs + (p.c.ids ? 1 : 0), (unsigned)((cols + kThreads * kCols - 1) / (kThreads * kCols)));
    fa_kv16_keep_kernel<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
