// Paged 4-bit KV cache: geometry, kernel parameters and launches.  The layout
// and the contracts are documented in include/fa_gb300.h.
#pragma once

#include <cuda_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace fa {

constexpr int kKv4MaxSlots = 65536;
constexpr int kKv4SharedSeqs = 2048;  // sequences of a reserve or fork that needs no workspace

// What every kernel on the cache reads.
struct Kv4Cache {
    uint8_t* pool;
    const int* table;
    const int* lens;
    const int* ids;  // slot of each sequence of the call, or null
    const float* k_scale;
    const float* v_scale;
    int num_pages, num_slots, table_width;
    int page_shift;  // log2(page_size)
    int Hkv;
    int* err;
    int* diag;
};

struct Kv4RowsParams {  // append and read
    const uint16_t* k_in;
    const uint16_t* v_in;
    uint16_t* k_out;
    uint16_t* v_out;
    const int* cu;
    int num_seqs, total;
    bool wide;  // the bf16 rows are 32-byte aligned
    int heads;  // append: KV heads of a warp
    Kv4Cache c;
};

struct Kv4AttnParams {
    const uint16_t* q;
    float* o;
    float* lse;
    float* part;  // workspace
    int B, Hq, Lq, group, R, causal;
    float scale;  // softmax_scale
    int fault;    // test hook: 1 = skip the first tile load of every warp
    Kv4Cache c;
};

struct Kv4PageParams {
    uint8_t* pool;
    int* table;
    int* lens;
    int* refs;
    const int* ids;    // slots (reserve, release), parents (fork)
    const int* other;  // new tokens (reserve), children (fork)
    int* info;
    int* ws;
    int n, num_pages, num_slots, table_width, page_shift, Hkv, D, layers;
    int* err;
};

cudaError_t launch_kv4_append(int D, const Kv4RowsParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_read(int D, const Kv4RowsParams& p, cudaStream_t stream);

// Workspace bytes of the attention on a device with num_sms SMs, and its
// launches (*launches kernels).
size_t kv4_attn_workspace(int D, int R, int num_sms);
cudaError_t launch_kv4_attn(int D, const Kv4AttnParams& p, int num_sms, cudaStream_t stream, int* launches);

size_t kv4_pages_workspace(int num_pages, int n);
cudaError_t launch_kv4_reserve(const Kv4PageParams& p, cudaStream_t stream);
cudaError_t launch_kv4_fork(const Kv4PageParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_release(const Kv4PageParams& p, cudaStream_t stream);
cudaError_t launch_kv4_compact(const Kv4PageParams& p, int num_sms, cudaStream_t stream);

}  // namespace fa
