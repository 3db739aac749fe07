// Rotary positions and the paged 16-bit KV cache: kernel parameters and
// launches.  Layouts and contracts are documented in include/fa_gb300.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace fa {

// What every kernel on the cache reads.  Page p holds K [Hkv][page_size][D],
// then V, in bf16.
struct Kv16Cache {
    uint16_t* pool;
    const int* table;
    const int* lens;
    const int* ids;  // slot of each sequence of the call, or null
    int num_pages, num_slots, table_width;
    int page_shift;  // log2(page_size)
    int Hkv;
    int* err;
    int* diag;
};

struct RotaryRows {  // [B][T][heads][D], strides in elements
    const void* x;
    void* y;
    long long xb, xt, xh, yb, yt, yh;
    int heads;
    bool in_place;
};

// Rotation of q and k rows; with `cache` k and v go into the cache (append).
struct RotaryParams {
    RotaryRows r[3];  // q, k, v
    const unsigned long long* freqs;
    const int* pos;   // null: the index along the tokens (append: in the cache)
    long long pos_b;  // positions from one batch to the next
    int B, T, D, R, start;
    float mscale;
    bool backward;
    const int* cu;  // append
    int num_seqs;
    Kv16Cache c;
};

struct Kv16KeepParams {
    const int* keep;
    const int* counts;
    const int* cu;
    int* back;
    int num_seqs, total, D, layers;
    long long layer_stride;  // elements
    Kv16Cache c;
};

struct Kv16AttnParams {
    uint16_t* o;
    float* lse;
    float* part;  // workspace
    const int* cu;
    const int* mask;  // bits of the drafted trees, or null
    int mask_words;
    int B, T, Hq, group;
    int npt;  // query tokens of a tile: 128 / group
    int rows; // rows of a part in the workspace
    int causal;
    float scale_log2;
    int fault;  // test hook: 1 = skip the first tile load of every block
    Kv16Cache c;
};

cudaError_t launch_rope(bool in_f32, bool out_f32, bool interleaved, const RotaryParams& p, int num_sms,
                        cudaStream_t stream);
cudaError_t launch_kv16_append(bool interleaved, const RotaryParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv16_keep(const Kv16KeepParams& p, cudaStream_t stream);

// Rows of a part in the workspace for T query tokens, workspace bytes, launch.
int kv16_attn_rows(long long T, int group);
size_t kv16_attn_workspace(int D, int rows, int num_sms);
cudaError_t launch_kv16_attn(int D, const CUtensorMap& q, const CUtensorMap& kv, const Kv16AttnParams& p, int num_sms,
                             cudaStream_t stream);

}  // namespace fa
