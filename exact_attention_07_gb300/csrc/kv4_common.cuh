// Device helpers of the 4-bit cache kernels: codes, scales, checked lookups.
#pragma once

#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx_sm103.cuh"

namespace fa {

// Two e2m1 codes of byte I of w to fp16 (low nibble in the low half): exact.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    if constexpr (I == 0)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(w));
    else
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(w));
    return r;
}

// Two e4m3 scales to fp16: exact (at most 448, at least 2^-9).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Slot and length of the call's sequence i; a bad slot or length is latched
// and counts as an empty sequence.
__device__ __forceinline__ int kv4_sequence(const Kv4Cache& c, int i, int& slot)
{
    slot = c.ids ? c.ids[i] : i;
    int len = -1;
    if (slot >= 0 && slot < c.num_slots) len = c.lens[slot];
    if (len < 0 || (long long)len > ((long long)c.table_width << c.page_shift)) {
        atomicOr(c.err, 2);
        slot = 0;
        len = 0;
    }
    return len;
}

// Byte offset of the unit of position pos of KV head h.
__device__ __forceinline__ long long kv4_unit(const Kv4Cache& c, int D, int page, int h, int pos)
{
    const int units = 1 << (c.page_shift - 4);
    return (((long long)page * c.Hkv + h) * units + ((pos >> 4) & (units - 1))) * (18 * D);
}

// A second kernel that is launched while the first still runs (programmatic
// dependent launch): its launch latency is hidden, and wait_for_primary()
// returns once the first has ended and its writes are visible.
__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 blocks, int threads, cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace fa
