// ssd_kv.h -- what the kernels of the serving loop share: status reports, the
// shape rules of the paged cache, and e4m3 conversion.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ssd.h"

namespace ssd {

__device__ __forceinline__ void report(int32_t *dev_status, int bits) {
    if (dev_status && bits) atomicOr(dev_status, bits);
}

inline bool kv_page_size_ok(int page_size) {
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

inline int log2_of(int pow2) {
    int s = 0;
    while ((1 << s) < pow2) ++s;
    return s;
}

inline bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Status of the launch just made.
inline int launched() { return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

// Sequences of a batch: those before the first whose tokens, cu[b] to cu[b + 1], would end before they begin.  What follows
// would name tokens of sequences before it.  For a whole block, room [1] for its use.
template <int kThreads>
__device__ __forceinline__ int sequences(const int32_t *cu, int B, int *room) {
    int fall = B;
#pragma unroll 8
    for (int b = threadIdx.x; b < B; b += kThreads)
        if (cu[b + 1] < cu[b]) fall = min(fall, b);
    if (!__syncthreads_or(fall < B)) return B;
    if (threadIdx.x == 0) *room = B;
    __syncthreads();
    if (fall < B) atomicMin(room, fall);
    __syncthreads();
    fall = *room;
    __syncthreads();
    return fall;
}

// Two values as e4m3, `lo` in the low byte: nearest, ties to even, magnitudes beyond
// 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes as halves (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t halves_of_e4m3x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}

}  // namespace ssd
