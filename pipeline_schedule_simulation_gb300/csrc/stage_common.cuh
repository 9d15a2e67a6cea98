// stage_common.cuh -- what the pipeline-stage operators (ppstage.h) share.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.cuh"
#include "ppstage.h"

namespace pps {

constexpr size_t kStageAlign = 256;
inline size_t stage_align(size_t x) { return (x + kStageAlign - 1) / kStageAlign * kStageAlign; }

// Carves a workspace in order; with a null base it only adds up the bytes.
struct Carve {
    unsigned char *base;
    size_t used = 0;
    template <class T>
    T *take(int64_t n) {
        T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += stage_align((size_t)n * sizeof(T));
        return p;
    }
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Rows that 16-byte accesses may read: base and row stride both multiples of
// 16 bytes (a single row needs only its base).
inline bool rows_aligned(const void *p, int64_t stride, int64_t rows, int elem) {
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || (stride * elem & 15) == 0);
}

int sm_count();  // of the current device

// Lets a kernel use `bytes` of dynamic shared memory, once per device (`ready`
// is the kernel's own).
template <class K>
int allow_smem(K kernel, int bytes, std::atomic<uint64_t> &ready) {
    int dev = 0;
    PPS_CUDA_TRY(cudaGetDevice(&dev));
    if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        PPS_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return PP_OK;
}

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Round to nearest even, as the type's conversion does.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return (uint32_t)__bfloat16_as_ushort(v.x) | (uint32_t)__bfloat16_as_ushort(v.y) << 16;
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace pps
