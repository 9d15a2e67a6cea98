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

// A launch that may start while the kernel before it on the stream is still
// running: the kernel calls after_previous() before it touches memory, which
// waits until that one is done.  cluster: blocks that form a cluster.
template <class... P, class... A>
int launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, int cluster,
                 const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
    cfg.attrs = at, cfg.numAttrs = cluster > 1 ? 2 : 1;
    PPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return PP_OK;
}
template <class... P, class... A>
int launch_after(void (*kernel)(P...), int64_t grid, int threads, int smem, cudaStream_t stream, int cluster,
                 const A &...args) {
    return launch_after(kernel, dim3((unsigned)grid), threads, smem, stream, cluster, args...);
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the kernel after this one take free places on the SMs and wait there.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// 2^x to 2 units in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The same with results below 2^-126 (a gradient may consist of them).
__device__ __forceinline__ float exp2_full(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace pps
