// stage_kept.cuh -- the 8-bit checkpoint format, used by every kernel that
// writes or reads one.
//
// 64 columns of a row share the step 2^e with e = floor(log2 a) - 6 for the
// largest magnitude a, so a / 2^e lies in [64, 128) and q = rint(x / 2^e) fits
// 8 bits: only a value that rounds to 128 is held as 127, half a step off like
// any other tie.  The error is at most half a step, a/128 at most.  A step that is a
// power of two costs up to one bit against a / 127, and makes q 2^e a bf16
// number: the backward pass multiplies exactly what was kept.
#pragma once

#include "stage_common.cuh"

namespace pps {

constexpr int kBlock = PP_STAGE_BLOCK;
constexpr int kMinExp = -126;  // keeps 2^e and 2^-e normal
constexpr int kNonfinite = PP_STAGE_NONFINITE;

__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of a block from its largest magnitude's bits (as a non-negative
// 32-bit float, so that whole-number order is magnitude order and NaN is
// largest).
__device__ __forceinline__ int block_exp(uint32_t amax_bits) {
    const int k = (int)(amax_bits >> 23);
    if (k == 255) return kNonfinite;
    const int e = k - 127 - 6;  // a subnormal magnitude (k = 0) falls under kMinExp as well
    return e < kMinExp ? kMinExp : e;
}

// q of one value given 2^-e (0 for a non-finite block).
__device__ __forceinline__ int quantize(float x, float inv) {
    const float r = fminf(fmaxf(rintf(x * inv), -127.f), 127.f);
    return inv == 0.f ? 0 : (int)r;
}

__device__ __forceinline__ float inv_step(int e) { return e == kNonfinite ? 0.f : two_to(-e); }
__device__ __forceinline__ float step_of(int e) { return e == kNonfinite ? __uint_as_float(0x7FC00000u) : two_to(e); }

// Packs the 8 consecutive columns that this lane holds; the 8 lanes of an
// aligned group of 8 hold one block (columns past the row's end are 0).
// Returns the 8 bytes and the exponent (the same in all 8 lanes).
__device__ __forceinline__ uint2 pack8(const float (&v)[8], int &e) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 4; o; o >>= 1) a = max(a, __shfl_xor_sync(~0u, a, o));
    e = block_exp(a);
    const float inv = inv_step(e);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(quantize(v[j], inv) & 0xFF) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}

// The 8 values that 8 bytes stand for.
__device__ __forceinline__ void unpack8(uint2 b, int e, float (&v)[8]) {
    const float step = step_of(e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = j < 4 ? b.x : b.y;
        v[j] = (float)(int8_t)(w >> (8 * (j & 3))) * step;
    }
}

// 8 consecutive elements at p, of which `left` exist (all 8 in the vector form).
template <bool VEC>
__device__ __forceinline__ void load8_bf16(const uint16_t *p, int64_t left, float (&v)[8]) {
    if (VEC && left >= 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? bf16_to_f32(p[j]) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8_bf16(uint16_t *p, int64_t left, const float (&v)[8]) {
    if (VEC && left >= 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(f32_to_bf16x2(v[0], v[1]), f32_to_bf16x2(v[2], v[3]),
                                                   f32_to_bf16x2(v[4], v[5]), f32_to_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = f32_to_bf16(v[j]);
    }
}
template <bool VEC>
__device__ __forceinline__ uint2 load8_bytes(const int8_t *p, int64_t left) {
    if (VEC && left >= 8) return *reinterpret_cast<const uint2 *>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < left) w[j >> 2] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}
template <bool VEC>
__device__ __forceinline__ void store8_bytes(int8_t *p, int64_t left, uint2 b) {
    if (VEC && left >= 8) {
        *reinterpret_cast<uint2 *>(p) = b;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = (int8_t)((j < 4 ? b.x : b.y) >> (8 * (j & 3)));
    }
}

// Checkpoint rows that 8-byte accesses may use.
inline bool kept_aligned(const void *q, int64_t stride, int64_t rows) {
    return ((uintptr_t)q & 7) == 0 && (rows <= 1 || (stride & 7) == 0);
}

int launch_unpack(const int8_t *q, int64_t stride_q, const int8_t *e, int64_t stride_e, int64_t T, int64_t H,
                  uint16_t *x, int64_t stride_x, cudaStream_t stream);

}  // namespace pps
