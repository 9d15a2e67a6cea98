// stage_kept.cuh -- the 8-bit checkpoint format, used by every kernel that
// writes or reads one.
//
// 64 columns of a row share the step 2^e with e = floor(log2 a) - 6 for the
// largest magnitude a, so a / 2^e lies in [64, 128) and q = rint(x / 2^e) fits
// 8 bits: only a value that rounds to 128 is held as 127, half a step off like
// any other tie.  The error is at most half a step, a/128 at most.  A step that is a
// power of two costs up to one bit against a / 127, and makes q 2^e a bf16
// number: the backward pass multiplies exactly what was kept.
// The step is 2^-126 at least, so that it is a normal number: where a < 2^-120
// the error is still up to 2^-127, and a block whose a is no more than that is
// held as zeros.
#pragma once

#include <cstring>

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

__device__ __forceinline__ float inv_step(int e) { return two_to(-e); }
__device__ __forceinline__ float step_of(int e) { return e == kNonfinite ? __uint_as_float(0x7FC00000u) : two_to(e); }

// 8 consecutive bf16 elements of a row, two to a word.
struct Raw8 {
    uint32_t w[4];
};
__device__ __forceinline__ void widen(const Raw8 &r, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(r.w[j]), v[2 * j + 1] = bf16_hi(r.w[j]);
}
__device__ __forceinline__ Raw8 narrow(const float (&v)[8]) {
    Raw8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = f32_to_bf16x2(v[2 * j], v[2 * j + 1]);
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // NaN wins
    __nv_bfloat162 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    const __nv_bfloat162 m = __hmax2_nan(x, y);
    uint32_t r;
    memcpy(&r, &m, 4);
    return r;
}

// Packs the 8 consecutive columns that this lane holds; the 8 lanes of an
// aligned group of 8 hold one block (columns past the row's end are 0).
// Returns the 8 bytes and the exponent (the same in all 8 lanes).
__device__ __forceinline__ uint2 pack8(const Raw8 &x, int &e) {
    uint32_t a = x.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < 4; ++j) a = max_bf16x2(a, x.w[j] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = 4; o; o >>= 1) a = max_bf16x2(a, __shfl_xor_sync(~0u, a, o));
    e = block_exp(max(a << 16, a & 0xFFFF0000u));
    // x / 2^e is exact, so that adding 1.5 * 2^23 rounds it to a whole number
    // (ties to even) that lies in the sum's low bits
    const float inv = e == kNonfinite ? 0.f : inv_step(e);
    constexpr float kRound = 12582912.f;
    if (e == kNonfinite) return make_uint2(0u, 0u);
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = __float_as_uint(fmaf(bf16_lo(x.w[j]), inv, kRound));
        const uint32_t hi = __float_as_uint(fmaf(bf16_hi(x.w[j]), inv, kRound));
        // the sums' low 16 bits are the whole numbers: two of them are held to +-127 at once
        b[j] = __vmins2(__vmaxs2(__byte_perm(lo, hi, 0x5410), 0xFF81FF81u), 0x007F007Fu);
    }
    return make_uint2(__byte_perm(b[0], b[1], 0x6420), __byte_perm(b[2], b[3], 0x6420));
}

// The 8 values that 8 bytes stand for, times `step`: a byte with its sign bit
// flipped becomes the low bits of 2^23, from which 2^23 + 128 is taken.
__device__ __forceinline__ void unpack8(uint2 b, float step, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = (j < 4 ? b.x : b.y) ^ 0x80808080u;
        v[j] = (__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + (j & 3))) - 8388736.f) * step;
    }
}

// 8 consecutive elements at p, of which `left` exist.  Unaligned ones are put
// together from the aligned words that hold them: a word with a byte of the
// row in it can be read whole, and no other is read.
template <bool VEC>
__device__ __forceinline__ Raw8 load8(const uint16_t *p, int64_t left) {
    Raw8 r{};
    if (VEC && left >= 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = w.x, r.w[1] = w.y, r.w[2] = w.z, r.w[3] = w.w;
    } else if (left > 0) {
        const uint32_t off = (uint32_t)((uintptr_t)p & 2) >> 1;  // halves before p in its word
        const uint32_t *a = reinterpret_cast<const uint32_t *>(p - off);
        const int n = left < 8 ? (int)left : 8;
        uint32_t w[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = 2 * j < n + (int)off ? a[j] : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.w[j] = __funnelshift_r(w[j], w[j + 1], 16 * off);
            if (2 * j + 1 >= n) r.w[j] &= 2 * j >= n ? 0u : 0xFFFFu;
        }
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, int64_t left, const Raw8 &r) {
    if (VEC && left >= 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = (uint16_t)(r.w[j >> 1] >> (16 * (j & 1)));
    }
}
template <bool VEC>
__device__ __forceinline__ void load8_bf16(const uint16_t *p, int64_t left, float (&v)[8]) {
    widen(load8<VEC>(p, left), v);
}
template <bool VEC>
__device__ __forceinline__ void store8_bf16(uint16_t *p, int64_t left, const float (&v)[8]) {
    store8<VEC>(p, left, narrow(v));
}
template <bool VEC>
__device__ __forceinline__ uint2 load8_bytes(const int8_t *p, int64_t left) {
    if (VEC && left >= 8) return *reinterpret_cast<const uint2 *>(p);
    if (left <= 0) return make_uint2(0u, 0u);
    const uint32_t off = (uint32_t)((uintptr_t)p & 3);
    const uint32_t *a = reinterpret_cast<const uint32_t *>(p - off);
    const int n = left < 8 ? (int)left : 8;
    uint32_t w[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) w[j] = 4 * j < n + (int)off ? a[j] : 0u;
    uint2 r = make_uint2(__funnelshift_r(w[0], w[1], 8 * off), __funnelshift_r(w[1], w[2], 8 * off));
    if (n < 8) {
        const uint64_t keep = (1ull << (8 * n)) - 1;
        r.x &= (uint32_t)keep, r.y &= (uint32_t)(keep >> 32);
    }
    return r;
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

// As panels or rows: element (t, c) at x[t*ld + (c/64)*panel + c%64].
int launch_unpack(const int8_t *q, int64_t stride_q, const int8_t *e, int64_t stride_e, int64_t T, int64_t H,
                  uint16_t *x, int64_t ld, int64_t panel, cudaStream_t stream);

}  // namespace pps
