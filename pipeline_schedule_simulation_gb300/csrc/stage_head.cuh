// stage_head.cuh -- what the kernels over a large vocabulary share: sums of
// exponentials, few tokens against the rows of w, operands as products read them.
#pragma once

#include "stage_kept.cuh"
#include "stage_product.cuh"

namespace pps {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

// The reference point of a sum of exponentials: the largest logit, or 0 where
// that is infinite (so that inf - inf never appears).
__device__ __forceinline__ float ref_of(float m) { return isinf(m) ? 0.f : m; }

// A sum of exponentials relative to ref_of(m), taken relative to `r` (an empty
// one stays empty).
__device__ __forceinline__ float rebase(float s, float m, float r) {
    return s == 0.f ? 0.f : s * exp2_fast((ref_of(m) - r) * kLog2e);
}

// x, or `least` where that is more; NaN stays.
__device__ __forceinline__ float not_below(float x, float least) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
    return y;
}
// Where a probability in 32 bits is 0 (e^-104), and its logarithm, which it is multiplied by, may be infinite.
constexpr float kNoLog = -128.f;

__device__ __forceinline__ bool inside(int64_t target, int64_t V) { return target >= 0 && target < V; }

// ---- few tokens: w is read once, by the row

// One or two tokens are two multiplications for every 2 bytes of w: a warp takes
// 4 rows of w at a time straight from memory, the lanes 8 columns each, against
// the tokens in shared memory as 32-bit floats.  Rows need no alignment (as a
// product, rows that TMA cannot load are copied first).  The loss of one token on
// 131072 x 4096 takes 167 us, 94 % of the measured bandwidth (275 us with rows of
// 4095), on 32000 x 2048 28 us with the join of the pieces, 34 us as a product.
// Four tokens are 313 us on 131072 x 4096 and 193 us as a product, so the limit
// is two.
constexpr int kFewTokens = 2, kFewFloats = 16384, kFewRows = 4, kFewWarps = 8, kFewBlocks = 4;

// The tokens into shared memory, [NT][2][chunks]: the two quads of each 8 columns apart.
template <int NT>
__device__ __forceinline__ void few_load(float4 *xs, const uint16_t *x, int64_t stride_x, int T, int H) {
    const int chunks = (H + 7) / 8;
    for (int i = threadIdx.x; i < NT * chunks; i += 32 * kFewWarps) {
        const int t = i / chunks, c = i - t * chunks;
        float v[8] = {};
        if (t < T) load8_bf16<false>(x + t * stride_x + c * 8, H - c * 8, v);
        xs[(2 * t) * chunks + c] = make_float4(v[0], v[1], v[2], v[3]);
        xs[(2 * t + 1) * chunks + c] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
}
// Products with rows first .. last-1 of w, a warp's, kFewRows at a time: take(v0, acc) with the lanes' parts of the sums
// (rows from `last` on are copies of the last).
template <int NT, bool VEC, class Take>
__device__ __forceinline__ void few_dots(const float4 *xs, const uint16_t *w, int64_t stride_w, int H, int64_t first,
                                           int64_t last, const Take &take) {
    const int chunks = (H + 7) / 8, lane = threadIdx.x & 31;
    for (int64_t v0 = first; v0 < last; v0 += kFewRows) {
        const uint16_t *row[kFewRows];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) row[r] = w + min(v0 + r, last - 1) * stride_w;
        float acc[kFewRows][NT] = {};
#pragma unroll 2
        for (int c = lane; c < chunks; c += 32) {
            Raw8 q[kFewRows];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) q[r] = load8<VEC>(row[r] + c * 8, H - c * 8);
            float4 a[NT], b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) a[t] = xs[2 * t * chunks + c], b[t] = xs[(2 * t + 1) * chunks + c];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                float u[8];
                widen(q[r], u);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float z = acc[r][t];
                    z = fmaf(u[0], a[t].x, z), z = fmaf(u[1], a[t].y, z), z = fmaf(u[2], a[t].z, z);
                    z = fmaf(u[3], a[t].w, z), z = fmaf(u[4], b[t].x, z), z = fmaf(u[5], b[t].y, z);
                    acc[r][t] = fmaf(u[7], b[t].w, fmaf(u[6], b[t].z, z));
                }
            }
        }
        take(v0, acc);
    }
}
// Logits of rows first .. last-1 of w: take(t, v, l) in all lanes, v ascending.
template <int NT, bool VEC, class Take>
__device__ __forceinline__ void few_logits(const float4 *xs, const uint16_t *w, int64_t stride_w, int H, int64_t first,
                                           int64_t last, const Take &take) {
    few_dots<NT, VEC>(xs, w, stride_w, H, first, last, [&](int64_t v0, const float (&acc)[kFewRows][NT]) {
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float l = acc[r][t];
#pragma unroll
                for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
                if (v0 + r < last) take(t, v0 + r, l);
            }
        }
    });
}

inline bool few_tokens(int64_t T, int64_t H) { return T <= kFewTokens && T * round_up(H, 8) <= kFewFloats; }

// Rows of w to a warp: all blocks run at once, as many to an SM as its 228 KB of
// shared memory hold (with the `own` bytes of its sums and what the SM takes for each).
inline int64_t few_rows(int64_t T, int64_t V, int64_t H, int64_t own) {
    const int64_t each = T * ceil_div(H, 8) * 32 + own + 1024, fit = 228 * 1024 / each;
    return ceil_div(V, (int64_t)sm_count() * (fit < kFewBlocks ? fit : kFewBlocks) * kFewWarps);
}

// ---- host side

inline int check_head(const void *x, int64_t sx, const void *w, int64_t sw, const void *target, int64_t T, int64_t V,
               int64_t H) {
    if (T < 0 || V < 1 || H < 1) return PP_ERR_ARG;
    if (T > PP_STAGE_MAX_ROWS || V > PP_STAGE_MAX_VOCAB || H > PP_STAGE_MAX_WIDTH) return PP_ERR_SIZE;
    if (!w || ((uintptr_t)w & 1) || sw < H) return PP_ERR_ARG;
    if (T > 0 && (!x || !target || ((uintptr_t)x & 1) || ((uintptr_t)target & 7) || sx < H)) return PP_ERR_ARG;
    return PP_OK;
}

// An operand as the products read it: in place, or as a copy whose rows start on
// 128 bytes.  Rows that TMA cannot load (not aligned to 16 bytes) are always
// copied.  Rows that it can but that straddle 128-byte lines make the loads
// slower; a copy costs 4 bytes an element and pays once enough row tiles of the
// other operand pass over it: w 50257 x 1000 takes 25 us to copy, and the loss
// of 777 tokens (4 row tiles) 94 us in place and 70 us from the copy.
constexpr int64_t kCopyFrom = 8;
struct Aligned {
    uint16_t *copy;  // null: in place
    Matrix at;
};
inline Aligned aligned(Carve &c, const uint16_t *p, int64_t stride, int64_t rows, int64_t H, int64_t passes) {
    const bool lines = rows <= 1 || (((uintptr_t)p & 127) == 0 && stride % 64 == 0);
    if (rows_aligned(p, stride, rows, 2) && (lines || passes < kCopyFrom)) return {nullptr, in_rows(p, stride)};
    const int64_t ld = round_up(H, 64);
    uint16_t *q = c.take<uint16_t>(rows * ld);
    return {q, in_rows(q, ld)};
}

inline int copy_if(const Aligned &a, const uint16_t *p, int64_t stride, int64_t rows, int64_t H, cudaStream_t stream) {
    return a.copy ? launch_copy_rows(p, stride, rows, H, nullptr, 0, nullptr, a.copy, a.at.ld, 64, stream) : PP_OK;
}

}  // namespace
}  // namespace pps
