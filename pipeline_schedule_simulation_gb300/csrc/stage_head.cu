// stage_head.cu -- softmax cross entropy of the last stage over a large
// vocabulary, and its gradients, without keeping the logits.
//
// Forward.  l = x w^T is taken tile by tile; of each token's part of a
// vocabulary tile (two pieces) only the largest logit and the sum of
// exponentials relative to it leave the product, and a second kernel joins the
// pieces of a token:
//   m = max_i m_i,  s = sum_i s_i e^(m_i - m),  lse = m + log s.
// Backward.  d = weight (softmax - onehot) is recomputed for a piece of the
// vocabulary at a time, as bf16 in the workspace, and both gradients take
// their product with it before the next piece:  dx += d w_piece,
// dw_piece = d^T x.  So the step is four products of 2 T V H, a third more
// than the gradients alone would need with the logits kept (4.3 GB in 32 bits
// at 8192 x 131072).
// d is rounded to bf16 before `scale`, by 2^-8 of each term at most: an operand
// of these products is 16 bits wide.  The many small terms' errors average out,
// but a token's term at its target, c (p - 1), is most of its gradient, and its
// error alone would put dx and dw of weighted tokens off by 2.4e-3 of their norm
// where the rounding of the results is 1.65e-3.  So what the rounding of that one
// term leaves over is kept in 32 bits and added where the products' results are
// finished: times the target's row of w to dx, times the token's row of x to the
// target's row of dw.
// Scores (GradEpi<true>, and a policy gradient through GradEpi<false>) take the
// same d and the same addition, but the argument is the loss's: on a peaked row the
// likeliest other column, or an entropy's terms, may be as large as the target's and
// stay rounded.  Logits six units wide put dx and dw off by 0.8e-3 of their norm before
// the results' own rounding (1.65e-3), 1.85e-3 with it; a row whose gradient is one
// such term by 1.65e-3, 2.3e-3 with it.  Two parts of 16 bits would hold d to 2^-16
// and take six products in place of four, forward included.
//
// The products bound both directions from a few hundred tokens on: 4096 tokens
// on 131072 x 4096 take 2.52 ms (1750 TFLOP/s; a cuBLAS product alone holds
// 1703 in a long loop on the same GPU, 1945 in a burst), the step of 8192 tokens
// 21.0 ms (1680 TFLOP/s over its four products).  For a few tokens reading w
// does: one token on 32000 x 2048 takes 28 us, its 131 MB alone 19 us.
#include <algorithm>

#include "stage_head.cuh"

namespace pps {
namespace {

struct StatsEpi {
    static constexpr bool kStore = false, kWhole = false;
    const int64_t *target;
    int64_t T, V;
    float2 *part;   // [pieces][T]: largest logit, sum of exponentials
    float *picked;  // [T]: the target's logit
    struct Row {
        int64_t target;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t) const { r.target = target[t]; }
    __device__ __forceinline__ void take(const Row &r, int64_t t, int n0, int end, int N, int piece,
                                         float (&v)[kRuns][32], float *) const {
        const int last = min(end, N);
        float top = kNegInf, s = 0.f;
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int n = n0 + i * kPieces * 32, cnt = min(32, last - n);
            if (cnt <= 0) break;
            if (cnt < 32) {  // columns that do not exist add nothing
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= cnt) v[i][j] = kNegInf;
            }
            float m[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[i][j]);
            const float was = top;
            top = fmaxf(fmaxf(top, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
            const float ref = ref_of(top);
            float e[4] = {rebase(s, was, ref), 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j) e[j & 3] += exp2_fast((v[i][j] - ref) * kLog2e);
            s = (e[0] + e[1]) + (e[2] + e[3]);
            const int64_t at = r.target - n;  // few rows have their target here
            if (at >= 0 && at < cnt) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (at == j) picked[t] = v[i][j];
            }
        }
        part[(int64_t)piece * T + t] = make_float2(top, s);
    }
};

// What a finished result gains from what the rounding of d left over; a product
// with an infinity or a NaN adds nothing (the rounded d has brought it already).
__device__ __forceinline__ float rest_times(float rest, float x) {
    const float c = rest * x;
    return fabsf(c) <= 3.402823466e38f ? c : 0.f;
}
// The same for 8 columns of a row of bf16, aligned.
__device__ __forceinline__ void add_rest(float (&b)[8], float rest, const uint16_t *row) {
    const uint4 q = *reinterpret_cast<const uint4 *>(row);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) b[2 * k] += rest_times(rest, bf16_lo(w[k])), b[2 * k + 1] += rest_times(rest, bf16_hi(w[k]));
}

// What the rounding leaves over is taken for nothing up to this share of the
// term, a sixteenth of the results' own rounding: so it is for every token
// without a weight whose target is improbable.
constexpr float kNoRest = 0x1p-12f;

// The other tokens of each target, as lists: head[v] is one, next[t] the one
// after t, -1 none.  Their order is that in which the blocks of the gradient's
// product run; what is taken from them does not depend on it.
struct Lists {
    int *head, *next;
};

// d of one piece of the vocabulary: columns v0 .., as bf16 (why, and what it costs:
// above).  ENT: with what reaches the logits through the entropy, so that
// d = c (p - onehot) + b p (log p + entropy).
template <bool ENT>
struct GradEpi {
    static constexpr bool kStore = false, kWhole = true;
    const int64_t *target;
    const float *lse, *weight;
    int64_t T, V, v0;
    uint16_t *d;  // in panels of T rows
    float *rest;  // [T]: what the rounding leaves over at the target
    Lists of;     // of the piece's columns; head null: not asked for
    const float *entropy, *dentropy;  // [T], ENT only
    struct Row {
        float lse, c, b, sum;  // sum: c + b entropy
        int64_t at;  // the target's column counted from the piece's first
        bool in;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t) const {
        const int64_t g = target[t];
        r.in = inside(g, V);
        r.c = weight ? weight[t] : 1.f;
        r.lse = lse[t];
        r.at = g - v0;
        if constexpr (ENT) {
            r.b = dentropy[t];
            r.sum = r.b != 0.f ? fmaf(r.b, entropy[t], r.c) : r.c;  // a row without that gradient is not asked for its entropy
        }
    }
    __device__ __forceinline__ void take(const Row &r, int64_t t, int n0, int end, int N, int, float (&v)[kRuns][32],
                                         float *) const {
        // whether the target is in one of these runs (past N it is the next piece's)
        const int64_t off = r.at - n0;
        const bool mine = r.in && off >= 0 && r.at < min(end, N) && (off & (kPieces * 32 - 1)) < 32;
        float left = 0.f;
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int n = n0 + i * kPieces * 32;
            if (n >= end) break;
            float p[32];
            const bool here = r.at >= n && r.at < n + 32;
            if constexpr (ENT) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float l = v[i][j] - r.lse;
                    p[j] = exp2_full(l * kLog2e) * fmaf(r.b, not_below(l, kNoLog), r.sum);
                }
                if (here) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (n + j == r.at) p[j] -= r.c;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) p[j] = exp2_full((v[i][j] - r.lse) * kLog2e);
                if (here) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (n + j == r.at) p[j] -= 1.f;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) p[j] *= r.c;
            }
            if (here && mine) {
                float x = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (n + j == r.at) x = p[j];
                left = x - bf16_to_f32(f32_to_bf16(x));
                // as good as exact, or an infinity or a NaN
                if (!(fabsf(left) > kNoRest * fabsf(x) && fabsf(left) <= 1e38f)) left = 0.f;
            }
            if (!r.in || n + 32 > N) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (!r.in || n + j >= N) p[j] = 0.f;
            }
            store_bf16(d + (int64_t)(n >> 6) * (T * 64) + t * 64 + (n & 63), p);
        }
        if (mine) rest[t] = left;
        if (left != 0.f && of.head) of.next[t] = atomicExch(of.head + r.at, (int)t);
    }
};

// dx: pieces add up in 32 bits; the last one adds what the rounding left over
// and writes the result.  A row that is left out is 0, whatever w holds.
struct DxEpi {
    static constexpr bool kStore = true, kWhole = false;
    static constexpr Side kSide = kEveryRow;
    float *acc;  // [T][ld_acc], ld_acc a multiple of 4
    uint16_t *dx;
    const int64_t *target;
    const float *rest;
    const uint16_t *w;  // rows aligned to 16 bytes
    int64_t V, ld_acc, ld, ld_w;
    float scale;
    bool first, last, vec;
    struct Row {
        int at;      // the target, -1 before the last piece and where the row is left out
        float rest;  // at the target
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t) const {
        const int64_t g = target[t];
        r.at = last && inside(g, V) ? (int)g : -1;
        r.rest = r.at >= 0 ? rest[t] : 0.f;
    }
    __device__ __forceinline__ Row of_lane(const Row &r, int lane) const {
        return {__shfl_sync(~0u, r.at, lane), __shfl_sync(~0u, r.rest, lane)};
    }
    __device__ __forceinline__ void finish(const Row &r, int64_t t, int64_t n, float (&v)[32]) const {
        float b[4][8] = {};
        if (!first) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 q = reinterpret_cast<const float4 *>(acc + t * ld_acc + n)[j];
                float *o = &b[j >> 1][4 * (j & 1)];
                o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w;
            }
        }
        if (r.rest != 0.f) {
            const uint16_t *row = w + r.at * ld_w + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) add_rest(b[j], r.rest, row + 8 * j);
        }
        const bool out = last && r.at < 0;
        const float c = last ? scale : 1.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = out ? 0.f : (v[j] + b[j >> 3][j & 7]) * c;
    }
    __device__ __forceinline__ bool narrow() const { return last; }
    __device__ __forceinline__ void row(int64_t t, int64_t n, const float (&v)[32]) const { store_bf16(dx + t * ld + n, v); }
    __device__ __forceinline__ void put(int64_t t, int64_t n, const float4 &v, int) const {
        store_quad(acc + t * ld_acc + n, v);
    }
    __device__ __forceinline__ float with(const Row &r, int64_t t, int64_t n) const {
        const float x = r.rest != 0.f ? bf16_to_f32(w[r.at * ld_w + n]) : 0.f;
        return (first ? 0.f : acc[t * ld_acc + n]) + rest_times(r.rest, x);
    }
    __device__ __forceinline__ void one(const Row &r, int64_t t, int64_t n, float v, float b, int) const {
        const float s = v + b;
        if (last) dx[t * ld + n] = r.at >= 0 ? f32_to_bf16(s * scale) : 0;
        else acc[t * ld_acc + n] = s;
    }
};

// dw.  A row with a list of tokens waits for what the rounding left over: as bf16
// it is also put aside in 32 bits, and written again by k_target_rows; in 32 bits
// it is added to there.  (The walk along the list here would hold up a warp's
// other 31 rows: the gradients of 777 weighted tokens on 50257 x 1000 took 314 us
// that way, 258 us this way, and 244 us without what is left over.)
struct DwEpi {
    static constexpr bool kStore = true, kWhole = false;
    static constexpr Side kSide = kSomeRows;
    uint16_t *dw16;  // one of the two
    float *dw32, *aside;
    const int *head;  // of the piece's rows
    int64_t ld, ld_aside;
    float scale;
    bool by_token, add, vec;
    struct Row {
        int aside;  // the row among those put aside, or -1
    };
    __device__ __forceinline__ void begin(Row &r, int64_t m) const {
        const int t = dw16 ? head[m] : -1;
        r.aside = t < 0 || by_token ? t : (int)m;
    }
    __device__ __forceinline__ bool apart(const Row &r) const { return r.aside >= 0; }
    __device__ __forceinline__ Row of_lane(const Row &r, int lane) const { return {__shfl_sync(~0u, r.aside, lane)}; }
    __device__ __forceinline__ void finish(const Row &r, int64_t m, int64_t n, float (&v)[32]) const {
        if (r.aside >= 0) {
            float *p = aside + r.aside * ld_aside + n;
#pragma unroll
            for (int j = 0; j < 8; ++j) store_quad(p + 4 * j, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= scale;
        if (add) add_f32(v, dw32 + m * ld + n);
    }
    __device__ __forceinline__ bool narrow() const { return dw16 != nullptr; }
    __device__ __forceinline__ void row(int64_t m, int64_t n, const float (&v)[32]) const { store_bf16(dw16 + m * ld + n, v); }
    __device__ __forceinline__ void put(int64_t m, int64_t n, const float4 &v, int) const { store_quad(dw32 + m * ld + n, v); }
    __device__ __forceinline__ float with(const Row &, int64_t m, int64_t n) const { return add ? dw32[m * ld + n] : 0.f; }
    __device__ __forceinline__ void one_apart(const Row &r, int64_t n, float v) const { aside[r.aside * ld_aside + n] = v; }
    __device__ __forceinline__ void one(const Row &, int64_t m, int64_t n, float v, float b, int) const {
        if (dw16) dw16[m * ld + n] = f32_to_bf16(v * scale);
        else dw32[m * ld + n] = v * scale + b;
    }
};

// A block finishes 2048 columns of a row of dw that has a list: its tokens' rows
// of x times what the rounding of d left over, added in the order of the tokens.
// With more than kListed tokens nothing is added: so many errors average out, to
// a third of one token's and less, and the walk stays short.  The kernel is a
// chain of loads, so all that a list of one token needs, as most are, is on its
// way before it is known whether there are more: 777 rows of 1000 take 4.7 us, 2048 of 2048 8 us.
constexpr int kListed = 8, kTargetThreads = 256;
struct TargetRows {
    const int64_t *target;
    const float *rest, *aside;
    const uint16_t *x;  // in panels of T rows
    Lists of;           // of the piece's rows
    int64_t T, v0, n, H, ld, ld_aside;
    uint16_t *dw16;
    float *dw32, scale;
    bool by_token, vec;
};
__global__ void __launch_bounds__(kTargetThreads) k_target_rows(const TargetRows a) {
    let_next_start();
    after_previous();
    const int64_t row = blockIdx.x, c = ((int64_t)blockIdx.y * kTargetThreads + threadIdx.x) * 8;
    if (c >= a.H) return;
    // by token: one of a list's tokens is its head; else every row is looked at
    const int64_t v = a.by_token ? a.target[row] - a.v0 : row;
    const float r0 = a.by_token ? a.rest[row] : 0.f;
    if (a.by_token && (v < 0 || v >= a.n || r0 == 0.f)) return;
    const int head = a.of.head[v], first = a.by_token ? (int)row : head;
    if (!a.by_token && head < 0) return;
    const uint16_t *x = a.x + (c >> 6) * (a.T * 64) + (c & 63);
    const auto add = [&](float (&s)[8], float r, const uint4 &q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) s[2 * k] += rest_times(r, bf16_lo(w[k])), s[2 * k + 1] += rest_times(r, bf16_hi(w[k]));
    };
    const uint4 q = *reinterpret_cast<const uint4 *>(x + (int64_t)first * 64);
    const float r = a.by_token ? r0 : a.rest[first];
    int u = a.of.next[first];
    // rows put aside are whole quads: of 8 columns the second 4 may not be there
    float4 p[2] = {};
    if (a.dw16) {
        const float *from = a.aside + row * a.ld_aside + c;
        p[0] = *reinterpret_cast<const float4 *>(from);
        if (c + 4 < a.H) p[1] = *reinterpret_cast<const float4 *>(from + 4);
    }
    if (head != first) return;
    float s[8] = {};
    if (u < 0) {
        add(s, r, q);
    } else {
        int t[kListed] = {first};
#pragma unroll
        for (int i = 1; i < kListed; ++i) {
            t[i] = 0x7FFFFFFF;
            if (u >= 0) t[i] = u, u = a.of.next[u];
        }
        const bool more = u >= 0;
#pragma unroll
        for (int i = 1; i < kListed; ++i)
#pragma unroll
            for (int j = i; j > 0; --j) {
                const int lo = min(t[j - 1], t[j]), hi = max(t[j - 1], t[j]);
                t[j - 1] = lo, t[j] = hi;
            }
#pragma unroll
        for (int i = 0; i < kListed; ++i)
            if (!more && t[i] != 0x7FFFFFFF) add(s, a.rest[t[i]], *reinterpret_cast<const uint4 *>(x + (int64_t)t[i] * 64));
    }
    if (a.dw16) {
        const float y[8] = {(p[0].x + s[0]) * a.scale, (p[0].y + s[1]) * a.scale, (p[0].z + s[2]) * a.scale,
                            (p[0].w + s[3]) * a.scale, (p[1].x + s[4]) * a.scale, (p[1].y + s[5]) * a.scale,
                            (p[1].z + s[6]) * a.scale, (p[1].w + s[7]) * a.scale};
        if (a.vec) store8_bf16<true>(a.dw16 + v * a.ld + c, a.H - c, y);
        else store8_bf16<false>(a.dw16 + v * a.ld + c, a.H - c, y);
    } else {
        float *o = a.dw32 + v * a.ld + c;
        if (a.vec && c + 8 <= a.H) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float4 &p = reinterpret_cast<float4 *>(o)[j];
                const float4 w = p;
                p = make_float4(fmaf(s[4 * j], a.scale, w.x), fmaf(s[4 * j + 1], a.scale, w.y),
                                fmaf(s[4 * j + 2], a.scale, w.z), fmaf(s[4 * j + 3], a.scale, w.w));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < a.H) o[j] = fmaf(s[j], a.scale, o[j]);
        }
    }
}

// ---- few tokens (few_logits): each warp keeps the statistics over its run of the
// vocabulary, a block is one piece.
template <int NT, bool VEC>
__global__ void __launch_bounds__(32 * kFewWarps, kFewBlocks) k_head_few(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                            int64_t stride_w, const int64_t *target, int T, int64_t V,
                                                            int H, int64_t rows, float2 *part, float *picked) {
    extern __shared__ float4 xs[];  // [NT][2][chunks]: the two quads of each 8 columns apart
    __shared__ float2 sh[kFewWarps][NT];
    let_next_start();
    after_previous();
    few_load<NT>(xs, x, stride_x, T, H);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = ((int64_t)blockIdx.x * kFewWarps + warp) * rows, last = min(first + rows, V);
    float m[NT], s[NT];
    int64_t want[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) m[t] = kNegInf, s[t] = 0.f, want[t] = t < T ? target[t] : -1;
    few_logits<NT, VEC>(xs, w, stride_w, H, first, last, [&](int t, int64_t v, float l) {
        const float top = fmaxf(m[t], l), ref = ref_of(top);
        s[t] = rebase(s[t], m[t], ref) + exp2_fast((l - ref) * kLog2e);
        m[t] = top;
        if (lane == 0 && want[t] == v) picked[t] = l;
    });
    if (lane == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) sh[warp][t] = make_float2(m[t], s[t]);
    }
    __syncthreads();
    if (threadIdx.x < T) {  // the warps' parts, in the order of the warps
        const int t = threadIdx.x;
        float top = kNegInf, sum = 0.f;
        for (int i = 0; i < kFewWarps; ++i) top = fmaxf(top, sh[i][t].x);
        const float ref = ref_of(top);
        for (int i = 0; i < kFewWarps; ++i) sum += rebase(sh[i][t].y, sh[i][t].x, ref);
        part[(int64_t)blockIdx.x * T + t] = make_float2(top, sum);
    }
}

// 8 tokens a block: 32 lanes along the pieces of each.  First the largest
// logit, then the sums relative to it.
__global__ void __launch_bounds__(256) k_head_join(const float2 *part, const float *picked, const int64_t *target,
                                                   int64_t pieces, int64_t T, int64_t V, float *loss, float *lse) {
    after_previous();
    __shared__ float2 sh[8][33];
    // 8 neighbouring tokens are read together; 32 runs of pieces for each
    const int col = threadIdx.x & 7, run = threadIdx.x >> 3;
    const int64_t t = (int64_t)blockIdx.x * 8 + col;
    float m = kNegInf, s = 0.f;
    if (t < T) {
        constexpr int kAhead = 8;
        for (int64_t i = run; i < pieces; i += 32 * kAhead) {
            float2 p[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t k = i + 32 * j;
                p[j] = k < pieces ? part[k * T + t] : make_float2(kNegInf, 0.f);
            }
            float mm = m;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) mm = fmaxf(mm, p[j].x);
            const float ref = ref_of(mm);
            s = rebase(s, m, ref);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) s += rebase(p[j].y, p[j].x, ref);
            m = mm;
        }
    }
    sh[col][run] = make_float2(m, s);
    __syncthreads();
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t u = (int64_t)blockIdx.x * 8 + row;
    const float2 q = sh[row][lane];
    m = q.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float ref = ref_of(m);
    s = rebase(q.y, q.x, ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0 && u < T) {
        const float l = ref + logf(s);
        if (lse) lse[u] = l;
        if (loss) loss[u] = inside(target[u], V) ? l - picked[u] : 0.f;
    }
}

// Columns of the vocabulary per piece of the backward pass: d of one piece is
// at most kPieceBytes up to 2^20 tokens.  A piece has 256 columns at least, so
// beyond them d takes 512 bytes a token (8.6 GB at 2^24).
constexpr int64_t kPieceBytes = 512ll << 20;
int64_t piece_of(int64_t T, int64_t V) {
    const int64_t cols = kPieceBytes / (2 * (T > 0 ? T : 1)) / 256 * 256;
    const int64_t most = 256 * 1024;
    int64_t p = cols < 256 ? 256 : cols > most ? most : cols;
    // equal pieces
    const int64_t n = ceil_div(V, p);
    return round_up(ceil_div(V, n), 256);
}

struct ForwardSpace {
    Aligned x, w;
    float2 *part;
    float *picked;
    bool few;
    ProductPlan plan;
    int64_t pieces;
    size_t bytes;
};
ForwardSpace forward_space(void *ws, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, int64_t T,
                           int64_t V, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    ForwardSpace s{};
    s.few = few_tokens(T, H);
    if (s.few) {
        s.pieces = ceil_div(V, few_rows(T, V, H, kFewWarps * kFewTokens * 8) * kFewWarps);
    } else {
        s.x = aligned(c, x, sx, T, H, ceil_div(V, 256));
        s.w = aligned(c, w, sw, V, H, ceil_div(T, 256));
        s.plan = plan_product(T, V, H, false, false);
        s.pieces = kPieces * s.plan.nt;
    }
    s.part = c.take<float2>(s.pieces * T);
    s.picked = c.take<float>(T);
    s.bytes = c.used;
    return s;
}

struct BackwardSpace {
    Aligned w;
    uint16_t *x, *d;  // in panels: x with the rows that are left out at 0, d of one piece
    float *acc, *parts, *rest, *aside;
    Lists of;
    int64_t piece, ld_acc;  // ld_acc: of the rows put aside too
    size_t bytes;
};
BackwardSpace backward_space(void *ws, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, int64_t T,
                             int64_t V, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    BackwardSpace s;
    s.piece = piece_of(T, V);
    s.ld_acc = round_up(H, 4);
    s.w = aligned(c, w, sw, V, H, ceil_div(T, 256));
    s.x = c.take<uint16_t>(T * round_up(H, 64));
    s.d = c.take<uint16_t>(T * s.piece);
    s.rest = c.take<float>(T);
    s.of = {c.take<int>(V), c.take<int>(T)};
    s.aside = c.take<float>((s.piece < V ? std::min(T, s.piece) : std::min(T, V)) * s.ld_acc);
    s.acc = c.take<float>(s.piece < V ? T * s.ld_acc : 0);
    int64_t parts = 0;  // the last piece may be shorter than the others
    for (const int64_t n : {s.piece < V ? s.piece : V, V - (V - 1) / s.piece * s.piece}) {
        parts = std::max(parts, part_floats(T, H, n));
        parts = std::max(parts, part_floats(n, H, T));
    }
    s.parts = c.take<float>(parts);
    s.bytes = c.used;
    return s;
}

}  // namespace
}  // namespace pps

using namespace pps;

extern "C" size_t pp_stage_head_forward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                  int64_t stride_w, int64_t T, int64_t V, int64_t H) {
    if (T < 1 || V < 1 || H < 1) return 0;
    return forward_space(nullptr, x, stride_x, w, stride_w, T, V, H).bytes;
}

extern "C" int pp_stage_head_forward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                     const int64_t *target, int64_t T, int64_t V, int64_t H, float *loss,
                                     float *lse, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const int rc = check_head(x, stride_x, w, stride_w, target, T, V, H);
    if (rc != PP_OK) return rc;
    if (T == 0) return PP_OK;
    if ((!loss && !lse) || ((uintptr_t)loss & 3) || ((uintptr_t)lse & 3)) return PP_ERR_ARG;
    const ForwardSpace s = forward_space(workspace, x, stride_x, w, stride_w, T, V, H);
    if (!workspace || ((uintptr_t)workspace & (kStageAlign - 1)) || workspace_bytes < s.bytes) return PP_ERR_ARG;
    int rp = PP_OK;
    if (s.few) {
        const bool vec = rows_aligned(w, stride_w, V, 2);
        const auto kernel = T == 1 ? (vec ? k_head_few<1, true> : k_head_few<1, false>)
                                   : (vec ? k_head_few<2, true> : k_head_few<2, false>);
        static std::atomic<uint64_t> ready[4];
        rp = allow_smem(kernel, kFewFloats * 4, ready[2 * (T - 1) + vec]);
        if (rp == PP_OK)
            rp = launch_after(kernel, s.pieces, 32 * kFewWarps, (int)(T * ceil_div(H, 8) * 32), stream, 1, x, stride_x, w,
                              stride_w, target, (int)T, V, (int)H, few_rows(T, V, H, kFewWarps * kFewTokens * 8), s.part, s.picked);
    } else {
        rp = copy_if(s.x, x, stride_x, T, H, stream);
        if (rp == PP_OK) rp = copy_if(s.w, w, stride_w, V, H, stream);
        if (rp == PP_OK)
            rp = launch_product<kRowsK, kRowsK>(s.x.at, s.w.at, T, V, H, StatsEpi{target, T, V, s.part, s.picked}, s.plan,
                                                stream);
    }
    if (rp != PP_OK) return rp;
    return launch_after(k_head_join, ceil_div(T, 8), 256, 0, stream, 1, (const float2 *)s.part, (const float *)s.picked,
                        target, s.pieces, T, V, loss, lse);
}

extern "C" size_t pp_stage_head_backward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                   int64_t stride_w, int64_t T, int64_t V, int64_t H) {
    if (T < 1 || V < 1 || H < 1) return 0;
    return backward_space(nullptr, x, stride_x, w, stride_w, T, V, H).bytes;
}

// entropy, dentropy: both null, or what GradEpi<true> reads.
static int head_backward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w, const int64_t *target,
                         const float *lse, const float *weight, const float *entropy, const float *dentropy, float scale,
                         int64_t T, int64_t V, int64_t H, uint16_t *dx, int64_t stride_dx, void *dw, int64_t stride_dw,
                         int dw_float, int dw_add, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const int rc = check_head(x, stride_x, w, stride_w, target, T, V, H);
    if (rc != PP_OK) return rc;
    if (!dw && (T > 0 && !dx)) return PP_ERR_ARG;
    if (dw && (stride_dw < H || ((uintptr_t)dw & (dw_float ? 3 : 1)) || (dw_add && !dw_float))) return PP_ERR_ARG;
    if (T > 0 && (!lse || ((uintptr_t)lse & 3) || ((uintptr_t)weight & 3) || (dx && (stride_dx < H || ((uintptr_t)dx & 1))))) return PP_ERR_ARG;
    if (T == 0) {  // no token: dw is 0, or what it was
        if (dw && !dw_add) {
            const size_t e = dw_float ? 4 : 2;
            PPS_CUDA_TRY(cudaMemset2DAsync(dw, stride_dw * e, 0, H * e, V, stream));
        }
        return PP_OK;
    }
    const BackwardSpace s = backward_space(workspace, x, stride_x, w, stride_w, T, V, H);
    if (!workspace || ((uintptr_t)workspace & (kStageAlign - 1)) || workspace_bytes < s.bytes) return PP_ERR_ARG;
    // with dw every list is emptied
    int rp = launch_copy_rows(x, stride_x, T, H, target, V, dw ? s.of.head : nullptr, s.x, 64, T * 64, stream);
    if (rp == PP_OK) rp = copy_if(s.w, w, stride_w, V, H, stream);
    const bool vec_dx = dx && rows_aligned(dx, stride_dx, T, 2), vec_dw = dw && rows_aligned(dw, stride_dw, V, dw_float ? 4 : 2);
    const Matrix xm = in_panels(s.x, T), d = in_panels(s.d, T);
    for (int64_t v0 = 0; v0 < V && rp == PP_OK; v0 += s.piece) {
        const int64_t n = V - v0 < s.piece ? V - v0 : s.piece;
        const Matrix wp = in_rows(s.w.at.p + v0 * s.w.at.ld, s.w.at.ld);
        const Lists of{dw ? s.of.head + v0 : nullptr, s.of.next};
        rp = dentropy ? whole_product<kPanelsK, kRowsK>(
                            xm, wp, T, n, H,
                            GradEpi<true>{target, lse, weight, T, V, v0, s.d, s.rest, of, entropy, dentropy}, stream)
                      : whole_product<kPanelsK, kRowsK>(
                            xm, wp, T, n, H,
                            GradEpi<false>{target, lse, weight, T, V, v0, s.d, s.rest, of, nullptr, nullptr}, stream);
        if (rp == PP_OK && dx) {
            const DxEpi epi{s.acc, dx, target, s.rest, s.w.at.p, V, s.ld_acc, stride_dx, s.w.at.ld, scale, v0 == 0,
                            v0 + n == V, vec_dx};
            // the copy's rows are whole panels; so are w's own if H is
            rp = s.w.copy || H % 64 == 0
                     ? product_in_parts<kPanelsK, kPanelsMN>(d, wp, T, H, n, epi, s.parts, stream)
                     : product_in_parts<kPanelsK, kRowsMN>(d, wp, T, H, n, epi, s.parts, stream);
        }
        if (rp == PP_OK && dw) {
            uint16_t *dw16 = dw_float ? nullptr : (uint16_t *)dw + v0 * stride_dw;
            float *dw32 = dw_float ? (float *)dw + v0 * stride_dw : nullptr;
            const bool by_token = T <= n;  // rows put aside: by their list's head, or all that the piece has
            const DwEpi epi{dw16, dw32, s.aside, of.head, stride_dw, s.ld_acc, scale, by_token, dw_add != 0, vec_dw};
            rp = product_in_parts<kPanelsMN, kPanelsMN>(d, xm, n, H, T, epi, s.parts, stream);
            if (rp == PP_OK)
                rp = launch_after(k_target_rows, dim3((unsigned)(by_token ? T : n), (unsigned)ceil_div(H, 8 * kTargetThreads)),
                                  kTargetThreads, 0, stream, 1,
                                  TargetRows{target, s.rest, s.aside, s.x, of, T, v0, n, H, stride_dw, s.ld_acc, dw16, dw32,
                                             scale, by_token, vec_dw});
        }
    }
    return rp;
}

extern "C" int pp_stage_head_backward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                      const int64_t *target, const float *lse, const float *weight, float scale,
                                      int64_t T, int64_t V, int64_t H, uint16_t *dx, int64_t stride_dx, void *dw,
                                      int64_t stride_dw, int dw_float, int dw_add, void *workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
    return head_backward(x, stride_x, w, stride_w, target, lse, weight, nullptr, nullptr, scale, T, V, H, dx, stride_dx, dw,
                         stride_dw, dw_float, dw_add, workspace, workspace_bytes, stream);
}

extern "C" size_t pp_stage_score_backward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                    int64_t stride_w, int64_t T, int64_t V, int64_t H) {
    return pp_stage_head_backward_workspace(x, stride_x, w, stride_w, T, V, H);
}

// logp is minus the loss: the loss's gradients, weighted with what reaches logp, and at the end minus that.
extern "C" int pp_stage_score_backward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                       const int64_t *target, const float *lse, const float *dlogp,
                                       const float *entropy, const float *dentropy, int64_t T, int64_t V, int64_t H,
                                       uint16_t *dx, int64_t stride_dx, void *dw, int64_t stride_dw, int dw_float,
                                       int dw_add, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (T > 0 && (!dlogp || (dentropy && !entropy) || ((uintptr_t)entropy & 3) || ((uintptr_t)dentropy & 3))) return PP_ERR_ARG;
    return head_backward(x, stride_x, w, stride_w, target, lse, dlogp, entropy, dentropy, -1.f, T, V, H, dx, stride_dx, dw,
                         stride_dw, dw_float, dw_add, workspace, workspace_bytes, stream);
}
