// stage_score.cu -- log probabilities of given tokens over a large vocabulary,
// with the entropy and the likeliest alternatives, without keeping the logits.
// (Their gradients are those of the loss, stage_head.cu.)
//
// As in the loss, l = x w^T is taken tile by tile and of each token's part of a
// tile (two pieces of up to 128 columns) only sums leave the product:
//   m = max l,   s = sum 2^q,   u = sum q 2^q   with q = (l - m) log2 e
// and, where alternatives are asked for, the logits that may be among the k
// largest.  A second kernel joins the pieces of a token:
//   lse = m + log s,   entropy = lse - sum p l = log s - u log 2 / s.
// Both terms of the entropy are positive, so nothing cancels.
//
// Alternatives.  A thread holds its piece in registers and writes the logits that
// reach a bound below which nothing can be among the token's k largest: k classes
// of runs of 32 columns each keep the largest logit that any of their runs has
// had, and the least of these k is such a bound, since k different logits reach
// it.  It rises as tiles finish; a thread reads it a tile ahead, and an old bound
// only lets through more.  So the order in which blocks run decides what is
// written, but not what is found.  Of 131072 columns some 660 are written for each
// token with 20 alternatives: 22 of a piece in the first tiles, one in ten pieces
// at the end.
//
// The product bounds it from a few hundred tokens on: 2048 tokens on 131072 x 4096
// take 1.12 ms (1960 TFLOP/s, the measured burst rate of a library product), 4096
// with 20 alternatives 2.31 ms (1905; the join of their pieces 0.07 ms of it).
// One token on 32000 x 2048 with 8 takes 32 us, its 131 MB alone 19; two on
// 131072 x 4096 187 us, 172 without alternatives.  333 tokens on 50257 x 1000 with
// 5 take 66 us, of which the product's loads 37: 3 row tiles, whose blocks each
// load 48 KB for 128 x 256 x 64 products.  Short rows leave the tiles' ends in
// sight: 8192 tokens on 131072 x 512 take 0.87 ms, 1.44 with 5 alternatives.
#include <algorithm>
#include <cmath>

#include "stage_head.cuh"

namespace pps {
namespace {

constexpr float kNaN = __builtin_nanf("");
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTop = PP_STAGE_MAX_TOP;
static_assert(kMaxTop <= 32);  // a lane to each

// Largest logit, s and u of a piece, as above; relative to ref_of(m).
struct Stats {
    float m, s, u;
};
constexpr float kNoExp = -200.f;  // 2^q is 0 from there on; q itself may be infinite

__device__ __forceinline__ Stats rebase(const Stats &a, float r) {
    if (a.s == 0.f) return {a.m, 0.f, 0.f};
    const float d = (ref_of(a.m) - r) * kLog2e, f = exp2_fast(d);
    return {a.m, a.s * f, f == 0.f ? 0.f : f * fmaf(a.s, d, a.u)};
}
__device__ __forceinline__ Stats add(const Stats &a, const Stats &b) {
    const float top = fmaxf(a.m, b.m), ref = ref_of(top);
    const Stats x = rebase(a, ref), y = rebase(b, ref);
    return {top, x.s + y.s, x.u + y.u};
}

// An alternative: its logit and its column.
struct Found {
    float l;
    int n;
};
__device__ __forceinline__ bool before(const Found &a, const Found &b) { return a.l > b.l || (a.l == b.l && a.n < b.n); }

// Floats as whole numbers of the same order, above 0 (which stands for no bound).  -0 is taken as 0: no float that is
// larger follows it, and the search below goes by a number's successor being above it.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return u == 0 ? kNegInf : __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// What the pieces' alternatives are written to.
struct Alternatives {
    int k, slots;     // slots: of a piece, k or more, even
    float guess;      // how far below the largest of 128 the k-th lies, in distances of the runs' largest (of normal numbers)
    int64_t pieces;
    uint8_t *count;   // [T][pieces]
    Found *found;     // [T][pieces][slots]; a piece's largest first
    uint32_t *least;  // [k + 1][T]: the classes' largest logits, as ordered(), and the bound; null where all tiles run at
                      // once (a call of 90 tokens on 3600 x 512 with 5 alternatives 28 us, 32 with it)
    bool sorted;      // pieces' alternatives are in order
    bool narrow;      // every second piece is empty
};

// The bound is taken from the classes in a token's first pieces, and then in the pieces of every kEvery-th column
// tile; the others read it as a word, a tile ahead (8192 tokens on 131072 x 512 with 5 alternatives 1.53 ms with the
// classes read in every tile, 1.50 like this).
constexpr int kYoung = 16, kEvery = 8;

template <bool TOP>
struct ScoreEpi {
    static constexpr bool kStore = false, kWhole = false;
    const int64_t *target;
    int64_t T, V;
    Stats *part;    // [pieces][T]
    float *picked;  // [T]: the target's logit
    Alternatives alt;
    struct Row {
        int64_t target;
        uint32_t least;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t) const {
        r.target = target[t];
        if constexpr (TOP) r.least = alt.least ? __ldcg(alt.least + (int64_t)alt.k * T + t) : 0;
    }
    __device__ __forceinline__ uint32_t least_of(int64_t t) const {
        uint32_t a = ~0u;
#pragma unroll
        for (int j = 0; j < kMaxTop; j += 8) {
            if (j >= alt.k) break;
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = j + i < alt.k ? __ldcg(alt.least + (j + i) * T + t) : ~0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) a = min(a, b[i]);
        }
        return a;
    }
    __device__ __forceinline__ void take(const Row &r, int64_t t, int n0, int end, int N, int piece,
                                         float (&v)[kRuns][32], float *own) const {
        const int last = min(end, N);
        float run[kRuns];  // largest logits of the runs
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int cnt = last - (n0 + i * kPieces * 32);
            run[i] = cnt >= 32 ? largest(v[i]) : largest_of(v[i], cnt);
        }
        if constexpr (TOP) take_out(r, t, n0, last, piece, run, v, own);
        Stats a{kNegInf, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int n = n0 + i * kPieces * 32, cnt = min(32, last - n);
            if (cnt <= 0) break;
            if (cnt < 32) {  // they add nothing
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= cnt) v[i][j] = kNegInf;
            }
            const float top = fmaxf(a.m, run[i]), ref = ref_of(top);
            const Stats b = rebase(a, ref);
            float2 e[2] = {{b.s, 0.f}, {0.f, 0.f}}, u[2] = {{b.u, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                float2 q = __fmul2_rn(__fadd2_rn({v[i][j], v[i][j + 1]}, {-ref, -ref}), {kLog2e, kLog2e});
                q = {not_below(q.x, kNoExp), not_below(q.y, kNoExp)};
                const float2 p = {exp2_fast(q.x), exp2_fast(q.y)};
                e[j >> 1 & 1] = __fadd2_rn(e[j >> 1 & 1], p);
                u[j >> 1 & 1] = __ffma2_rn(p, q, u[j >> 1 & 1]);
            }
            a = {top, (e[0].x + e[0].y) + (e[1].x + e[1].y), (u[0].x + u[0].y) + (u[1].x + u[1].y)};
            const int64_t at = r.target - n;  // few rows have their target here
            if (at >= 0 && at < cnt) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (at == j) picked[t] = v[i][j];
            }
        }
        part[(int64_t)piece * T + t] = a;
    }
    static __device__ __forceinline__ float largest(const float (&v)[32]) {  // NaN only where all are
        float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
        return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    }
    static __device__ __forceinline__ float largest_of(const float (&v)[32], int cnt) {  // of the first ones
        float m = kNaN;
#pragma unroll
        for (int j = 0; j < 31; ++j) m = fmaxf(m, j < cnt ? v[j] : kNaN);
        return m;
    }
    // The columns of a run that exist and reach a bound, as bits.
    static __device__ __forceinline__ uint32_t reaching(float bound, const float (&v)[32], int cnt) {
        uint32_t b[4] = {};
#pragma unroll
        for (int j = 0; j < 32; ++j) b[j & 3] |= v[j] >= bound ? 1u << j : 0u;
        return ((b[0] | b[1]) | (b[2] | b[3])) & (cnt >= 32 ? ~0u : (1u << max(cnt, 0)) - 1);
    }
    // What reaches the bound is written.  Where that is more than there are slots, the bound is raised
    // by bisection until it leaves k or a few more; among equals at such a bound the first columns are written.
    // A lane's run goes through its own shared memory, so that what is written is found by its number: a branch for each
    // of 128 registers takes 80000 cycles a tile, most of them waiting for instructions.
    __device__ __forceinline__ void take_out(const Row &r, int64_t t, int n0, int last, int piece, const float (&run)[kRuns],
                                             const float (&v)[kRuns][32], float *own) const {
        const int64_t at = t * alt.pieces + piece;
        const float top = fmaxf(fmaxf(run[0], run[1]), fmaxf(run[2], run[3]));
        uint32_t low = r.least;
        if (alt.least && (low == 0 || piece < kYoung || piece / kPieces % kEvery == 0)) {
            low = max(low, least_of(t));
            if (low > r.least) atomicMax(alt.least + (int64_t)alt.k * T + t, low);
        }
        const float least = from_ordered(low);
        int c = 0;
        if (top >= least) {
            constexpr int kAll = kRuns * 32;
            uint32_t lo = ordered(least), hi = max(ordered(top), lo);
            uint32_t in[kRuns], equal[kRuns] = {};  // what is written; and what only for the first columns
            // without a bound the first guess goes by how far the runs' largest lie apart
            float down = alt.guess * (top - fminf(fminf(run[0], run[1]), fminf(run[2], run[3])));
            int n = kAll + 1;  // what reaches lo; not known yet
            for (int i = 0;; ++i) {
                uint32_t u;
                if (n > kAll) {
                    u = least == kNegInf && i < 4 ? min(max(ordered(top - down), lo), hi) : lo;
                    down *= 2;
                } else if (lo == hi) {
                    u = hi + 1;
                } else {
                    const float mid = 0.5f * (from_ordered(lo) + from_ordered(hi));
                    u = i < 12 && isfinite(mid) ? min(max(ordered(mid), lo + 1), hi) : lo + (hi - lo + 1) / 2;
                }
                const float bound = from_ordered(u);
                uint32_t b[kRuns];
                int q = 0;
#pragma unroll
                for (int r = 0; r < kRuns; ++r) {
                    b[r] = 0;
                    if (run[r] >= bound) b[r] = reaching(bound, v[r], last - (n0 + r * kPieces * 32));
                    q += __popc(b[r]);
                }
                // Above the bound that leaves too many: these, and as many equals as there is room for.  They are fewer
                // than k (at hi + 1, none or what a larger bound was tried for), so that all written have a slot.
                if (u > hi) {
#pragma unroll
                    for (int r = 0; r < kRuns; ++r) equal[r] = in[r] & ~b[r], in[r] = b[r];
                    n = q;
                    break;
                }
                if (u == lo || q >= alt.k) {
                    lo = u, n = q;
#pragma unroll
                    for (int r = 0; r < kRuns; ++r) in[r] = b[r];
                    if (n <= alt.slots) break;
                } else {
                    hi = u - 1;
                }
            }
            // the largest comes first, so that the join may leave the others unread
            Found *to = alt.found + at * alt.slots;
            int room = alt.slots - n;
            bool led = false;
            c = 1;
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                if (equal[i]) {
                    while (__popc(equal[i]) > room) equal[i] &= ~(0x80000000u >> __clz(equal[i]));
                    room -= __popc(equal[i]);
                    in[i] |= equal[i];
                }
                if (in[i]) {
                    const bool more = in[i] & (in[i] - 1);  // one alone is the run's largest
                    if (more) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) own[j * 32] = v[i][j];
                    }
                    for (uint32_t b = in[i]; b; b &= b - 1) {
                        const int j = __ffs(b) - 1;
                        const Found f{more ? own[j * 32] : run[i], n0 + i * kPieces * 32 + j};
                        const bool first = !led && f.l == top;
                        to[first ? 0 : c] = f;
                        if (first) led = true;
                        else ++c;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kRuns; ++i)
                if (alt.least && run[i] > least) atomicMax(alt.least + (int64_t)((piece * kRuns + i) % alt.k) * T + t, ordered(run[i]));
        }
        alt.count[at] = (uint8_t)c;
    }
};
static_assert(kRuns == 4);

// ---- few tokens (few_dots): a block's logits go to shared memory, and when all are
// there its threads take the statistics and each logit's place; a block is one
// piece.  (With both in the loop over the rows of w, in all lanes, two tokens on
// 131072 x 4096 with 8 alternatives took 211 us, 169 without those.)
constexpr int kFewMost = 1024;  // rows of w to a block

// Sums over the warp's lanes of M values; lane i ends with that of value i / (32 / M).
template <int M>
__device__ __forceinline__ float sum_apart(const float (&v)[M], int lane) {
    float x[M];
#pragma unroll
    for (int i = 0; i < M; ++i) x[i] = v[i];
    int o = 16;
#pragma unroll
    for (int h = M / 2; h >= 1; h /= 2, o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = upper ? x[i] : x[i + h], keep = upper ? x[i + h] : x[i];
            x[i] = keep + __shfl_xor_sync(~0u, give, o);
        }
    }
#pragma unroll
    for (; o; o >>= 1) x[0] += __shfl_xor_sync(~0u, x[0], o);
    return x[0];
}

template <int NT, bool VEC, bool TOP>
__global__ void __launch_bounds__(32 * kFewWarps, kFewBlocks)
    k_score_few(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w, const int64_t *target, int T,
                int64_t V, int H, int64_t rows, Stats *part, float *picked, const Alternatives alt) {
    extern __shared__ float4 xs[];
    __shared__ float4 quads[NT][kFewMost / 4];
    __shared__ float tops[NT][kFewWarps];
    __shared__ float2 sums[NT][kFewWarps];
    let_next_start();
    after_previous();
    few_load<NT>(xs, x, stride_x, T, H);
    constexpr int kThreads = 32 * kFewWarps, M = kFewRows * NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * kFewWarps * rows, from = first + warp * rows;
    const int all = (int)min(V - first, kFewWarps * rows);
    const auto l = [&](int t) { return reinterpret_cast<float *>(quads[t]); };
    few_dots<NT, VEC>(xs, w, stride_w, H, from, min(from + rows, V), [&](int64_t v0, const float (&acc)[kFewRows][NT]) {
        float v[M];
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = acc[i / NT][i % NT];
        const float sum = sum_apart<M>(v, lane);
        const int i = lane / (32 / M), r = i / NT, t = i % NT;  // M runs of lanes have a value each
        if (lane % (32 / M) == 0 && v0 + r < from + rows && v0 + r < V) l(t)[v0 - first + r] = sum;
    });
    if (threadIdx.x < 4 && all + threadIdx.x < kFewMost) {  // whole quads are read: no comparison finds NaN
#pragma unroll
        for (int t = 0; t < NT; ++t) l(t)[all + threadIdx.x] = kNaN;
    }
    __syncthreads();
    float m[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = kNegInf;
        for (int i = threadIdx.x; i < all; i += kThreads) m[t] = fmaxf(m[t], l(t)[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m[t] = fmaxf(m[t], __shfl_xor_sync(~0u, m[t], o));
        if (lane == 0) tops[t][warp] = m[t];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i) m[t] = fmaxf(m[t], tops[t][i]);
        const float ref = ref_of(m[t]);
        const int64_t at = t < T ? target[t] - first : -1;
        float s = 0.f, u = 0.f;
        for (int i = threadIdx.x; i < all; i += kThreads) {
            const float q = not_below((l(t)[i] - ref) * kLog2e, kNoExp), p = exp2_fast(q);
            s += p, u = fmaf(p, q, u);
            if (i == at) picked[t] = l(t)[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o), u += __shfl_xor_sync(~0u, u, o);
        if (lane == 0) sums[t][warp] = make_float2(s, u);
    }
    __syncthreads();
    if (threadIdx.x < T) {
        Stats a{m[0], 0.f, 0.f};
#pragma unroll
        for (int t = 1; t < NT; ++t)
            if (threadIdx.x == t) a.m = m[t];
        for (int i = 0; i < kFewWarps; ++i) a.s += sums[threadIdx.x][i].x, a.u += sums[threadIdx.x][i].y;
        part[(int64_t)blockIdx.x * T + threadIdx.x] = a;
    }
    if constexpr (TOP) {
        for (int t = 0; t < T; ++t) {
            const int64_t at = (int64_t)t * alt.pieces + blockIdx.x;
            const float *mine = reinterpret_cast<const float *>(quads[t]);
            int numbers = 0;
            for (int i0 = 0; i0 < all; i0 += kThreads) {
                const int i = i0 + threadIdx.x;
                const float f = i < all ? mine[i] : kNaN;
                numbers += __syncthreads_count(f == f);
                if (f != f) continue;
                int place = 0;
                for (int j = 0; j < all; j += 4) {
                    const float4 g = quads[t][j / 4];
                    place += (g.x > f || (g.x == f && j < i)) + (g.y > f || (g.y == f && j + 1 < i)) +
                             (g.z > f || (g.z == f && j + 2 < i)) + (g.w > f || (g.w == f && j + 3 < i));
                }
                if (place < alt.k) alt.found[at * alt.slots + place] = {f, (int)first + i};
            }
            if (threadIdx.x == 0) alt.count[at] = (uint8_t)min(numbers, alt.k);
        }
    }
}

// ---- the join

// With many tokens a block takes 8, a warp's lanes the pieces of each; with few a
// block takes one.  First the largest logit, then the sums relative to it, then of
// the alternatives those that reach the k-th of the lanes' largest logits (as many
// different logits do), a lane whose pieces have none left out.
// The first gives 32 lanes to a token, the second 256.  With alternatives (80
// registers: three such blocks to an SM) a token is so much to look through that
// the second stays ahead beyond the blocks that run at once.  Whole calls on
// 32000 x 256 with 5 and with 20, a block to a token against 8 tokens a block: one
// token 11.3 / 16.9 and 13.6 / 45.5 us, 456 41.6 / 48.3 and 56 / 76, 608 (four to an
// SM) 54.9 / 54.8 and 73 / 85, 900 71 / 69 and 89 / 96, 2048 127 / 109 and 162 / 142.
// Without alternatives a token is two sums: one 7.8 / 8.7 us, 3 10.4 / 10.7, 64
// 14.8 / 11.1 (on 131072 x 64 3 tokens 18.2 / 19.5, 4 19.8 / 19.5, 16 32.4 / 20.6).
constexpr int kOneToSM = 4, kOneAlone = 3;  // up to so many tokens a block each: to an SM with alternatives, in all without
constexpr int kJoinThreads = 256;

// The i-th of a lane's pieces: every 32nd, or both of every 32nd tile where a tile's second piece is empty (tiles of up
// to 32 columns): half of the lanes would have nothing else, and no k largest logits to take a bound from (16 tokens on
// 3000 x 64 with 20 alternatives 149 us by that, 22 like this; both of each tile always: 900 tokens 127 us, 43).
__device__ __forceinline__ int piece_of_lane(bool narrow, int lane, int i) {
    return narrow ? 64 * (i >> 1) + 2 * lane + (i & 1) : 32 * i + lane;
}

// Alternatives that a warp sorts at a time, and a block: all that pass the bound, but for many equals (with as many
// alternatives as lanes some hundred do).
constexpr int kKept = 256, kKeptOfBlock = 512;

// Of the n entries in shared memory, MOST at most, the first k, in order, by THREADS threads (a warp, or the block).
template <int THREADS, int MOST>
__device__ __forceinline__ int sort_kept(Found *kept, int n, int k, int thread) {
    constexpr int kEach = MOST / THREADS;
    const auto sync = [] {
        if (THREADS == 32) __syncwarp();
        else __syncthreads();
    };
    Found f[kEach];
    int place[kEach];
    sync();
#pragma unroll
    for (int i = 0; i < kEach; ++i) f[i] = kept[i * THREADS + thread], place[i] = 0;
    for (int j = 0; j < n; ++j) {
        const Found g = kept[j];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i * THREADS < n) place[i] += before(g, f[i]);
    }
    sync();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (i * THREADS + thread < n && place[i] < k) kept[place[i]] = f[i];
    sync();
    return min(n, k);
}

// How many alternatives a piece has; no more than its slots, should its block have given up and written nothing.
__device__ __forceinline__ int count_of(const Alternatives &alt, int64_t at) { return min((int)alt.count[at], alt.slots); }

struct JoinArgs {
    const Stats *part;
    const float *picked;
    const int64_t *target;
    int64_t pieces, T, V;
    float *logp, *lse, *entropy, *top_logp;
    int64_t *top_index;
};

// A warp collects and sorts the alternatives that reach `least` of one token's pieces; lanes with `skip` have none.
__device__ __forceinline__ int collect(const Alternatives &alt, int64_t pieces, int64_t t, float least, bool skip, Found *mine,
                                       int lane) {
    const int k = alt.k, slots = alt.slots;
    const Found *found = alt.found + t * pieces * slots;
    int n = 0;
    constexpr int kAhead = 4;
    for (int64_t p0 = 0; p0 < pieces; p0 += 32 * kAhead) {
        int counts[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int64_t p = p0 + piece_of_lane(alt.narrow, lane, h);
            counts[h] = !skip && p < pieces ? count_of(alt, t * pieces + p) : 0;
        }
        // slots are even in number, so that two are 16 aligned bytes
        uint4 ahead[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
            if (counts[h] > 0)
                ahead[h] = *reinterpret_cast<const uint4 *>(found + (p0 + piece_of_lane(alt.narrow, lane, h)) * slots);
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const Found *from = found + (p0 + piece_of_lane(alt.narrow, lane, h)) * slots;
            uint4 q = ahead[h];
            const int c = counts[h] > 0 && __uint_as_float(q.x) >= least ? counts[h] : 0;
            for (int e = 0; __any_sync(~0u, e < c); e += 2) {
                if (e > 0 && e < c) q = *reinterpret_cast<const uint4 *>(from + e);
                const Found f[2] = {{e < c ? __uint_as_float(q.x) : kNaN, (int)q.y}, {e + 1 < c ? __uint_as_float(q.z) : kNaN, (int)q.w}};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool is = f[i].l >= least;
                    const uint32_t in = __ballot_sync(~0u, is);
                    if (is) mine[n + __popc(in & ((1u << lane) - 1))] = f[i];
                    n += __popc(in);
                    if (n > kKept - 32) {
                        n = sort_kept<32, kKept>(mine, n, k, lane);
                        least = fmaxf(least, mine[k - 1].l);
                    }
                }
            }
        }
    }
    return sort_kept<32, kKept>(mine, n, k, lane);
}

template <bool TOP, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, TOP ? 3 : 4) k_score_join(const JoinArgs a, const Alternatives alt) {
    constexpr int kGroups = kJoinThreads / ROWS;  // threads of a token
    __shared__ Stats sh[ROWS][kGroups + 1];
    constexpr int kMost = ROWS == 1 ? kKeptOfBlock : kKept;
    __shared__ Found keep[TOP ? ROWS : 1][TOP ? kMost : 1];
    __shared__ int kept;
    const bool narrow = TOP && alt.narrow;
    let_next_start();
    after_previous();
    constexpr int kCounts = TOP && ROWS == 1 ? 4 : 1;
    [[maybe_unused]] int counts[kCounts] = {};  // of the first pieces of one token's thread, on their way already
    if constexpr (TOP && ROWS == 1) {
#pragma unroll
        for (int j = 0; j < kCounts; ++j) {
            const int p = threadIdx.x + j * kGroups;
            if (p < a.pieces) counts[j] = count_of(alt, blockIdx.x * a.pieces + p);
        }
    }
    // neighbouring tokens are read together
    const int col = threadIdx.x % ROWS, run = threadIdx.x / ROWS;
    const int64_t t = (int64_t)blockIdx.x * ROWS + col;
    Stats x{kNegInf, 0.f, 0.f};
    if (t < a.T) {
        // of one token, a thread's pieces are those of every 256th place; of eight, a lane's
        constexpr int kAhead = ROWS == 1 ? 4 : 8;
        for (int64_t i = 0; i < a.pieces; i += kGroups * kAhead) {
            Stats p[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t k = i + (ROWS == 1 ? run + kGroups * j : piece_of_lane(narrow, run, j));
                p[j] = k < a.pieces ? a.part[k * a.T + t] : Stats{kNegInf, 0.f, 0.f};
            }
            float top = x.m;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) top = fmaxf(top, p[j].m);
            const float ref = ref_of(top);
            x = rebase(x, ref);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const Stats y = rebase(p[j], ref);
                x.s += y.s, x.u += y.u;
            }
            x.m = top;
        }
    }
    sh[col][run] = x;
    if (threadIdx.x == 0) kept = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = ROWS == 1 ? 0 : warp;
    const int64_t u = (int64_t)blockIdx.x * ROWS + row;
    // a token's warp adds its parts up
    x = sh[row][ROWS == 1 ? piece_of_lane(narrow, lane, 0) : lane];
#pragma unroll
    for (int i = 1; i < kGroups / 32; ++i) x = add(x, sh[row][piece_of_lane(narrow, lane, i)]);
    float m = x.m;
    const float of_lane = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float ref = ref_of(m);
    x = rebase(x, ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        x.s += __shfl_xor_sync(~0u, x.s, o);
        x.u += __shfl_xor_sync(~0u, x.u, o);
    }
    if (u >= a.T) return;
    const float logs = logf(x.s), lse = ref + logs;
    if (lane == 0 && (ROWS > 1 || warp == 0)) {
        if (a.lse) a.lse[u] = lse;
        if (a.entropy) a.entropy[u] = logs - x.u * kLn2 / x.s;
        if (a.logp) a.logp[u] = inside(a.target[u], a.V) ? a.picked[u] - lse : 0.f;
    }
    if constexpr (TOP) {
        const int k = alt.k;
        Found *mine = keep[row];
        int n, place = 0;
        // k different logits reach the k-th of the lanes' largest
        for (int i = 0; i < 32; ++i) {
            const float b = __shfl_sync(~0u, of_lane, i);
            place += b > of_lane || (b == of_lane && i < lane);
        }
        float least = __shfl_sync(~0u, of_lane, __ffs(__ballot_sync(~0u, place == k - 1)) - 1);
        if (ROWS > 1) {
            if (alt.least)
                least = fmaxf(least, from_ordered(__reduce_min_sync(~0u, lane < k ? alt.least[lane * a.T + u] : ~0u)));
            n = collect(alt, a.pieces, u, least, !(of_lane >= least), mine, lane);
        } else {
            // the largest of this thread's pieces, which it looks through if any is large enough
            const auto look = [&](int64_t p, int c) {
                const Found *from = alt.found + (u * a.pieces + p) * alt.slots;
                for (int e = 0; e < c; e += 2) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(from + e);
                    const Found f[2] = {{__uint_as_float(q.x), (int)q.y}, {__uint_as_float(q.z), (int)q.w}};
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (e + i < c && f[i].l >= least) {
                            const int to = atomicAdd(&kept, 1);
                            if (to < kMost) mine[to] = f[i];
                        }
                    if (f[0].l < least && (e == 0 || alt.sorted)) break;
                }
            };
            if (sh[0][threadIdx.x].m >= least) {
#pragma unroll
                for (int j = 0; j < kCounts; ++j) look(threadIdx.x + j * kGroups, counts[j]);
                for (int64_t p = threadIdx.x + kCounts * kGroups; p < a.pieces; p += kGroups) look(p, count_of(alt, u * a.pieces + p));
            }
            __syncthreads();
            n = kept;
            if (n <= kMost) {
                n = sort_kept<kJoinThreads, kMost>(mine, n, k, threadIdx.x);
            } else if (warp == 0) {  // many equals
                n = collect(alt, a.pieces, u, least, !(of_lane >= least), mine, lane);
            }
            if (warp) return;
        }
        if (lane < k) {
            // a row with fewer numbers than that has a NaN
            a.top_logp[u * k + lane] = lane < n ? mine[lane].l - lse : kNaN;
            a.top_index[u * k + lane] = lane < n ? mine[lane].n : -1;
        }
    }
}

__global__ void __launch_bounds__(256) k_no_bounds(uint32_t *least, int64_t n) {
    let_next_start();
    after_previous();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) least[i] = 0;
}

// Rows of w to a warp of few tokens.
int64_t score_rows(int64_t T, int64_t V, int64_t H) {
    return std::min<int64_t>(few_rows(T, V, H, T * (kFewMost * 4 + kFewWarps * 12)), kFewMost / kFewWarps);
}

// Tokens are taken so many at a time that what their pieces leave takes about
// kLeftBytes (256 tokens at least): with 20 alternatives a piece leaves up to
// 205 bytes of a token, which 131072 columns make 210 KB.
constexpr int64_t kLeftBytes = 1ll << 30;
constexpr int kMoreSlots = 4;

struct ScoreSpace {
    Aligned x, w;
    Stats *part;
    float *picked;
    Alternatives alt;
    bool few;
    int64_t rows, each;  // rows of w to a warp of few tokens; tokens at a time
    size_t bytes;
};
int64_t pieces_of(int64_t T, int64_t V, int64_t H) { return kPieces * plan_product(T, V, H, false, false).nt; }
ScoreSpace score_space(void *ws, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, int64_t T, int64_t V,
                       int64_t H, int k) {
    Carve c{static_cast<unsigned char *>(ws)};
    ScoreSpace s{};
    s.few = few_tokens(T, H);
    s.alt.sorted = s.few;
    s.alt.k = k, s.alt.slots = ((s.few ? k : k + kMoreSlots) + 1) & ~1;
    s.alt.guess = 0.5f + 0.32f * std::sqrt((float)k);
    s.each = T;
    int64_t pieces;
    if (s.few) {
        s.rows = score_rows(T, V, H);
        pieces = ceil_div(V, s.rows * kFewWarps);
    } else {
        s.x = aligned(c, x, sx, T, H, ceil_div(V, 256));
        s.w = aligned(c, w, sw, V, H, ceil_div(T, 256));
        pieces = pieces_of(T, V, H);
        const int64_t left = pieces * ((int64_t)sizeof(Stats) + (k ? 1 + s.alt.slots * (int64_t)sizeof(Found) : 0));
        const int64_t most = std::max<int64_t>(kLeftBytes / left, 256);
        if (T > most) {
            s.each = std::min(T, round_up(ceil_div(T, ceil_div(T, most)), 256));
            pieces = std::max(pieces_of(s.each, V, H), pieces_of((T - 1) % s.each + 1, V, H));
        }
    }
    s.alt.pieces = pieces;  // the most
    s.part = c.take<Stats>(pieces * s.each);
    s.picked = c.take<float>(s.each);
    if (k) {
        s.alt.found = c.take<Found>(pieces * s.each * s.alt.slots);
        s.alt.count = c.take<uint8_t>(pieces * s.each);
        if (!s.few) s.alt.least = c.take<uint32_t>((k + 1) * s.each);
    }
    s.bytes = c.used;
    return s;
}

template <bool TOP>
int score(const ScoreSpace &s, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, const int64_t *target,
          int64_t T, int64_t V, int64_t H, float *logp, float *lse, float *entropy, float *top_logp, int64_t *top_index,
          cudaStream_t stream) {
    const int k = s.alt.k;
    int rc = PP_OK;
    if (!s.few) {
        rc = copy_if(s.x, x, sx, T, H, stream);
        if (rc == PP_OK) rc = copy_if(s.w, w, sw, V, H, stream);
    }
    for (int64_t t0 = 0; t0 < T && rc == PP_OK; t0 += s.each) {
        const int64_t n = std::min(s.each, T - t0);
        Alternatives alt = s.alt;
        if (s.few) {
            const bool vec = rows_aligned(w, sw, V, 2);
            const auto kernel = n == 1 ? (vec ? k_score_few<1, true, TOP> : k_score_few<1, false, TOP>)
                                       : (vec ? k_score_few<2, true, TOP> : k_score_few<2, false, TOP>);
            static std::atomic<uint64_t> ready[4];
            rc = allow_smem(kernel, kFewFloats * 4, ready[2 * (n - 1) + vec]);
            if (rc == PP_OK)
                rc = launch_after(kernel, alt.pieces, 32 * kFewWarps, (int)(n * ceil_div(H, 8) * 32), stream, 1, x, sx, w, sw,
                                  target, (int)n, V, (int)H, s.rows, s.part, s.picked, alt);
        } else {
            const ProductPlan plan = plan_product(n, V, H, false, false);
            alt.pieces = kPieces * plan.nt;
            alt.narrow = plan.tile_n <= 32;
            if (plan.mt * plan.nt * plan.cg <= sm_count()) alt.least = nullptr;
            if (TOP && alt.least) rc = launch_after(k_no_bounds, ceil_div(n * (k + 1), 256), 256, 0, stream, 1, alt.least, n * (k + 1));
            if (rc == PP_OK)
                rc = launch_product<kRowsK, kRowsK>(in_rows(s.x.at.p + t0 * s.x.at.ld, s.x.at.ld), s.w.at, n, V, H,
                                                    ScoreEpi<TOP>{target + t0, n, V, s.part, s.picked, alt}, plan, stream);
        }
        const auto from = [&](auto *p, int64_t each) { return p ? p + t0 * each : p; };
        const bool one = n <= (TOP ? kOneToSM * (int64_t)sm_count() : kOneAlone);
        if (rc == PP_OK)
            rc = launch_after(one ? k_score_join<TOP, 1> : k_score_join<TOP, 8>, one ? n : ceil_div(n, 8), kJoinThreads, 0,
                              stream, 1,
                              JoinArgs{s.part, s.picked, target + t0, alt.pieces, n, V, from(logp, 1), from(lse, 1),
                                       from(entropy, 1), from(top_logp, k), from(top_index, k)},
                              alt);
    }
    return rc;
}

}  // namespace
}  // namespace pps

using namespace pps;

extern "C" size_t pp_stage_score_forward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                   int64_t stride_w, int64_t T, int64_t V, int64_t H, int64_t top) {
    if (T < 1 || V < 1 || H < 1 || top < 0 || top > kMaxTop) return 0;
    return score_space(nullptr, x, stride_x, w, stride_w, T, V, H, (int)top).bytes;
}

extern "C" int pp_stage_score_forward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                      const int64_t *target, int64_t T, int64_t V, int64_t H, int64_t top, float *logp,
                                      float *lse, float *entropy, float *top_logp, int64_t *top_index, void *workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
    const int rc = check_head(x, stride_x, w, stride_w, target, T, V, H);
    if (rc != PP_OK) return rc;
    if (top < 0 || top > V) return PP_ERR_ARG;
    if (top > kMaxTop) return PP_ERR_SIZE;
    if (T == 0) return PP_OK;
    if ((!logp && !lse && !entropy && !top) || (((uintptr_t)logp | (uintptr_t)lse | (uintptr_t)entropy) & 3)) return PP_ERR_ARG;
    if (top && (!top_logp || !top_index || ((uintptr_t)top_logp & 3) || ((uintptr_t)top_index & 7))) return PP_ERR_ARG;
    const ScoreSpace s = score_space(workspace, x, stride_x, w, stride_w, T, V, H, (int)top);
    if (!workspace || ((uintptr_t)workspace & (kStageAlign - 1)) || workspace_bytes < s.bytes) return PP_ERR_ARG;
    return (top ? score<true> : score<false>)(s, x, stride_x, w, stride_w, target, T, V, H, logp, lse, entropy, top_logp,
                                              top_index, stream);
}
