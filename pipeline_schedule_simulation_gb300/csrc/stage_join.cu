// stage_join.cu -- the norm after a block, its gate, the residual scale and
// sum, and the norm before the next block, forward and backward.
//
// A block of threads holds a whole row in registers, so each input is read
// once and each output written once: forward moves 8 bytes an element (10 with
// both checkpoints), backward 10 from checkpoints and 12 from bf16, and memory
// bounds both.  Both directions need two sums over the row, one after the
// other, and a block that loads a row, sums and only then loads the next leaves
// the memory idle while it sums.  So long runs of rows come through a ring in
// shared memory that bulk copies keep filled, several rows ahead of the
// arithmetic; few or unaligned rows are loaded directly, by as many blocks as
// there are rows, and narrow rows (up to 512 columns) are taken by a warp each.
// One GB300, 16384 x 8192: forward 168 us (6.4 TB/s, 94 % of the measured copy
// rate), with both checkpoints 228 us (87 %; the packing's instructions issue in
// two thirds of all cycles), backward from bf16 273 us (87 %), from checkpoints
// 228 us (86 %), the column sums among them.  16384 x 512 by warps: forward 13 us (75 %).
#include <atomic>

#include "stage_kept.cuh"
#include "stage_ring.cuh"

namespace pps {
namespace {

// Sum over the block; every thread gets it.  `sh` holds one value per warp and
// must not be in use by an earlier call that some thread may still be reading:
// callers alternate between two.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 128; ++i) {
        const float4 p = reinterpret_cast<const float4 *>(sh)[i];
        s += (p.x + p.y) + (p.z + p.w);
    }
    return s;
}

struct Kept {
    int8_t *q, *e;
    int64_t sq, se;
};

struct JoinForward {
    const uint16_t *x, *f, *w_post, *w_pre, *gate;
    int64_t sx, sf, sg, rows_per_gate;
    float alpha, eps;
    int64_t T;
    int H;
    uint16_t *y, *h;
    int64_t sy, sh;
    float *rstd_post, *rstd_pre;
    Kept ky, kf;
};

// NT threads hold NV vectors of 8 columns each: H <= 8 * NT * NV.
template <int NT, int NV, bool VEC, bool KEEP>
__global__ void __launch_bounds__(NT) k_join_forward(const JoinForward a) {
    __shared__ __align__(16) float sh[2][32];
    let_next_start();
    after_previous();
    const float inv_h = 1.f / (float)a.H;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const uint16_t *g = a.gate ? a.gate + (a.rows_per_gate > 0 ? t / a.rows_per_gate : 0) * a.sg : nullptr;
        float f[NV][8], y[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8;
            const int left = a.H - c;
            load8_bf16<VEC>(a.f + t * a.sf + (left > 0 ? c : 0), left, f[i]);
            load8_bf16<VEC>(a.x + t * a.sx + (left > 0 ? c : 0), left, y[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += f[i][j] * f[i][j];
        }
        const float r1 = rsqrtf(block_sum<NT>(ss, sh[0]) * inv_h + a.eps);
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
                int e;
                const uint2 b = pack8(narrow(f[i]), e);  // f came as bf16: nothing is lost
                if (left > 0) {
                    store8_bytes<VEC>(a.kf.q + t * a.kf.sq + c, left, b);
                    if ((threadIdx.x & 7) == 0) a.kf.e[t * a.kf.se + c / kBlock] = (int8_t)e;
                }
            }
        }
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
            float w[8];
            load8_bf16<VEC>(a.w_post + (left > 0 ? c : 0), left, w);
            if (g) {
                float gv[8];
                load8_bf16<VEC>(g + (left > 0 ? c : 0), left, gv);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= gv[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[i][j] = a.alpha * y[i][j] + w[j] * (f[i][j] * r1);
                ss += y[i][j] * y[i][j];
            }
            if (left > 0) store8_bf16<VEC>(a.y + t * a.sy + c, left, y[i]);
        }
        const float r2 = rsqrtf(block_sum<NT>(ss, sh[1]) * inv_h + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
            float w[8];
            load8_bf16<VEC>(a.w_pre + (left > 0 ? c : 0), left, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= y[i][j] * r2;
            if (left > 0) store8_bf16<VEC>(a.h + t * a.sh + c, left, w);
            if (KEEP) {
                int e;
                const uint2 b = pack8(narrow(y[i]), e);  // y as its next reader sees it
                if (left > 0) {
                    store8_bytes<VEC>(a.ky.q + t * a.ky.sq + c, left, b);
                    if ((threadIdx.x & 7) == 0) a.ky.e[t * a.ky.se + c / kBlock] = (int8_t)e;
                }
            }
        }
        if (threadIdx.x == 0) {
            a.rstd_post[t] = r1;
            a.rstd_pre[t] = r2;
        }
    }
}

constexpr int kNarrow = 512;  // widths up to this: a warp to a row, kWarps rows a block at once
constexpr int kWarps = 8;

// Threads of a ring block for this width: two vectors of 8 columns each (one up
// to 1024 columns), in whole warps; 0 where a row is too wide.
int ring_threads(int64_t H) { return H > 8192 ? 0 : (int)round_up(ceil_div(H, H <= 1024 ? 8 : 16), 32); }

// Rows are shared out in items: a run of rows of one gate group, so that an
// item's column sums belong to one gate row.
struct Items {
    int64_t rows_per_gate, groups, rows, per_group, count;
};
Items items_of(int64_t T, int64_t H, int64_t rows_per_gate) {
    Items it;
    it.rows_per_gate = rows_per_gate > 0 && rows_per_gate < T ? rows_per_gate : T;
    it.groups = ceil_div(T, it.rows_per_gate);
    // one run of rows for each block that is resident on the GPU (two to an SM
    // where rows are too wide for the ring)
    const int threads = ring_threads(H);
    const int64_t want = (int64_t)sm_count() * (H <= kNarrow ? (H <= 256 ? 4 : 2) : threads ? 512 / threads : 2);
    it.rows = ceil_div(T, want);
    if (H <= kNarrow && it.rows < kWarps) it.rows = kWarps;
    if (it.rows > it.rows_per_gate) it.rows = it.rows_per_gate;
    it.per_group = ceil_div(it.rows_per_gate, it.rows);
    it.count = it.groups * it.per_group;
    return it;
}

struct JoinBackward {
    const uint16_t *dh, *dy, *y, *f, *w_post, *w_pre, *gate;
    int64_t sdh, sdy, sy, sf, sg;
    Kept ky, kf;
    const float *rstd_post, *rstd_pre;
    float alpha;
    int64_t T;
    int H;
    uint16_t *dx, *df;
    int64_t sdx, sdf;
    float *part_pre, *part_post;  // [items][ld]: sum dh n2, sum d n1
    int64_t ld;
    Items it;
};

template <bool VEC, bool PACKED>
__device__ __forceinline__ void load_saved(const uint16_t *p, int64_t s, const Kept &k, int64_t t, int c, int left,
                                           float (&v)[8]) {
    if (PACKED) {
        if (left > 0) unpack8(load8_bytes<VEC>(k.q + t * k.sq + c, left), step_of(k.e[t * k.se + c / kBlock]), v);
        // past the row's end a block's bytes are 0, and so is a value unless the block is not finite
        if (left < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= left) v[j] = 0.f;
        }
    } else {
        load8_bf16<VEC>(p + t * s + (left > 0 ? c : 0), left, v);
    }
}

template <int NT, int NV, bool VEC, bool PACKED>
__global__ void __launch_bounds__(NT) k_join_backward(const JoinBackward a) {
    __shared__ __align__(16) float sh[2][32];
    let_next_start();
    after_previous();
    const float inv_h = 1.f / (float)a.H;
    const int64_t group = blockIdx.x / a.it.per_group, part = blockIdx.x % a.it.per_group;
    const int64_t first = group * a.it.rows_per_gate + part * a.it.rows;
    int64_t last = min(first + a.it.rows, (group + 1) * a.it.rows_per_gate);
    last = min(last, a.T);
    const uint16_t *g = a.gate ? a.gate + group * a.sg : nullptr;
    float sum_pre[NV][8] = {}, sum_post[NV][8] = {};
    for (int64_t t = first; t < last; ++t) {
        const float r1 = a.rstd_post[t], r2 = a.rstd_pre[t];
        float n2[NV][8], d[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
            float w[8];
            load8_bf16<VEC>(a.dh + t * a.sdh + (left > 0 ? c : 0), left, d[i]);
            load_saved<VEC, PACKED>(a.y, a.sy, a.ky, t, c, left, n2[i]);
            load8_bf16<VEC>(a.w_pre + (left > 0 ? c : 0), left, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n2[i][j] *= r2;
                sum_pre[i][j] += d[i][j] * n2[i][j];
                d[i][j] *= w[j];
                ss += d[i][j] * n2[i][j];
            }
        }
        const float m2 = block_sum<NT>(ss, sh[0]) * inv_h;
        float n1[NV][8];
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
            float u[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = r2 * (d[i][j] - n2[i][j] * m2);
            if (a.dy) {
                load8_bf16<VEC>(a.dy + t * a.sdy + (left > 0 ? c : 0), left, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] += u[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = a.alpha * d[i][j];
            if (left > 0) store8_bf16<VEC>(a.dx + t * a.sdx + c, left, u);
            load_saved<VEC, PACKED>(a.f, a.sf, a.kf, t, c, left, n1[i]);
            load8_bf16<VEC>(a.w_post + (left > 0 ? c : 0), left, w);
            if (g) {
                load8_bf16<VEC>(g + (left > 0 ? c : 0), left, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= u[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n1[i][j] *= r1;
                sum_post[i][j] += d[i][j] * n1[i][j];
                d[i][j] *= w[j];
                ss += d[i][j] * n1[i][j];
            }
        }
        const float m1 = block_sum<NT>(ss, sh[1]) * inv_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * NT + (int)threadIdx.x) * 8, left = a.H - c;
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = r1 * (d[i][j] - n1[i][j] * m1);
            if (left > 0) store8_bf16<VEC>(a.df + t * a.sdf + c, left, u);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + (int)threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < a.H) {
                a.part_pre[blockIdx.x * a.ld + c + j] = sum_pre[i][j];
                a.part_post[blockIdx.x * a.ld + c + j] = sum_post[i][j];
            }
    }
}

// ---- narrow rows: a warp to a row

// H <= 256 * NV: sums need no other warp, and a block of 8 warps has 8 rows in
// flight (a block of threads to a row would leave most of them idle).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <int NV, bool VEC, bool KEEP>
__global__ void __launch_bounds__(32 * kWarps) k_join_forward_narrow(const JoinForward a) {
    let_next_start();
    after_previous();
    const float inv_h = 1.f / (float)a.H;
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const uint16_t *g = a.gate ? a.gate + (a.rows_per_gate > 0 ? t / a.rows_per_gate : 0) * a.sg : nullptr;
        Raw8 fr[NV];
        float y[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c, at = left > 0 ? c : 0;
            fr[i] = load8<VEC>(a.f + t * a.sf + at, left);
            load8_bf16<VEC>(a.x + t * a.sx + at, left, y[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8];
            widen(fr[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += f[j] * f[j];
        }
        const float r1 = rsqrtf(warp_sum(ss) * inv_h + a.eps);
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c, at = left > 0 ? c : 0;
            float w[8], f[8];
            load8_bf16<VEC>(a.w_post + at, left, w);
            if (g) {
                load8_bf16<VEC>(g + at, left, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= f[j];
            }
            widen(fr[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[i][j] = a.alpha * y[i][j] + w[j] * (f[j] * r1);
                ss += y[i][j] * y[i][j];
            }
            const Raw8 yr = narrow(y[i]);
            if (left > 0) store8<VEC>(a.y + t * a.sy + c, left, yr);
            if (KEEP) {
                int ey, ef;
                const uint2 by = pack8(yr, ey), bf = pack8(fr[i], ef);
                if (left > 0) {
                    store8_bytes<VEC>(a.ky.q + t * a.ky.sq + c, left, by);
                    store8_bytes<VEC>(a.kf.q + t * a.kf.sq + c, left, bf);
                    if ((lane & 7) == 0) {
                        a.ky.e[t * a.ky.se + c / kBlock] = (int8_t)ey;
                        a.kf.e[t * a.kf.se + c / kBlock] = (int8_t)ef;
                    }
                }
            }
        }
        const float r2 = rsqrtf(warp_sum(ss) * inv_h + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c;
            if (left > 0) {
                float w[8];
                load8_bf16<VEC>(a.w_pre + c, left, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= y[i][j] * r2;
                store8_bf16<VEC>(a.h + t * a.sh + c, left, w);
            }
        }
        if (lane == 0) {
            a.rstd_post[t] = r1;
            a.rstd_pre[t] = r2;
        }
    }
}

template <int NV, bool VEC, bool PACKED>
__global__ void __launch_bounds__(32 * kWarps, NV == 1 ? 4 : 2) k_join_backward_narrow(const JoinBackward a) {
    let_next_start();
    after_previous();
    __shared__ float sums[2][kWarps][NV * 256];
    const float inv_h = 1.f / (float)a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t group = blockIdx.x / a.it.per_group, part = blockIdx.x % a.it.per_group;
    const int64_t first = group * a.it.rows_per_gate + part * a.it.rows;
    int64_t last = min(first + a.it.rows, (group + 1) * a.it.rows_per_gate);
    last = min(last, a.T);
    float sum_pre[NV][8] = {}, sum_post[NV][8] = {};
    for (int64_t t = first + warp; t < last; t += kWarps) {
        const float r1 = a.rstd_post[t], r2 = a.rstd_pre[t];
        Raw8 dr[NV], ur[NV];
        float n2[NV][8], n1[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c, at = left > 0 ? c : 0;
            dr[i] = load8<VEC>(a.dh + t * a.sdh + at, left);
            ur[i] = a.dy ? load8<VEC>(a.dy + t * a.sdy + at, left) : Raw8{};
            load_saved<VEC, PACKED>(a.y, a.sy, a.ky, t, c, left, n2[i]);
            load_saved<VEC, PACKED>(a.f, a.sf, a.kf, t, c, left, n1[i]);
        }
        float d[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c, at = left > 0 ? c : 0;
            float w[8];
            widen(dr[i], d[i]);
            load8_bf16<VEC>(a.w_pre + at, left, w);  // from the L1 cache: registers are what limits this kernel
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n2[i][j] *= r2;
                n1[i][j] *= r1;
                sum_pre[i][j] += d[i][j] * n2[i][j];
                d[i][j] *= w[j];
                ss += d[i][j] * n2[i][j];
            }
        }
        const float m2 = warp_sum(ss) * (inv_h * r2);
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c, at = left > 0 ? c : 0;
            float u[8], gw[8];
            widen(ur[i], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[i][j] = fmaf(r2, d[i][j], fmaf(-m2, n2[i][j], u[j]));
                u[j] = a.alpha * d[i][j];
            }
            if (left > 0) store8_bf16<VEC>(a.dx + t * a.sdx + c, left, u);
            load8_bf16<VEC>(a.w_post + at, left, gw);
            if (a.gate) {
                load8_bf16<VEC>(a.gate + group * a.sg + at, left, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) gw[j] *= u[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum_post[i][j] += d[i][j] * n1[i][j];
                d[i][j] *= gw[j];
                ss += d[i][j] * n1[i][j];
            }
        }
        const float m1 = warp_sum(ss) * (inv_h * r1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 32 + lane) * 8, left = a.H - c;
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = fmaf(r1, d[i][j], -m1 * n1[i][j]);
            if (left > 0) store8_bf16<VEC>(a.df + t * a.sdf + c, left, u);
        }
    }
    // the warps' sums, in the order of the warps
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sums[0][warp][(i * 32 + lane) * 8 + j] = sum_pre[i][j];
            sums[1][warp][(i * 32 + lane) * 8 + j] = sum_post[i][j];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += 32 * kWarps) {
        float p = 0.f, q = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) p += sums[0][w][c], q += sums[1][w][c];
        a.part_pre[blockIdx.x * a.ld + c] = p;
        a.part_post[blockIdx.x * a.ld + c] = q;
    }
}

// ---- rows through a ring.  FULL: the row's columns are all of the block's
// vectors, and no vector's end is looked at (16384 x 8192 backward from
// checkpoints: 216 us, 267 us with the looks).

// Shared memory of one block: a header with a barrier for each stage, then the stages.
constexpr int kRingHeader = 128;

__device__ __forceinline__ Raw8 ring_raw(const unsigned char *stage, uint32_t at, int c) {
    const uint4 w = *reinterpret_cast<const uint4 *>(stage + at + 2 * c);
    return Raw8{{w.x, w.y, w.z, w.w}};
}

// A vector past the row's end (ok false) reads as zeros, without a branch: what
// it would read is put aside, not skipped.
__device__ __forceinline__ Raw8 ring_raw(const unsigned char *stage, uint32_t at, int c, bool ok) {
    Raw8 r = ring_raw(stage, at, ok ? c : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = ok ? r.w[j] : 0u;
    return r;
}

template <int NT, int NV, bool KEEP, bool FULL>
__global__ void __launch_bounds__(NT, 1024 / NT) k_join_forward_ring(const JoinForward a, const int stages) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float sh[2][32];
    __shared__ RingState state;
    const int nt = blockDim.x;  // a whole number of warps, NT at most
    if (threadIdx.x < 64) sh[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;  // also for the warps that are not there
    let_next_start();
    after_previous();
    const uint32_t row_bytes = 2u * a.H;
    Ring<2> ring{tc::smem_u32(smem) + kRingHeader, tc::smem_u32(smem), 2 * row_bytes, stages,
                 {{(const unsigned char *)a.f, 2 * a.sf, row_bytes, 0}, {(const unsigned char *)a.x, 2 * a.sx, row_bytes, row_bytes}}};
    const float inv_h = 1.f / (float)a.H;
    if (threadIdx.x == 0) {
        ring.init(&state);
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + (int64_t)i * gridDim.x < a.T) ring.load(&state, blockIdx.x + (int64_t)i * gridDim.x, i, 0);
    }
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    const int c0 = (int)threadIdx.x * 8;
    uint16_t *py = a.y + blockIdx.x * a.sy + c0, *ph = a.h + blockIdx.x * a.sh + c0;
    int8_t *qf = a.kf.q + blockIdx.x * a.kf.sq + c0, *ef = a.kf.e + blockIdx.x * a.kf.se + c0 / kBlock;
    int8_t *qy = a.ky.q + blockIdx.x * a.ky.sq + c0, *ey = a.ky.e + blockIdx.x * a.ky.se + c0 / kBlock;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const unsigned char *stage = smem + kRingHeader + slot * ring.stage_bytes;
        const uint16_t *g = a.gate ? a.gate + (a.rows_per_gate > 0 ? t / a.rows_per_gate : 0) * a.sg : nullptr;
        // a wait that runs out is recorded; the block then goes through its rows without data, and loads no more
        tc::mbar_wait(ring.bars + 8 * slot, parity, &state.stop, 5);
        Raw8 fr[NV];
        float y[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            const bool ok = FULL || c < a.H;
            fr[i] = ring_raw(stage, 0, c, ok);
            widen(ring_raw(stage, row_bytes, c, ok), y[i]);
            float f[8];
            widen(fr[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += f[j] * f[j];
        }
        const float r1 = rsqrtf(block_sum<NT>(ss, sh[0]) * inv_h + a.eps);
        // every thread has read the stage
        if (threadIdx.x == 0 && t + (int64_t)stages * gridDim.x < a.T)
            ring.refill(&state, t + (int64_t)stages * gridDim.x, slot, parity);
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + (int)threadIdx.x) * 8;
                int e;
                const uint2 b = pack8(fr[i], e);
                if (FULL || c < a.H) {
                    *reinterpret_cast<uint2 *>(qf + i * nt * 8) = b;
                    if ((threadIdx.x & 7) == 0) ef[i * nt * 8 / kBlock] = (int8_t)e;
                }
            }
        }
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            const bool ok = FULL || c < a.H;
            const int at = ok ? c : 0;
            float w[8], f[8];
            load8_bf16<true>(a.w_post + at, 8, w);
            if (g) {
                load8_bf16<true>(g + at, 8, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= f[j];
            }
            // past the row's end column 0 was read: no weight, which an infinity or a NaN there would not be times 0
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = ok ? w[j] : 0.f;
            widen(fr[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[i][j] = a.alpha * y[i][j] + w[j] * (f[j] * r1);
                ss += y[i][j] * y[i][j];
            }
            const Raw8 yr = narrow(y[i]);
            if (ok) store8<true>(py + i * nt * 8, 8, yr);
            if (KEEP) {
                int e;
                const uint2 b = pack8(yr, e);  // y as its next reader sees it
                if (ok) {
                    *reinterpret_cast<uint2 *>(qy + i * nt * 8) = b;
                    if ((threadIdx.x & 7) == 0) ey[i * nt * 8 / kBlock] = (int8_t)e;
                }
            }
        }
        const float r2 = rsqrtf(block_sum<NT>(ss, sh[1]) * inv_h + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            if (FULL || c < a.H) {
                float w[8];
                load8_bf16<true>(a.w_pre + c, 8, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= y[i][j] * r2;
                store8_bf16<true>(ph + i * nt * 8, 8, w);
            }
        }
        if (threadIdx.x == 0) {
            a.rstd_post[t] = r1;
            a.rstd_pre[t] = r2;
        }
        py += gridDim.x * a.sy, ph += gridDim.x * a.sh;
        if (KEEP) {
            qf += gridDim.x * a.kf.sq, ef += gridDim.x * a.kf.se;
            qy += gridDim.x * a.ky.sq, ey += gridDim.x * a.ky.se;
        }
        if (++slot == stages) slot = 0, parity ^= 1;
    }
    if (threadIdx.x == 0) ring.finish(&state);
}

template <int NT, int NV, bool PACKED, bool FULL>
__global__ void __launch_bounds__(NT, 512 / NT) k_join_backward_ring(const JoinBackward a, const int stages) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float sh[2][32];
    __shared__ RingState state;
    const int nt = blockDim.x;  // a whole number of warps, NT at most
    if (threadIdx.x < 64) sh[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;  // also for the warps that are not there
    let_next_start();
    after_previous();
    const uint32_t wide = 2u * a.H, saved = PACKED ? (uint32_t)a.H : wide, at_dy = wide + 2 * saved;
    Ring<4> ring{tc::smem_u32(smem) + kRingHeader, tc::smem_u32(smem), at_dy + (a.dy ? wide : 0), stages,
                 {{(const unsigned char *)a.dh, 2 * a.sdh, wide, 0},
                  {PACKED ? (const unsigned char *)a.ky.q : (const unsigned char *)a.y, PACKED ? a.ky.sq : 2 * a.sy, saved, wide},
                  {PACKED ? (const unsigned char *)a.kf.q : (const unsigned char *)a.f, PACKED ? a.kf.sq : 2 * a.sf, saved,
                   wide + saved},
                  {(const unsigned char *)a.dy, 2 * a.sdy, a.dy ? wide : 0, at_dy}}};
    const float inv_h = 1.f / (float)a.H;
    const int64_t group = blockIdx.x / a.it.per_group, part = blockIdx.x % a.it.per_group;
    const int64_t first = group * a.it.rows_per_gate + part * a.it.rows;
    int64_t last = min(first + a.it.rows, (group + 1) * a.it.rows_per_gate);
    last = min(last, a.T);
    if (threadIdx.x == 0) {
        ring.init(&state);
        for (int i = 0; i < stages; ++i)
            if (first + i < last) ring.load(&state, first + i, i, 0);
    }
    // the weights of this thread's columns stay in registers: the item has one gate row
    Raw8 w_pre[NV];
    float gw[NV][8], sum_pre[NV][8] = {}, sum_post[NV][8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + (int)threadIdx.x) * 8, left = FULL ? 8 : a.H - c, at = left > 0 ? c : 0;
        w_pre[i] = load8<true>(a.w_pre + at, left);
        load8_bf16<true>(a.w_post + at, left, gw[i]);
        if (a.gate) {
            float u[8];
            load8_bf16<true>(a.gate + group * a.sg + at, left, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) gw[i][j] *= u[j];
        }
    }
    // what is read beside the ring is read a row ahead
    float r1 = 0.f, r2 = 0.f, next1 = 0.f, next2 = 0.f;
    int ey[NV] = {}, ef[NV] = {};
    const int c0 = (int)threadIdx.x * 8;
    const int8_t *py = a.ky.e + first * a.ky.se + c0 / kBlock, *pf = a.kf.e + first * a.kf.se + c0 / kBlock;
    const auto ahead = [&](int64_t t) {
        next1 = a.rstd_post[t], next2 = a.rstd_pre[t];
        if (PACKED) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (FULL || c0 + i * nt * 8 < a.H) ey[i] = py[i * nt * 8 / kBlock], ef[i] = pf[i * nt * 8 / kBlock];
            py += a.ky.se, pf += a.kf.se;
        }
    };
    uint16_t *px = a.dx + first * a.sdx + c0, *pd = a.df + first * a.sdf + c0;
    if (first < last) ahead(first);
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    for (int64_t t = first; t < last; ++t) {
        const unsigned char *stage = smem + kRingHeader + slot * ring.stage_bytes;
        float step_y[NV], step_f[NV];
        r1 = next1, r2 = next2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            step_y[i] = PACKED ? step_of(ey[i]) * r2 : r2;
            step_f[i] = PACKED ? step_of(ef[i]) * r1 : r1;
        }
        if (t + 1 < last) ahead(t + 1);
        tc::mbar_wait(ring.bars + 8 * slot, parity, &state.stop, 6);
        const auto norm = [&](uint32_t at, int c, bool ok, float step, float (&n)[8]) {
            if (PACKED) {
                uint2 q = *reinterpret_cast<const uint2 *>(stage + at + (ok ? c : 0));
                q.x = ok ? q.x : 0u, q.y = ok ? q.y : 0u;
                unpack8(q, step, n);
            } else {
                widen(ring_raw(stage, at, c, ok), n);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[j] *= step;
            }
        };
        float n2[NV][8], d[NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            const bool ok = FULL || c < a.H;
            float w[8];
            norm(wide, c, ok, step_y[i], n2[i]);
            widen(ring_raw(stage, 0, c, ok), d[i]);
            widen(w_pre[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum_pre[i][j] += d[i][j] * n2[i][j];
                d[i][j] *= w[j];
                ss += d[i][j] * n2[i][j];
            }
        }
        const float m2 = block_sum<NT>(ss, sh[0]) * (inv_h * r2);
        float n1[NV][8];
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            const bool ok = FULL || c < a.H;
            float u[8];
            if (a.dy) {
                widen(ring_raw(stage, at_dy, c, ok), u);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = fmaf(r2, d[i][j], fmaf(-m2, n2[i][j], u[j]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = fmaf(r2, d[i][j], -m2 * n2[i][j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = a.alpha * d[i][j];
            if (ok) store8_bf16<true>(px + i * nt * 8, 8, u);
            norm(wide + saved, c, ok, step_f[i], n1[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum_post[i][j] += d[i][j] * n1[i][j];
                d[i][j] *= gw[i][j];
                ss += d[i][j] * n1[i][j];
            }
        }
        const float m1 = block_sum<NT>(ss, sh[1]) * (inv_h * r1);
        // every thread has read the stage
        if (threadIdx.x == 0 && t + stages < last) ring.refill(&state, t + stages, slot, parity);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            if (FULL || c < a.H) {
                float u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = fmaf(r1, d[i][j], -m1 * n1[i][j]);
                store8_bf16<true>(pd + i * nt * 8, 8, u);
            }
        }
        px += a.sdx, pd += a.sdf;
        if (++slot == stages) slot = 0, parity ^= 1;
    }
    if (threadIdx.x == 0) ring.finish(&state);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + (int)threadIdx.x) * 8;
        if (FULL || c < a.H) {
            float *p = a.part_pre + blockIdx.x * a.ld + c, *q = a.part_post + blockIdx.x * a.ld + c;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                reinterpret_cast<float4 *>(p)[j] =
                    make_float4(sum_pre[i][4 * j], sum_pre[i][4 * j + 1], sum_pre[i][4 * j + 2], sum_pre[i][4 * j + 3]);
                reinterpret_cast<float4 *>(q)[j] =
                    make_float4(sum_post[i][4 * j], sum_post[i][4 * j + 1], sum_post[i][4 * j + 2], sum_post[i][4 * j + 3]);
            }
        }
    }
}

// Blocks on an SM and stages that each has.
struct RingPlan {
    int threads, blocks, stages;
    size_t smem;
};
RingPlan ring_plan(int64_t H, int64_t stage_bytes, int threads_on_sm) {
    RingPlan p{ring_threads(H), 0, 0, 0};
    if (!p.threads) return p;
    p.blocks = threads_on_sm / p.threads;
    const int64_t each = 220 * 1024 / p.blocks - 1024 - kRingHeader;
    p.stages = (int)(each / stage_bytes < kMaxStages ? each / stage_bytes : kMaxStages);
    if (p.stages < 2) p.threads = 0;
    p.smem = kRingHeader + p.stages * stage_bytes;
    return p;
}

// Column sums of the items' parts, in a fixed order: blockIdx.y = 0 joins all
// items (the part of the norm after the block weighted by its group's gate), the
// others a gate group each.  8 quads of columns and 32 runs of items a block,
// each run four items at a time.
__global__ void __launch_bounds__(256) k_join_columns(const float *part_pre, const float *part_post, Items it, int H,
                                                      int64_t ld, const uint16_t *w_post, const uint16_t *gate,
                                                      int64_t sg, float *dw_post, float *dw_pre, float *dgate,
                                                      int64_t sdg) {
    after_previous();
    __shared__ float s0[32][33], s1[32][33];
    constexpr int kAhead = 4;
    const int quad = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int h = blockIdx.x * 32 + quad * 4;  // rows of the parts are whole quads
    const bool all = blockIdx.y == 0;
    for (int64_t g = all ? 0 : blockIdx.y - 1; g < (all ? 1 : it.groups); g += all ? 1 : gridDim.y - 1) {
        const int64_t from = all ? 0 : g * it.per_group, to = all ? it.count : (g + 1) * it.per_group;
        float a[4] = {}, b[4] = {};
        if (h < H) {
            for (int64_t i = from + row; i < to; i += 32 * kAhead) {
                float4 p[kAhead], r[kAhead];
                float u[kAhead][4];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int64_t j = i + 32 * k;
                    const bool in = j < to;
                    p[k] = in ? *reinterpret_cast<const float4 *>(part_post + j * ld + h) : make_float4(0.f, 0.f, 0.f, 0.f);
                    r[k] = in && all ? *reinterpret_cast<const float4 *>(part_pre + j * ld + h)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                    const uint16_t *gr = gate + j / it.per_group * sg + h;
#pragma unroll
                    for (int c = 0; c < 4; ++c) u[k][c] = in && all && gate && h + c < H ? bf16_to_f32(gr[c]) : 1.f;
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    a[0] += r[k].x, a[1] += r[k].y, a[2] += r[k].z, a[3] += r[k].w;
                    b[0] += p[k].x * u[k][0], b[1] += p[k].y * u[k][1], b[2] += p[k].z * u[k][2], b[3] += p[k].w * u[k][3];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s0[row][quad * 4 + j] = a[j], s1[row][quad * 4 + j] = b[j];
        __syncthreads();
        // 8 lanes to a column, 4 runs each
        const int col = threadIdx.x >> 3, hh = blockIdx.x * 32 + col;
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) sa += s0[quad * 4 + j][col], sb += s1[quad * 4 + j][col];
#pragma unroll
        for (int o = 4; o; o >>= 1) {
            sa += __shfl_xor_sync(~0u, sa, o);
            sb += __shfl_xor_sync(~0u, sb, o);
        }
        if (quad == 0 && hh < H) {
            if (all) {
                dw_pre[hh] = sa;
                dw_post[hh] = sb;
            } else {
                dgate[g * sdg + hh] = sb * bf16_to_f32(w_post[hh]);
            }
        }
        __syncthreads();
    }
}

template <bool VEC, bool KEEP>
int forward_by_width(const JoinForward &a, unsigned grid, cudaStream_t s) {
    if (a.H <= kNarrow) {
        const int64_t want = ceil_div(a.T, kWarps), most = (int64_t)sm_count() * 8;
        const int64_t g = want < most ? want : most;
        return a.H <= 256 ? launch_after(k_join_forward_narrow<1, VEC, KEEP>, g, 32 * kWarps, 0, s, 1, a)
                          : launch_after(k_join_forward_narrow<2, VEC, KEEP>, g, 32 * kWarps, 0, s, 1, a);
    }
    if (a.H <= 1024) return launch_after(k_join_forward<128, 1, VEC, KEEP>, grid, 128, 0, s, 1, a);
    if (a.H <= 2048) return launch_after(k_join_forward<256, 1, VEC, KEEP>, grid, 256, 0, s, 1, a);
    if (a.H <= 4096) return launch_after(k_join_forward<512, 1, VEC, KEEP>, grid, 512, 0, s, 1, a);
    if (a.H <= 8192) return launch_after(k_join_forward<512, 2, VEC, KEEP>, grid, 512, 0, s, 1, a);
    return launch_after(k_join_forward<1024, 2, VEC, KEEP>, grid, 1024, 0, s, 1, a);
}

template <bool VEC, bool PACKED>
int backward_by_width(const JoinBackward &a, cudaStream_t s) {
    const unsigned grid = (unsigned)a.it.count;
    if (a.H <= kNarrow)
        return a.H <= 256 ? launch_after(k_join_backward_narrow<1, VEC, PACKED>, grid, 32 * kWarps, 0, s, 1, a)
                          : launch_after(k_join_backward_narrow<2, VEC, PACKED>, grid, 32 * kWarps, 0, s, 1, a);
    if (a.H <= 1024) return launch_after(k_join_backward<128, 1, VEC, PACKED>, grid, 128, 0, s, 1, a);
    if (a.H <= 2048) return launch_after(k_join_backward<256, 1, VEC, PACKED>, grid, 256, 0, s, 1, a);
    if (a.H <= 4096) return launch_after(k_join_backward<512, 1, VEC, PACKED>, grid, 512, 0, s, 1, a);
    if (a.H <= 8192) return launch_after(k_join_backward<512, 2, VEC, PACKED>, grid, 512, 0, s, 1, a);
    return launch_after(k_join_backward<1024, 2, VEC, PACKED>, grid, 1024, 0, s, 1, a);
}

template <class K, class A>
int launch_ring(K kernel, const A &a, const RingPlan &p, unsigned grid, std::atomic<uint64_t> &ready, cudaStream_t s) {
    const int rc = allow_smem(kernel, 226 * 1024, ready);
    if (rc != PP_OK) return rc;
    return launch_after(kernel, grid, p.threads, (int)p.smem, s, 1, a, p.stages);
}

template <bool KEEP>
int forward_ring(const JoinForward &a, const RingPlan &p, cudaStream_t s) {
    static std::atomic<uint64_t> ready[8];
    // 512 columns are a whole number of warps, whatever the vectors
    const int64_t most = (int64_t)sm_count() * p.blocks;
    const unsigned grid = (unsigned)(a.T < most ? a.T : most);
    const bool full = a.H % 512 == 0;
    if (a.H <= 1024)
        return full ? launch_ring(k_join_forward_ring<128, 1, KEEP, true>, a, p, grid, ready[0], s)
                    : launch_ring(k_join_forward_ring<128, 1, KEEP, false>, a, p, grid, ready[1], s);
    if (a.H <= 2048)
        return full ? launch_ring(k_join_forward_ring<128, 2, KEEP, true>, a, p, grid, ready[2], s)
                    : launch_ring(k_join_forward_ring<128, 2, KEEP, false>, a, p, grid, ready[3], s);
    if (a.H <= 4096)
        return full ? launch_ring(k_join_forward_ring<256, 2, KEEP, true>, a, p, grid, ready[4], s)
                    : launch_ring(k_join_forward_ring<256, 2, KEEP, false>, a, p, grid, ready[5], s);
    return full ? launch_ring(k_join_forward_ring<512, 2, KEEP, true>, a, p, grid, ready[6], s)
                : launch_ring(k_join_forward_ring<512, 2, KEEP, false>, a, p, grid, ready[7], s);
}

template <bool PACKED>
int backward_ring(const JoinBackward &a, const RingPlan &p, cudaStream_t s) {
    static std::atomic<uint64_t> ready[8];
    // 512 columns are a whole number of warps, whatever the vectors
    const unsigned grid = (unsigned)a.it.count;
    const bool full = a.H % 512 == 0;
    if (a.H <= 1024)
        return full ? launch_ring(k_join_backward_ring<128, 1, PACKED, true>, a, p, grid, ready[0], s)
                    : launch_ring(k_join_backward_ring<128, 1, PACKED, false>, a, p, grid, ready[1], s);
    if (a.H <= 2048)
        return full ? launch_ring(k_join_backward_ring<128, 2, PACKED, true>, a, p, grid, ready[2], s)
                    : launch_ring(k_join_backward_ring<128, 2, PACKED, false>, a, p, grid, ready[3], s);
    if (a.H <= 4096)
        return full ? launch_ring(k_join_backward_ring<256, 2, PACKED, true>, a, p, grid, ready[4], s)
                    : launch_ring(k_join_backward_ring<256, 2, PACKED, false>, a, p, grid, ready[5], s);
    return full ? launch_ring(k_join_backward_ring<512, 2, PACKED, true>, a, p, grid, ready[6], s)
                : launch_ring(k_join_backward_ring<512, 2, PACKED, false>, a, p, grid, ready[7], s);
}

int check_join(int64_t T, int64_t H) {
    if (T < 0 || H < 1) return PP_ERR_ARG;
    if (T > PP_STAGE_MAX_ROWS || H > PP_STAGE_MAX_JOIN_WIDTH) return PP_ERR_SIZE;
    return PP_OK;
}
bool bad_rows(const void *p, int64_t stride, int64_t H) { return !p || ((uintptr_t)p & 1) || stride < H; }
bool bad_kept(const Kept &k, int64_t H) { return !k.q || !k.e || k.sq < H || k.se < ceil_div(H, kBlock); }

struct BackSpace {
    float *pre, *post;
    int64_t ld;
    size_t bytes;
};
BackSpace back_space(void *ws, const Items &it, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    BackSpace s;
    s.ld = round_up(H, 8);
    s.pre = c.take<float>(it.count * s.ld);
    s.post = c.take<float>(it.count * s.ld);
    s.bytes = c.used;
    return s;
}

}  // namespace
}  // namespace pps

using namespace pps;

extern "C" int pp_stage_join_forward(const uint16_t *x, int64_t stride_x, const uint16_t *f, int64_t stride_f,
                                     const uint16_t *w_post, const uint16_t *w_pre, const uint16_t *gate,
                                     int64_t stride_gate, int64_t rows_per_gate, float alpha, float eps, int64_t T,
                                     int64_t H, uint16_t *y, int64_t stride_y, uint16_t *h, int64_t stride_h,
                                     float *rstd_post, float *rstd_pre, int8_t *y_q, int64_t stride_yq, int8_t *y_e,
                                     int64_t stride_ye, int8_t *f_q, int64_t stride_fq, int8_t *f_e, int64_t stride_fe,
                                     cudaStream_t stream) {
    const int rc = check_join(T, H);
    if (rc != PP_OK) return rc;
    if (T == 0) return PP_OK;
    const bool keep = y_q || y_e || f_q || f_e;
    JoinForward a{x, f, w_post, w_pre, gate, stride_x, stride_f, stride_gate, rows_per_gate, alpha, eps, T, (int)H,
                  y, h, stride_y, stride_h, rstd_post, rstd_pre,
                  Kept{y_q, y_e, stride_yq, stride_ye}, Kept{f_q, f_e, stride_fq, stride_fe}};
    if (bad_rows(x, stride_x, H) || bad_rows(f, stride_f, H) || bad_rows(w_post, H, H) || bad_rows(w_pre, H, H) ||
        bad_rows(y, stride_y, H) || bad_rows(h, stride_h, H) || (gate && bad_rows(gate, stride_gate, H)) ||
        !rstd_post || !rstd_pre || ((uintptr_t)rstd_post & 3) || ((uintptr_t)rstd_pre & 3) || !(eps >= 0.f) ||
        (keep && (bad_kept(a.ky, H) || bad_kept(a.kf, H))))
        return PP_ERR_ARG;
    const bool vec = rows_aligned(x, stride_x, T, 2) && rows_aligned(f, stride_f, T, 2) &&
                     rows_aligned(w_post, H, 1, 2) && rows_aligned(w_pre, H, 1, 2) && rows_aligned(y, stride_y, T, 2) &&
                     rows_aligned(h, stride_h, T, 2) && (!gate || rows_aligned(gate, stride_gate, 2, 2)) &&
                     (!keep || (kept_aligned(y_q, stride_yq, T) && kept_aligned(f_q, stride_fq, T)));
    // the ring pays from about two rows a block on
    const RingPlan p = ring_plan(H, 4 * H, 1024);
    if (vec && p.threads && H > kNarrow && H % 8 == 0 && T >= 2 * (int64_t)sm_count() * p.blocks) {
        return keep ? forward_ring<true>(a, p, stream) : forward_ring<false>(a, p, stream);
    }
    const int64_t most = (int64_t)sm_count() * 16;
    const unsigned grid = (unsigned)(T < most ? T : most);
    if (vec) return keep ? forward_by_width<true, true>(a, grid, stream) : forward_by_width<true, false>(a, grid, stream);
    return keep ? forward_by_width<false, true>(a, grid, stream) : forward_by_width<false, false>(a, grid, stream);
}

extern "C" size_t pp_stage_join_backward_workspace(int64_t T, int64_t H, int64_t rows_per_gate) {
    if (T < 1 || H < 1) return 0;
    return back_space(nullptr, items_of(T, H, rows_per_gate), H).bytes;
}

extern "C" int pp_stage_join_backward(const uint16_t *dh, int64_t stride_dh, const uint16_t *dy, int64_t stride_dy,
                                      const uint16_t *y, int64_t stride_y, const uint16_t *f, int64_t stride_f,
                                      const int8_t *y_q, int64_t stride_yq, const int8_t *y_e, int64_t stride_ye,
                                      const int8_t *f_q, int64_t stride_fq, const int8_t *f_e, int64_t stride_fe,
                                      const float *rstd_post, const float *rstd_pre, const uint16_t *w_post,
                                      const uint16_t *w_pre, const uint16_t *gate, int64_t stride_gate,
                                      int64_t rows_per_gate, float alpha, int64_t T, int64_t H, uint16_t *dx,
                                      int64_t stride_dx, uint16_t *df, int64_t stride_df, float *dw_post, float *dw_pre,
                                      float *dgate, int64_t stride_dgate, void *workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
    const int rc = check_join(T, H);
    if (rc != PP_OK) return rc;
    if (!dw_post || !dw_pre || ((uintptr_t)dw_post & 3) || ((uintptr_t)dw_pre & 3) || (!gate != !dgate) ||
        (dgate && (((uintptr_t)dgate & 3) || stride_dgate < H)))
        return PP_ERR_ARG;
    if (T == 0) {  // no gate group has a row
        PPS_CUDA_TRY(cudaMemsetAsync(dw_post, 0, H * 4, stream));
        PPS_CUDA_TRY(cudaMemsetAsync(dw_pre, 0, H * 4, stream));
        return PP_OK;
    }
    const bool packed = y_q || y_e || f_q || f_e;
    const Items it = items_of(T, H, rows_per_gate);
    const BackSpace s = back_space(workspace, it, H);
    JoinBackward a{dh, dy, y, f, w_post, w_pre, gate, stride_dh, stride_dy, stride_y, stride_f, stride_gate,
                   Kept{const_cast<int8_t *>(y_q), const_cast<int8_t *>(y_e), stride_yq, stride_ye},
                   Kept{const_cast<int8_t *>(f_q), const_cast<int8_t *>(f_e), stride_fq, stride_fe},
                   rstd_post, rstd_pre, alpha, T, (int)H, dx, df, stride_dx, stride_df, s.pre, s.post, s.ld, it};
    if (bad_rows(dh, stride_dh, H) || (dy && bad_rows(dy, stride_dy, H)) || bad_rows(w_post, H, H) ||
        bad_rows(w_pre, H, H) || (gate && bad_rows(gate, stride_gate, H)) || bad_rows(dx, stride_dx, H) ||
        bad_rows(df, stride_df, H) || !rstd_post || !rstd_pre || ((uintptr_t)rstd_post & 3) ||
        ((uintptr_t)rstd_pre & 3))
        return PP_ERR_ARG;
    if (packed ? (y || f || bad_kept(a.ky, H) || bad_kept(a.kf, H)) : (bad_rows(y, stride_y, H) || bad_rows(f, stride_f, H)))
        return PP_ERR_ARG;
    if (!workspace || ((uintptr_t)workspace & (kStageAlign - 1)) || workspace_bytes < s.bytes) return PP_ERR_ARG;
    const bool vec = rows_aligned(dh, stride_dh, T, 2) && (!dy || rows_aligned(dy, stride_dy, T, 2)) &&
                     rows_aligned(w_post, H, 1, 2) && rows_aligned(w_pre, H, 1, 2) &&
                     (!gate || rows_aligned(gate, stride_gate, 2, 2)) && rows_aligned(dx, stride_dx, T, 2) &&
                     rows_aligned(df, stride_df, T, 2) &&
                     (packed ? kept_aligned(y_q, stride_yq, T) && kept_aligned(f_q, stride_fq, T)
                             : rows_aligned(y, stride_y, T, 2) && rows_aligned(f, stride_f, T, 2));
    const RingPlan p = ring_plan(H, (dy ? 4 : 2) * H + (packed ? 2 : 4) * H, 512);
    // bulk copies take whole 16 bytes
    const bool whole = packed ? H % 16 == 0 && rows_aligned(y_q, stride_yq, T, 1) && rows_aligned(f_q, stride_fq, T, 1)
                              : H % 8 == 0;
    int rr;
    if (vec && whole && p.threads && H > kNarrow && it.rows >= 2)
        rr = packed ? backward_ring<true>(a, p, stream) : backward_ring<false>(a, p, stream);
    else if (vec) rr = packed ? backward_by_width<true, true>(a, stream) : backward_by_width<true, false>(a, stream);
    else rr = packed ? backward_by_width<false, true>(a, stream) : backward_by_width<false, false>(a, stream);
    if (rr != PP_OK) return rr;
    const dim3 grid((unsigned)ceil_div(H, 32), 1 + (gate ? (unsigned)(it.groups < 1024 ? it.groups : 1024) : 0));
    return launch_after(k_join_columns, grid, 256, 0, stream, 1, (const float *)s.pre, (const float *)s.post, it, (int)H,
                        s.ld, w_post, gate, stride_gate, dw_post, dw_pre, dgate, stride_dgate);
}
