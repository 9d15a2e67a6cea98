// stage_head.cu -- softmax cross entropy of the last stage over a large
// vocabulary, and its gradients, without keeping the logits.
//
// Forward.  l = x w^T is taken tile by tile; of each (token, vocabulary tile)
// only the largest logit and the sum of exponentials relative to it leave the
// product, and a second kernel joins the tiles of a token:
//   m = max_i m_i,  s = sum_i s_i e^(m_i - m),  lse = m + log s.
// Backward.  d = weight (softmax - onehot) is recomputed for a piece of the
// vocabulary at a time, as bf16 in the workspace, and both gradients take
// their product with it before the next piece:  dx += d w_piece,
// dw_piece = d^T x.
#include <algorithm>

#include "stage_product.cuh"

namespace pps {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

// The reference point of a sum of exponentials: the largest logit, or 0 where
// that is infinite (so that inf - inf never appears).
__device__ __forceinline__ float ref_of(float m) { return isinf(m) ? 0.f : m; }

// Joins (m, s) with (m2, s2): sums of exponentials relative to ref_of(m).
__device__ __forceinline__ void join_stats(float &m, float &s, float m2, float s2) {
    const float mm = fmaxf(m, m2), r = ref_of(mm);
    // an empty part (m = -inf, s = 0) adds nothing
    const float a = s == 0.f ? 0.f : s * exp2f((ref_of(m) - r) * kLog2e);
    const float b = s2 == 0.f ? 0.f : s2 * exp2f((ref_of(m2) - r) * kLog2e);
    m = mm;
    s = a + b;
}

__device__ __forceinline__ bool inside(int64_t target, int64_t V) { return target >= 0 && target < V; }

struct StatsEpi {
    static constexpr bool kWhole = false;
    const int64_t *target;
    int64_t T, V;
    float2 *part;   // [column tiles][T]: largest logit, sum of exponentials
    float *picked;  // [T]: the target's logit
    struct Row {
        float m, s;
        int64_t target;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t, int) const {
        r.m = kNegInf;
        r.s = 0.f;
        r.target = target ? target[t] : -1;
    }
    __device__ __forceinline__ void chunk(Row &r, int64_t t, int64_t n, int cnt, const float (&v)[32]) const {
        float m = kNegInf, s = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cnt) m = fmaxf(m, v[j]);
        const float ref = ref_of(m);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cnt) s += exp2f((v[j] - ref) * kLog2e);
        join_stats(r.m, r.s, m, s);
        if (r.target >= n && r.target < n + cnt) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (r.target == n + j) picked[t] = v[j];
        }
    }
    __device__ __forceinline__ void end(Row &r, int64_t t, int64_t tile) const {
        part[tile * T + t] = make_float2(r.m, r.s);
    }
};

// d of one piece: columns v0 .. of the vocabulary, as bf16.
struct GradEpi {
    static constexpr bool kWhole = true;
    const int64_t *target;
    const float *lse, *weight;
    int64_t T, V, v0;
    uint16_t *d;  // in panels of T rows
    struct Row {
        float lse, c;
        int64_t at;  // the target's column counted from the piece's first
        bool in;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t, int) const {
        const int64_t g = target[t];
        r.in = inside(g, V);
        r.c = weight ? weight[t] : 1.f;
        r.lse = lse[t];
        r.at = g - v0;
    }
    __device__ __forceinline__ void chunk(Row &r, int64_t t, int64_t n, int cnt, const float (&v)[32]) const {
        float p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            p[j] = exp2f((v[j] - r.lse) * kLog2e);
            if (n + j == r.at) p[j] -= 1.f;
            p[j] = r.in && j < cnt ? p[j] * r.c : 0.f;
        }
        store_bf16(d + (n >> 6) * (T * 64) + t * 64 + (n & 63), 32, true, p);
    }
    __device__ __forceinline__ void end(Row &, int64_t, int64_t) const {}
};

// dx: pieces add up in 32 bits; the last one writes the result.
struct DxEpi {
    static constexpr bool kWhole = false;
    float *acc;  // [T][ld_acc]
    uint16_t *dx;
    const int64_t *target;
    int64_t V, ld_acc, ld;
    float scale;
    bool first, last, vec;
    struct Row {
        bool in;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t t, int) const { r.in = inside(target[t], V); }
    __device__ __forceinline__ void chunk(Row &r, int64_t t, int64_t n, int cnt, const float (&v)[32]) const {
        float s[32];
        if (first) {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = v[j];
        } else {
            load_f32(acc + t * ld_acc + n, cnt, true, s);
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] += v[j];
        }
        if (last) {  // a row that is left out is 0, whatever w holds
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = r.in ? s[j] * scale : 0.f;
            store_bf16(dx + t * ld + n, cnt, vec, s);
        } else {
            store_f32(acc + t * ld_acc + n, cnt, true, s);
        }
    }
    __device__ __forceinline__ void end(Row &, int64_t, int64_t) const {}
};

struct DwEpi {
    static constexpr bool kWhole = false;
    uint16_t *dw16;  // one of the two
    float *dw32;
    int64_t ld;
    float scale;
    bool add, vec;
    struct Row {};
    __device__ __forceinline__ void begin(Row &, int64_t, int) const {}
    __device__ __forceinline__ void chunk(Row &, int64_t m, int64_t n, int cnt, const float (&v)[32]) const {
        float s[32];
        if (dw32 && add) {
            load_f32(dw32 + m * ld + n, cnt, vec, s);
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] += v[j] * scale;
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = v[j] * scale;
        }
        if (dw32) store_f32(dw32 + m * ld + n, cnt, vec, s);
        else store_bf16(dw16 + m * ld + n, cnt, vec, s);
    }
    __device__ __forceinline__ void end(Row &, int64_t, int64_t) const {}
};

// One block of 32 tokens: 32 lanes along the tiles for each token.
__global__ void __launch_bounds__(1024) k_head_join(const float2 *part, const float *picked, const int64_t *target,
                                                    int64_t tiles, int64_t T, int64_t V, float *loss, float *lse) {
    __shared__ float2 sh[32][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    float m = kNegInf, s = 0.f;
    if (t < T)
        for (int64_t i = row; i < tiles; i += 32) {
            const float2 p = part[i * T + t];
            join_stats(m, s, p.x, p.y);
        }
    sh[row][lane] = make_float2(m, s);
    __syncthreads();
    // token blockIdx*32 + row: its 32 parts across the warp, always in the same order
    const int64_t u = (int64_t)blockIdx.x * 32 + row;
    m = sh[lane][row].x;
    s = sh[lane][row].y;
#pragma unroll
    for (int o = 16; o; o >>= 1) join_stats(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
    if (lane == 0 && u < T) {
        const float l = ref_of(m) + logf(s);
        if (lse) lse[u] = l;
        if (loss) loss[u] = inside(target[u], V) ? l - picked[u] : 0.f;
    }
}

// Columns of the vocabulary per piece of the backward pass: d of one piece is
// at most kPieceBytes.
constexpr int64_t kPieceBytes = 512ll << 20;
int64_t piece_of(int64_t T, int64_t V) {
    const int64_t cols = kPieceBytes / (2 * (T > 0 ? T : 1)) / 256 * 256;
    const int64_t most = 256 * 1024;
    int64_t p = cols < 256 ? 256 : cols > most ? most : cols;
    // equal pieces
    const int64_t n = ceil_div(V, p);
    return round_up(ceil_div(V, n), 256);
}

int check_head(const void *x, int64_t sx, const void *w, int64_t sw, const void *target, int64_t T, int64_t V,
               int64_t H) {
    if (T < 0 || V < 1 || H < 1) return PP_ERR_ARG;
    if (T > PP_STAGE_MAX_ROWS || V > PP_STAGE_MAX_VOCAB || H > PP_STAGE_MAX_WIDTH) return PP_ERR_SIZE;
    if (!w || ((uintptr_t)w & 1) || sw < H) return PP_ERR_ARG;
    if (T > 0 && (!x || !target || ((uintptr_t)x & 1) || ((uintptr_t)target & 7) || sx < H)) return PP_ERR_ARG;
    return PP_OK;
}

// An operand as the products read it: in place, or as an aligned copy in rows.
struct Aligned {
    uint16_t *copy;  // null: in place
    Matrix at;
};
Aligned aligned(Carve &c, const uint16_t *p, int64_t stride, int64_t rows, int64_t H) {
    if (rows_aligned(p, stride, rows, 2)) return {nullptr, in_rows(p, stride)};
    const int64_t ld = round_up(H, 64);
    uint16_t *q = c.take<uint16_t>(rows * ld);
    return {q, in_rows(q, ld)};
}

struct ForwardSpace {
    Aligned x, w;
    float2 *part;
    float *picked;
    int64_t tiles;
    size_t bytes;
};
ForwardSpace forward_space(void *ws, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, int64_t T,
                           int64_t V, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    ForwardSpace s;
    s.x = aligned(c, x, sx, T, H);
    s.w = aligned(c, w, sw, V, H);
    s.tiles = plan_product(T, V, H).nt;
    s.part = c.take<float2>(s.tiles * T);
    s.picked = c.take<float>(T);
    s.bytes = c.used;
    return s;
}

struct BackwardSpace {
    Aligned w;
    uint16_t *x, *d;  // in panels: x with the rows that are left out at 0, d of one piece
    float *acc, *parts;
    int64_t piece, ld_acc;
    size_t bytes;
};
BackwardSpace backward_space(void *ws, const uint16_t *x, int64_t sx, const uint16_t *w, int64_t sw, int64_t T,
                             int64_t V, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    BackwardSpace s;
    s.piece = piece_of(T, V);
    s.ld_acc = round_up(H, 32);
    s.w = aligned(c, w, sw, V, H);
    s.x = c.take<uint16_t>(T * round_up(H, 64));
    s.d = c.take<uint16_t>(T * s.piece);
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

int copy_if(const Aligned &a, const uint16_t *p, int64_t stride, int64_t rows, int64_t H, cudaStream_t stream) {
    return a.copy ? launch_copy_rows(p, stride, rows, H, nullptr, 0, a.copy, a.at.ld, 64, stream) : PP_OK;
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
    int rp = copy_if(s.x, x, stride_x, T, H, stream);
    if (rp == PP_OK) rp = copy_if(s.w, w, stride_w, V, H, stream);
    if (rp == PP_OK)
        rp = launch_product<kRowsK, kRowsK>(s.x.at, s.w.at, T, V, H, StatsEpi{target, T, V, s.part, s.picked}, stream);
    if (rp != PP_OK) return rp;
    k_head_join<<<(unsigned)ceil_div(T, 32), 1024, 0, stream>>>(s.part, s.picked, target, s.tiles, T, V, loss,
                                                                lse);
    PPS_CUDA_TRY(cudaGetLastError());
    return PP_OK;
}

extern "C" size_t pp_stage_head_backward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w,
                                                   int64_t stride_w, int64_t T, int64_t V, int64_t H) {
    if (T < 1 || V < 1 || H < 1) return 0;
    return backward_space(nullptr, x, stride_x, w, stride_w, T, V, H).bytes;
}

extern "C" int pp_stage_head_backward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                      const int64_t *target, const float *lse, const float *weight, float scale,
                                      int64_t T, int64_t V, int64_t H, uint16_t *dx, int64_t stride_dx, void *dw,
                                      int64_t stride_dw, int dw_float, int dw_add, void *workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
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
    int rp = launch_copy_rows(x, stride_x, T, H, target, V, s.x, 64, T * 64, stream);
    if (rp == PP_OK) rp = copy_if(s.w, w, stride_w, V, H, stream);
    const bool vec_dx = dx && rows_aligned(dx, stride_dx, T, 2), vec_dw = dw && rows_aligned(dw, stride_dw, V, dw_float ? 4 : 2);
    const Matrix xm = in_panels(s.x, T), d = in_panels(s.d, T);
    for (int64_t v0 = 0; v0 < V && rp == PP_OK; v0 += s.piece) {
        const int64_t n = V - v0 < s.piece ? V - v0 : s.piece;
        const Matrix wp = in_rows(s.w.at.p + v0 * s.w.at.ld, s.w.at.ld);
        rp = launch_product<kPanelsK, kRowsK>(xm, wp, T, n, H, GradEpi{target, lse, weight, T, V, v0, s.d}, stream);
        if (rp == PP_OK && dx) {
            const DxEpi epi{s.acc, dx, target, V, s.ld_acc, stride_dx, scale, v0 == 0, v0 + n == V, vec_dx};
            // the copy's rows are whole panels; so are w's own if H is
            rp = s.w.copy || H % 64 == 0
                     ? product_in_parts<kPanelsK, kPanelsMN>(d, wp, T, H, n, epi, s.parts, stream)
                     : product_in_parts<kPanelsK, kRowsMN>(d, wp, T, H, n, epi, s.parts, stream);
        }
        if (rp == PP_OK && dw)
            rp = product_in_parts<kPanelsMN, kPanelsMN>(
                d, xm, n, H, T,
                DwEpi{dw_float ? nullptr : (uint16_t *)dw + v0 * stride_dw,
                      dw_float ? (float *)dw + v0 * stride_dw : nullptr, stride_dw, scale, dw_add != 0, vec_dw},
                s.parts, stream);
    }
    return rp;
}
