// stage_kept.cu -- activation checkpoints in 8 bits and the weight gradient
// taken from them.
//
// Packing and unpacking move 3 bytes an element and are bound by memory:
// 16384 x 8192 on one GB300 in 67 us and 73 us, 88 % and 81 % of the measured
// copy rate.  The weight gradient dw = add + dy^T v is a tensor-core product
// over the tokens; v is unpacked first into panels of the workspace (3 bytes
// an element, 32 us of the 711-728 us that 8192^3 takes), exactly, since every
// value of a checkpoint is a bf16 number.  Both operands lie with their tokens
// apart (MN-major), which the MMA reads as they are.
#include "stage_kept.cuh"
#include "stage_product.cuh"

namespace pps {
namespace {

// A thread takes one unit of 8 columns of kRows consecutive rows and has all
// their loads in flight at once: the kernels are one pass over memory.  A warp
// is 32 consecutive units of a row, then of the next kRows rows; units are
// counted in 32 bits where that is enough (I), for the one division.
constexpr int kRows = 4, kThreads = 256;
constexpr int64_t kManyUnits = 1ll << 31;  // from here on 64 bits

// 8 lanes to a block of 64 columns.
template <bool VEC, class I>
__global__ void __launch_bounds__(kThreads) k_pack(const uint16_t *x, int64_t stride_x, int64_t T, int64_t H, int8_t *q,
                                                   int64_t stride_q, int8_t *e, int64_t stride_e) {
    let_next_start();
    after_previous();
    const I per = (I)((H + kBlock - 1) / kBlock * 8), u = (I)blockIdx.x * kThreads + threadIdx.x, g = u / per;
    const int64_t t = (int64_t)g * kRows, c = (int64_t)(u - g * per) * 8;
    // threads past the last unit go on with nothing: whole warps shuffle
    const int rows = t < T ? (int)(T - t < kRows ? T - t : kRows) : 0;
    const int left = H - c > 8 ? 8 : (int)(H - c);
    const uint16_t *px = x + t * stride_x + c;
    int8_t *pq = q + t * stride_q + c, *pe = e + t * stride_e + c / kBlock;
    Raw8 r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        r[i] = Raw8{};
        if (i < rows && left > 0) r[i] = load8<VEC>(px + i * stride_x, left);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        int ex;
        const uint2 b = pack8(r[i], ex);
        if (i < rows) {
            if (left > 0) store8_bytes<VEC>(pq + i * stride_q, left, b);
            if ((c & (kBlock - 1)) == 0) pe[i * stride_e] = (int8_t)ex;
        }
    }
}

template <bool VEC, class I>
__global__ void __launch_bounds__(kThreads) k_unpack(const int8_t *q, int64_t stride_q, const int8_t *e,
                                                     int64_t stride_e, int64_t T, int64_t H, uint16_t *x, int64_t ld,
                                                     int64_t panel) {
    let_next_start();
    after_previous();
    const I per = (I)((H + 7) / 8), u = (I)blockIdx.x * kThreads + threadIdx.x, g = u / per;
    const int64_t t = (int64_t)g * kRows, c = (int64_t)(u - g * per) * 8;
    if (t >= T) return;
    const int rows = (int)(T - t < kRows ? T - t : kRows), left = H - c > 8 ? 8 : (int)(H - c);
    const int8_t *pq = q + t * stride_q + c, *pe = e + t * stride_e + c / kBlock;
    uint16_t *px = x + t * ld + c / kBlock * panel + c % kBlock;
    uint2 b[kRows];
    int ex[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (i < rows) {
            b[i] = load8_bytes<VEC>(pq + i * stride_q, left);
            ex[i] = pe[i * stride_e];
        }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (i < rows) {
            float v[8];
            unpack8(b[i], step_of(ex[i]), v);
            store8_bf16<VEC>(px + i * ld, left, v);
        }
}

struct WgradEpi : NoRow {
    static constexpr bool kStore = true, kWhole = false;
    const float *add;
    float *dw;
    int64_t ld_add, ld;
    bool vec;
    __device__ __forceinline__ void finish(const Row &, int64_t m, int64_t n, float (&v)[32]) const {
        if (add) add_f32(v, add + m * ld_add + n);
    }
    __device__ __forceinline__ bool narrow() const { return false; }
    __device__ __forceinline__ void row(int64_t, int64_t, const float (&)[32]) const {}
    __device__ __forceinline__ void put(int64_t m, int64_t n, const float4 &v, int) const { store_quad(dw + m * ld + n, v); }
    __device__ __forceinline__ float with(const Row &, int64_t m, int64_t n) const { return add ? add[m * ld_add + n] : 0.f; }
    __device__ __forceinline__ void one(const Row &, int64_t m, int64_t n, float v, float b, int) const { dw[m * ld + n] = b + v; }
};

bool bad_kept(const int8_t *q, int64_t sq, const int8_t *e, int64_t se, int64_t H) {
    return !q || !e || sq < H || se < ceil_div(H, kBlock);
}

struct WgradSpace {
    uint16_t *v;   // what the checkpoint stands for, in panels
    uint16_t *dy;  // an aligned copy of dy in panels, or null
    float *parts;
    size_t bytes;
};
WgradSpace wgrad_space(void *ws, const uint16_t *dy, int64_t stride_dy, int64_t T, int64_t N, int64_t H) {
    Carve c{static_cast<unsigned char *>(ws)};
    WgradSpace s;
    s.v = c.take<uint16_t>(T * round_up(H, 64));
    s.dy = rows_aligned(dy, stride_dy, T, 2) ? nullptr : c.take<uint16_t>(T * round_up(N, 64));
    s.parts = c.take<float>(part_floats(N, H, T));
    s.bytes = c.used;
    return s;
}

}  // namespace

int launch_unpack(const int8_t *q, int64_t stride_q, const int8_t *e, int64_t stride_e, int64_t T, int64_t H,
                  uint16_t *x, int64_t ld, int64_t panel, cudaStream_t stream) {
    const int64_t units = ceil_div(T, kRows) * ceil_div(H, 8), grid = ceil_div(units, kThreads);
    const bool vec = rows_aligned(x, ld, T, 2) && kept_aligned(q, stride_q, T);
    const auto kernel = units < kManyUnits ? (vec ? k_unpack<true, uint32_t> : k_unpack<false, uint32_t>)
                                           : (vec ? k_unpack<true, int64_t> : k_unpack<false, int64_t>);
    return launch_after(kernel, grid, kThreads, 0, stream, 1, q, stride_q, e, stride_e, T, H, x, ld, panel);
}

}  // namespace pps

using namespace pps;

static int check_kept(int64_t T, int64_t H) {
    if (T < 0 || H < 1) return PP_ERR_ARG;
    if (T > PP_STAGE_MAX_ROWS || H > PP_STAGE_MAX_WIDTH) return PP_ERR_SIZE;
    return PP_OK;
}

extern "C" int pp_stage_pack(const uint16_t *x, int64_t stride_x, int64_t T, int64_t H, int8_t *q, int64_t stride_q,
                             int8_t *e, int64_t stride_e, cudaStream_t stream) {
    const int rc = check_kept(T, H);
    if (rc != PP_OK) return rc;
    if (T == 0) return PP_OK;
    if (!x || ((uintptr_t)x & 1) || stride_x < H || bad_kept(q, stride_q, e, stride_e, H)) return PP_ERR_ARG;
    const int64_t units = ceil_div(T, kRows) * ceil_div(H, kBlock) * 8, grid = ceil_div(units, kThreads);
    const bool vec = rows_aligned(x, stride_x, T, 2) && kept_aligned(q, stride_q, T);
    const auto kernel = units < kManyUnits ? (vec ? k_pack<true, uint32_t> : k_pack<false, uint32_t>)
                                           : (vec ? k_pack<true, int64_t> : k_pack<false, int64_t>);
    return launch_after(kernel, grid, kThreads, 0, stream, 1, x, stride_x, T, H, q, stride_q, e, stride_e);
}

extern "C" int pp_stage_unpack(const int8_t *q, int64_t stride_q, const int8_t *e, int64_t stride_e, int64_t T,
                               int64_t H, uint16_t *x, int64_t stride_x, cudaStream_t stream) {
    const int rc = check_kept(T, H);
    if (rc != PP_OK) return rc;
    if (T == 0) return PP_OK;
    if (!x || ((uintptr_t)x & 1) || stride_x < H || bad_kept(q, stride_q, e, stride_e, H)) return PP_ERR_ARG;
    return launch_unpack(q, stride_q, e, stride_e, T, H, x, stride_x, kBlock, stream);
}

extern "C" size_t pp_stage_weight_grad_workspace(const uint16_t *dy, int64_t stride_dy, int64_t T, int64_t N,
                                                 int64_t H) {
    if (T < 1 || N < 1 || H < 1) return 0;
    return wgrad_space(nullptr, dy, stride_dy, T, N, H).bytes;
}

extern "C" int pp_stage_weight_grad(const uint16_t *dy, int64_t stride_dy, const int8_t *q, int64_t stride_q,
                                    const int8_t *e, int64_t stride_e, int64_t T, int64_t N, int64_t H,
                                    const float *add, int64_t stride_add, float *dw, int64_t stride_dw,
                                    void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const int rc = check_kept(T, H);
    if (rc != PP_OK) return rc;
    if (N < 1) return PP_ERR_ARG;
    if (N > PP_STAGE_MAX_VOCAB) return PP_ERR_SIZE;
    if (!dw || ((uintptr_t)dw & 3) || stride_dw < H) return PP_ERR_ARG;
    if (add && (((uintptr_t)add & 3) || stride_add < H || (add == dw && stride_add != stride_dw))) return PP_ERR_ARG;
    if (T == 0) {
        if (!add) PPS_CUDA_TRY(cudaMemset2DAsync(dw, stride_dw * 4, 0, H * 4, N, stream));
        else if (add != dw)
            PPS_CUDA_TRY(cudaMemcpy2DAsync(dw, stride_dw * 4, add, stride_add * 4, H * 4, N, cudaMemcpyDeviceToDevice,
                                           stream));
        return PP_OK;
    }
    if (!dy || ((uintptr_t)dy & 1) || stride_dy < N || bad_kept(q, stride_q, e, stride_e, H)) return PP_ERR_ARG;
    const WgradSpace s = wgrad_space(workspace, dy, stride_dy, T, N, H);
    if (!workspace || ((uintptr_t)workspace & (kStageAlign - 1)) || workspace_bytes < s.bytes) return PP_ERR_ARG;
    const bool copy = !rows_aligned(dy, stride_dy, T, 2);
    int rp = launch_unpack(q, stride_q, e, stride_e, T, H, s.v, kBlock, T * kBlock, stream);
    if (rp == PP_OK && copy) rp = launch_copy_rows(dy, stride_dy, T, N, nullptr, 0, nullptr, s.dy, kBlock, T * kBlock, stream);
    if (rp != PP_OK) return rp;
    const bool vec = rows_aligned(dw, stride_dw, N, 4) && (!add || rows_aligned(add, stride_add, N, 4));
    const WgradEpi epi{{}, add, dw, stride_add, stride_dw, vec};
    const Matrix v = in_panels(s.v, T);
    if (copy) return product_in_parts<kPanelsMN, kPanelsMN>(in_panels(s.dy, T), v, N, H, T, epi, s.parts, stream);
    if (N % 64 == 0)
        return product_in_parts<kPanelsMN, kPanelsMN>(in_rows(dy, stride_dy), v, N, H, T, epi, s.parts, stream);
    return product_in_parts<kRowsMN, kPanelsMN>(in_rows(dy, stride_dy), v, N, H, T, epi, s.parts, stream);
}
