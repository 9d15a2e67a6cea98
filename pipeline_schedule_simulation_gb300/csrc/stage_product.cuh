// stage_product.cuh -- matrix products of the pipeline-stage operators on the
// tensor cores.
//
// C[m][n] = sum_k A(m,k) B(n,k) over bf16 operands, summed in 32 bits in TMEM,
// handed to an epilogue row by row instead of being stored:
//   typename Epi::Row  what a row keeps between its pieces
//   begin(row, m, part)  a row m of the tile starts (part: which part of K)
//   chunk(row, m, n, cnt, v)  columns n .. n+cnt-1 (cnt <= 32) of row m
//   end(row, m, tile)  the row's piece of column tile `tile` is done
//   kWhole             the columns go on to the next multiple of 64, with cnt <= 0
//                      past the last one
// Each (row, column tile) is handed over by one thread, in column order.
//
// Persistent blocks, one to an SM: a warp loads 64-deep slices of A and B by
// TMA into a ring of six, a thread issues the MMAs of a tile into one of two
// TMEM accumulators, four warps take the other accumulator through the
// epilogue.  Operands come K-major or MN-major as they lie in memory; both
// forms use the 128-byte swizzle.  What the library lays out itself lies in
// panels of 64 columns (128 bytes), each panel's rows one after the other, so
// that a box is one run of memory in either form.
//
// CG = 2: a pair of blocks shares a tile of 256 x 256: each holds half of A
// and half of B, so that a slice costs each SM 32 KB of loads for 256 x 256 x
// 64 products of the pair; a lone block needs 48 KB for half of that.
// CG = 1: a block takes a tile of 128 x 128, with the same loads: for products
// with so few tiles that more of them are worth more than fast ones.
#pragma once

#include "stage_common.cuh"
#include "stage_tc.cuh"

namespace pps {

// A matrix of bf16: element (row, col) at p[row*ld + (col/64)*panel + col%64].
// Rows in memory: panel = 64 and ld their stride (aligned to 16 bytes); panels:
// ld = 64 and panel their stride, the last panel's columns padded with zeros.
struct Matrix {
    const uint16_t *p;
    int64_t ld, panel;
};
inline Matrix in_rows(const uint16_t *p, int64_t ld) { return {p, ld, 64}; }
inline Matrix in_panels(const uint16_t *p, int64_t rows) { return {p, 64, rows * 64}; }

// How an operand lies: rows along k (K-major), rows along m or n (MN-major),
// panels in either use.  MN-major rows whose columns are whole panels are
// loaded as panels.
enum Form { kRowsK, kRowsMN, kPanelsK, kPanelsMN };
__host__ __device__ constexpr bool is_mn(Form f) { return f == kRowsMN || f == kPanelsMN; }

// One stage's half of an operand: 128 of its rows (m or n) from i0, slice k.
template <int CG, Form F>
__device__ __forceinline__ void load_half(uint32_t to, const CUtensorMap *map, int i0, int k, uint32_t bar) {
    if (F == kRowsK) tc::tma_load<CG>(to, map, k * 64, i0, 0, bar);
    if (F == kPanelsK) tc::tma_load<CG>(to, map, 0, i0, k, bar);
    if (F == kPanelsMN) tc::tma_load<CG>(to, map, 0, k * 64, i0 / 64, bar);
    if (F == kRowsMN) {
        tc::tma_load<CG>(to, map, i0, k * 64, 0, bar);
        tc::tma_load<CG>(to + 8192, map, i0 + 64, k * 64, 0, bar);
    }
}

constexpr int kTileK = 64, kHalf = 128;  // a block holds 128 rows of A and 128 of B
constexpr int kStages = 6;
constexpr int kBytesHalf = kHalf * kTileK * 2, kBytesStage = 2 * kBytesHalf;
constexpr int kProductSmem = kStages * kBytesStage + 1024;
constexpr int kProductThreads = 256;

struct ProductShape {
    int M, N, K;
    int mt, nt;    // tiles
    int group;     // row tiles that are taken together
    int splits;    // parts of K
    int k_blocks;  // slices of K in each part (the last may have fewer)
};

// Tile number -> (row tile, column tile): `group` row tiles at a time run
// through all column tiles, so that their slices of A stay in the L2 cache.
__device__ __forceinline__ void tile_at(const ProductShape &s, int64_t i, int &m, int &n) {
    const int64_t per = (int64_t)s.group * s.nt;
    const int g = (int)(i / per), first = g * s.group;
    const int rows = min(s.group, s.mt - first), r = (int)(i - g * per);
    m = first + r % rows;
    n = r / rows;
}

template <class Epi, Form FA, Form FB, int CG>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const ProductShape s, const Epi epi) {
    constexpr int kTileN = kHalf * CG;
    constexpr bool A_MN = is_mn(FA), B_MN = is_mn(FB);
    constexpr uint32_t kCols = 2 * kTileN;  // TMEM columns: two accumulators
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int stop;
    const uint32_t ring = (tc::smem_u32(raw) + 1023) & ~1023u;
    const uint32_t full = tc::smem_u32(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? tc::cluster_rank() : 0;
    const int64_t tiles = (int64_t)s.mt * s.nt * s.splits, first = blockIdx.x / CG, step = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(acc_full + 8 * i, 1);
            tc::mbar_init(acc_empty + 8 * i, 4 * CG);
        }
        tc::mbar_init(drained, 1);
        stop = 0;
        tc::fence_barrier_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    if (warp == 2) tc::tmem_alloc<CG>(tc::smem_u32(&tmem_at), kCols);
    tc::fence_before();
    __syncthreads();
    if (CG == 2) tc::cluster_sync();  // the other block's barriers are ready
    tc::fence_after();
    const uint32_t tmem = tmem_at;
    const int all_blocks = (s.K + kTileK - 1) / kTileK;

    if (warp == 0) {
        if (lane == 0) {
            int64_t it = 0;
            bool ok = true;
            for (int64_t t = first; t < tiles && ok; t += step) {
                const int part = (int)(t % s.splits);
                int m, n;
                tile_at(s, t / s.splits, m, n);
                const int m0 = (m * CG + (int)rank) * kHalf, n0 = (n * CG + (int)rank) * kHalf;
                const int k0 = part * s.k_blocks, k1 = min(k0 + s.k_blocks, all_blocks);
                for (int k = k0; k < k1; ++k, ++it) {
                    const int st = (int)(it % kStages);
                    if (!tc::mbar_wait(empty + 8 * st, (uint32_t)(it / kStages + 1) & 1, &stop, 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = ring + st * kBytesStage, b = a + kBytesHalf;
                    // a pair's loads all count on the first block's barrier
                    const uint32_t bar = CG == 2 ? tc::in_block(full + 8 * st, 0) : full + 8 * st;
                    if (rank == 0) tc::mbar_expect(full + 8 * st, CG * kBytesStage);
                    load_half<CG, FA>(a, &map_a, m0, k, bar);
                    load_half<CG, FB>(b, &map_b, n0, k, bar);
                }
            }
            // after giving up: the copies still in flight land before the block ends
            if (!ok) {
                if (rank == 0)
                    for (int64_t j = it > kStages ? it - kStages : 0; j < it; ++j)
                        tc::mbar_drain(full + 8 * (int)(j % kStages), (uint32_t)(j / kStages) & 1);
                else
                    tc::let_land();
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = tc::instr_desc(kHalf * CG, kTileN, A_MN, B_MN);
            // 16 k further: 32 bytes along a K-major row, two groups of 8 k in the MN-major form
            constexpr uint32_t step_a = A_MN ? 2048 : 32, step_b = B_MN ? 2048 : 32;
            int64_t it = 0;
            int j = 0;
            bool ok = true;
            for (int64_t t = first; t < tiles && ok; t += step, ++j) {
                const int part = (int)(t % s.splits);
                const int k0 = part * s.k_blocks, k1 = min(k0 + s.k_blocks, all_blocks);
                const int buf = j & 1;
                if (!tc::mbar_wait(acc_empty + 8 * buf, (uint32_t)((j >> 1) + 1) & 1, &stop, 2)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                for (int k = k0; k < k1; ++k, ++it) {
                    const int st = (int)(it % kStages);
                    if (!tc::mbar_wait(full + 8 * st, (uint32_t)(it / kStages) & 1, &stop, 3)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t a = ring + st * kBytesStage, b = a + kBytesHalf;
#pragma unroll
                    for (int kk = 0; kk < kTileK / 16; ++kk)
                        tc::mma<CG>(tmem + buf * kTileN, tc::smem_desc(a + kk * step_a, A_MN ? 8192 : 16, 1024),
                                    tc::smem_desc(b + kk * step_b, B_MN ? 8192 : 16, 1024), idesc, k > k0 || kk > 0);
                    tc::mma_commit<CG>(empty + 8 * st);
                }
                if (ok) tc::mma_commit<CG>(acc_full + 8 * buf);
            }
            // the MMAs have finished before TMEM is given back
            tc::mma_commit<CG>(drained);
            tc::mbar_drain(drained, 0);
        }
    } else if (warp >= 4) {
        const int quarter = warp - 4;
        const int wide = Epi::kWhole ? (s.N + 63) & ~63 : s.N;
        int j = 0;
        for (int64_t t = first; t < tiles; t += step, ++j) {
            const int part = (int)(t % s.splits);
            int mt, nt;
            tile_at(s, t / s.splits, mt, nt);
            const int buf = j & 1;
            const int64_t m = (int64_t)(mt * CG + (int)rank) * kHalf + quarter * 32 + lane;
            const bool live = m < s.M;
            typename Epi::Row row;
            if (live) epi.begin(row, m, part);
            // lanes give up one by one: the warp goes on together
            const bool ok = tc::mbar_wait(acc_full + 8 * buf, (uint32_t)(j >> 1) & 1, &stop, 4);
            if (!__all_sync(~0u, ok)) break;
            tc::fence_after();
            for (int c = 0; c < kTileN && nt * kTileN + c < wide; c += 32) {
                float v[32];
                tc::tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * kTileN + c, v);
                const int n = nt * kTileN + c, left = s.N - n;
                if (live) epi.chunk(row, m, n, left < 32 ? left : 32, v);
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) tc::mbar_arrive_at(tc::in_block(acc_empty + 8 * buf, 0));
                else tc::mbar_arrive(acc_empty + 8 * buf);
            }
            if (live) epi.end(row, m, nt);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (CG == 2) tc::cluster_sync();  // neither block ends while the other may still signal it
    tc::fence_after();
    if (warp == 2) tc::tmem_free<CG>(tmem, kCols);
}

// ---- host side

// The map of an operand of `rows` x `cols` as it lies in memory, for boxes of
// box_rows x 64 x box_panels.
int encode_map(CUtensorMap *map, const Matrix &m, int64_t rows, int64_t cols, bool panels, int box_rows,
               int box_panels);

// I: the operand's extent along m or n, K along k.
template <Form F>
int map_of(CUtensorMap *map, const Matrix &m, int64_t I, int64_t K) {
    if (F == kRowsK) return encode_map(map, m, I, K, false, kHalf, 1);
    if (F == kPanelsK) return encode_map(map, m, I, K, true, kHalf, 1);
    if (F == kPanelsMN) return encode_map(map, m, K, I, true, 64, 2);
    return encode_map(map, m, K, I, false, 64, 1);
}

// How a product is cut: pairs of blocks from the point on where lone blocks'
// tiles would not all fit on the SMs at once, and K in parts where there are
// still fewer tiles than SMs (each part has at least 4 slices, none is empty).
struct ProductPlan {
    int cg, splits;
    int64_t mt, nt;
};
inline ProductPlan plan_product(int64_t M, int64_t N, int64_t K) {
    const int64_t sms = sm_count(), blocks = ceil_div(K, kTileK);
    ProductPlan p;
    p.cg = M > kHalf && ceil_div(M, kHalf) * ceil_div(N, kHalf) > sms ? 2 : 1;
    p.mt = ceil_div(M, kHalf * p.cg), p.nt = ceil_div(N, kHalf * p.cg);
    int64_t s = sms / p.cg / (p.mt * p.nt > 0 ? p.mt * p.nt : 1);
    if (s > blocks / 4) s = blocks / 4;
    p.splits = s <= 1 ? 1 : (int)ceil_div(blocks, ceil_div(blocks, s));
    return p;
}

// A product without parts of K, whatever the plan says of them: its column
// tiles are plan_product()'s.
template <Form FA, Form FB, class Epi>
int launch_product(const Matrix &A, const Matrix &B, int64_t M, int64_t N, int64_t K, const Epi &epi,
                   cudaStream_t stream, int splits = 1) {
    if (M <= 0 || N <= 0 || K <= 0) return PP_ERR_INTERNAL;
    CUtensorMap ma, mb;
    int rc = map_of<FA>(&ma, A, M, K);
    if (rc == PP_OK) rc = map_of<FB>(&mb, B, N, K);
    if (rc != PP_OK) return rc;
    const ProductPlan p = plan_product(M, N, K);
    ProductShape s;
    s.M = (int)M, s.N = (int)N, s.K = (int)K;
    s.mt = (int)p.mt, s.nt = (int)p.nt;
    s.splits = splits;
    s.k_blocks = (int)ceil_div(ceil_div(K, kTileK), splits);
    s.group = s.mt < 16 ? s.mt : 16;
    const int64_t tiles = p.mt * p.nt * splits, most = sm_count() / p.cg;
    const unsigned grid = (unsigned)(tiles < most ? tiles : most) * p.cg;
    static std::atomic<uint64_t> ready[2];
    if (p.cg == 1) {
        rc = allow_smem(k_product<Epi, FA, FB, 1>, kProductSmem, ready[0]);
        if (rc != PP_OK) return rc;
        k_product<Epi, FA, FB, 1><<<grid, kProductThreads, kProductSmem, stream>>>(ma, mb, s, epi);
        PPS_CUDA_TRY(cudaGetLastError());
        return PP_OK;
    }
    rc = allow_smem(k_product<Epi, FA, FB, 2>, kProductSmem, ready[1]);
    if (rc != PP_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(kProductThreads), cfg.dynamicSmemBytes = kProductSmem;
    cfg.stream = stream;
    cudaLaunchAttribute pair;
    pair.id = cudaLaunchAttributeClusterDimension;
    pair.val.clusterDim.x = 2, pair.val.clusterDim.y = 1, pair.val.clusterDim.z = 1;
    cfg.attrs = &pair, cfg.numAttrs = 1;
    PPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_product<Epi, FA, FB, 2>, ma, mb, s, epi));
    return PP_OK;
}

// Parts of K: each part's sums apart, [part][M][ld].  Epilogues are local to
// their translation unit, and so are the kernels and attribute flags made from
// them.
namespace {
struct PartEpi {
    static constexpr bool kWhole = false;
    float *parts;
    int64_t M, ld;
    struct Row {
        float *p;
    };
    __device__ __forceinline__ void begin(Row &r, int64_t m, int part) const { r.p = parts + (part * M + m) * ld; }
    __device__ __forceinline__ void chunk(Row &r, int64_t, int64_t n, int cnt, const float (&v)[32]) const {
        // ld is a multiple of 32: the columns past the last one are there to be written
        float4 *p = reinterpret_cast<float4 *>(r.p + n);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    __device__ __forceinline__ void end(Row &, int64_t, int64_t) const {}
};
}  // namespace

// Adds the parts up, always in the same order, and hands them to the epilogue.
template <class Epi>
__global__ void __launch_bounds__(128) k_join_parts(const float *parts, int splits, int64_t M, int64_t N, int64_t ld,
                                                    const Epi epi) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, per = ld / 32;
    const int64_t m = i / per, n = i % per * 32;
    if (m >= M || n >= N) return;
    float v[32] = {};
    for (int s = 0; s < splits; ++s) {
        const float4 *p = reinterpret_cast<const float4 *>(parts + (s * M + m) * ld + n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 q = p[j];
            v[4 * j] += q.x, v[4 * j + 1] += q.y, v[4 * j + 2] += q.z, v[4 * j + 3] += q.w;
        }
    }
    typename Epi::Row row;
    epi.begin(row, m, 0);
    epi.chunk(row, m, n, N - n < 32 ? (int)(N - n) : 32, v);
    epi.end(row, m, 0);
}

// Floats of scratch memory that product_in_parts needs.
inline int64_t part_floats(int64_t M, int64_t N, int64_t K) {
    const int s = plan_product(M, N, K).splits;
    return s > 1 ? s * M * round_up(N, 32) : 0;
}

// A product whose K is shared out where there are too few tiles for the SMs.
template <Form FA, Form FB, class Epi>
int product_in_parts(const Matrix &A, const Matrix &B, int64_t M, int64_t N, int64_t K, const Epi &epi, float *parts,
                     cudaStream_t stream) {
    const int splits = plan_product(M, N, K).splits;
    if (splits == 1) return launch_product<FA, FB>(A, B, M, N, K, epi, stream);
    const int64_t ld = round_up(N, 32);
    const int rc = launch_product<FA, FB>(A, B, M, N, K, PartEpi{parts, M, ld}, stream, splits);
    if (rc != PP_OK) return rc;
    k_join_parts<Epi><<<(unsigned)ceil_div(M * (ld / 32), 128), 128, 0, stream>>>(parts, splits, M, N, ld, epi);
    PPS_CUDA_TRY(cudaGetLastError());
    return PP_OK;
}

// 32 columns of a row as bf16, or added to / stored as 32-bit floats.
__device__ __forceinline__ void store_bf16(uint16_t *p, int cnt, bool vec, const float (&v)[32]) {
    if (vec && cnt == 32) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4 *>(p)[j] =
                make_uint4(f32_to_bf16x2(v[8 * j], v[8 * j + 1]), f32_to_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                           f32_to_bf16x2(v[8 * j + 4], v[8 * j + 5]), f32_to_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cnt) p[j] = f32_to_bf16(v[j]);
    }
}
__device__ __forceinline__ void load_f32(const float *p, int cnt, bool vec, float (&v)[32]) {
    if (vec && cnt == 32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 q = reinterpret_cast<const float4 *>(p)[j];
            v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = j < cnt ? p[j] : 0.f;
    }
}
__device__ __forceinline__ void store_f32(float *p, int cnt, bool vec, const float (&v)[32]) {
    if (vec && cnt == 32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            reinterpret_cast<float4 *>(p)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cnt) p[j] = v[j];
    }
}

// A copy of rows at any stride and alignment as panels (or aligned rows), the
// last panel's columns past H as zeros; with `target`, a row whose target is
// outside 0..V-1 becomes 0.
int launch_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H, const int64_t *target, int64_t V,
                     uint16_t *out, int64_t ld, int64_t panel, cudaStream_t stream);

}  // namespace pps
