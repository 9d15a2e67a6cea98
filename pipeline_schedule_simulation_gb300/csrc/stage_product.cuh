// stage_product.cuh -- matrix products of the pipeline-stage operators.
//
// C[m][n] = sum_k A(m,k) B(n,k) over bf16 operands, summed in 32 bits, handed
// to an epilogue row by row instead of being stored:
//   typename Epi::Row  what a row keeps between its pieces
//   begin(row, m)      a row m of the tile starts
//   chunk(row, m, n, cnt, v)  columns n .. n+cnt-1 (cnt <= 32) of row m
//   end(row, m, tile)  the row's piece of column tile `tile` is done
// Each (row, column tile) is handed over by one thread, in column order.
#pragma once

#include "stage_common.cuh"

namespace pps {

// An operand: element (i, k) at p[i*ld + k] (k_major) or p[k*ld + i].
struct Operand {
    const uint16_t *p;
    int64_t ld;
    bool k_major;
    __device__ __forceinline__ uint16_t at(int64_t i, int64_t k) const {
        return k_major ? p[i * ld + k] : p[k * ld + i];
    }
};

constexpr int kTileN = 64;  // columns of one column tile

// One 64 x 64 tile per block, 4 x 4 elements per thread, 16 k at a time.
template <class Epi>
__global__ void __launch_bounds__(256) k_product(Operand A, Operand B, int64_t M, int64_t N, int64_t K, Epi epi) {
    __shared__ float sa[16][65], sb[16][65], sc[64][65];
    const int64_t mt = (M + 63) / 64, tile = blockIdx.x / mt;
    const int64_t m0 = blockIdx.x % mt * 64, n0 = tile * kTileN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            // consecutive threads follow the operand's contiguous direction
            const int ra = A.k_major ? i >> 4 : i & 63, ka = A.k_major ? i & 15 : i >> 6;
            const int rb = B.k_major ? i >> 4 : i & 63, kb = B.k_major ? i & 15 : i >> 6;
            sa[ka][ra] = m0 + ra < M && k0 + ka < K ? bf16_to_f32(A.at(m0 + ra, k0 + ka)) : 0.f;
            sb[kb][rb] = n0 + rb < N && k0 + kb < K ? bf16_to_f32(B.at(n0 + rb, k0 + kb)) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[ty + 16 * i][tx + 16 * j] = acc[i][j];
    __syncthreads();
    const int64_t m = m0 + threadIdx.x;
    if (threadIdx.x >= 64 || m >= M) return;
    typename Epi::Row row;
    epi.begin(row, m);
    for (int c = 0; c < kTileN && n0 + c < N; c += 32) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = sc[threadIdx.x][c + j];
        const int64_t left = N - n0 - c;
        epi.chunk(row, m, n0 + c, left < 32 ? (int)left : 32, v);
    }
    epi.end(row, m, tile);
}

inline int64_t column_tiles(int64_t N) { return ceil_div(N, kTileN); }

template <class Epi>
int launch_product(const Operand &A, const Operand &B, int64_t M, int64_t N, int64_t K, const Epi &epi,
                   cudaStream_t stream) {
    if (M <= 0 || N <= 0) return PP_OK;
    const int64_t blocks = ceil_div(M, 64) * column_tiles(N);
    if (blocks > 0x7FFFFFFF) return PP_ERR_SIZE;
    k_product<Epi><<<(unsigned)blocks, 256, 0, stream>>>(A, B, M, N, K, epi);
    PPS_CUDA_TRY(cudaGetLastError());
    return PP_OK;
}

}  // namespace pps
