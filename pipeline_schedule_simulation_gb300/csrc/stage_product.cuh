// stage_product.cuh -- matrix products of the pipeline-stage operators on the
// tensor cores.
//
// C[m][n] = sum_k A(m,k) B(n,k) over bf16 operands, summed in 32 bits in TMEM
// and handed to an epilogue instead of being stored.  Epilogues that store C
// (kStore), with columns in quads where `vec` says that rows are aligned and one
// by one otherwise (part: which part of K):
//   finish(row, m, n, v)   columns n .. n+31 of row m: scaled, added, in place
//   narrow()               whether rows are stored as bf16:
//   row(m, n, v)           then 32 finished columns at once,
//   put(m, n, v, part)     else four
//   with(row, m, n)        what one column is added to
//   one(row, m, n, v, b, part)  one column, from the sum and that to memory
// The others get a row as a thread has it.  A row's part of a column tile is two
// pieces, the even and the odd runs of 32 columns.  All of them:
//   typename Epi::Row  what a row needs beside its sums
//   begin(row, m)      loads that
// and those that store C:
//   kSide              which rows use that: kNoRow, kSomeRows, kEveryRow
//   of_lane(row, lane) another lane's
//   apart(row), one_apart(row, n, v)  (kSomeRows) those rows, and what is done with
//                      one column of such a row beside one()
// and those that do not:
//   take(row, m, n0, end, N, piece, v, own)  one piece: run i is the columns from
//                      n0 + 64 i on, below `end` and (what exists) N; own: 32 floats
//                      of shared memory of the lane's own, one every 32
//   kWhole             runs go on to the next multiple of 64 past N, and none is
//                      cut by a tile's end
//
// Persistent blocks, one to an SM: a warp loads 64-deep slices of A and B by
// TMA into a ring, a thread issues the MMAs of a tile into one of two TMEM
// accumulators, eight warps take the other accumulator through the epilogue.
// Operands come K-major or MN-major as they lie in memory; both forms use the
// 128-byte swizzle.  What the library lays out itself lies in panels of 64
// columns (128 bytes), each panel's rows one after the other, so that a box is
// one run of memory in either form.
//
// The tensor cores add up in 32 bits but cut the sum off below its last bit at
// every step, so a long sum shrinks: by about 6e-7 of itself over 1024 k where
// the terms have one sign, and in proportion to that length.  A sum is therefore
// taken in runs of 2048 k: each run goes to the other accumulator, and the
// epilogue's threads, which hold the tile in registers, add the runs up with
// rounding.  A run lasts 16384 cycles, taking it over less than a tenth of that,
// beside the next run; it costs nothing that can be measured (4096 x 131072 x
// 4096 in 2.55 ms with and without), and the log-sum-exp of 4096-wide logits is
// off by 5e-7 of itself instead of 1.2e-6.
//
// CG = 2: a pair of blocks shares a tile of 256 x 256: each holds half of A
// and half of B, so that a slice costs each SM 32 KB of loads for its half of
// 256 x 256 x 64 products.
// CG = 1: a block takes a tile of 128 rows and 16 to 256 columns, chosen so
// that the tiles fill the SMs: for products with few tiles, and for few rows,
// where reading B is all that counts.
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

// One slice k of an operand's rows (m or n) from i0 on, as many as the map's box holds
// (MN-major rows: `rows`, a multiple of 64, in boxes of 64).
template <int CG, Form F>
__device__ __forceinline__ void load_slice(uint32_t to, const CUtensorMap *map, int i0, int rows, int k, uint32_t bar) {
    if (F == kRowsK) tc::tma_load<CG>(to, map, k * 64, i0, 0, bar);
    if (F == kPanelsK) tc::tma_load<CG>(to, map, 0, i0, k, bar);
    if (F == kPanelsMN) tc::tma_load<CG>(to, map, 0, k * 64, i0 / 64, bar);
    if (F == kRowsMN)
        for (int i = 0; i < rows; i += 64) tc::tma_load<CG>(to + i * 128, map, i0 + i, k * 64, 0, bar);
}

constexpr int kTileK = 64, kHalf = 128;  // a block holds 128 rows of A
constexpr int kBytesA = kHalf * kTileK * 2;
constexpr int kRingBytes = 6 * 2 * kBytesA;  // 192 KB
template <int CG>
struct RingOf {
    static constexpr int kRowsB = CG == 2 ? 128 : 256;  // most rows of B in a block
    static constexpr int kStageBytes = kBytesA + kRowsB * kTileK * 2, kStages = kRingBytes / kStageBytes;
};
constexpr int kEpilogueWarps = 8, kProductThreads = 128 + 32 * kEpilogueWarps;
constexpr int kPieces = kEpilogueWarps / 4;  // pieces of a row's part of a tile
constexpr int kRuns = 256 / 32 / kPieces;    // runs of 32 columns in a piece
constexpr int kTurnBytes = 32 * 32 * 4;  // a warp's run of columns, turned for storing
constexpr int kProductSmem = kRingBytes + 1024 + kEpilogueWarps * kTurnBytes;
constexpr int kAccStride = 256;  // TMEM columns of an accumulator
constexpr int kRun = 32;         // slices (2048 k) that one accumulator adds up
// Registers: the epilogue's 8 warps take what the first 4 can spare.
constexpr int kLaunchRegs = 168, kFewRegs = 64, kManyRegs = 216;
static_assert(128 * kFewRegs + 32 * kEpilogueWarps * kManyRegs <= kProductThreads * kLaunchRegs);

struct ProductShape {
    int M, N, K;
    int tile_n;    // columns of a tile
    int mt, nt;    // tiles
    int group;     // row tiles that are taken together
    int splits;    // parts of K
    int k_blocks;  // slices of K in each part (the last may have fewer)
};

// Tile number -> (row tile, column tile): `group` row tiles at a time run
// through all column tiles, so that their slices of A stay in the L2 cache.
__device__ __forceinline__ void tile_at(const ProductShape &s, uint32_t i, int &m, int &n) {
    const uint32_t per = (uint32_t)s.group * s.nt, g = i / per;
    const int first = (int)g * s.group, rows = min(s.group, s.mt - first), r = (int)(i - g * per);
    m = first + r % rows;
    n = r / rows;
}

// Four columns of a row, aligned.
__device__ __forceinline__ void store_quad(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }

// 32 columns of a row as bf16, aligned.
__device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        reinterpret_cast<uint4 *>(p)[j] =
            make_uint4(f32_to_bf16x2(v[8 * j], v[8 * j + 1]), f32_to_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                       f32_to_bf16x2(v[8 * j + 4], v[8 * j + 5]), f32_to_bf16x2(v[8 * j + 6], v[8 * j + 7]));
}

// 32 columns of a row, aligned, added to what `to` holds, all loaded first.
__device__ __forceinline__ void add_f32(float (&v)[32], const float *to) {
    float4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = reinterpret_cast<const float4 *>(to)[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[4 * j] += b[j].x, v[4 * j + 1] += b[j].y, v[4 * j + 2] += b[j].z, v[4 * j + 3] += b[j].w;
}

// For epilogues that need nothing beside a row's sums.
enum Side { kNoRow, kSomeRows, kEveryRow };
struct NoRow {
    static constexpr Side kSide = kNoRow;
    struct Row {};
    __device__ __forceinline__ void begin(Row &, int64_t) const {}
};

// 32 rows x 32 columns, a row to a lane.  Each lane finishes its row's values
// (what they are added to comes in whole lines that way); then they are turned
// through the warp's shared memory and stored along the rows, 4 rows at once,
// where the lanes' own stores would be 16 bytes of 32 rows each: the weight
// gradient of 512 tokens on 8192 x 8192 takes 84 us into new memory, 142 us by
// the lanes.  (32 columns of bf16 are half a line either way; by the lanes they
// are 16 bytes a store, turned 8: those stay with the lanes.)  Unaligned rows
// are turned too, a column to a lane, 8 rows on their way at once.
template <class Epi>
__device__ __forceinline__ void store_run(const Epi &epi, const typename Epi::Row &side, float4 *turn, int lane, int64_t m0,
                                          int64_t M, int n, int end, int part, float (&v)[32]) {
    if (m0 >= M) return;
    const bool whole = epi.vec && end - n >= 32;
    if (whole && m0 + lane < M) epi.finish(side, m0 + lane, n, v);
    if (whole && epi.narrow()) {
        if (m0 + lane < M) epi.row(m0 + lane, n, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        turn[lane * 8 + (j ^ (lane & 7))] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    if (whole) {
        const int at = lane & 7, row = lane >> 3;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + row;
            const float4 x = turn[r * 8 + (at ^ (r & 7))];
            if (m0 + r < M) epi.put(m0 + r, n + 4 * at, x, part);
        }
    } else {
        const float *one = reinterpret_cast<const float *>(turn);
        const int rows = n + lane < end ? (M - m0 < 32 ? (int)(M - m0) : 32) : 0;
        const auto sum_of = [&](int r) { return one[r * 32 + ((lane >> 2) ^ (r & 7)) * 4 + (lane & 3)]; };
        for (int r0 = 0; r0 < (Epi::kSide == kEveryRow ? 32 : rows); r0 += 8) {
            [[maybe_unused]] typename Epi::Row of[8];
            float b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (Epi::kSide == kEveryRow) of[k] = epi.of_lane(side, r0 + k);
                b[k] = r0 + k < rows ? epi.with(of[k], m0 + r0 + k, n + lane) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + k;
                const float x = sum_of(r);
                if (r < rows) epi.one(of[k], m0 + r, n + lane, x, b[k], part);
            }
        }
        if constexpr (Epi::kSide == kSomeRows) {
            uint32_t apart = __ballot_sync(~0u, m0 + lane < M && epi.apart(side));
            for (; apart; apart &= apart - 1) {
                const int r = __ffs(apart) - 1;
                const typename Epi::Row its = epi.of_lane(side, r);
                if (r < rows) epi.one_apart(its, n + lane, sum_of(r));
            }
        }
    }
    __syncwarp();
}

// A place in a ring of N: the slot, and the parity of its current round.
template <int N>
struct Place {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) slot = 0, round ^= 1;
    }
    __device__ __forceinline__ void back() {
        if (--slot < 0) slot = N - 1, round ^= 1;
    }
};

template <class Epi, Form FA, Form FB, int CG>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const ProductShape s, const Epi epi) {
    constexpr bool A_MN = is_mn(FA), B_MN = is_mn(FB);
    constexpr int kStages = RingOf<CG>::kStages, kStageBytes = RingOf<CG>::kStageBytes;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_at;
    __shared__ int stop;
    const uint32_t ring = (tc::smem_u32(raw) + 1023) & ~1023u;
    const uint32_t full = tc::smem_u32(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? tc::cluster_rank() : 0;
    const int rows_b = s.tile_n / CG;
    const uint32_t tiles = (uint32_t)s.mt * s.nt * s.splits, first = blockIdx.x / CG, step = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(acc_full + 8 * i, 1);
            tc::mbar_init(acc_empty + 8 * i, kEpilogueWarps * CG);
        }
        tc::mbar_init(drained, 1);
        stop = 0;
        tc::fence_barrier_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    if (warp == 2) tc::tmem_alloc<CG>(tc::smem_u32(&tmem_at), 2 * kAccStride);
    tc::fence_before();
    __syncthreads();
    if (CG == 2) tc::cluster_sync();  // the other block's barriers are ready
    tc::fence_after();
    const uint32_t tmem = tmem_at;
    let_next_start();
    after_previous();
    const int all_blocks = (s.K + kTileK - 1) / kTileK;

    if (warp < 4) {
        tc::give_registers<kFewRegs>();
        if (warp == 0) {
            if (lane == 0) {
                Place<kStages> at;
                int loaded = 0;  // slots that have been filled, up to all of them
                bool ok = true;
                for (uint32_t t = first; t < tiles && ok; t += step) {
                    const int part = (int)(t % s.splits);
                    int m, n;
                    tile_at(s, t / s.splits, m, n);
                    const int m0 = (m * CG + (int)rank) * kHalf, n0 = n * s.tile_n + (int)rank * rows_b;
                    const int k0 = part * s.k_blocks, k1 = min(k0 + s.k_blocks, all_blocks);
                    for (int k = k0; k < k1; ++k, at.next()) {
                        const int st = at.slot;
                        if (!tc::mbar_wait(empty + 8 * st, at.round ^ 1, &stop, 1)) {
                            ok = false;
                            break;
                        }
                        const uint32_t a = ring + st * kStageBytes, b = a + kBytesA;
                        // a pair's loads all count on the first block's barrier
                        const uint32_t bar = CG == 2 ? tc::in_block(full + 8 * st, 0) : full + 8 * st;
                        if (rank == 0) tc::mbar_expect(full + 8 * st, CG * (kBytesA + rows_b * kTileK * 2));
                        load_slice<CG, FA>(a, &map_a, m0, kHalf, k, bar);
                        load_slice<CG, FB>(b, &map_b, n0, rows_b, k, bar);
                        if (loaded < kStages) ++loaded;
                    }
                }
                // after giving up: the copies still in flight land before the block ends
                if (!ok) {
                    if (rank == 0)
                        for (; loaded > 0; --loaded) {
                            at.back();
                            tc::mbar_drain(full + 8 * at.slot, at.round);
                        }
                    else
                        tc::let_land();
                }
            }
        } else if (warp == 1) {
            if (lane == 0 && rank == 0) {
                const uint32_t idesc = tc::instr_desc(kHalf * CG, s.tile_n, A_MN, B_MN);
                // 16 k further: 32 bytes along a K-major row, two groups of 8 k in the MN-major form
                constexpr uint32_t step_a = A_MN ? 2048 : 32, step_b = B_MN ? 2048 : 32;
                Place<kStages> at;
                Place<2> run;
                bool ok = true;
                for (uint32_t t = first; t < tiles && ok; t += step) {
                    const int part = (int)(t % s.splits);
                    const int k0 = part * s.k_blocks, k1 = min(k0 + s.k_blocks, all_blocks);
                    for (int r0 = k0; r0 < k1 && ok; r0 += kRun, run.next()) {
                        const int buf = run.slot, r1 = min(r0 + kRun, k1);
                        if (!tc::mbar_wait(acc_empty + 8 * buf, run.round ^ 1, &stop, 2)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        for (int k = r0; k < r1; ++k, at.next()) {
                            const int st = at.slot;
                            if (!tc::mbar_wait(full + 8 * st, at.round, &stop, 3)) {
                                ok = false;
                                break;
                            }
                            tc::fence_after();
                            const uint32_t a = ring + st * kStageBytes, b = a + kBytesA;
#pragma unroll
                            for (int kk = 0; kk < kTileK / 16; ++kk)
                                tc::mma<CG>(tmem + buf * kAccStride, tc::smem_desc(a + kk * step_a, A_MN ? 8192 : 16, 1024),
                                            tc::smem_desc(b + kk * step_b, B_MN ? 8192 : 16, 1024), idesc,
                                            k > r0 || kk > 0);
                            tc::mma_commit<CG>(empty + 8 * st);
                        }
                        if (ok) tc::mma_commit<CG>(acc_full + 8 * buf);
                    }
                }
                // the MMAs have finished before TMEM is given back
                tc::mma_commit<CG>(drained);
                tc::mbar_drain(drained, 0);
            }
        }
    } else {
        tc::take_registers<kManyRegs>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int wide = Epi::kWhole ? (s.N + 63) & ~63 : s.N;
        Place<2> run;
        bool ok = true;
        // what a row needs beside its sums is loaded a tile ahead, or where results are stored (and the stores of the
        // tile before are still on their way) before the wait for the sums
        typename Epi::Row next{};
        const auto begin_next = [&](uint32_t t) {
            if constexpr (!Epi::kStore) {
                if (t >= tiles) return;
                int mt, nt;
                tile_at(s, t / s.splits, mt, nt);
                const int64_t m = (int64_t)(mt * CG + (int)rank) * kHalf + quarter * 32 + lane;
                if (m < s.M) epi.begin(next, m);
            }
        };
        begin_next(first);
        for (uint32_t t = first; t < tiles && ok; t += step) {
            const int part = (int)(t % s.splits);
            int mt, nt;
            tile_at(s, t / s.splits, mt, nt);
            const int64_t m = (int64_t)(mt * CG + (int)rank) * kHalf + quarter * 32 + lane;
            const int first_n = nt * s.tile_n, n0 = first_n + half * 32, n1 = min(first_n + s.tile_n, wide);
            const int k0 = part * s.k_blocks, k1 = min(k0 + s.k_blocks, all_blocks);
            const bool live = m < s.M;
            typename Epi::Row row = next;
            if constexpr (Epi::kStore)
                if (live) epi.begin(row, m);
            uint32_t sum[kRuns][32];  // floats, as the loads give them
            for (int r0 = k0; r0 < k1; r0 += kRun, run.next()) {
                const int buf = run.slot;
                // lanes give up one by one: the warp goes on together
                ok = __all_sync(~0u, tc::mbar_wait(acc_full + 8 * buf, run.round, &stop, 4));
                if (!ok) break;
                tc::fence_after();
                const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + buf * kAccStride + half * 32;
                if (r0 > k0) {
#pragma unroll
                    for (int i = 0; i < kRuns; ++i)
                        if (n0 + i * kPieces * 32 < n1) {
                            uint32_t v[32];
                            tc::tmem_load32(acc + i * kPieces * 32, v);
                            tc::tmem_wait();
                            tc::tmem_loaded(v);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                sum[i][c] = __float_as_uint(__uint_as_float(sum[i][c]) + __uint_as_float(v[c]));
                        }
                } else {
                    // nothing else is in these registers yet: all loads at once
#pragma unroll
                    for (int i = 0; i < kRuns; ++i)
                        if (n0 + i * kPieces * 32 < n1) tc::tmem_load32(acc + i * kPieces * 32, sum[i]);
                    tc::tmem_wait();
#pragma unroll
                    for (int i = 0; i < kRuns; ++i) tc::tmem_loaded(sum[i]);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) tc::mbar_arrive_at(tc::in_block(acc_empty + 8 * buf, 0));
                    else tc::mbar_arrive(acc_empty + 8 * buf);
                }
            }
            float v[kRuns][32];
#pragma unroll
            for (int i = 0; i < kRuns; ++i)
#pragma unroll
                for (int c = 0; c < 32; ++c) v[i][c] = __uint_as_float(sum[i][c]);
            float4 *turn = reinterpret_cast<float4 *>(raw + (ring - tc::smem_u32(raw)) + kRingBytes + (warp - 4) * kTurnBytes);
            if constexpr (Epi::kStore) {
                if (ok) {
                    const int64_t m_first = m - lane;
                    const int end = min(n1, s.N);
#pragma unroll
                    for (int i = 0; i < kRuns; ++i) {
                        const int n = n0 + i * kPieces * 32;
                        if (n < n1) store_run(epi, row, turn, lane, m_first, s.M, n, end, part, v[i]);
                    }
                }
            } else {
                begin_next(t + step);
                if (ok && live) epi.take(row, m, n0, n1, s.N, kPieces * nt + half, v, reinterpret_cast<float *>(turn) + lane);
                __syncwarp();
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (CG == 2) tc::cluster_sync();  // neither block ends while the other may still signal it
    tc::fence_after();
    if (warp == 2) tc::tmem_free<CG>(tmem, 2 * kAccStride);
}

// ---- host side

// The map of an operand of `rows` x `cols` as it lies in memory, for boxes of
// box_rows x 64 x box_panels.
int encode_map(CUtensorMap *map, const Matrix &m, int64_t rows, int64_t cols, bool panels, int box_rows,
               int box_panels);

// I: the operand's extent along m or n, K along k; `rows` of I in a box.
template <Form F>
int map_of(CUtensorMap *map, const Matrix &m, int64_t I, int64_t K, int rows) {
    if (F == kRowsK) return encode_map(map, m, I, K, false, rows, 1);
    if (F == kPanelsK) return encode_map(map, m, I, K, true, rows, 1);
    if (F == kPanelsMN) return encode_map(map, m, K, I, true, 64, rows / 64);
    return encode_map(map, m, K, I, false, 64, 1);
}

// How a product is cut.  A slice of 64 k costs a pair of blocks 512 cycles
// (its 256 x 256 x 64 products), a lone block with n columns 256 + 2n (its
// loads, 64 bytes a cycle); a tile costs some slices more for its start and
// end, a part of K its sums written and read again.  The cheapest of: pairs;
// lone blocks with as many columns as fill the SMs once, twice, ... (a
// multiple of 16, of 64 where B is MN-major or the epilogue takes whole
// columns); each whole, and with K in as many parts (of at least 4 slices) as
// fill the SMs.
struct ProductPlan {
    int cg, splits, tile_n;
    int64_t mt, nt;
};
ProductPlan plan_product(int64_t M, int64_t N, int64_t K, bool by_64, bool may_split);

template <Form FA, Form FB, class Epi>
int launch_product(const Matrix &A, const Matrix &B, int64_t M, int64_t N, int64_t K, const Epi &epi,
                   const ProductPlan &p, cudaStream_t stream) {
    if (M <= 0 || N <= 0 || K <= 0) return PP_ERR_INTERNAL;
    if (p.mt * p.nt * p.splits > 0x7FFFFFFF) return PP_ERR_SIZE;  // tiles are counted in 32 bits
    CUtensorMap ma, mb;
    int rc = map_of<FA>(&ma, A, M, K, kHalf);
    if (rc == PP_OK) rc = map_of<FB>(&mb, B, N, K, p.tile_n / p.cg);
    if (rc != PP_OK) return rc;
    ProductShape s;
    s.M = (int)M, s.N = (int)N, s.K = (int)K;
    s.tile_n = p.tile_n;
    s.mt = (int)p.mt, s.nt = (int)p.nt;
    s.splits = p.splits;
    s.k_blocks = (int)ceil_div(ceil_div(K, kTileK), p.splits);
    s.group = s.mt < 16 ? s.mt : 16;
    const int64_t tiles = p.mt * p.nt * p.splits, most = sm_count() / p.cg, grid = (tiles < most ? tiles : most) * p.cg;
    static std::atomic<uint64_t> ready[2];
    const auto kernel = p.cg == 1 ? k_product<Epi, FA, FB, 1> : k_product<Epi, FA, FB, 2>;
    if (!ready[p.cg - 1].load(std::memory_order_relaxed)) {
        // the epilogue's warps would wait forever for registers that the launch does not have
        cudaFuncAttributes fa;
        PPS_CUDA_TRY(cudaFuncGetAttributes(&fa, kernel));
        if (fa.numRegs < kLaunchRegs) return PP_ERR_INTERNAL;
    }
    rc = allow_smem(kernel, kProductSmem, ready[p.cg - 1]);
    if (rc != PP_OK) return rc;
    return launch_after(kernel, grid, kProductThreads, kProductSmem, stream, p.cg, ma, mb, s, epi);
}

// A product that is not to be cut along K: its epilogue takes whole sums.
template <Form FA, Form FB, class Epi>
int whole_product(const Matrix &A, const Matrix &B, int64_t M, int64_t N, int64_t K, const Epi &epi,
                  cudaStream_t stream) {
    return launch_product<FA, FB>(A, B, M, N, K, epi, plan_product(M, N, K, true, false), stream);
}

// Parts of K: each part's sums apart, [part][M][ld].  Epilogues are local to
// their translation unit, and so are the kernels and attribute flags made from
// them.
namespace {
struct PartEpi : NoRow {
    static constexpr bool kStore = true, kWhole = false;
    static constexpr bool vec = true;
    float *parts;
    int64_t M, ld;  // ld is a multiple of 4
    __device__ __forceinline__ bool narrow() const { return false; }
    __device__ __forceinline__ void finish(const Row &, int64_t, int64_t, float (&)[32]) const {}
    __device__ __forceinline__ void row(int64_t, int64_t, const float (&)[32]) const {}
    __device__ __forceinline__ void put(int64_t m, int64_t n, const float4 &v, int part) const {
        *reinterpret_cast<float4 *>(parts + (part * M + m) * ld + n) = v;
    }
    __device__ __forceinline__ float with(const Row &, int64_t, int64_t) const { return 0.f; }
    __device__ __forceinline__ void one(const Row &, int64_t m, int64_t n, float v, float, int part) const {
        parts[(part * M + m) * ld + n] = v;
    }
};
}  // namespace

// Adds the parts up, always in the same order, and hands them to the epilogue:
// 64 quads of columns a block, 4 threads to a quad.
template <class Epi>
__global__ void __launch_bounds__(256) k_join_parts(const float *parts, int splits, int64_t M, int64_t N, int64_t ld,
                                                    const Epi epi) {
    let_next_start();
    after_previous();
    __shared__ float4 sh[4][64];
    const int q = threadIdx.x & 63, run = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 64 + q, per = ld / 4;
    const int64_t m = i / per, n = (i - m * per) * 4;
    const bool in = m < M && n < N;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    // what the sums are added to is on its way beside the parts
    typename Epi::Row row{};
    float b[4] = {};
    if (!run && in) {
        epi.begin(row, m);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < N) b[j] = epi.with(row, m, n + j);
    }
    if (in) {
        const float4 *p = reinterpret_cast<const float4 *>(parts + m * ld + n);
#pragma unroll 4
        for (int s = run; s < splits; s += 4) {
            const float4 x = p[s * (M * ld / 4)];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
    }
    sh[run][q] = v;
    __syncthreads();
    if (run || !in) return;
#pragma unroll
    for (int r = 1; r < 4; ++r) {
        const float4 x = sh[r][q];
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < N) {
            if constexpr (Epi::kSide == kSomeRows)
                if (epi.apart(row)) epi.one_apart(row, n + j, x[j]);
            epi.one(row, m, n + j, x[j], b[j], 0);
        }
}

// Floats of scratch memory that product_in_parts needs (B is MN-major there).
inline int64_t part_floats(int64_t M, int64_t N, int64_t K) {
    const int s = plan_product(M, N, K, true, true).splits;
    return s > 1 ? s * M * round_up(N, 4) : 0;
}

// A product whose K is shared out where that is cheaper.
template <Form FA, Form FB, class Epi>
int product_in_parts(const Matrix &A, const Matrix &B, int64_t M, int64_t N, int64_t K, const Epi &epi, float *parts,
                     cudaStream_t stream) {
    static_assert(is_mn(FB));
    const ProductPlan p = plan_product(M, N, K, true, true);
    if (p.splits == 1) return launch_product<FA, FB>(A, B, M, N, K, epi, p, stream);
    const int64_t ld = round_up(N, 4);
    const int rc = launch_product<FA, FB>(A, B, M, N, K, PartEpi{{}, parts, M, ld}, p, stream);
    if (rc != PP_OK) return rc;
    return launch_after(k_join_parts<Epi>, ceil_div(M * (ld / 4), 64), 256, 0, stream, 1, (const float *)parts, p.splits, M,
                        N, ld, epi);
}

// A copy of rows at any stride and alignment as panels (or aligned rows), the
// last panel's columns past H as zeros; with `target`, a row whose target is
// outside 0..V-1 becomes 0, and the V words from `clear` (null: none) become -1.
int launch_copy_rows(const uint16_t *x, int64_t stride, int64_t T, int64_t H, const int64_t *target, int64_t V,
                     int *clear, uint16_t *out, int64_t ld, int64_t panel, cudaStream_t stream);

}  // namespace pps
