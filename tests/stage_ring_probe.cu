// One block that takes rows through the library's ring (stage_ring.cuh) as the
// kernels of the join do, with a short limit on its waits.  A row's barrier can
// be told of 16 bytes that no copy brings, so that the wait for it runs out.
#include "stage_ring.cuh"

namespace pps {
int register_wait_reader(WaitReader *) { return 0; }

constexpr int kThreads = 64, kStages = kMaxStages, kHeader = 128;

// out[t]: the sum of row t's words, 0 for rows after the one held up.
// issued: rows asked for.  landed[i]: whether the last copy into slot i had landed when the block ended.
__global__ void __launch_bounds__(kThreads) k_probe(const uint32_t *in, int rows, int words, int held, unsigned long long limit,
                                                    uint32_t *out, uint32_t *issued, uint32_t *landed) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RingState state;
    __shared__ uint32_t sum;
    const uint32_t bytes = 4u * words;
    const Ring<1> ring{tc::smem_u32(smem) + kHeader, tc::smem_u32(smem), bytes, kStages,
                       {{(const unsigned char *)in, bytes, bytes, 0}}};
    const auto hold = [&](int row, int slot) {
        if (row == held)
            asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(ring.bars + 8 * slot) : "memory");
    };
    int n = 0;
    if (threadIdx.x == 0) {
        ring.init(&state);
        for (int i = 0; i < kStages && i < rows; ++i) hold(i, i), ring.load(&state, i, i, 0), n = i + 1;
    }
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    for (int t = 0; t < rows; ++t) {
        if (threadIdx.x == 0) sum = 0;
        __syncthreads();
        const bool came = tc::mbar_wait(ring.bars + 8 * slot, parity, &state.stop, 5, limit);
        const uint32_t *row = reinterpret_cast<const uint32_t *>(smem + kHeader + slot * bytes);
        uint32_t s = 0;
        for (int i = threadIdx.x; came && i < words; i += kThreads) s += row[i];
        atomicAdd(&sum, s);
        __syncthreads();
        if (threadIdx.x == 0) {
            out[t] = held >= 0 && t >= held ? 0 : sum;
            if (t + kStages < rows) {
                hold(t + kStages, slot);
                ring.refill(&state, t + kStages, slot, parity);
                n += !state.stop;
            }
        }
        if (++slot == kStages) slot = 0, parity ^= 1;
    }
    if (threadIdx.x == 0) {
        ring.finish(&state, limit);
        *issued = n;
        for (int i = 0; i < kStages; ++i) landed[i] = i < n && tc::mbar_try(ring.bars + 8 * i, ((n - 1 - i) / kStages) & 1);
    }
}
}  // namespace pps

using namespace pps;

// Returns the CUDA status; *record is what a wait that ran out left.
extern "C" int ring_probe(const uint32_t *in, int rows, int words, int held, unsigned long long limit, uint32_t *out,
                          uint32_t *issued, uint32_t *landed, uint64_t *record) {
    k_probe<<<1, kThreads, kHeader + kStages * 4 * words>>>(in, rows, words, held, limit, out, issued, landed);
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return (int)e;
    return take_wait_failure(record);
}
