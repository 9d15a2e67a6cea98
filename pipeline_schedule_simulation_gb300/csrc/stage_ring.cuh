// stage_ring.cuh -- rows that one block takes one after the other, brought into
// a ring in shared memory by bulk copies several rows ahead of the arithmetic.
#pragma once

#include "stage_tc.cuh"

namespace pps {

constexpr int kMaxStages = 4;

// What the block's threads share beside the ring's barriers: whether a wait of
// theirs ran out, and for each slot the parity of the round that it was filled
// for last (-1: never).
struct RingState {
    int stop, round[kMaxStages];
};

// A row is `parts` bulk copies into the ring's next stage.
struct RowPart {
    const unsigned char *p;
    int64_t stride;  // bytes
    uint32_t bytes, at;
};
template <int PARTS>
struct Ring {
    uint32_t base, bars, stage_bytes;
    int stages;
    RowPart part[PARTS];

    // The rest are calls of the loading thread.
    __device__ __forceinline__ void init(RingState *st) const {
        st->stop = 0;
        for (int i = 0; i < kMaxStages; ++i) st->round[i] = -1;
        for (int i = 0; i < stages; ++i) tc::mbar_init(bars + 8 * i, 1);
        tc::fence_barrier_init();
    }
    __device__ __forceinline__ void load(RingState *st, int64_t row, int slot, uint32_t round) const {
        const uint32_t bar = bars + 8 * slot, to = base + slot * stage_bytes;
        tc::mbar_expect(bar, stage_bytes);
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
            if (part[i].bytes) tc::bulk_load(to + part[i].at, part[i].p + row * part[i].stride, part[i].bytes, bar);
        st->round[slot] = (int)round;
    }
    // Fills a slot again that every thread has read in the round of this parity, unless a wait of the block has run
    // out: one of this thread's that did has set `stop`, so no slot is filled whose last copy may still be in flight.
    __device__ __forceinline__ void refill(RingState *st, int64_t row, int slot, uint32_t round) const {
        if (*(volatile int *)&st->stop) return;
        tc::fence_async();
        load(st, row, slot, round ^ 1);
    }
    // Before the block ends.  If a wait ran out, the copies still in flight land (each waited for with a limit again),
    // so that none writes to shared memory that has become another block's.
    __device__ __forceinline__ void finish(const RingState *st, unsigned long long limit = tc::kWaitNs) const {
        if (!*(volatile const int *)&st->stop) return;  // every copy has been waited for
        for (int i = 0; i < stages; ++i)
            if (st->round[i] >= 0) tc::mbar_drain(bars + 8 * i, (uint32_t)st->round[i], limit);
    }
};

}  // namespace pps
