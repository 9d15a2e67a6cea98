// stage_waits.h -- the records of waits that ran out: a word in each
// translation unit's device memory, read and cleared from the host.  Host code
// only.
#pragma once

#include <cstdint>
#include <mutex>

namespace pps {

// How one translation unit's word is read and cleared: 0, or the CUDA error that kept it from that.
struct WaitReader {
    int (*take)(uint64_t *word);
    WaitReader *next;
};

class WaitRecords {
public:
    void add(WaitReader *r) {
        std::lock_guard<std::mutex> lk(mu_);
        r->next = first_;
        first_ = r;
    }
    // The first record found.  A word that cannot be read is an error, not "no failure"; the others are taken all the same.
    int take(uint64_t *record) {
        std::lock_guard<std::mutex> lk(mu_);
        *record = 0;
        int rc = 0;
        for (const WaitReader *r = first_; r; r = r->next) {
            uint64_t word = 0;
            const int e = r->take(&word);
            if (e && !rc) rc = e;
            if (!*record) *record = word;
        }
        return rc;
    }

private:
    std::mutex mu_;
    WaitReader *first_ = nullptr;
};

}  // namespace pps
