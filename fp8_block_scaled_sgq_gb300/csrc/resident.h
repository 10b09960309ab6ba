// How many CTAs of a kernel an SM holds: asked once a device, by whichever call
// comes first there.  Only an answer is kept, so that a question which failed is
// put again by the next call.
#pragma once
#include <atomic>

namespace sgq {

class Resident {
    std::atomic<int> kept_[64] = {};

public:
    // ask(): the number, or 0 where it cannot be told.  0: as ask(), or no such device.
    template <typename Ask>
    int on(int dev, Ask ask) {
        if (dev < 0 || dev >= 64) return 0;
        int n = kept_[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
        n = ask();
        if (n > 0) kept_[dev].store(n, std::memory_order_relaxed);
        return n > 0 ? n : 0;
    }
};

}  // namespace sgq
