// Work that is done once for each device of the process (plain C++).
#pragma once

#include <stdint.h>

#include <atomic>

namespace sgi {

// For settings that belong to a device, like a kernel's attributes: runs set()
// on the first call for a device and returns its result; later calls return 0
// at once, unless set() failed (a result other than 0), which is not
// remembered.  Threads that come first at the same time may each run set(), so
// it has to be harmless to repeat.  Devices from 64 run it on every call.
class OncePerDevice {
public:
    template <typename F>
    auto operator()(int device, F set) -> decltype(set()) {
        const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
        if (done_.load(std::memory_order_acquire) & bit) return decltype(set())(0);
        const auto result = set();
        if (result == decltype(result)(0)) done_.fetch_or(bit, std::memory_order_release);
        return result;
    }

private:
    std::atomic<uint64_t> done_{0};
};

}  // namespace sgi
