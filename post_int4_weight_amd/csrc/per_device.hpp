// What a process sets up once on each device that it uses. Plain C++, no HIP.
#pragma once

#include <atomic>
#include <cstdint>

namespace ptq {

// once(device, ask): ask() where it has not yet succeeded on this device (on one past the 64 that are remembered: always).
// Threads may come at once, and may then ask twice.
class PerDevice {
    std::atomic<uint64_t> done{0};

public:
    template <typename Ask>
    int once(int device, Ask&& ask) {
        const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
        if (done.load(std::memory_order_acquire) & bit) return 0;
        const int status = ask();
        if (status == 0) done.fetch_or(bit, std::memory_order_release);
        return status;
    }
};

}  // namespace ptq
