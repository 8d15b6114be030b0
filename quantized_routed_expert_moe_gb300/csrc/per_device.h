// What a process works out once per device, for calls from any host thread.
#pragma once

#include <atomic>

namespace moe {

// A positive number per device, kept once `make` has given it; 0 is a failure and is not
// kept. Threads that ask at the same time may each work it out, to the same result. Devices
// past the last of the table work it out every time.
class PerDevice {
public:
    static constexpr int kDevices = 16;
    template <class F>
    int get(int device, F make) {
        if (device < 0 || device >= kDevices) return make();
        int v = kept_[device].load(std::memory_order_acquire);
        if (v > 0) return v;
        v = make();
        if (v > 0) kept_[device].store(v, std::memory_order_release);
        return v;
    }

private:
    std::atomic<int> kept_[kDevices] = {};
};

}  // namespace moe
