// per_device.h -- what the host works out once for every CUDA device of the process: a
// kernel's attributes and a device's sizes hold for the device that was current when they
// were set or read.  No CUDA header is needed here.
#pragma once

#include <atomic>

namespace pkv {

// One positive int per device, made by the first call that needs it.  Host threads may call
// together: two that come first both make the value, which has to be the same.
class PerDevice {
public:
    // *value = this device's; make(value) returns 0 or an error, which is returned and not remembered.
    template <class F>
    int get(int device, int* value, F make) {
        const bool kept = device >= 0 && device < kDevices;
        if (kept && (*value = made_[device].load(std::memory_order_acquire)) > 0) return 0;
        const int e = make(value);
        if (e == 0 && kept) made_[device].store(*value, std::memory_order_release);
        return e;
    }

private:
    static constexpr int kDevices = 64;   // a device past them is asked every time
    std::atomic<int> made_[kDevices]{};
};

}  // namespace pkv
