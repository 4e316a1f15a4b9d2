// per_device.cuh -- a number that is found out once for each device (plain
// C++: no CUDA call of its own).
#pragma once

#include <atomic>

namespace rlscan {
namespace seq {

// get(device, find): what find() gave on the device's first call, a positive
// number; anything else is a failure, which the next call tries again.  Two
// threads may both come first: they find the same.
class PerDevice {
public:
    static constexpr int kDevices = 64;

    template <class F>
    int get(int device, F find)
    {
        if (device < 0 || device >= kDevices) return find();
        int v = known_[device].load(std::memory_order_relaxed);
        if (v <= 0) {
            v = find();
            if (v > 0) known_[device].store(v, std::memory_order_relaxed);
        }
        return v;
    }

private:
    std::atomic<int> known_[kDevices] = {};
};

}  // namespace seq
}  // namespace rlscan
