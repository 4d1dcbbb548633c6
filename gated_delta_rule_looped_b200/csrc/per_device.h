// per_device.h -- a number that is found once for each GPU and kept (internal).
#pragma once

#include <atomic>

namespace lt2 {

class PerDevice {
public:
    // The number of device `dev`: kept, or what find() gives (above 0; anything else is not kept).
    template <typename F>
    int get(int dev, F find)
    {
        const bool keep = dev >= 0 && dev < kDevices;
        int n = keep ? kept_[dev].load(std::memory_order_relaxed) : 0;
        if (n > 0) return n;
        n = find();
        if (keep && n > 0) kept_[dev].store(n, std::memory_order_relaxed);
        return n;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> kept_[kDevices] = {};
};

}  // namespace lt2
