// per_device.h -- what the host has set up once on each device of the process.
#pragma once

#include <atomic>

namespace moe_host {

// A number by device, 0 before it is known: a kernel's attributes, and what follows from them, belong to
// a device's copy of the kernel.
class PerDevice {
  public:
    // The number reaches value: raise(value) sets it on the current device where it is still smaller, and says
    // whether that worked.
    template <typename Raise>
    bool reach(int device, int value, Raise raise) {
        if (device < 0 || device >= MOST) return raise(value);
        if (value <= at_[device].load(std::memory_order_acquire)) return true;
        if (!raise(value)) return false;
        at_[device].store(value, std::memory_order_release);
        return true;
    }

    // The number, made on the current device by make() the first time (0: it could not be made).
    template <typename Make>
    int get(int device, Make make) {
        if (device < 0 || device >= MOST) return make();
        int v = at_[device].load(std::memory_order_acquire);
        if (v == 0) at_[device].store(v = make(), std::memory_order_release);
        return v;
    }

  private:
    static constexpr int MOST = 64;
    std::atomic<int> at_[MOST] = {};
};

}  // namespace moe_host
