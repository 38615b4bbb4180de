// Host-side settings and answers that are kept per device and may be asked for
// by several threads at once.  Plain C++ (no CUDA header).
#pragma once

#include <atomic>
#include <mutex>

namespace as {

constexpr int KEPT_DEVICES = 64;  // devices above are asked every time

// A device setting that is only ever raised.  raise() returns 0, or what
// set(value) returned.  One thread sets at a time, and never to less than what
// is recorded, so that the setting is at least the recorded value.
class RaisedLimit {
  public:
    template <typename Set>
    int raise(int dev, int value, Set &&set)
    {
        const bool kept = dev >= 0 && dev < KEPT_DEVICES;
        if (kept && at_[dev].load(std::memory_order_acquire) >= value) return 0;
        std::lock_guard<std::mutex> lock(mutex_);
        if (kept && at_[dev].load(std::memory_order_relaxed) >= value) return 0;
        const int e = set(value);
        if (e == 0 && kept) at_[dev].store(value, std::memory_order_release);
        return e;
    }

  private:
    std::atomic<int> at_[KEPT_DEVICES] = {};
    std::mutex mutex_;
};

// A non-negative answer about a device.  Threads that ask first may both
// compute it (to the same value).
class DeviceAnswer {
  public:
    template <typename Ask>
    int get(int dev, Ask &&ask)
    {
        const bool kept = dev >= 0 && dev < KEPT_DEVICES;
        const int known = kept ? plus_one_[dev].load(std::memory_order_relaxed) : 0;
        if (known) return known - 1;
        const int answer = ask();
        if (kept) plus_one_[dev].store(answer + 1, std::memory_order_relaxed);
        return answer;
    }

  private:
    std::atomic<int> plus_one_[KEPT_DEVICES] = {};
};

}  // namespace as
