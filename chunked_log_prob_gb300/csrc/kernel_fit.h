// What the host knows of a kernel on each device: whether it has been opted in to
// large shared memory there (an attribute of the device), and how many of its
// CTAs fit an SM, of the last launch shape. Plain C++; safe between threads.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace grpo {

constexpr int kMaxDevices = 64;

class KernelFit {
 public:
  // The kept answer for this device and shape; false: none.
  bool find(int device, int threads, size_t smem, int* ctas) const {
    if (!known(device)) return false;
    const uint64_t seen = last_[device].load(std::memory_order_relaxed);
    if ((seen & ~uint64_t{0xff}) != key(threads, smem)) return false;
    *ctas = static_cast<int>(seen & 0xff);
    return true;
  }
  void keep(int device, int threads, size_t smem, int ctas) {
    if (known(device) && ctas >= 0 && ctas <= 0xff)
      last_[device].store(key(threads, smem) | static_cast<uint64_t>(ctas),
                          std::memory_order_relaxed);
  }
  bool opted_in(int device) const {
    return known(device) && opted_[device].load(std::memory_order_relaxed);
  }
  void set_opted_in(int device) {
    if (known(device)) opted_[device].store(true, std::memory_order_relaxed);
  }

 private:
  static bool known(int device) { return device >= 0 && device < kMaxDevices; }
  // Of up to 1024 threads and 227 KB; never 0, which stands for nothing kept.
  static uint64_t key(int threads, size_t smem) {
    return (static_cast<uint64_t>(smem) << 24) | (static_cast<uint64_t>(threads) << 8);
  }
  std::atomic<uint64_t> last_[kMaxDevices] = {};
  std::atomic<bool> opted_[kMaxDevices] = {};
};

}  // namespace grpo
