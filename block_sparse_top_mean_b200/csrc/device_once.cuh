// A record of the devices on which something was done once.  Devices from 64 on are never
// recorded (the work is done again each time there), so they cannot stand for another.
#pragma once

#include <stdint.h>

#include <atomic>

namespace msa {

class DeviceOnce {
 public:
  bool done(int dev) const { return (bits_.load(std::memory_order_relaxed) & bit(dev)) != 0; }
  void mark(int dev) { bits_.fetch_or(bit(dev), std::memory_order_relaxed); }

 private:
  static uint64_t bit(int dev) { return dev >= 0 && dev < 64 ? 1ull << dev : 0; }
  std::atomic<uint64_t> bits_{0};
};

}  // namespace msa
