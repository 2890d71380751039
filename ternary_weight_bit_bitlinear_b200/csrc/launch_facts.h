// launch_facts.h -- what a launcher looks up once per device and keeps: facts
// that several host threads may ask for, and set, at once.  Two threads that
// look the same fact up store the same value, so no lock is needed, but each
// fact is one atomic word.
#pragma once

#include <atomic>
#include <cstdint>

namespace blh {

using FlagFact = std::atomic<bool>;   // a kernel attribute has been set
using CountFact = std::atomic<int>;   // 0: not looked up yet

// The value that belongs to the last key (positive) asked about.  Key and value
// are one word: a thread never finds its key with the value of another's.
class KeyedFact {
 public:
  bool get(int key, int* value) const {
    const uint64_t w = word_.load(std::memory_order_relaxed);
    *value = static_cast<int>(static_cast<uint32_t>(w));
    return static_cast<int>(w >> 32) == key;
  }
  void set(int key, int value) {
    word_.store(static_cast<uint64_t>(static_cast<uint32_t>(key)) << 32 |
                    static_cast<uint32_t>(value),
                std::memory_order_relaxed);
  }

 private:
  std::atomic<uint64_t> word_{0};
};

}  // namespace blh
