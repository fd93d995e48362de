// State that belongs to a device and is set or asked once for each: a kernel's
// attributes and its resident clusters hold for the device that was current, and
// a process may use several.  Nothing of CUDA here.
#pragma once

#include <atomic>

namespace gb300 {

constexpr int MAX_DEVICES = 64;

// The device of the library call in progress on this thread (set as the call
// looks up its device's state; 0 before any).
int call_device();

// A step that has to succeed once on each device (two threads may both take it).
class OncePerDevice {
 public:
  // `step` on the first call for device dev and on those after a failure
  template <class E, class F>
  E run(int dev, E ok, F step) {
    if (done_[dev].load(std::memory_order_acquire)) return ok;
    const E e = step();
    if (e == ok) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<bool> done_[MAX_DEVICES] = {};
};

// A count asked of each device once.
class CountPerDevice {
 public:
  // the count that `ask` gave for device dev; a negative one (it failed) is not
  // kept and counts as none
  template <class F>
  int get(int dev, F ask) {
    int kept = kept_[dev].load(std::memory_order_relaxed);
    if (kept == 0) {
      const int n = ask();
      if (n < 0) return 0;
      kept = n + 1;
      kept_[dev].store(kept, std::memory_order_relaxed);
    }
    return kept - 1;
  }

 private:
  std::atomic<int> kept_[MAX_DEVICES] = {};  // one more than the count; 0: not asked
};

}  // namespace gb300
