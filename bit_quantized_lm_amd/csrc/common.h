// Internal helpers shared by the host and device translation units of the
// draft-head library (not part of the public ABI).
#pragma once

#include <stdint.h>

#include <atomic>

namespace dh {

// What has to be done once on every device before a kernel runs there. Calls of
// several threads may meet in the first one and do it twice, so it has to bear that;
// what failed (a result other than `good`) is tried again by the next call.
class OncePerDevice {
 public:
  template <class Result, class F>
  Result run(int device, Result good, F&& f) {
    const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;   // beyond: every time
    if (done_.load(std::memory_order_acquire) & bit) return good;
    const Result r = f();
    if (r == good) done_.fetch_or(bit, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// Record `msg` as the calling thread's last error and return `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear the calling thread's last error and return DH_OK.
int ok();

}  // namespace dh
