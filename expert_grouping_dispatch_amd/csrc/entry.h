// Helpers of the C entry points: pointer and size checks, the gfx950 device
// check, and the status of a launch.
#pragma once

#include <atomic>
#include <cstdlib>
#include <cstring>

#include "internal.h"
#include "moe_route.h"

namespace moe {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_device_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The kernels are written for gfx950 only; any other device is rejected
// rather than run on code built for another target.  For tests of this
// rejection, MOE_ROUTE_ASSUME_ARCH (when set) stands in for the device's
// architecture name.
inline int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  int state = dev < kMaxDevices ? g_device_ok[dev].load(std::memory_order_relaxed) : 0;
  if (state == 0) {
    hipDeviceProp_t prop;
    state = 2;
    if (hipGetDeviceProperties(&prop, dev) == hipSuccess) {
      const char* forced = std::getenv("MOE_ROUTE_ASSUME_ARCH");
      const char* a = forced != nullptr ? forced : prop.gcnArchName;
      if (std::strncmp(a, "gfx950", 6) == 0 && (a[6] == '\0' || a[6] == ':')) state = 1;
    }
    if (dev < kMaxDevices) g_device_ok[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? MOE_OK : MOE_ERR_UNSUPPORTED_DEVICE;
}

inline int launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

inline bool slots_ok(int64_t n_rows, int32_t top_k) {
  if (n_rows < 0 || top_k < 1 || top_k > MOE_MAX_TOP_K) return false;
  return n_rows <= int64_t(0xFFFFFFFEu) / top_k;  // every slot index and position < sentinel
}

}  // namespace moe
