// What the library's host files share: the calling thread's last error and the
// device guard.
#pragma once

#include <hip/hip_runtime.h>

namespace microadam {

// Records code and message for the calling thread and returns code.
__attribute__((visibility("hidden"))) int fail(int code, const char *fmt, ...);
__attribute__((visibility("hidden"))) void clear_error();

// Device guard: runs with the given device current, restores afterwards.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) { ok = false; return; }
    if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

}  // namespace microadam
