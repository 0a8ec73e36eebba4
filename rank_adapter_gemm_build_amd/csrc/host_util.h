// Helpers shared by the host sources of the C ABI: error reporting, the device of a
// call, kernel timing.  Defined in api.cpp.
#pragma once

#include <hip/hip_runtime_api.h>

#include "common.h"

namespace rax {

// Record the calling thread's error message; both return the status to hand back.
lora_status fail(lora_status code, const char* fmt, ...);
lora_status ok();
lora_status hip_fail(hipError_t e, const char* what);

// Make `device` current for the scope, restoring the previous device after.
struct DeviceGuard {
  int prev = -1;
  hipError_t err = hipSuccess;
  explicit DeviceGuard(int device) {
    err = hipGetDevice(&prev);
    if (err == hipSuccess && prev != device) err = hipSetDevice(device);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

lora_status check_device(int device);

// Events for the next launch of `kernel` (none unless timing is enabled)
KTimer timer_for(int kernel);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace rax
