// Host helpers shared by the C ABI's entry points: the error text, the device
// check and the pointer checks. Defined in api.cpp.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe_api {

constexpr int kMaxDevices = 64;

// Stores the text moe_last_error() returns on this thread; returns `status`.
moe_status fail(moe_status status, const char* fmt, ...);
// MOE_OK if the current device is gfx950.
moe_status check_device();
moe_status launched(hipError_t err, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace moe_api

#define REQUIRE_PTR(p)                                                           \
  do {                                                                           \
    if (!(p)) return moe_api::fail(MOE_EINVAL, "%s is NULL", #p);                \
    if (!moe_api::aligned16(p))                                                  \
      return moe_api::fail(MOE_EALIGN, "%s is not 16-byte aligned", #p);         \
  } while (0)
