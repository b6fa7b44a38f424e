// Host helpers shared by the C ABI's entry points: the error text, the device
// check and the pointer checks. Defined in api.cpp.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_int8.h"

namespace moe_api {

constexpr int kMaxDevices = 64;

// Stores the text moe_last_error() returns on this thread; returns `status`.
moe_status fail(moe_status status, const char* fmt, ...);
// MOE_OK if the current device is gfx950.
moe_status check_device();
moe_status launched(hipError_t err, const char* what);

// The routing's sizes, and a layer's: H and I multiples of hmod and imod, 32-bit offsets.
moe_status check_route_dims(int32_t T, int32_t E, int32_t k);
moe_status check_shape(const moe_shape* s, int hmod, int imod);

inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }


// Arrays of a call: no output may overlap an input or another output.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
  bool out;
};
template <int N>
moe_status check_overlap(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i) {
    if (!s[i].out || !s[i].p || !s[i].bytes) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = a + s[i].bytes;
    for (int j = 0; j < N; ++j) {
      if (j == i || (s[j].out && j < i) || !s[j].p || !s[j].bytes) continue;
      const uintptr_t c = reinterpret_cast<uintptr_t>(s[j].p), d = c + s[j].bytes;
      if (a < d && c < b) return fail(MOE_EINVAL, "%s overlaps %s in memory", s[i].name, s[j].name);
    }
  }
  return MOE_OK;
}
inline size_t values(int64_t rows, int64_t cols, int type) {
  return static_cast<size_t>(rows) * cols * (type == MOE_F32 ? 4 : type == MOE_INT8 ? 1 : 2);
}

}  // namespace moe_api

#define REQUIRE_PTR(p)                                                           \
  do {                                                                           \
    if (!(p)) return moe_api::fail(MOE_EINVAL, "%s is NULL", #p);                \
    if (!moe_api::aligned16(p))                                                  \
      return moe_api::fail(MOE_EALIGN, "%s is not 16-byte aligned", #p);         \
  } while (0)
