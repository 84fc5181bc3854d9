// What the files of the C ABI share: the status helpers and argument checks
// (defined in api.cpp). Every check that can be made on the host runs before
// the first HIP call.
#pragma once

#include <cstdint>
#include <limits>

#include "w8a8.h"   // include/ is on the include path
#include "internal.hpp"

#define W8A8_API extern "C" __attribute__((visibility("default")))

namespace w8a8 {
namespace api {

constexpr int64_t kMaxRows = std::numeric_limits<int32_t>::max();

// Records the thread's error text and returns s.
w8a8_status_t fail(w8a8_status_t s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns W8A8_OK.
w8a8_status_t ok();
// Whether the current device can run the library.
w8a8_status_t check_device();
// The status of a launch.
w8a8_status_t launched(hipError_t e, const char *what);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace api
}  // namespace w8a8
