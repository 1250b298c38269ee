// Host-side helpers shared by the library's translation units: error details
// (per thread, read back by fp8_gemm_strerror), argument checks, the device
// check and the launch status.  Defined in fp8_gemm.hip unless inline.
#pragma once

#include <stdint.h>

#include "../../include/fp8_gemm.h"

namespace fp8g_host __attribute__((visibility("hidden"))) {

// Record the detail of a failure and return its status; ok() clears it.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

// FP8G_OK when the current device is one this library is built for.
int check_device();

// The status of the kernel launch just made.
int launch_status(const char *what);

constexpr int64_t kMaxRowStride = (int64_t(1) << 23) - 16;   // keeps 256 rows of offsets below 2^31

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool dtype_ok(int d) { return d == FP8G_E4M3 || d == FP8G_E5M2; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace fp8g_host
