// What the C ABI's sources share: the calling thread's last error, the device check and
// the argument checks' helpers.  abi.cpp defines the functions.
#pragma once

#include "w4a8_moe.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {
namespace abi {

// records the error detail of the calling thread and returns status
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// clears it
int ok();
// W4A8_OK if the current device is a gfx950; fills the error detail otherwise
int check_device();
// the status of a launch
int launched(hipError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMaxRows = (int64_t)1 << 31;   // row indices are int32

}  // namespace abi
}  // namespace w4a8
