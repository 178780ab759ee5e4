// What the C ABI files share: error reporting, the device's properties and the checks of
// an output epilogue (defined in api.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "launch.h"

namespace w4 {

// Record the message of a failure on this thread and return `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear this thread's message and return W4_OK.
int ok();
int launched(hipError_t e, const char* what);
DeviceCaps device_caps();
// Output epilogue over outc columns from the caller's bias, dtype and segments (validated).
int make_epi(int64_t outc, int64_t M, const void* bias, int out_dtype, const w4_out_seg* segs, int nsegs, Epi* ep);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace w4
