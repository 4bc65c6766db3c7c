// The status text of the C entry points: one description per thread, set by
// every call.
#pragma once

#include <hip/hip_runtime.h>

#include "dspark.h"

namespace dspark {

// Stores the description of a refusal and returns its status.
dspark_status fail(dspark_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
dspark_status ok();
// DSPARK_E_LAUNCH with the runtime's text, or ok().
dspark_status launched(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dspark
