// Host-side helpers shared by the two halves of the C ABI (api.cpp for
// moe.h, api_train.cpp for moe_train.h); defined in api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include "moe.h"

namespace moe {

constexpr int32_t kAlignMaxExperts = 1024;

// Sets moe_last_error() to the formatted message and returns `st`.
moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears moe_last_error().
moe_status ok();
// MOE_OK when the current device is a gfx950.
moe_status check_device();
// A HIP runtime result as a status.
moe_status hip_status(hipError_t err, const char* what);

}  // namespace moe
