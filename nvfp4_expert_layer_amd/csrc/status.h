// Status and device helpers shared by the host files (defined in engine.cpp).
#pragma once
#include <hip/hip_runtime.h>

namespace moe {

// Records the message for moe_nvfp4_last_error and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();                                              // clears the message, returns OK
int hip_status(hipError_t e, const char* where);       // OK, or MOE_NVFP4_ERR_HIP with a message
int current_arch_ok(int* dev_out);                     // OK iff the current device is gfx950
int cu_count(int dev, int* out);                       // compute units of the current device `dev`

}  // namespace moe
