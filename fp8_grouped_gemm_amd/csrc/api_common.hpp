// What the C ABI sources share: the thread's error message, the device check and the
// argument-check macro (defined in api.cpp).
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/moe.h"

namespace moe {

// Stores the message that moe_last_error() returns on this thread; returns `status`.
__attribute__((format(printf, 2, 3))) int fail(int status, const char* fmt, ...);
// MOE_OK if device `dev` is a gfx950
int check_device(int dev);
// the current device must be gfx950; fills the CU count
int current_device(int* cus);
int hip_status(hipError_t e, const char* what);

}  // namespace moe

#define REQUIRE(cond, ...) \
  do {                     \
    if (!(cond)) return moe::fail(MOE_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)
