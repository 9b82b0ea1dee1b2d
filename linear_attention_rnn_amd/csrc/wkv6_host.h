// What the library's C ABI layers share on the host: the calling thread's
// error text (wkv6_last_error) and the per-device workspace pool.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include <string>

namespace wkv6 {

// Sets the calling thread's error text; returns `status`.
int set_error(int status, const std::string& msg);

// Workspace in stream order from the current device's pool (hipFreeAsync
// gives it back).
hipError_t workspace_alloc(void** p, size_t bytes, hipStream_t stream);

}  // namespace wkv6
