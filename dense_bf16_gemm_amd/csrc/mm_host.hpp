// mm_host.hpp -- host helpers shared by the C ABI's sources: the error string,
// argument checks and the device's attributes.  Defined in mm_api.hip.
#pragma once

#include <stdint.h>

#include <string>

#include "../../include/mm.h"

#define MM_HIDDEN __attribute__((visibility("hidden")))

namespace mmh {

// Leaves `msg` for mm_last_error and returns `s`.
MM_HIDDEN mm_status fail(mm_status s, const std::string& msg);

// Whether two byte ranges share a byte (never with a null pointer or no bytes).
MM_HIDDEN bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes);

// Compute units of the current device (cached per device).
MM_HIDDEN mm_status device_cus(int* cus);

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace mmh
