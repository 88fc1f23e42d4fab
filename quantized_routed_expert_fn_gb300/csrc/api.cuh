// api.cuh -- host helpers shared by the C ABI's translation units.
#pragma once

#include <cstddef>

namespace moe {

// Records the message moe_last_error() returns on this thread; returns code.
int fail(int code, const char *fmt, ...);

// Limit of every bounded device wait: MOE_TIMEOUT_MS (default 1000).
unsigned long long timeout_ns();

bool overlap(const void *a, size_t na, const void *b, size_t nb);

}  // namespace moe
