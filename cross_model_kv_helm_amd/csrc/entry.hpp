// entry.hpp — what the library's C entry points share: the per-thread error
// text, the argument checks' arithmetic and the device gate.  Defined in
// api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace helm::entry {

constexpr size_t kAlign = 256;   // of every workspace and of the pieces inside one
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Records the text helm_last_error() returns; returns `status`.
__attribute__((format(printf, 2, 3))) int fail(int status, const char* fmt, ...);
void clear_error();
bool mul_ok(int64_t& acc, int64_t f);
bool overlaps(const void* a, int64_t na, const void* b, int64_t nb);
int device_gate(int device);
int launch_status(hipError_t e, const char* what);

}  // namespace helm::entry
