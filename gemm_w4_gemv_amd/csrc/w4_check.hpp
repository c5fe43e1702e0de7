// Argument checks and error reporting shared by the C-ABI files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w4.h"

namespace w4 {

// Records the message that w4_last_error() returns on this thread (w4_api.hip).
w4_status fail(w4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline w4_status hip_fail(hipError_t err, const char* what) {
    return fail(W4_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(err), (int)err);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

}  // namespace w4
