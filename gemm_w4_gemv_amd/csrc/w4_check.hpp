// Argument checks and error reporting shared by the C-ABI files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

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
inline bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return true;
    return false;
}
inline bool any_overlap(std::initializer_list<Range> outs) {
    for (const Range& a : outs)
        for (const Range& b : outs)
            if (&a != &b && overlap(a, b)) return true;
    return false;
}

// Bytes from the first to past the last value of ``rows`` rows of ``wide`` values.
inline Range rows_range(const void* p, int64_t rows, int64_t stride, int64_t wide, size_t value = 2) {
    return range(p, p && rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)wide) * value : 0);
}

}  // namespace w4
