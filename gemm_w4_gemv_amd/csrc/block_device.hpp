// Eight neighbouring values of a row in a lane: one 16-byte load of BF16.
#pragma once

#include "w4_device.hpp"

namespace w4 {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8_t widen(const u32x4_t& w) {
    f32x8_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
    return v;
}
__device__ __forceinline__ u32x4_t narrow(const f32x8_t& v) {
    return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// Loads and stores that with kApart go past the caches' ways of keeping what is
// read or written once.
template <bool kApart, typename T>
__device__ __forceinline__ void put(T* p, const T& v) {
    if constexpr (kApart) {
        __builtin_nontemporal_store(v, p);
    } else {
        *p = v;
    }
}
template <bool kApart, typename T>
__device__ __forceinline__ T take(const T* p) {
    if constexpr (kApart) {
        return __builtin_nontemporal_load(p);
    } else {
        return *p;
    }
}

}  // namespace w4
