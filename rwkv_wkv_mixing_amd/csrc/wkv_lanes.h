// What the delta-rule and norm kernels share: float32 and bf16 values, and sums over the lanes of a wave without a
// trip through LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wkv {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
// a and b rounded to bf16, a in the lower half
__device__ __forceinline__ uint32_t pk2(float a, float b) {
    const f2 p = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf2));
}

template <int Ctrl>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), Ctrl, 0xf, 0xf, true));
}

// x summed over the aligned groups of `lanes` lanes (a power of two, the same for the whole wave), to all
// of them.  The partners are lane ^ 1, lane ^ 2, then the mirrored lane of the 8 and of the 16 (whose
// halves are already uniform), then the other row of 16 and the other half of the wave: both partners add
// the same two numbers, so every lane gets the same bits.
__device__ __forceinline__ float sum_lanes(float x, int lanes) {
    if (lanes > 1) x += dpp<0xB1>(x);    // quad_perm [1, 0, 3, 2]
    if (lanes > 2) x += dpp<0x4E>(x);    // quad_perm [2, 3, 0, 1]
    if (lanes > 4) x += dpp<0x141>(x);   // row_half_mirror
    if (lanes > 8) x += dpp<0x140>(x);   // row_mirror
    if (lanes > 16) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if (lanes > 32) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return x;
}

// x summed over the four lanes l, l + 16, l + 32, l + 48
__device__ __forceinline__ float sum_rows(float x) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

}  // namespace wkv
