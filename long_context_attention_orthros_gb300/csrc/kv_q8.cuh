// kv_q8.cuh -- the 8-bit KV cache: one row (d values of one KV head) is held as d codes
// (e4m3 or int8) and one exponent e, and stands for code * 2^e.
//
// e is the smallest whole number with max|x| 2^-e <= M (M = 448 for e4m3, 127 for int8),
// clamped to [-126, 127] and 0 for a row of zeros; the codes are x 2^-e rounded to nearest
// even.  A power of two makes x 2^-e exact in fp32 (so every implementation of the definition
// gives the same codes) and code 2^e exact in bf16 (4 and 7 significant bits; only below
// bf16's smallest value is it rounded).  A value that is not finite has no code: the row's e
// then comes from its finite values, an e4m3 code of it is NaN, an int8 code is the nearest
// end of the range (0 for a NaN), and ORTHROS_DEVERR_RANGE is set.
#pragma once

#include <cuda_fp16.h>

#include "serve.cuh"

namespace orthros {

// exponent of a row whose largest finite |x| is amax
template <int CODE>
__device__ __forceinline__ int q8_exponent(float amax)
{
    constexpr int TOP = CODE == ORTHROS_KV_E4M3 ? 8 : 6;  // M = (1 + f) 2^TOP
    constexpr uint32_t MANT = CODE == ORTHROS_KV_E4M3 ? 0x600000u : 0x7e0000u;  // f: 0.75 and 63/64, as fp32 bits
    const uint32_t u = __float_as_uint(amax);
    if (u == 0u)
        return 0;
    // a subnormal amax has the field 0: its exponent is below the clamp all the same
    const int e = static_cast<int>(u >> 23) - 127 - TOP + ((u & 0x7fffffu) > MANT ? 1 : 0);
    return e < -126 ? -126 : e;
}

// 2^n for a whole n in [-127, 127]
__device__ __forceinline__ float q8_pow2(int n)
{
    return __uint_as_float(n > -127 ? static_cast<uint32_t>(127 + n) << 23 : 0x400000u);
}

// codes of two finite values already scaled by 2^-e, in the low 16 bits (a in the lowest byte)
template <int CODE>
__device__ __forceinline__ uint32_t q8_codes2_finite(float a, float b)
{
    if constexpr (CODE == ORTHROS_KV_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    } else {
        return (static_cast<uint32_t>(__float2int_rn(a)) & 0xffu) | (static_cast<uint32_t>(__float2int_rn(b)) & 0xffu) << 8;
    }
}

// the same for any two values: what is not finite becomes NaN (e4m3), the end of the range or 0 (int8)
template <int CODE>
__device__ __forceinline__ uint32_t q8_codes2(float a, float b)
{
    if constexpr (CODE == ORTHROS_KV_E4M3) {
        // the conversion saturates, so that infinities are made NaN first
        if (!(fabsf(a) < __int_as_float(0x7f800000)))
            a = __int_as_float(0x7fffffff);
        if (!(fabsf(b) < __int_as_float(0x7f800000)))
            b = __int_as_float(0x7fffffff);
        return q8_codes2_finite<CODE>(a, b);
    } else {
        const uint32_t r = q8_codes2_finite<CODE>(fminf(fmaxf(a, -127.f), 127.f), fminf(fmaxf(b, -127.f), 127.f));
        return (a == a ? r & 0xffu : 0u) | (b == b ? r & 0xff00u : 0u);
    }
}

// the two low (hi = false) or high codes of a word as fp16
template <int CODE>
__device__ __forceinline__ uint32_t q8_half2(uint32_t w, bool hi)
{
    if constexpr (CODE == ORTHROS_KV_E4M3) {
        uint32_t r;
        const uint16_t two = static_cast<uint16_t>(hi ? w >> 16 : w & 0xffffu);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
        return r;
    } else {
        // 0x6400 | u is 1024 + u: with u = code + 128, subtract 1152
        const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, hi ? 0x4342 : 0x4140);
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(1152.f));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
}

}  // namespace orthros
