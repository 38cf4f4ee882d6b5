// Conversions between float32, fp16 and e4m3 (four significant bits, 448 at
// most, no infinities). Every e4m3 value is an fp16 one.
#pragma once

#include "common.cuh"

namespace tpk {

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint16_t x) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) {
    float2 r;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(x));
    return r;
}

// log2 of a positive normal number, to 2^-22 beside its exponent.
__device__ __forceinline__ float log2_of(float x) {
    const int bits = __float_as_int(x);
    return (float)((bits >> 23) - 127) + __log2f(__int_as_float((bits & 0x007FFFFF) | 0x3F800000));
}

// Two float32 values as e4m3, to nearest even, beyond 448 as 448 (infinities too).
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace tpk
