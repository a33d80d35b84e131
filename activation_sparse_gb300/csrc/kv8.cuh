// kv8.cuh -- device helpers of a cache in 8 bits: e4m3 codes, and scale bytes
// that are biased exponents.
#pragma once

#include <cuda_fp16.h>

#include "kv.cuh"

namespace si {

constexpr float kE4m3Max = 448.0f;  // 1.75 * 2^8
constexpr int kScaleNaN = 255;

// What a scale byte stands for, within the cache's limits (never a subnormal).
__device__ __forceinline__ float scale_of(int byte, int lo, int hi) {
    return byte == kScaleNaN ? __int_as_float(0x7FC00000) : __int_as_float(min(max(byte, lo), hi) << 23);
}

// The scale byte of a row whose largest magnitude is top: the least power of two whose 448-fold reaches it.
__device__ __forceinline__ int scale_byte_for(float top, int lo, int hi) {
    const int bits = __float_as_int(top);  // >= 0
    if (bits >= 0x7F800000) return kScaleNaN;
    const int e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000);  // 448's fraction; a subnormal is below every lo
    return min(max(e, lo), hi);
}

// Two codes from two floats, to nearest, what exceeds 448 becomes 448; a in the low byte.
__device__ __forceinline__ uint32_t code2(float a, float b) {
    uint16_t w;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(b), "f"(a));
    return w;
}

// Two codes (the low 16 bits) as two fp16, exactly.
__device__ __forceinline__ uint32_t halves(uint16_t codes) {
    uint32_t w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(codes));
    return w;
}

__device__ __forceinline__ bool code_nan(uint32_t code) { return (code & 0x7Fu) == 0x7Fu; }

}  // namespace si
