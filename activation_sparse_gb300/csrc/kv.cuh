// kv.cuh -- device helpers of the key/value cache's kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kv.h"

namespace si {

// Wait site of the tree attention, beside those in common.cuh.
constexpr unsigned kSiteAttend = 6u << 8;

// a / b for 0 <= a, 0 < b, exact: a float quotient and its correction, a
// third of an integer division's instructions.
__device__ __forceinline__ int div_of(int a, int b) {
    int q = (int)__fdividef((float)a, (float)b);
    int r = a - q * b;
    while (r < 0) r += b, --q;
    while (r >= b) r -= b, ++q;
    return q;
}

template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(bf_lo(w), bf_hi(w));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t w;
    if (FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        w = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        w = *reinterpret_cast<const uint32_t*>(&h);
    }
    return w;
}

// cos and sin of a pair's angle: the position times its turns, in 64-bit fixed point that wraps to the fraction of a
// turn (exact for any int32 position).
__device__ __forceinline__ float2 turned(long long pos, unsigned long long turn) {
    // signed fraction in half turns: [-1, 1)
    const float x = (float)(int32_t)(uint32_t)(((unsigned long long)pos * turn) >> 32) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c, s);
}

// SMs of the current device (0: cannot be asked).
inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

}  // namespace si
