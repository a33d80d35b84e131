// kv.cuh -- device helpers of the key/value cache's kernels.
#pragma once

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

// SMs of the current device (0: cannot be asked).
inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

}  // namespace si
