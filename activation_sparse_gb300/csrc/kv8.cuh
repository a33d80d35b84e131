// kv8.cuh -- device helpers of a cache in 8 bits: e4m3 codes, and scale bytes
// that are biased exponents.
#pragma once

#include <cuda_fp16.h>

#include "kv.cuh"

namespace si {

constexpr int kScaleNaN = 255;

// What a scale byte stands for, within the cache's limits (never a subnormal).
__device__ __forceinline__ float scale_of(int byte, int lo, int hi) {
    return byte == kScaleNaN ? __int_as_float(0x7FC00000) : __int_as_float(min(max(byte, lo), hi) << 23);
}

// The exponent of what a scale byte stands for.
__device__ __forceinline__ float exponent_of(int byte, int lo, int hi) {
    return byte == kScaleNaN ? __int_as_float(0x7FC00000) : (float)(min(max(byte, lo), hi) - 127);
}

// The scale byte of a row whose largest magnitude is top: the least power of two whose 448-fold (1.75 * 2^8) reaches it.
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

// The four codes of a word as fp16, exactly: bytes 0, 1 and 2, 3.
__device__ __forceinline__ void halves4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Byte offset of 16-byte unit `unit` of row `row` in a tile of rows of DP codes; XORed so that the eight rows of an
// ldmatrix lie in different banks (two rows of 64 codes share the banks' 128 bytes).
template <int DP>
__device__ __forceinline__ uint32_t tile8_at(int row, int unit) {
    const int swap = DP == 64 ? (row >> 1) & 3 : row & 7;
    return (uint32_t)(row * DP + ((unit ^ swap) * 16));
}

// As Copy, for rows of codes: a warp copies WK keys of every tile, lane i % WK holding the slot of key i. A sweep's rows are
// neighbours, and PERIOD sweeps are eight rows: their places in the tile then differ by eight rows' bytes alone.
template <int DP, int WK = 16>
struct Copy8 {
    static constexpr int UNITS = DP / 16;
    static constexpr int AT_ONCE = 32 / UNITS;
    static constexpr int SWEEPS = WK / AT_ONCE;
    static constexpr int PERIOD = 8 / AT_ONCE;
    static __device__ __forceinline__ int row(int lane, int j) { return j * AT_ONCE + lane / UNITS; }
    static __device__ __forceinline__ void slots(int held, int lane, int (&slot)[SWEEPS]) {
#pragma unroll
        for (int j = 0; j < SWEEPS; ++j) slot[j] = __shfl_sync(0xFFFFFFFFu, held, row(lane, j));
    }
    // Where this lane's unit of the first sweeps' rows lies in the tile, and so that of sweep j.
    uint32_t at[PERIOD];
    __device__ __forceinline__ Copy8(int lane, int own0) {
#pragma unroll
        for (int j = 0; j < PERIOD; ++j) at[j] = tile8_at<DP>(own0 + row(lane, j), lane % UNITS);
    }
    __device__ __forceinline__ uint32_t place(int j) const { return at[j % PERIOD] + j / PERIOD * 8 * DP; }
};

// Where a lane's row of an ldmatrix of sixteen keys (0-7, 8-15 of a unit, then of the next unit) lies in a tile, for every
// two units; the next sixteen keys' lie 16 * DP bytes on.
template <int DP>
struct Load8 {
    uint32_t at[DP / 32];
    __device__ __forceinline__ Load8(int lane, int own0) {
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) at[i] = tile8_at<DP>(own0 + (lane & 15), 2 * i + (lane >> 4));
    }
    __device__ __forceinline__ uint32_t place(int u, int m) const { return at[u / 2] + m * 16 * DP; }
};

// d += a (16 x 16) * b (16 x 8)
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This lane's eight elements of a query row of D elements (nullptr: zeros), which the DP / 8 lanes of a group share.
template <int DP>
__device__ __forceinline__ uint4 query_load(const uint16_t* row, int D, int lane) {
    const int u = lane % (DP / 8);
    return row && u * 8 < D ? *reinterpret_cast<const uint4*>(row + u * 8) : make_uint4(0, 0, 0, 0);
}

// The same as fp16. fp16 queries are taken as they are; bf16 ones times the power of two that brings the row's largest into
// 2^14 .. 2^15, so that all down to 2^-29 of it is exact and what lies below good to 2^-39 of it: `down` undoes it. A
// row that is not finite stays as it is.
template <int DP>
__device__ __forceinline__ uint4 query_half(uint4 val, bool fp16, float& down) {
    down = 1.0f;
    if (fp16) return val;
    uint32_t w[4] = {val.x, val.y, val.z, val.w};
    uint32_t top = 0;  // the largest exponent
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7F80u, w[i] >> 16 & 0x7F80u));
#pragma unroll
    for (int o = 1; o < DP / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const int e = (int)(top >> 7), f = min(268 - e, 253);
    const float up = e < 255 ? __int_as_float(f << 23) : 1.0f;
    if (e < 255) down = __int_as_float((254 - f) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<true>(bf_lo(w[i]) * up, bf_hi(w[i]) * up);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A product's sum, up to 2^32, times a query row's `down` and the key's scale: past 2^64 `down` is taken in two parts, one
// on either side of the scale, which may bring the score back into fp32's range.
constexpr float kSteep = 18446744073709551616.0f;
__device__ __forceinline__ float rest_of(float down) { return fmaxf(down * (1.0f / kSteep), 1.0f); }

__device__ __forceinline__ bool code_nan(uint32_t code) { return (code & 0x7Fu) == 0x7Fu; }

}  // namespace si
