// append8.cu -- rotary append into a cache of e4m3 codes.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kAppendThreads = 256;

template <bool FP16>
__device__ __forceinline__ void widen8(const uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<FP16>(u[i]);
        f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
}

// Eight pairs in place: (x[i], y[i]) where the layout is half-split, else (x[0], x[1]), ..., (y[6], y[7]).
__device__ __forceinline__ void rotate8f(float (&x)[8], float (&y)[8], const float2* cs, bool interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 c = cs[i];
        float& p = !interleaved ? x[i] : i < 4 ? x[(2 * i) & 7] : y[(2 * i) & 7];
        float& r = !interleaved ? y[i] : i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7];
        const float a = p, b = r;
        p = a * c.x - b * c.y;
        r = b * c.x + a * c.y;
    }
}

template <bool FP16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(pack2<FP16>(f[0], f[1]), pack2<FP16>(f[2], f[3]), pack2<FP16>(f[4], f[5]), pack2<FP16>(f[6], f[7]));
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
    const uint32_t a = code2(f[0] * inv, f[1] * inv), b = code2(f[2] * inv, f[3] * inv);
    const uint32_t c = code2(f[4] * inv, f[5] * inv), d = code2(f[6] * inv, f[7] * inv);
    return make_uint2(a | b << 16, c | d << 16);
}

__device__ __forceinline__ unsigned size_of(const float (&f)[8]) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);  // NaN above infinity above all
    return m;
}

// One block per token, as the append in 16 bits. A key or value row of a head
// is a group of 2^group lanes, 16 elements a lane (eight pairs; the elements
// past the pairs eight a lane), so that its largest magnitude is a few
// shuffles. The row is scaled and rounded from the fp32 values.
template <bool FP16>
__global__ void __launch_bounds__(kAppendThreads)
    k_kv_append8(const __grid_constant__ KvAppendParams P, const __grid_constant__ RopeTable R, int group) {
    __shared__ float2 cs[kRopeMaxPairs];
    grid_launch_dependents();
    grid_dependency_wait();
    const long long tok = blockIdx.x;
    const int b = (int)(blockIdx.x / (unsigned)P.T), t = (int)(blockIdx.x - (unsigned)b * (unsigned)P.T);
    const int np = R.n_pairs, tid = threadIdx.x;
    for (int i = tid; i < np; i += kAppendThreads) cs[i] = turned(P.pos[tok * R.n_axes + R.axis[i]], R.turn[i]);
    const KvView& C = P.c;
    const int D = C.D, Hkv = C.Hkv;
    const int len = C.len[b];
    const bool fits = len >= 0 && len <= C.cap - P.T;
    if (!fits && tid == 0) atomicOr(P.err, SI_DEVERR_CACHE);
    const int32_t* list = C.table ? C.table + b * C.tb + len + t : nullptr;
    __syncthreads();

    const int rot = np / 8;                       // lanes of a head's pairs
    const int tail = (D - 2 * np) / 8;            // 16-byte units past them
    if (fits) {
        const uint16_t* k = static_cast<const uint16_t*>(P.k) + b * P.kb + t * P.kt;
        const uint16_t* v = static_cast<const uint16_t*>(P.v) + b * P.vb + t * P.vt;
        const int part = tid & ((1 << group) - 1);
        for (int base = 0; base < 2 * Hkv; base += kAppendThreads >> group) {
            const int task = base + (tid >> group);
            const bool is_v = task >= Hkv;
            const int head = is_v ? task - Hkv : task;
            const long long slot = task >= 2 * Hkv ? -1 : list ? list[head * C.th] : len + t;
            const bool on = slot >= 0 && slot < C.n_slots;
            if (!on && task < 2 * Hkv && part == 0) atomicOr(P.err, SI_DEVERR_CACHE);
            float x[8] = {}, y[8] = {};
            int o0 = -1, o1 = -1;                 // places of x and y in the row
            if (on) {
                const uint16_t* src = is_v ? v + head * P.vh : k + head * P.kh;
                if (is_v) {
                    if (part < D / 16) o0 = part * 16, o1 = o0 + 8;
                } else if (part < rot) {
                    o0 = R.interleaved ? part * 16 : part * 8;
                    o1 = R.interleaved ? o0 + 8 : np + o0;
                } else if (part < rot + tail) {
                    o0 = 2 * np + (part - rot) * 8;
                }
                if (o0 >= 0) widen8<FP16>(*reinterpret_cast<const uint4*>(src + o0), x);
                if (o1 >= 0) widen8<FP16>(*reinterpret_cast<const uint4*>(src + o1), y);
                if (!is_v && part < rot) rotate8f(x, y, cs + part * 8, R.interleaved);
            }
            uint8_t* scale = is_v ? C.v_scale + b * C.vcb + head * C.vch : C.k_scale + b * C.kcb + head * C.kch;
            int byte = kScaleNaN;
            if (C.block_shift == 0) {
                unsigned m = max(size_of(x), size_of(y));
                for (int o = 1; o < 1 << group; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                byte = scale_byte_for(__uint_as_float(m), C.e_lo, C.e_hi);
                if (on && part == 0) scale[slot] = (uint8_t)byte;
            } else if (on) {
                byte = scale[slot >> C.block_shift];
                if (byte != kScaleNaN) byte = min(max(byte, C.e_lo), C.e_hi);
            }
            if (!on) continue;
            const float inv = __int_as_float((254 - byte) << 23);  // 2^(127 - byte)
            uint2 cx = make_uint2(0, 0), cy = cx;
            if (byte != kScaleNaN) cx = codes8(x, inv), cy = codes8(y, inv);
            uint8_t* dst = is_v ? static_cast<uint8_t*>(const_cast<void*>(C.v)) + b * C.vb + head * C.vh + slot * C.vs
                                : static_cast<uint8_t*>(const_cast<void*>(C.k)) + b * C.kb + head * C.kh + slot * C.ks;
            if (o0 >= 0) *reinterpret_cast<uint2*>(dst + o0) = cx;
            if (o1 >= 0) *reinterpret_cast<uint2*>(dst + o1) = cy;
            if (!is_v && part == 0 && C.acc) C.acc[b * C.ab + head * C.ah + slot] = 0.0f;
        }
    }

    const int per_q = rot + tail;
    const uint16_t* q = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt;
    uint16_t* qo = static_cast<uint16_t*>(P.q_out) + tok * P.Hq * D;
    for (int u = tid; u < P.Hq * per_q; u += kAppendThreads) {
        const int head = div_of(u, per_q), part = u - head * per_q;
        const uint16_t* src = q + head * P.qh;
        uint16_t* dst = qo + (long long)head * D;
        if (part >= rot) {
            const int o = 2 * np + (part - rot) * 8;
            *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
        } else {
            const int o0 = R.interleaved ? part * 16 : part * 8, o1 = R.interleaved ? o0 + 8 : np + o0;
            float x[8], y[8];
            widen8<FP16>(*reinterpret_cast<const uint4*>(src + o0), x);
            widen8<FP16>(*reinterpret_cast<const uint4*>(src + o1), y);
            rotate8f(x, y, cs + part * 8, R.interleaved);
            *reinterpret_cast<uint4*>(dst + o0) = narrow8<FP16>(x);
            *reinterpret_cast<uint4*>(dst + o1) = narrow8<FP16>(y);
        }
    }
}

}  // namespace

cudaError_t launch_kv_append8(const KvAppendParams& P, const RopeTable& R, cudaStream_t st) {
    const int np = R.n_pairs, lanes = np / 8 + (P.c.D - 2 * np) / 8;  // of a key's row: at most 31; a value's takes fewer
    int group = 0;
    while ((1 << group) < lanes || (1 << group) < P.c.D / 16) ++group;
    void* args[3] = {const_cast<KvAppendParams*>(&P), const_cast<RopeTable*>(&R), &group};
    const void* fn = P.c.fp16 ? reinterpret_cast<const void*>(&k_kv_append8<true>)
                              : reinterpret_cast<const void*>(&k_kv_append8<false>);
    return launch(fn, dim3((unsigned)((long long)P.c.B * P.T), 1, 1), kAppendThreads, 0, args, st);
}

}  // namespace si
