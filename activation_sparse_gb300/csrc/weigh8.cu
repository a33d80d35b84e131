// weigh8.cu -- the attention weight that each key of a cache of e4m3 codes received.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kWarps = 4;

// A warp a key: it walks the rows that count.
__global__ void __launch_bounds__(32 * kWarps) k_kv_accumulate8(const __grid_constant__ AttendParams P) {
    grid_launch_dependents();
    grid_dependency_wait();
    const KvView& C = P.c;
    const int lane = threadIdx.x & 31, D = C.D, T = P.T;
    const int b = blockIdx.y / C.Hkv, h = blockIdx.y % C.Hkv;
    const int len = C.len[b];
    if (len < 0 || len > C.cap - T) {
        if (threadIdx.x == 0) atomicOr(P.err, SI_DEVERR_CACHE);
        return;
    }
    const int32_t* list = C.table ? C.table + b * C.tb + h * C.th : nullptr;
    const unsigned long long want = P.rows ? P.rows[b] : ~0ull;
    for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < len + T; i += gridDim.x * kWarps) {
        const long long slot = list ? list[i] : i;
        if (slot < 0 || slot >= C.n_slots) {
            if (lane == 0) atomicOr(P.err, SI_DEVERR_CACHE);
            continue;
        }
        const uint8_t* k = static_cast<const uint8_t*>(C.k) + b * C.kb + h * C.kh + slot * C.ks;
        const float sk = scale_of(C.k_scale[b * C.kcb + h * C.kch + (slot >> C.block_shift)], C.e_lo, C.e_hi);
        float kf[8], w = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t c = lane + 32 * e < D ? halves(k[lane + 32 * e]) : 0;
            kf[e] = __half2float(__low2half(*reinterpret_cast<const __half2*>(&c)));
        }
        for (int t = 0; t < T; ++t) {
            const unsigned long long word = word_of(P.mask, T, b, t);
            if (!(want >> t & 1) || word == 0 || (i >= len && !(word >> (i - len) & 1))) continue;
            for (int g = 0; g < P.G; ++g) {
                const float lse = P.lse[((long long)b * T + t) * P.Hq + h * P.G + g];
                const uint16_t* q = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)(h * P.G + g) * P.qh;
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (lane + 32 * e < D) s += kf[e] * (C.fp16 ? widen<true>(q[lane + 32 * e]) : widen<false>(q[lane + 32 * e]));
                s = warp_sum(s) * sk;
                if (lse != -INFINITY) w += ex2(__fadd_rn(__fmul_rn(s, P.scale), -lse) * kLog2e);
            }
        }
        const long long at = b * C.ab + h * C.ah + slot;
        if (lane == 0) P.acc_out[at] = C.acc[at] + w;
    }
}

}  // namespace

cudaError_t launch_kv_accumulate8(const AttendParams& P, cudaStream_t st) {
    const int blocks = (int)(((long long)P.c.cap + kWarps - 1) / kWarps);
    if ((long long)P.c.B * P.c.Hkv > 65535) return cudaErrorInvalidValue;
    void* args[1] = {const_cast<AttendParams*>(&P)};
    return launch(reinterpret_cast<const void*>(&k_kv_accumulate8), dim3(blocks < 4096 ? blocks : 4096, P.c.B * P.c.Hkv, 1),
                  32 * kWarps, 0, args, st);
}

}  // namespace si
