// attend8.cu -- tree attention over a cache of e4m3 codes.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kWarps = 4;

// A warp a query row: it walks the list, each lane with its share of the
// elements, and keeps the running maximum and sum of the softmax.
__global__ void __launch_bounds__(32 * kWarps) k_tree_attention8(const __grid_constant__ AttendParams P) {
    grid_launch_dependents();
    grid_dependency_wait();
    const KvView& C = P.c;
    const int lane = threadIdx.x & 31, D = C.D, T = P.T;
    const long long id = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (id >= (long long)C.B * T * P.Hq) return;
    const int hq = (int)(id % P.Hq), t = (int)(id / P.Hq % T), b = (int)(id / P.Hq / T), h = hq / P.G;
    const int len = C.len[b];
    const bool fits = len >= 0 && len <= C.cap - T;
    if (!fits && lane == 0) atomicOr(P.err, SI_DEVERR_CACHE);
    const unsigned long long word = fits ? word_of(P.mask, T, b, t) : 0;
    const uint16_t* q = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + hq * P.qh;
    const int32_t* list = C.table ? C.table + b * C.tb + h * C.th : nullptr;
    const uint8_t* k = static_cast<const uint8_t*>(C.k) + b * C.kb + h * C.kh;
    const uint8_t* v = static_cast<const uint8_t*>(C.v) + b * C.vb + h * C.vh;
    const uint8_t* ksc = C.k_scale + b * C.kcb + h * C.kch;
    const uint8_t* vsc = C.v_scale + b * C.vcb + h * C.vch;
    float qf[8], o[8] = {}, top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = lane + 32 * i;
        qf[i] = d < D ? P.c.fp16 ? widen<true>(q[d]) : widen<false>(q[d]) : 0.0f;
    }
    auto code_of = [](uint8_t c) {
        const uint32_t w = halves(c);
        return __half2float(__low2half(*reinterpret_cast<const __half2*>(&w)));
    };
    for (int i = 0; word && i < len + T; ++i) {
        if (i >= len && !(word >> (i - len) & 1)) continue;
        const long long slot = list ? list[i] : i;
        if (slot < 0 || slot >= C.n_slots) {
            if (lane == 0) atomicOr(P.err, SI_DEVERR_CACHE);
            continue;
        }
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < D) s += qf[e] * code_of(k[slot * C.ks + lane + 32 * e]);
        s = warp_sum(s) * scale_of(ksc[slot >> C.block_shift], C.e_lo, C.e_hi);
        const float high = fmaxf(top, s), shift = high == -INFINITY ? 0.0f : high, c2 = P.scale * kLog2e;
        const float keep = ex2((top - shift) * c2), p = ex2((s - shift) * c2);
        const float w = p * scale_of(vsc[slot >> C.block_shift], C.e_lo, C.e_hi);
        top = high;
        sum = sum * keep + p;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < D) o[e] = o[e] * keep + w * code_of(v[slot * C.vs + lane + 32 * e]);
    }
    const bool empty = word == 0 || sum == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = lane + 32 * e;
        if (d >= D) continue;
        const float x = empty ? 0.0f : o[e] * inv;
        static_cast<uint16_t*>(P.out)[id * D + d] = (uint16_t)(C.fp16 ? pack<true>(x, x) : pack<false>(x, x));
    }
    if (P.lse && lane == 0) P.lse[id] = empty ? -INFINITY : lse_of(top, P.scale, sum);
}

}  // namespace

cudaError_t launch_tree_attention8(const AttendParams& P, cudaStream_t st) {
    const long long blocks = ((long long)P.c.B * P.T * P.Hq + kWarps - 1) / kWarps;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    void* args[1] = {const_cast<AttendParams*>(&P)};
    return launch(reinterpret_cast<const void*>(&k_tree_attention8), dim3((unsigned)blocks, 1, 1), 32 * kWarps, 0, args, st);
}

}  // namespace si
