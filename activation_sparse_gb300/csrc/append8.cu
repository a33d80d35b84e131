// append8.cu -- rotary append into a cache of e4m3 codes.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

// 8192 tokens of 32 + 8 + 8 heads of 128 / of 64 with 64, 96, 128, 192 and 256 threads a token: 42.3, 40.6, 40.1, 42.4, 49.5 /
// 23.1, 22.7, 26.0, 28.3, 33.5 us.
constexpr int kAppendThreads = 96;

// Sixteen elements of a row as they were loaded: eight pairs, (x[i], y[i]) where the layout is half-split and (x[0], x[1]),
// ..., (y[6], y[7]) where it is interleaved.
template <bool FP16>
struct Lane {
    uint32_t x[4], y[4];

    // Pairs 2i and 2i + 1, turned (cs: cos and sin of the eight pairs; nullptr: not turned).
    __device__ __forceinline__ void two(int i, const float2* cs, bool interleaved, float2& p, float2& r) const {
        if (interleaved) {
            p = unpack2<FP16>(i < 2 ? x[2 * i & 3] : y[2 * i & 3]);
            r = unpack2<FP16>(i < 2 ? x[(2 * i + 1) & 3] : y[(2 * i + 1) & 3]);
        } else {
            const float2 a = unpack2<FP16>(x[i]), b = unpack2<FP16>(y[i]);
            p = make_float2(a.x, b.x), r = make_float2(a.y, b.y);
        }
        if (cs) {
            const float2 c = cs[2 * i], d = cs[2 * i + 1];
            p = make_float2(p.x * c.x - p.y * c.y, p.y * c.x + p.x * c.y);
            r = make_float2(r.x * d.x - r.y * d.y, r.y * d.x + r.x * d.y);
        }
    }
};

__device__ __forceinline__ unsigned size_of(float2 p) {  // NaN above infinity above all
    return max(__float_as_uint(p.x) & 0x7FFFFFFFu, __float_as_uint(p.y) & 0x7FFFFFFFu);
}

// One block per token, as the append in 16 bits. A row of a head is a group of
// 2^group lanes, 16 elements a lane (eight pairs; the elements past the pairs
// eight a lane), so that a key's or value's largest magnitude is a few
// shuffles. Rows are scaled and rounded from the fp32 values, which are made
// twice, for the magnitude and for the codes: the elements stay as they were
// loaded meanwhile, half of the registers. Bound by memory and the chain of
// loads (position, slot, row): 8192 tokens of 32 + 8 + 8 heads of 128 take 40.6
// us, 4.5 TB/s, 0.68 of what a plain copy reaches.
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
    const int D = C.D, Hkv = C.Hkv, Hq = P.Hq;
    const int len = C.len[b];
    const bool fits = len >= 0 && len <= C.cap - P.T;
    if (!fits && tid == 0) atomicOr(P.err, SI_DEVERR_CACHE);
    const int32_t* list = C.table ? C.table + b * C.tb + len + t : nullptr;
    __syncthreads();

    const int rot = np / 8;                       // lanes of a head's pairs
    const int tail = (D - 2 * np) / 8;            // 16-byte units past them
    const int part = tid & ((1 << group) - 1), heads = Hq + 2 * Hkv;
    const bool inter = R.interleaved;
    for (int base = 0; base < heads; base += kAppendThreads >> group) {
        // queries, then keys, then values
        const int row = base + (tid >> group);
        const bool is_q = row < Hq, is_v = row >= Hq + Hkv;
        const int head = is_q ? row : is_v ? row - Hq - Hkv : row - Hq;
        long long slot = 0;
        bool on = row < heads;
        if (on && !is_q) {
            slot = !fits ? -1 : list ? list[head * C.th] : len + t;
            on = slot >= 0 && slot < C.n_slots;
            if (!on && fits && part == 0) atomicOr(P.err, SI_DEVERR_CACHE);
        }
        const bool turns = !is_v && part < rot;
        int o0 = -1, o1 = -1;                     // places of x and y in the row
        if (on) {
            if (is_v) {
                if (part < D / 16) o0 = part * 16, o1 = o0 + 8;
            } else if (part < rot) {
                o0 = inter ? part * 16 : part * 8;
                o1 = inter ? o0 + 8 : np + o0;
            } else if (part < rot + tail) {
                o0 = 2 * np + (part - rot) * 8;
            }
        }
        Lane<FP16> e = {};
        const uint16_t* src = is_q ? static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)head * P.qh
                              : is_v ? static_cast<const uint16_t*>(P.v) + b * P.vb + t * P.vt + (long long)head * P.vh
                                     : static_cast<const uint16_t*>(P.k) + b * P.kb + t * P.kt + (long long)head * P.kh;
        if (o0 >= 0) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + o0);
            e.x[0] = w.x, e.x[1] = w.y, e.x[2] = w.z, e.x[3] = w.w;
        }
        if (o1 >= 0) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + o1);
            e.y[0] = w.x, e.y[1] = w.y, e.y[2] = w.z, e.y[3] = w.w;
        }
        const float2* c = turns ? cs + part * 8 : nullptr;
        const bool pairs = inter && turns;        // else x and y hold two stretches side by side
        if (is_q && on) {
            uint16_t* dst = static_cast<uint16_t*>(P.q_out) + (tok * Hq + head) * D;
            if (turns) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 p, r;
                    e.two(i, c, pairs, p, r);
                    if (inter) {
                        (i < 2 ? e.x : e.y)[2 * i & 3] = pack2<FP16>(p.x, p.y);
                        (i < 2 ? e.x : e.y)[(2 * i + 1) & 3] = pack2<FP16>(r.x, r.y);
                    } else {
                        e.x[i] = pack2<FP16>(p.x, r.x), e.y[i] = pack2<FP16>(p.y, r.y);
                    }
                }
            }
            if (o0 >= 0) *reinterpret_cast<uint4*>(dst + o0) = make_uint4(e.x[0], e.x[1], e.x[2], e.x[3]);
            if (o1 >= 0) *reinterpret_cast<uint4*>(dst + o1) = make_uint4(e.y[0], e.y[1], e.y[2], e.y[3]);
        }
        if (!__any_sync(0xFFFFFFFFu, on && !is_q)) continue;
        uint8_t* scale = is_v ? C.v_scale + b * C.vcb + head * C.vch : C.k_scale + b * C.kcb + head * C.kch;
        int byte = kScaleNaN;
        if (C.block_shift == 0) {
            unsigned m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 p, r;
                e.two(i, c, pairs, p, r);
                m = max(m, max(size_of(p), size_of(r)));
            }
            for (int o = 1; o < 1 << group; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            byte = scale_byte_for(__uint_as_float(m), C.e_lo, C.e_hi);
            if (on && !is_q && part == 0) scale[slot] = (uint8_t)byte;
        } else if (on && !is_q) {
            byte = scale[slot >> C.block_shift];
            if (byte != kScaleNaN) byte = min(max(byte, C.e_lo), C.e_hi);
        }
        if (!on || is_q) continue;
        const float inv = __int_as_float((254 - byte) << 23);  // 2^(127 - byte)
        uint32_t code[4] = {};                    // of x, then of y
        if (byte != kScaleNaN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 p, r;
                e.two(i, c, pairs, p, r);
                if (pairs) {
                    code[i] = code2(p.x * inv, p.y * inv) | code2(r.x * inv, r.y * inv) << 16;
                } else {
                    code[i / 2] |= code2(p.x * inv, r.x * inv) << (i % 2 * 16);
                    code[2 + i / 2] |= code2(p.y * inv, r.y * inv) << (i % 2 * 16);
                }
            }
        }
        uint8_t* dst = is_v ? static_cast<uint8_t*>(const_cast<void*>(C.v)) + b * C.vb + head * C.vh + slot * C.vs
                            : static_cast<uint8_t*>(const_cast<void*>(C.k)) + b * C.kb + head * C.kh + slot * C.ks;
        if (o1 == o0 + 8 && o0 >= 0) {
            *reinterpret_cast<uint4*>(dst + o0) = make_uint4(code[0], code[1], code[2], code[3]);
        } else {
            if (o0 >= 0) *reinterpret_cast<uint2*>(dst + o0) = make_uint2(code[0], code[1]);
            if (o1 >= 0) *reinterpret_cast<uint2*>(dst + o1) = make_uint2(code[2], code[3]);
        }
        if (!is_v && part == 0 && C.acc) C.acc[b * C.ab + head * C.ah + slot] = 0.0f;
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
