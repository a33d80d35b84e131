// kv.cu -- the key/value cache's bookkeeping kernels: rotary append of new
// tokens, and acceptance with eviction by accumulated attention weight.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace si {

namespace {

// ------------------------------------------------------------------ append

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

// Eight pairs: half-split layout takes a = x[0..7], b = x[n_pairs ..]; the
// interleaved one has (a, b) alternating through both vectors.
template <bool FP16>
__device__ __forceinline__ void rotate8(uint4& x, uint4& y, const float2* cs, bool interleaved) {
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (interleaved) {
            const float2 p = unpack2<FP16>(xw[i]), r = unpack2<FP16>(yw[i]);
            const float2 c = cs[i], d = cs[4 + i];
            xw[i] = pack2<FP16>(p.x * c.x - p.y * c.y, p.y * c.x + p.x * c.y);
            yw[i] = pack2<FP16>(r.x * d.x - r.y * d.y, r.y * d.x + r.x * d.y);
        } else {
            const float2 a = unpack2<FP16>(xw[i]), b = unpack2<FP16>(yw[i]);
            const float2 c = cs[2 * i], d = cs[2 * i + 1];
            xw[i] = pack2<FP16>(a.x * c.x - b.x * c.y, a.y * d.x - b.y * d.y);
            yw[i] = pack2<FP16>(b.x * c.x + a.x * c.y, b.y * d.x + a.y * d.y);
        }
    }
}

constexpr int kAppendThreads = 256;

// One block per token. The angle of pair i is pos * inv_freq turns taken in
// 64-bit fixed point (the product wraps to the fraction of a turn, exact for
// any int32 position); cos and sin of the token's pairs are made once, in
// shared memory, for its Hq + Hkv heads. Bound by memory: every element is
// read and written once, in 16-byte units.
template <bool FP16>
__global__ void __launch_bounds__(kAppendThreads)
    k_kv_append(const __grid_constant__ KvAppendParams P, const __grid_constant__ RopeTable R) {
    __shared__ float2 cs[kRopeMaxPairs];
    grid_launch_dependents();
    grid_dependency_wait();
    const long long tok = blockIdx.x;
    const int b = (int)(tok / P.T), t = (int)(tok % P.T);
    const int np = R.n_pairs;
    for (int i = threadIdx.x; i < np; i += kAppendThreads) {
        const long long pos = P.pos[tok * R.n_axes + R.axis[i]];
        const unsigned long long turn = (unsigned long long)pos * R.turn[i];
        // signed fraction in half turns: [-1, 1)
        const float x = (float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
        float s, c;
        sincospif(x, &s, &c);
        cs[i] = make_float2(c, s);
    }
    const KvView& C = P.c;
    const int D = C.D, Hkv = C.Hkv;
    const int len = C.len[b];
    const bool fits = len >= 0 && len <= C.cap - P.T;
    if (!fits && threadIdx.x == 0) atomicOr(P.err, SI_DEVERR_CACHE);
    const int32_t* list = C.table ? C.table + b * C.tb + len + t : nullptr;
    if (C.acc && fits) {
        for (int h = threadIdx.x; h < Hkv; h += kAppendThreads) {
            const long long slot = list ? list[h * C.th] : len + t;
            if (slot >= 0 && slot < C.n_slots) C.acc[b * C.ab + h * C.ah + slot] = 0.0f;
        }
    }
    __syncthreads();

    const int rot = np / 8;                       // 16-pair-element units of a rotated head
    const int tail = (D - 2 * np) / 8;            // 16-byte units past the rotated part
    const int per_qk = rot + tail, per_v = D / 8;
    const int n_qk = (P.Hq + Hkv) * per_qk;
    const int n_units = n_qk + Hkv * per_v;
    const uint16_t* q = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt;
    const uint16_t* k = static_cast<const uint16_t*>(P.k) + b * P.kb + t * P.kt;
    const uint16_t* v = static_cast<const uint16_t*>(P.v) + b * P.vb + t * P.vt;
    uint16_t* qo = static_cast<uint16_t*>(P.q_out) + tok * P.Hq * D;
    for (int u = threadIdx.x; u < n_units; u += kAppendThreads) {
        const uint16_t* src;
        uint16_t* dst;
        int part;
        const bool is_v = u >= n_qk;
        int head = is_v ? (u - n_qk) / per_v : u / per_qk;
        part = is_v ? (u - n_qk) - head * per_v : u - head * per_qk;
        if (!is_v && head < P.Hq) {
            src = q + head * P.qh;
            dst = qo + (long long)head * D;
        } else {
            if (!is_v) head -= P.Hq;
            if (!fits) continue;
            const long long slot = list ? list[head * C.th] : len + t;
            if (slot < 0 || slot >= C.n_slots) {
                atomicOr(P.err, SI_DEVERR_CACHE);
                continue;
            }
            src = is_v ? v + head * P.vh : k + head * P.kh;
            dst = is_v ? static_cast<uint16_t*>(const_cast<void*>(C.v)) + b * C.vb + head * C.vh + slot * C.vs
                       : static_cast<uint16_t*>(const_cast<void*>(C.k)) + b * C.kb + head * C.kh + slot * C.ks;
        }
        if (is_v || part >= rot) {
            const int o = is_v ? part * 8 : 2 * np + (part - rot) * 8;
            *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
        } else {
            const int o0 = R.interleaved ? part * 16 : part * 8;
            const int o1 = R.interleaved ? o0 + 8 : np + o0;
            uint4 x = *reinterpret_cast<const uint4*>(src + o0);
            uint4 y = *reinterpret_cast<const uint4*>(src + o1);
            rotate8<FP16>(x, y, cs + part * 8, R.interleaved);
            *reinterpret_cast<uint4*>(dst + o0) = x;
            *reinterpret_cast<uint4*>(dst + o1) = y;
        }
    }
}

// ------------------------------------------------------------------- evict

constexpr int kEvictBins = 2048;
constexpr int kEvictChunk = 24576;  // entries a CTA holds at most: 8 bytes each in shared memory
constexpr int kEvictBatch = 8;      // entries a thread loads at once: two dependent loads each

struct EvictShared {
    unsigned hist[3][kEvictBins];  // one per radix pass: peers read them while the next is filled
    unsigned warp_a[32], warp_b[32];
    unsigned total_a, total_b;     // this CTA's strict and tied counts, read by the peers
    unsigned bin, left, whole;
    int last;
};

// Larger weight <=> larger key, -0 and +0 alike, NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0u : value_key(w); }

// One cluster per list: it holds the whole candidate list (slot and key) in
// the shared memory of its CTAs, finds the key of the last survivor by a
// radix selection over 11 + 11 + 10 bits (each pass sums the CTAs' histograms
// through distributed shared memory), and writes the stable partition.
// Everything is read before the first cluster barrier and written after it,
// so the list may be edited in place.
template <int kEvictThreads>
__global__ void __launch_bounds__(kEvictThreads, 1024 / kEvictThreads) k_kv_evict(const __grid_constant__ KvEvictParams P, int chunk_cap) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    EvictShared& S = *reinterpret_cast<EvictShared*>(smem_raw);
    int32_t* slots = reinterpret_cast<int32_t*>(smem_raw + sizeof(EvictShared));
    uint32_t* keys = reinterpret_cast<uint32_t*>(slots + chunk_cap);
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    constexpr int kEvictWarps = kEvictThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 3 * kEvictBins / 4; i += kEvictThreads)
        reinterpret_cast<uint4*>(&S.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    // what the warps before this one have counted (warp sums in v[0 .. warps - 1])
    auto before_warp = [&](const unsigned* v) {
        return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? v[lane] : 0u);
    };
    grid_launch_dependents();
    grid_dependency_wait();

    const int row = blockIdx.x / CS;
    const int h = row % P.Hkv, lb = row / P.Hkv, b = lb % P.B, l = lb / P.B;
    const int32_t* table = P.table + l * P.tl + b * P.tb + h * P.th;
    int32_t* out = P.table_out + l * P.ol + b * P.ob + h * P.oh;
    const float* acc = P.acc ? P.acc + l * P.al + b * P.ab + h * P.ah : nullptr;
    const int T = P.T;
    const int len = P.len[lb];
    const bool bad = len < 0 || len > P.cap - T;
    int np = P.n_path ? P.n_path[b] : T;
    bool path_bad = np < 0 || np > T;
    unsigned long long taken = 0;  // accepted nodes, where a path names them
    if (P.path && !path_bad) {
        unsigned lo = 0, hi = 0;
        bool out_of_range = false;
        for (int i = lane; i < np; i += 32) {
            const int node = P.path[(long long)b * T + i];
            if (node < 0 || node >= T) out_of_range = true;
            else if (node < 32) lo |= 1u << node;
            else hi |= 1u << (node - 32);
        }
        lo = __reduce_or_sync(0xFFFFFFFFu, lo);
        hi = __reduce_or_sync(0xFFFFFFFFu, hi);
        taken = (unsigned long long)hi << 32 | lo;
        path_bad = __any_sync(0xFFFFFFFFu, out_of_range) || __popcll(taken) != np;
    }
    if (path_bad) np = 0, taken = 0;
    if ((bad || path_bad) && rank == 0 && tid == 0)
        atomicOr(P.err, (bad ? SI_DEVERR_CACHE : 0u) | (path_bad ? SI_DEVERR_COUNT : 0u));
    const bool named = P.path && !path_bad;
    const int n = bad ? 0 : len + np;
    const int used = bad ? 0 : len + T;           // entries this call may reorder
    const bool evict = P.budget > 0 && n > P.budget;
    const int n_new = bad ? len : (evict ? P.budget : n);

    // this CTA's candidates [c0, c1)
    const int chunk = ((n + CS - 1) / CS + 31) & ~31;
    const int c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk), m = c1 - c0;
    const int lo_c = P.sinks, hi_c = n - P.recent;  // candidates outside [lo_c, hi_c) are safe
    unsigned need = evict ? (unsigned)(P.budget - P.sinks - P.recent) : 0u;
    bool bad_slot = false;
    for (int i0 = tid; i0 < m; i0 += kEvictThreads * kEvictBatch) {
        int slot[kEvictBatch];
        float w[kEvictBatch];
#pragma unroll
        for (int j = 0; j < kEvictBatch; ++j) {
            const int c = c0 + i0 + j * kEvictThreads;
            int at = c;
            if (c >= len && c < c1 && named) at = len + P.path[(long long)b * T + c - len];
            slot[j] = c < c1 ? table[at] : 0;
        }
        if (evict) {
#pragma unroll
            for (int j = 0; j < kEvictBatch; ++j) {
                const bool ok = slot[j] >= 0 && slot[j] < P.n_slots;
                bad_slot |= !ok;
                w[j] = ok ? acc[slot[j]] : __int_as_float(0x7FC00000);
            }
        }
#pragma unroll
        for (int j = 0; j < kEvictBatch; ++j) {
            const int i = i0 + j * kEvictThreads, c = c0 + i;
            if (i >= m) continue;
            slots[i] = slot[j];
            if (!evict) continue;
            const uint32_t key = weight_key(w[j]);
            keys[i] = key;
            if (need > 0 && c >= lo_c && c < hi_c) atomicAdd(&S.hist[0][key >> 21], 1u);
        }
    }
    if (bad_slot) atomicOr(P.err, SI_DEVERR_CACHE);
    int rejected = -1;  // slot of the node that this thread puts behind the candidates
    if (rank == 0 && named && tid < T && !(taken >> tid & 1)) rejected = bad ? -1 : table[len + tid];
    cluster.sync();

    if (!evict) {
        for (int i = tid; i < m; i += kEvictThreads)
            if (!P.in_place || c0 + i >= len) out[c0 + i] = slots[i];
    } else {
        uint32_t prefix = 0xFFFFFFFFu, tie_need = 0;  // need = 0: no key lies above, no tie is taken
        if (need > 0) {
            prefix = 0;
            tie_need = 0xFFFFFFFFu;
            int shift = 21, width = 11;
            uint32_t done = 0;  // mask of the bits fixed so far
            for (int pass = 0; pass < 3; ++pass) {
                unsigned* hist = S.hist[pass];
                const int bins = 1 << width;
                if (pass > 0) {  // the first was counted as the weights came in
                    for (int i = tid; i < m; i += kEvictThreads) {
                        const int c = c0 + i;
                        const uint32_t key = keys[i];
                        if (((key ^ prefix) & done) == 0 && c >= lo_c && c < hi_c)
                            atomicAdd(&hist[key >> shift & (bins - 1)], 1u);
                    }
                    cluster.sync();
                }
                // every CTA sums all histograms: a few bins a thread, highest bin first
                constexpr int kMaxPer = kEvictBins / kEvictThreads;
                const int per = bins / kEvictThreads;
                unsigned cnt[kMaxPer] = {};
                for (int r = 0; r < CS; ++r) {
                    const unsigned* peer = cluster.map_shared_rank(hist, r);
#pragma unroll
                    for (int j = 0; j < kMaxPer; ++j)
                        if (j < per) cnt[j] += peer[bins - 1 - (tid * per + j)];
                }
                unsigned mine = 0;
#pragma unroll
                for (int j = 0; j < kMaxPer; ++j) mine += cnt[j];
                unsigned incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (lane == 31) S.warp_a[warp] = incl;
                __syncthreads();
                const unsigned before = incl - mine + before_warp(S.warp_a);
                if (before < need && before + mine >= need) {
                    unsigned above = before;
#pragma unroll
                    for (int j = 0; j < kMaxPer; ++j) {
                        if (above < need && above + cnt[j] >= need) {
                            S.bin = bins - 1 - (tid * per + j);
                            S.left = need - above;
                            S.whole = cnt[j] == need - above;
                            above = 0xFFFFFFFFu;
                        } else if (above != 0xFFFFFFFFu) {
                            above += cnt[j];
                        }
                    }
                }
                __syncthreads();
                prefix |= S.bin << shift;
                done |= (uint32_t)(bins - 1) << shift;
                need = S.left;
                if (S.whole) break;  // the bin is taken whole: every key >= prefix survives
                if (pass == 2) tie_need = need;
                width = pass == 0 ? 11 : 10;
                shift -= width;
                __syncthreads();
            }
        }
        // strict survivors and ties per warp segment, then per CTA
        const int seg = (((m + kEvictWarps - 1) / kEvictWarps) + 31) & ~31;
        const int s0 = min(m, warp * seg), s1 = min(m, s0 + seg);
        unsigned n_strict = 0, n_tie = 0;
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane, c = c0 + i;
            const bool in = i < s1;
            const uint32_t key = in ? keys[i] : 0u;
            const bool safe = in && (c < lo_c || c >= hi_c);
            n_strict += __popc(__ballot_sync(0xFFFFFFFFu, safe || (in && key > prefix)));
            n_tie += __popc(__ballot_sync(0xFFFFFFFFu, in && !safe && key == prefix));
        }
        __syncthreads();
        if (lane == 0) S.warp_a[warp] = n_strict, S.warp_b[warp] = n_tie;
        __syncthreads();
        const unsigned warps_a = before_warp(S.warp_a), warps_b = before_warp(S.warp_b);
        if (warp == kEvictWarps - 1 && lane == 0) S.total_a = warps_a + n_strict, S.total_b = warps_b + n_tie;
        cluster.sync();
        unsigned strict = 0, tie = 0;
        for (int r = 0; r < rank; ++r) {
            strict += *cluster.map_shared_rank(&S.total_a, r);
            tie += *cluster.map_shared_rank(&S.total_b, r);
        }
        strict += warps_a, tie += warps_b;
        unsigned kept = strict + min(tie, tie_need);  // survivors before this warp's segment
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane, c = c0 + i;
            const bool in = i < s1;
            const uint32_t key = in ? keys[i] : 0u;
            const bool safe = in && (c < lo_c || c >= hi_c);
            const bool tied = in && !safe && key == prefix;
            const unsigned ties = __ballot_sync(0xFFFFFFFFu, tied);
            const bool keep = safe || (in && key > prefix) || (tied && tie + __popc(ties & lanemask_lt()) < tie_need);
            const unsigned keeps = __ballot_sync(0xFFFFFFFFu, keep);
            const int pos = (int)(kept + __popc(keeps & lanemask_lt()));
            if (in) out[keep ? pos : P.budget + (c - pos)] = slots[i];
            tie += __popc(ties);
            kept += __popc(keeps);
        }
    }
    if (rejected >= 0) out[n + tid - __popcll(taken & ((1ull << tid) - 1))] = rejected;
    if (!P.in_place) {
        // what this call does not reorder: unaccepted nodes that stay behind the candidates, free slots
        const int from = named ? used : n;
        for (int i = from + rank * kEvictThreads + tid; i < P.cap; i += CS * kEvictThreads) out[i] = table[i];
        if (h == 0 && rank == 0 && tid == 0) P.len_out[lb] = n_new;
    } else if (rank == 0) {
        // the other heads' clusters still read len: the last cluster of the grid writes the new ones
        unsigned* len_new = P.ticket + 1;
        if (tid == 0) {
            if (h == 0) len_new[lb] = (unsigned)n_new;
            __threadfence();
            S.last = atomicAdd(P.ticket, 1u) == (unsigned)(P.L * P.B * P.Hkv) - 1u;
        }
        __syncthreads();
        if (S.last) {
            __threadfence();
            for (int i = tid; i < P.L * P.B; i += kEvictThreads) P.len_out[i] = (int)__ldcg(len_new + i);
            if (tid == 0) *P.ticket = 0;
        }
    }
    cluster.sync();  // peers may still read this CTA's totals
}

cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, int cluster, void** args, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& P, const RopeTable& R, cudaStream_t st) {
    void* args[2] = {const_cast<KvAppendParams*>(&P), const_cast<RopeTable*>(&R)};
    const void* fn = P.c.fp16 ? reinterpret_cast<const void*>(&k_kv_append<true>)
                              : reinterpret_cast<const void*>(&k_kv_append<false>);
    return launch(fn, dim3((unsigned)((long long)P.c.B * P.T), 1, 1), kAppendThreads, 0, 1, args, st);
}

cudaError_t launch_kv_evict(const KvEvictParams& P, cudaStream_t st) {
    const long long rows = (long long)P.L * P.B * P.Hkv;
    int cs = 1;
    while ((P.cap + cs - 1) / cs > kEvictChunk) cs *= 2;
    // few lists: more CTAs a list, down to 2048 entries each
    while (cs < 8 && (P.cap + cs - 1) / cs > 2048 && rows * cs < 304) cs *= 2;
    int chunk = (((P.cap + cs - 1) / cs) + 31) & ~31;
    const bool wide = chunk > 6144;
    const size_t smem = sizeof(EvictShared) + (size_t)chunk * 8;
    cudaError_t e = wide ? allow_max_smem(k_kv_evict<1024>) : allow_max_smem(k_kv_evict<256>);
    if (e != cudaSuccess) return e;
    void* args[2] = {const_cast<KvEvictParams*>(&P), &chunk};
    const void* fn = wide ? reinterpret_cast<const void*>(&k_kv_evict<1024>)
                          : reinterpret_cast<const void*>(&k_kv_evict<256>);
    return launch(fn, dim3((unsigned)(rows * cs), 1, 1), wide ? 1024 : 256, smem, cs, args, st);
}

}  // namespace si
