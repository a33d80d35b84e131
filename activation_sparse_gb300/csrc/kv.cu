// kv.cu -- the key/value cache's bookkeeping kernels: rotary append of new
// tokens, and acceptance with eviction by accumulated attention weight.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <cstring>

#include "kv.cuh"

namespace cg = cooperative_groups;

namespace si {

namespace {

// ------------------------------------------------------------------ append

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
// read and written once, in 16-byte units. 8192 tokens of 32 + 8 + 8 heads of
// 128 take 41 us (a plain copy of the same bytes 33); what carries it is the
// eight blocks an SM: elements loaded ahead of the angles (48 registers, five
// blocks) took 54 us, and through shared memory a token ahead 46.
template <bool FP16>
__global__ void __launch_bounds__(kAppendThreads)
    k_kv_append(const __grid_constant__ KvAppendParams P, const __grid_constant__ RopeTable R) {
    __shared__ float2 cs[kRopeMaxPairs];
    grid_launch_dependents();
    grid_dependency_wait();
    const long long tok = blockIdx.x;
    const int b = (int)(blockIdx.x / (unsigned)P.T), t = (int)(blockIdx.x - (unsigned)b * (unsigned)P.T);
    const int np = R.n_pairs;
    for (int i = threadIdx.x; i < np; i += kAppendThreads) {
        const long long pos = P.pos[tok * R.n_axes + R.axis[i]];
        cs[i] = turned(pos, R.turn[i]);
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
        int head = is_v ? div_of(u - n_qk, per_v) : div_of(u, per_qk);
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
constexpr int kEvictChunk = 24576;  // candidates a CTA holds at most: a key each in shared memory
constexpr int kEvictBatch = 8;      // entries a thread loads at once: two dependent loads each

struct alignas(16) EvictShared {
    unsigned hist[kEvictBins];
    unsigned warp_a[32], warp_b[32];
    unsigned total_a, total_b;     // this CTA's strict and tied counts, read by the peers
    unsigned found[3][3];          // per pass: bin, how many of it survive, whether that is all of it
    int last;
};

// Larger weight <=> larger key, -0 and +0 alike, NaN below everything. Keys
// of weights lie strictly between kKeyNone (no candidate) and kKeySafe (kept
// whatever its weight).
constexpr uint32_t kKeyNone = 0u, kKeyNaN = 1u, kKeySafe = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? kKeyNaN : value_key(w); }

// One cluster per list. It holds the candidates' keys in the shared memory of
// its CTAs, finds the key of the last survivor by a radix selection over 11 +
// 11 + 10 bits, and writes the stable partition. In each pass the CTAs add
// their non-empty bins to the first CTA's histogram (a list's weights fall
// into few bins: a few hundred words, where reading every peer's histogram
// moved 8 KB a peer); the first CTA finds the bin and tells the others. The
// slots are read again for the partition, so that more CTAs share an SM; in
// place they are all read before the last cluster barrier and written after
// it. Bound by latency (a chain of three loads: length, slot, weight; then
// barriers) and for long lists by the weights' gather: four bytes of every
// 32-byte sector, 0.6 sectors a cycle and SM.
template <int THREADS, bool IN_PLACE>
__global__ void __launch_bounds__(THREADS, (IN_PLACE ? 512 : 1536) / THREADS > 0 ? (IN_PLACE ? 512 : 1536) / THREADS : 1)
    k_kv_evict(const __grid_constant__ KvEvictParams P) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    EvictShared& S = *reinterpret_cast<EvictShared*>(smem_raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(EvictShared));
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto clear = [&]() {
        for (int i = tid; i < kEvictBins / 4; i += THREADS)
            reinterpret_cast<uint4*>(S.hist)[i] = make_uint4(0, 0, 0, 0);
    };
    auto all_sync = [&]() {
        if (CS > 1) cluster.sync();
        else __syncthreads();
    };
    // what the warps before this one have counted (warp sums in v[0 .. WARPS - 1])
    auto before_warp = [&](const unsigned* v) {
        return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? v[lane] : 0u);
    };
    clear();
    all_sync();  // the first CTA's histogram is clear before a peer adds to it
    grid_launch_dependents();
    grid_dependency_wait();

    const int row = blockIdx.x / CS;
    const int h = row % P.Hkv, lb = row / P.Hkv, b = lb % P.B, l = lb / P.B;
    const int32_t* table = P.table + l * P.tl + b * P.tb + h * P.th;
    int32_t* out = P.table_out + l * P.ol + b * P.ob + h * P.oh;
    const float* acc = P.acc ? P.acc + l * P.al + b * P.ab + h * P.ah : nullptr;
    const int T = P.T;
    // What does not wait for the length goes out with it: the path, and where one CTA has the whole list its
    // first entries past the sinks (a list has cap entries whatever its length).
    int early[kEvictBatch];
#pragma unroll
    for (int j = 0; j < kEvictBatch; ++j) {
        const unsigned i = (unsigned)P.sinks + tid + j * THREADS;  // any sinks without a budget
        early[j] = CS == 1 && i < (unsigned)P.cap ? table[i] : 0;
    }
    const int path_lo = P.path && lane < T ? P.path[(long long)b * T + lane] : 0;
    const int path_hi = P.path && lane + 32 < T ? P.path[(long long)b * T + lane + 32] : 0;
    const int len = P.len[lb];
    const bool bad = len < 0 || len > P.cap - T;
    int np = P.n_path ? P.n_path[b] : T;
    bool path_bad = np < 0 || np > T;
    unsigned long long taken = 0;  // accepted nodes, where a path names them
    if (P.path && !path_bad) {
        unsigned lo = 0, hi = 0;
        bool out_of_range = false;
        for (int i = lane; i < np; i += 32) {
            const int node = i < 32 ? path_lo : path_hi;
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
    const bool named = P.path && !path_bad && !bad;  // a list out of bounds is left as it is
    const int n = bad ? 0 : len + np;
    const int used = bad ? 0 : len + T;           // entries this call may reorder
    const bool evict = P.budget > 0 && n > P.budget;
    const int n_new = bad ? len : (evict ? P.budget : n);

    // this CTA's candidates [c0, c1); the chunk is padded to whole sets of 128
    const int chunk = ((n + CS - 1) / CS + 127) & ~127;
    const int c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk), m = c1 - c0;
    const int lo_c = P.sinks, hi_c = n - P.recent;  // candidates outside [lo_c, hi_c) are safe
    const unsigned n_slots = (unsigned)P.n_slots;
    auto entry_of = [&](int c) {  // list entry of candidate c
        return named && c >= len ? len + P.path[(long long)b * T + c - len] : c;
    };
    bool bad_slot = false;
    if (evict) {
        // The safe ones at either end are kept whatever they weigh: nothing is read for them.
        const int safe_lo = min(m, max(0, lo_c - c0)), safe_hi = max(safe_lo, min(m, hi_c - c0));
        for (int i = tid; i < ((m + 127) & ~127); i += THREADS)
            if (i < safe_lo || i >= safe_hi) keys[i] = i < m ? kKeySafe : kKeyNone;
        if (tid == 0 && m > safe_hi - safe_lo) atomicAdd(&S.hist[kKeySafe >> 21], (unsigned)(m - (safe_hi - safe_lo)));
        // candidates whose entry is their own index, then accepted nodes, in path order
        const int by_table = min(safe_hi, max(safe_lo, (named ? len : n) - c0));
        for (int i0 = safe_lo + tid; i0 < by_table; i0 += THREADS * kEvictBatch) {
            int slot[kEvictBatch];
            float w[kEvictBatch];
#pragma unroll
            for (int j = 0; j < kEvictBatch; ++j) {
                const int i = i0 + j * THREADS;
                slot[j] = i >= by_table ? 0 : CS == 1 && i0 == P.sinks + tid ? early[j] : table[c0 + i];
            }
#pragma unroll
            for (int j = 0; j < kEvictBatch; ++j) {
                const bool ok = (unsigned)slot[j] < n_slots;
                bad_slot |= !ok;
                w[j] = acc[ok ? slot[j] : 0];
            }
#pragma unroll
            for (int j = 0; j < kEvictBatch; ++j) {
                const int i = i0 + j * THREADS;
                if (i >= by_table) break;
                const uint32_t key = weight_key(w[j]);
                keys[i] = key;
                atomicAdd(&S.hist[key >> 21], 1u);
            }
        }
        for (int i = by_table + tid; i < safe_hi; i += THREADS) {
            const int slot = table[entry_of(c0 + i)];
            const bool ok = (unsigned)slot < n_slots;
            bad_slot |= !ok;
            const uint32_t key = weight_key(acc[ok ? slot : 0]);
            keys[i] = key;
            atomicAdd(&S.hist[key >> 21], 1u);
        }
    }
    if (bad_slot) atomicOr(P.err, SI_DEVERR_CACHE);
    int rejected = -1;  // slot of the node that this thread puts behind the candidates
    if (rank == 0 && named && tid < T && !(taken >> tid & 1)) rejected = table[len + tid];

    if (!evict) {
        if (IN_PLACE) {
            // live entries stay; accepted nodes (at most 64) may change places
            const int c = len + tid;
            const bool moves = rank == 0 && named && c < n;
            const int slot = moves ? table[entry_of(c)] : 0;
            all_sync();
            if (moves) out[c] = slot;
        } else {
            for (int c = c0 + tid; c < c1; c += THREADS) out[c] = table[entry_of(c)];
        }
    } else {
        const int quads = ((m + 127) & ~127) / 4;
        const uint4* keys4 = reinterpret_cast<const uint4*>(keys);
        unsigned need = (unsigned)P.budget;
        uint32_t prefix = 0, tie_need = 0xFFFFFFFFu;
        uint32_t done = 0;  // mask of the bits fixed so far
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bins = pass < 2 ? 2048 : 1024;
            if (pass > 0) {  // the first was counted as the weights came in
                clear();
                __syncthreads();
                if (CS > 1) cluster.barrier_arrive();  // clear: peers may add to it
                for (int i = tid; i < quads; i += THREADS) {
                    const uint4 k = keys4[i];
                    if (((k.x ^ prefix) & done) == 0) atomicAdd(&S.hist[k.x >> shift & (bins - 1)], 1u);
                    if (((k.y ^ prefix) & done) == 0) atomicAdd(&S.hist[k.y >> shift & (bins - 1)], 1u);
                    if (((k.z ^ prefix) & done) == 0) atomicAdd(&S.hist[k.z >> shift & (bins - 1)], 1u);
                    if (((k.w ^ prefix) & done) == 0) atomicAdd(&S.hist[k.w >> shift & (bins - 1)], 1u);
                }
                if (CS > 1) cluster.barrier_wait();
            }
            if (rank > 0) {
                __syncthreads();
                unsigned* lead = cluster.map_shared_rank(S.hist, 0);
                for (int i = tid; i < bins; i += THREADS)
                    if (const unsigned c = S.hist[i]) atomicAdd(lead + i, c);
            }
            all_sync();
            if (rank == 0) {
                // a few bins a thread, highest first: the one where the count from the top reaches need
                constexpr int kMaxPer = kEvictBins / THREADS;
                const int per = bins / THREADS;
                unsigned cnt[kMaxPer], mine = 0;
#pragma unroll
                for (int j = 0; j < kMaxPer; ++j) {
                    cnt[j] = j < per ? S.hist[bins - 1 - (tid * per + j)] : 0;
                    mine += cnt[j];
                }
                unsigned incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (lane == 31) S.warp_a[warp] = incl;
                __syncthreads();
                unsigned above = incl - mine + before_warp(S.warp_a);
                if (above < need && above + mine >= need) {
#pragma unroll
                    for (int j = 0; j < kMaxPer; ++j) {
                        if (above < need && above + cnt[j] >= need) {
                            for (int r = 0; r < CS; ++r) {
                                unsigned* f = cluster.map_shared_rank(S.found[pass], r);
                                f[0] = bins - 1 - (tid * per + j);
                                f[1] = need - above;
                                f[2] = cnt[j] == need - above;
                            }
                            above = need;
                        } else {
                            above += cnt[j];
                        }
                    }
                }
            }
            all_sync();
            prefix |= S.found[pass][0] << shift;
            done |= (uint32_t)(bins - 1) << shift;
            need = S.found[pass][1];
            if (S.found[pass][2]) break;  // the bin is taken whole: every key >= prefix survives
            if (pass == 2) tie_need = need;
        }
        // Keys above the prefix survive, keys equal to it while tie_need lasts. Counts of both per warp
        // segment (whole sets of 128 candidates, four a lane), then per CTA; packed as strict | ties << 16.
        const int sets = quads / 32, per_warp = (sets + WARPS - 1) / WARPS;
        const int s0 = min(sets, warp * per_warp), s1 = min(sets, s0 + per_warp);
        auto classes = [&](const uint4& k) {
            return (unsigned)((k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix)) |
                   (unsigned)((k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix)) << 16;
        };
        unsigned both = 0;
        for (int q = s0; q < s1; ++q) both += classes(keys4[q * 32 + lane]);
        const unsigned n_strict = __reduce_add_sync(0xFFFFFFFFu, both & 0xFFFFu);
        const unsigned n_tie = __reduce_add_sync(0xFFFFFFFFu, both >> 16);
        if (lane == 0) S.warp_a[warp] = n_strict, S.warp_b[warp] = n_tie;
        __syncthreads();
        const unsigned warps_a = before_warp(S.warp_a), warps_b = before_warp(S.warp_b);
        unsigned strict = warps_a, tie = warps_b;
        if (CS > 1) {
            if (warp == WARPS - 1 && lane == 0) S.total_a = warps_a + n_strict, S.total_b = warps_b + n_tie;
            cluster.sync();
            unsigned a = 0, t2 = 0;
            if (lane < rank) {
                a = *cluster.map_shared_rank(&S.total_a, lane);
                t2 = *cluster.map_shared_rank(&S.total_b, lane);
            }
            strict += __reduce_add_sync(0xFFFFFFFFu, a);
            tie += __reduce_add_sync(0xFFFFFFFFu, t2);
        }
        // A set again, now a candidate a lane four times over: the writes of a warp are runs of the output.
        auto read_set = [&](int q, int (&slot)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = c0 + q * 128 + e * 32 + lane;
                slot[e] = c < c1 ? table[entry_of(c)] : 0;
            }
        };
        unsigned kept = strict + min(tie, tie_need);  // survivors before the next 32 candidates
        auto write_set = [&](int q, const int (&slot)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = q * 128 + e * 32 + lane, c = c0 + i;
                const uint32_t key = keys[i];
                const unsigned ties = __ballot_sync(0xFFFFFFFFu, key == prefix);
                const bool keep = key > prefix || (key == prefix && tie + __popc(ties & lanemask_lt()) < tie_need);
                const unsigned keeps = __ballot_sync(0xFFFFFFFFu, keep && c < c1);
                const int pos = (int)(kept + __popc(keeps & lanemask_lt()));
                if (c < c1) out[keep ? pos : P.budget + (c - pos)] = slot[e];
                tie += __popc(ties);
                kept += __popc(keeps);
            }
        };
        if (IN_PLACE) {
            constexpr int kMost = kEvictChunk / 128 / (512 / 32);  // sets a warp has at most
            int slot[kMost][4];
#pragma unroll
            for (int q = 0; q < kMost; ++q)
                if (s0 + q < s1) read_set(s0 + q, slot[q]);
            all_sync();
#pragma unroll
            for (int q = 0; q < kMost; ++q)
                if (s0 + q < s1) write_set(s0 + q, slot[q]);
        } else {
            for (int q = s0; q < s1; ++q) {
                int slot[4];
                read_set(q, slot);
                write_set(q, slot);
            }
        }
    }
    if (rejected >= 0) out[n + tid - __popcll(taken & ((1ull << tid) - 1))] = rejected;
    if (!IN_PLACE) {
        // what this call does not reorder: unaccepted nodes that stay behind the candidates, free slots
        const int from = named ? used : n;
        for (int i = from + rank * THREADS + tid; i < P.cap; i += CS * THREADS) out[i] = table[i];
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
            for (int i = tid; i < P.L * P.B; i += THREADS) P.len_out[i] = (int)__ldcg(len_new + i);
            if (tid == 0) *P.ticket = 0;
        }
    }
    if (CS > 1) cluster.sync();  // peers may still read this CTA's totals
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

template <int THREADS, bool IN_PLACE>
cudaError_t launch_evict(const KvEvictParams& P, unsigned ctas, int cs, size_t smem, cudaStream_t st) {
    const auto kern = k_kv_evict<THREADS, IN_PLACE>;
    const cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    void* args[1] = {const_cast<KvEvictParams*>(&P)};
    return launch(reinterpret_cast<const void*>(kern), dim3(ctas, 1, 1), THREADS, smem, cs, args, st);
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
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    // CTAs a list (at most eight, the portable cluster). Few enough candidates each that three CTAs share an
    // SM where eight CTAs can do that (64 lists of up to 100001: 73 us, 96 with twice the candidates each). Where
    // the lists alone do not fill the GPU, lists above 6144 are split down to 3200 each: a cluster's barriers
    // cost 2 us, a CTA's further thousand candidates 1 (eight lists of 3000, whole / in two: 7.5 / 8.8 us;
    // of 8000, in two / in four: 12.1 / 10.6; 128 lists of 4096, whole / in four: 14.5 / 18.1).
    int cs = 1;
    auto each = [&]() { return ((P.cap + cs - 1) / cs + 127) & ~127; };
    while (cs < 8 && (each() > 12544 || (P.cap > 6144 && each() > 3200 && rows * cs <= sms))) cs *= 2;
    const int chunk = each();
    if (chunk > kEvictChunk) return cudaErrorInvalidValue;
    // 512 threads where the CTAs all run at once, three an SM, or hold much each; else 256, of which six fit.
    // 512 / 256: eight lists of 1025 5.9 / 6.6 us, 256 of 4096 16.0 / 22.4, 320 of 2000 12.6 / 15.1, 448 of 2000
    // 12.5 / 11.6, 896 of 2000 22.3 / 16.3, of 4096 28.9 / 25.1, of 6000 36.1 / 48.8.
    const bool wide = chunk > 5120 || rows * cs <= 3 * sms;
    const size_t smem = sizeof(EvictShared) + (size_t)chunk * 4;
    if (P.in_place)
        return wide ? launch_evict<512, true>(P, (unsigned)(rows * cs), cs, smem, st)
                    : launch_evict<256, true>(P, (unsigned)(rows * cs), cs, smem, st);
    return wide ? launch_evict<512, false>(P, (unsigned)(rows * cs), cs, smem, st)
                : launch_evict<256, false>(P, (unsigned)(rows * cs), cs, smem, st);
}

}  // namespace si
