// logprobs.cu -- log probabilities, entropy and best alternatives of rows of logits.
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "attend.cuh"

namespace cg = cooperative_groups;

namespace si {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostCtas = 8;  // of a row: the portable cluster
constexpr int kBatch = 4;     // 16-byte units a thread has under way

template <int DTYPE>
struct Unit {
    static constexpr int N = DTYPE == SI_FP32 ? 4 : 8;  // logits
    static constexpr int kSize = 16 / N;
    static constexpr int kWord = N / 4;                 // logits of a word
    static constexpr uint32_t kNone = DTYPE == SI_FP32 ? 0xFF800000u : DTYPE == SI_FP16 ? 0xFC00FC00u : 0xFF80FF80u;  // -inf
    static __device__ __forceinline__ float2 pair(uint32_t w) {  // of the types of 16 bits
        return unpack2<DTYPE == SI_FP16>(w);
    }
    static __device__ __forceinline__ float logit(const void* row, long long i) {
        if (DTYPE == SI_FP32) return static_cast<const float*>(row)[i];
        return widen<DTYPE == SI_FP16>(static_cast<const uint16_t*>(row)[i]);
    }
    // element for element; NaN where either is
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        if (DTYPE == SI_FP32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else if (DTYPE == SI_FP16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // element for element; NaN where both are
    static __device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) {
        uint32_t d;
        if (DTYPE == SI_FP32) asm("min.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else if (DTYPE == SI_FP16) asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
};

// NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Larger logit <=> larger key, -0 and +0 alike, every NaN the same and above all; then the lower id. Never 0.
__device__ __forceinline__ unsigned long long order_of(float x, int id) {
    const uint32_t key = x != x ? 0xFFFFFFFFu : value_key(x);
    return (unsigned long long)key << 32 | (uint32_t)~id;
}

// The logit of an order (any NaN for NaN).
__device__ __forceinline__ float logit_of(unsigned long long order) {
    const uint32_t key = (uint32_t)(order >> 32);
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// What a set of logits gives: the largest m, s = sum of 2^e and u = sum of e 2^e, e = (x - m) c in powers of two.
struct Sums {
    float m, s, u;
};

// Of both sets. A power below 2^-1000 is 0, whatever it multiplies.
__device__ __forceinline__ Sums both_of(const Sums a, const Sums b, float c) {
    const float m = max_nan(a.m, b.m);
    const float da = fmaxf((a.m - m) * c, -1000.0f), db = fmaxf((b.m - m) * c, -1000.0f);
    const float fa = a.m == -INFINITY ? 0.0f : ex2(da), fb = b.m == -INFINITY ? 0.0f : ex2(db);
    return Sums{m, fa * a.s + fb * b.s, fa * (a.u + da * a.s) + fb * (b.u + db * b.s)};
}

__device__ __forceinline__ Sums shuffled(const Sums a, int o) {
    return Sums{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o), __shfl_xor_sync(0xFFFFFFFFu, a.u, o)};
}

// A warp's 32 values, falling by lane, of 32 in any order.
__device__ __forceinline__ unsigned long long sorted(unsigned long long v, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2) {
            const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, v, j);
            const bool first = (lane & j) == 0, falling = (lane & k) == 0;
            v = (first == falling) == (v > other) ? v : other;
        }
    return v;
}

// The 32 largest of two falling rows, falling; `other` comes rising.
__device__ __forceinline__ unsigned long long merged(unsigned long long v, unsigned long long other, int lane) {
    v = v > other ? v : other;
#pragma unroll
    for (int j = 16; j > 0; j /= 2) {
        const unsigned long long x = __shfl_xor_sync(0xFFFFFFFFu, v, j);
        v = ((lane & j) == 0) == (v > x) ? v : x;
    }
    return v;
}

struct Shared {
    unsigned long long lists[kWarps][32];       // falling rows, a warp's each
    unsigned long long peers[kMostCtas][32];    // the first CTA's: those of the row's CTAs
    Sums sums[kWarps], peer_sums[kMostCtas];
    int chosen[32], n_chosen;
};

// The block's 32 largest in lists[0], of falling rows of its warps (all threads; begins and ends with a barrier).
__device__ __forceinline__ void gather(Shared& S, unsigned long long list, int warp, int lane) {
    __syncthreads();
    S.lists[warp][lane] = list;
#pragma unroll
    for (int w = 1; w < kWarps; w *= 2) {
        __syncthreads();
        if (warp % (2 * w) == 0) S.lists[warp][lane] = list = merged(list, S.lists[warp + w][31 - lane], lane);
    }
    __syncthreads();
}

// A cluster a row, its 16-byte units dealt to the CTAs in equal stretches and
// to a CTA's threads in turn. One pass: a thread keeps the largest logit so
// far, where it was, and the sums relative to it, which are rescaled when it
// grows (a few times a row).
// The K largest: at most K threads of a CTA can have them, the ones whose own
// largest are the K largest of those; only their logits are looked at again,
// a warp a thread, so no order of the logits costs more than K threads' share.
// 2048 rows of 131072 bf16 take 88 us, 6.1 TB/s, 0.91 of what a plain copy
// reaches (fp32 164, 6.5 TB/s; with eight alternatives 102, with 32 128: every
// thread looks for its largest once more, and the candidates); one row of 32768
// fp32 with eight alternatives 5.4 on the GPU (of 262144, 7.8), 7.6 to 9 with the
// host's call; 128 rows of 50001 with four alternatives 12.4, of which the
// alternatives are 4.5: sorts and merges of a block's threads, and a cluster
// barrier. (Where the search for the place of a maximum that grew is done at once,
// in every batch some lane of a warp has one: 124 us for 96.)
template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 4) k_token_logprobs(const __grid_constant__ LogprobsParams P) {
    using U = Unit<DTYPE>;
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = P.V;
    if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
    grid_launch_dependents();
    grid_dependency_wait();
    const long long n = blockIdx.x / CS;
    const uint8_t* const row = static_cast<const uint8_t*>(P.x) + n * P.stride * U::kSize;
    // logits before the first whole unit, units, and logits behind the last: the first CTA's threads take one of those each
    const int head = min(V, (int)(-(reinterpret_cast<intptr_t>(row) / U::kSize) & (U::N - 1)));
    const int units = (V - head) / U::N, tail = V - head - units * U::N;
    const int u0 = (int)((long long)units * rank / CS), u1 = (int)((long long)units * (rank + 1) / CS);
    const uint4* const body = reinterpret_cast<const uint4*>(row + (long long)head * U::kSize);
    const bool has_head = rank == 0 && tid < head, has_tail = rank == 0 && tid < tail;
    const float c = P.inv_t * kLog2e;

    Sums a{-INFINITY, 0.0f, 0.0f};
    uint64_t s2 = 0, u2 = 0;  // what belongs to a.s and a.u, in two sums each
    // where the largest was first: a logit, or -2 - j of the unit j that has it (-1: the thread has none)
    int best = has_head ? tid : u0 + tid < u1 ? -2 - (u0 + tid) : has_tail ? head + units * U::N + tid : -1;
    auto grow = [&](float top) {
        if (a.m != -INFINITY) {
            const float d = fmaxf((a.m - top) * c, -1000.0f), f = ex2(d);
            u2 = mul2(fma2(both(d, d), s2, u2), both(f, f));
            s2 = mul2(s2, both(f, f));
            a.u = f * (a.u + d * a.s);
            a.s *= f;
        }
        a.m = top;
    };
    auto one = [&](float x, int id) {
        if (!(x <= a.m) && a.m == a.m) best = id, grow(x);
        const float e = fmaxf((x - (a.m == -INFINITY ? 0.0f : a.m)) * c, -200.0f), p = ex2(e);
        a.s += p;
        a.u = fmaf(p, e, a.u);
    };
    uint4 next[kBatch];  // under way while the ones before are summed
    auto load = [&](int j) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            next[i] = make_uint4(U::kNone, U::kNone, U::kNone, U::kNone);
            if (j + i * kThreads < u1) next[i] = body[j + i * kThreads];
        }
    };
    load(u0 + tid);
    // the first CTA's tokens: trips to memory of their own
    const bool has_target = rank == 0 && tid < P.M;
    const int target = has_target ? P.targets[n * P.M + tid] : -1;
    const float target_x = target >= 0 && target < V ? U::logit(row, target) : -INFINITY;
    if (has_head) one(U::logit(row, tid), tid);
    for (int j = u0 + tid; j < u1; j += kBatch * kThreads) {
        uint32_t w[4 * kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            w[4 * i] = next[i].x, w[4 * i + 1] = next[i].y, w[4 * i + 2] = next[i].z, w[4 * i + 3] = next[i].w;
        load(j + kBatch * kThreads);
        uint32_t unit[kBatch], hi = 0, lo = w[0];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            unit[i] = U::larger(U::larger(w[4 * i], w[4 * i + 1]), U::larger(w[4 * i + 2], w[4 * i + 3]));
            hi = i ? U::larger(hi, unit[i]) : unit[0];
        }
#pragma unroll
        for (int i = 1; i < 4 * kBatch; ++i) lo = U::smaller(lo, w[i]);
        auto across = [](uint32_t v) {  // a word's largest
            if (DTYPE == SI_FP32) return __uint_as_float(v);
            const float2 p = U::pair(v);
            return max_nan(p.x, p.y);
        };
        const float top = across(hi);
        const float2 l = U::pair(lo);
        const float low = DTYPE == SI_FP32 ? __uint_as_float(lo) : fminf(l.x, l.y);
        if (!(top <= a.m) && a.m == a.m) {  // it grows, or is NaN now
#pragma unroll
            for (int i = kBatch - 1; i >= 0; --i) {
                // For one alternative the batch will do: few threads look again.
                if (P.K < 2 && i > 0) continue;
                const float x = across(unit[i]);
                if (P.K < 2 || x == top || x != x) best = -2 - (j + i * kThreads);
            }
            grow(top);
        }
        const float base = a.m == -INFINITY ? 0.0f : a.m;
        const uint64_t base2 = both(-base, -base), c2 = both(c, c);
        const bool far = !((low - base) * c >= -1000.0f);  // -inf among them, or nearly: e's are bounded, 0 * -inf is NaN
        auto sum = [&](auto bounded) {
#pragma unroll
            for (int i = 0; i < 4 * kBatch; i += 2 / U::kWord) {
                float2 x;
                if (DTYPE == SI_FP32) x = make_float2(__uint_as_float(w[i]), __uint_as_float(w[(i + 1) % (4 * kBatch)]));
                else x = U::pair(w[i]);
                uint64_t e2 = mul2(add2(both(x.x, x.y), base2), c2);
                float e0, e1;
                split(e2, e0, e1);
                if (bounded.value) {
                    e0 = fmaxf(e0, -200.0f), e1 = fmaxf(e1, -200.0f);
                    e2 = both(e0, e1);
                }
                const uint64_t p2 = both(ex2(e0), ex2(e1));
                s2 = add2(s2, p2);
                u2 = fma2(p2, e2, u2);
            }
        };
        if (far) sum(std::true_type());
        else sum(std::false_type());
    }
    if (has_tail) one(U::logit(row, head + units * U::N + tid), head + units * U::N + tid);
    {
        float x, y;
        split(s2, x, y);
        a.s += x + y;
        split(u2, x, y);
        a.u += x + y;
    }
    const float own = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = both_of(a, shuffled(a, o), c);
    if (lane == 0) S.sums[warp] = a;
    if (tid == 0) S.n_chosen = 0;
    if (P.K < 2) __syncthreads();
    bool wanted = P.K > 0 && best != -1;
    if (P.K == 1) {  // of threads whose largest is the block's
        float top = S.sums[0].m;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = max_nan(top, S.sums[w].m);
        wanted = wanted && (own == top || own != own);
    }
    if (wanted && best < -1) {  // the first such logit of that unit, or of its batch
        const int unit = -2 - best;
        best = head + unit * U::N;  // where all are -inf
        bool found = false;
#pragma unroll 1
        for (int k = 0; k < kBatch && !found && unit + k * kThreads < u1; ++k) {
            const uint4 v = body[unit + k * kThreads];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const int first = head + (unit + k * kThreads) * U::N;
            auto is = [&](float x, int i) {
                if (x == own || (own != own && x != x)) best = first + i, found = true;
            };
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                if (DTYPE == SI_FP32) {
                    is(__uint_as_float(w[i]), i);
                } else {
                    const float2 x = U::pair(w[i]);
                    is(x.y, 2 * i + 1);
                    is(x.x, 2 * i);
                }
            }
        }
    }
    const unsigned long long mine = wanted ? order_of(own, best) : 0;
    if (P.K == 1) {
        unsigned long long most = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long x = __shfl_xor_sync(0xFFFFFFFFu, most, o);
            most = most > x ? most : x;
        }
        if (lane == 0) S.lists[warp][0] = most;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWarps; ++w) most = most > S.lists[w][0] ? most : S.lists[w][0];
            S.lists[0][0] = most;
        }
        __syncwarp();
    } else if (P.K > 0) {
        gather(S, sorted(mine, lane), warp, lane);
        {
            const unsigned long long least = S.lists[0][P.K - 1];  // 0: fewer threads have any
            if (mine != 0 && mine >= least) S.chosen[atomicAdd(&S.n_chosen, 1)] = tid;
            __syncthreads();
            unsigned long long list = 0, bar = least;
            // takes what the lanes have that is not below the bar
            auto insert = [&](unsigned long long v) {
                for (unsigned who = __ballot_sync(0xFFFFFFFFu, v != 0 && v >= bar); who; who &= who - 1) {
                    const unsigned long long x = __shfl_sync(0xFFFFFFFFu, v, __ffs(who) - 1);
                    const int at = __popc(__ballot_sync(0xFFFFFFFFu, list > x));
                    const unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, list, 1);
                    list = lane < at ? list : lane == at ? x : before;
                }
                const unsigned long long last = __shfl_sync(0xFFFFFFFFu, list, P.K - 1);
                bar = last > least ? last : least;
            };
            const float least_x = least ? logit_of(least) : -INFINITY;
            for (int i = warp; i < S.n_chosen; i += kWarps) {
                const int t = S.chosen[i], its = u0 + t < u1 ? (u1 - u0 - t + kThreads - 1) / kThreads : 0;  // units
                if (rank == 0 && (t < head || t < tail)) {
                    const int id = lane == 0 && t < head ? t : lane == 1 && t < tail ? head + units * U::N + t : -1;
                    insert(id < 0 ? 0 : order_of(U::logit(row, id), id));
                }
                for (int k0 = 0; k0 < its; k0 += 32) {
                    uint4 w = make_uint4(U::kNone, U::kNone, U::kNone, U::kNone);
                    if (k0 + lane < its) w = body[u0 + t + (k0 + lane) * kThreads];
                    const uint32_t hi = U::larger(U::larger(w.x, w.y), U::larger(w.z, w.w));
                    float top = __uint_as_float(hi);
                    if (DTYPE != SI_FP32) {
                        const float2 h = U::pair(hi);
                        top = max_nan(h.x, h.y);
                    }
                    for (unsigned who = __ballot_sync(0xFFFFFFFFu, k0 + lane < its && !(top < least_x)); who; who &= who - 1) {
                        const int l = __ffs(who) - 1, e = lane % U::N;
                        const uint32_t x = __shfl_sync(0xFFFFFFFFu, w.x, l), y = __shfl_sync(0xFFFFFFFFu, w.y, l);
                        const uint32_t z = __shfl_sync(0xFFFFFFFFu, w.z, l), v = __shfl_sync(0xFFFFFFFFu, w.w, l);
                        const int at = e / U::kWord;
                        const uint32_t mine_w = at == 0 ? x : at == 1 ? y : at == 2 ? z : v;
                        float f = __uint_as_float(mine_w);
                        if (DTYPE != SI_FP32) {
                            const float2 p = U::pair(mine_w);
                            f = e % 2 ? p.y : p.x;
                        }
                        insert(lane < U::N ? order_of(f, head + (u0 + t + (k0 + l) * kThreads) * U::N + e) : 0);
                    }
                }
            }
            gather(S, list, warp, lane);
        }
    }
    // the row's CTAs to the first one, which runs
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
        Sums all = S.sums[0];
        for (int w = 1; w < kWarps; ++w) all = both_of(all, S.sums[w], c);
        Shared& first = *cluster.map_shared_rank(&S, 0);
        if (lane == 0) first.peer_sums[rank] = all;
        if (P.K > 0) first.peers[rank][lane] = S.lists[0][lane];
    }
    if (CS > 1) cluster.sync();
    else __syncthreads();
    if (rank != 0) return;
    a = S.peer_sums[0];
    for (int r = 1; r < CS; ++r) a = both_of(a, S.peer_sums[r], c);
    const bool none = a.m == -INFINITY, odd = a.m != a.m || a.m == INFINITY;
    const float rest = logf(a.s);
    auto logp_of = [&](float x) { return odd ? NAN : none ? -INFINITY : (x - a.m) * P.inv_t - rest; };
    if (tid == 0 && P.entropy) P.entropy[n] = odd ? NAN : none ? 0.0f : rest - 0.693147180559945309f * (a.u / a.s);
    if (has_target) P.logp[n * P.M + tid] = target >= 0 && target < V ? logp_of(target_x) : -INFINITY;
    for (int m = tid + kThreads; m < P.M; m += kThreads) {
        const int id = P.targets[n * P.M + m];
        P.logp[n * P.M + m] = id >= 0 && id < V ? logp_of(U::logit(row, id)) : -INFINITY;
    }
    if (P.K > 0) {
        if (CS > 1) gather(S, warp < CS && lane < P.K ? S.peers[warp][lane] : 0, warp, lane);
        if (tid < P.K) {
            const unsigned long long order = S.lists[0][tid];
            P.top_ids[n * P.K + tid] = (int)~(uint32_t)order;
            P.top_logp[n * P.K + tid] = logp_of(logit_of(order));
        }
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobsParams& P, cudaStream_t st) {
    const void* fn = P.dtype == SI_FP32   ? reinterpret_cast<const void*>(&k_token_logprobs<SI_FP32>)
                     : P.dtype == SI_FP16 ? reinterpret_cast<const void*>(&k_token_logprobs<SI_FP16>)
                                          : reinterpret_cast<const void*>(&k_token_logprobs<SI_BF16>);
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const long long bytes = (long long)P.V * (P.dtype == SI_FP32 ? 4 : 2);
    // CTAs of a row: as many as all rows together fill the GPU with, four an SM, where each has a unit a thread. 128 rows of
    // 50001 with one / two / four / eight: 19.4 / 15.0 / 12.4 / 17.7 us; 2048 of 131072 with one / two: 88.3 / 100.3. (Eight
    // units a thread under way and three CTAs an SM: 14.3 and 132; blocks of 128 threads, eight an SM: 12.3 and 88.8.)
    int cs = 1;
    while (cs < kMostCtas && (long long)P.N * cs * 2 <= 4ll * sms && bytes / (2 * cs) >= 16 * kThreads) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P.N * (unsigned)cs, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[1] = {const_cast<LogprobsParams*>(&P)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace si
