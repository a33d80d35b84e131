// attend.cuh -- what the cache attention's kernels share: the schedule that
// deals a launch's tiles of keys to its CTAs, the gathered copies, and the
// warp-level matrix instructions.
#pragma once

#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "kv.cuh"

namespace si {
namespace {

constexpr int KT = 64;             // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- primitives

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// the same without the choice
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// d += a (16 x 16) * b (16 x 8), fp32 accumulators
template <bool FP16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (FP16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 lanes at once.
__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void split(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// fp16's normal range ends at 2^-14: beside one key that has nearly all of the weight, the others' weights, all of the
// output where that key's value is small, would keep a few bits each (3000 keys at e^-14 of the largest: 4 % off).
// So fp16 weights are taken times 2^15, the most that the type holds, and their sums come out the same power
// larger; the output's quotient does not see it. Where a row's maximum may be outgrown by 2^kLazy before its
// weights are rescaled, the power is that much less. bf16 has fp32's range.
template <bool FP16, bool LAZY>
struct Weights {
    static constexpr int kLazy = !LAZY ? 0 : FP16 ? 4 : 8;
    static constexpr float kUp = FP16 ? 15 - kLazy : 0;  // added to the exponent
    static constexpr float kDown = FP16 ? 1.0f / (1 << (15 - kLazy)) : 1.0f;  // of the sums
};

// log of sum * exp(scale * score). The product is rounded by itself, as where a key's weight is taken: whatever
// the scores' size, scale * score and lse then differ by log(sum) alone.
__device__ __forceinline__ float lse_of(float score, float scale, float sum) {
    return __fadd_rn(__fmul_rn(score, scale), logf(sum));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
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

template <bool FP16>
__device__ __forceinline__ bool not_finite(uint16_t w) {
    return FP16 ? (w & 0x7C00u) == 0x7C00u : (w & 0x7F80u) == 0x7F80u;
}

template <bool FP16>
__device__ __forceinline__ float widen(uint16_t w) {
    if (FP16) return __half2float(*reinterpret_cast<const __half*>(&w));
    return __uint_as_float((uint32_t)w << 16);
}

// Byte offset of 16-byte unit `unit` of row `row` in a tile of rows of DP
// 16-bit elements; the unit index is XORed with the row's low bits so that
// the eight rows of an ldmatrix lie in different banks.
template <int DP>
__device__ __forceinline__ uint32_t tile_at(int row, int unit) {
    return (uint32_t)(row * (DP * 2) + ((unit ^ (row & 7)) * 16));
}

// --------------------------------------------------------------- schedule

// The lists of one launch: `groups` lists a sequence (cache heads x row
// blocks), each of tiles_of(tot[b]) tiles, in flat order.
struct Plan {
    int* len;         // [B] live keys (0 where the sequence is out of bounds)
    int* tot;         // [B] live keys + new nodes (0 likewise)
    int* first;       // [B + 1] flat index of the sequence's first tile
    int* part;        // [B + 1] first part of the sequence, where lists are cut by themselves
    int* cut;         // [1] tiles a part has at most there; 0: CTAs' shares run across lists

    static constexpr int words(int B) { return 4 * B + 3; }
    __device__ __forceinline__ Plan(int* at, int B)
        : len(at), tot(at + B), first(at + 2 * B), part(at + 3 * B + 1), cut(at + 4 * B + 2) {}
};

// K: keys a tile, here and below.
template <int K = KT>
__device__ __forceinline__ int tiles_of(int tot) {
    return tot > K ? (tot + K - 1) / K : 1;
}

// Fills the plan for `ctas` CTAs (all threads; ends with a barrier). Lengths
// are read once.
//
// A list is cut into parts, one CTA each, or the CTAs' shares run across the
// lists' ends. Running across balances any set of lists, but a CTA then
// finishes two lists, and every piece of a list costs it about PIECE tiles'
// time (queries in, partial rows out). So lists are cut by themselves where
// the longest part and one piece take less than an even share and two. A part
// has at least LEAST tiles. (Where every tile can have a CTA of its own, both ways
// are the same and the shorter one is taken: 1000 keys of codes 9.7 -> 8.9 us.)
template <int THREADS, int LEAST, int PIECE, int K = KT>
__device__ void make_plan(const KvView& C, int T, int groups, int ctas, const Plan& p, unsigned* err, bool report) {
    if (C.B == 1) {
        // The same for one sequence, by one thread: the general way's code alone, cold in the instruction
        // cache at every launch, takes 1.3 us of a short call.
        if (threadIdx.x == 0) {
            const int len = C.len[0];
            const bool ok = len >= 0 && len <= C.cap - T;
            if (!ok && report) atomicOr(err, SI_DEVERR_CACHE);
            const int tot = ok ? len + T : 0, n = tiles_of<K>(tot), total = n * groups;
            int q = 0;
            if (PIECE > 0 && groups <= ctas && (LEAST > 1 || total > ctas)) {
                const int even = max(LEAST, div_of(total + ctas - 1, ctas)), m = div_of(ctas, groups);
                q = max(even, div_of(n + m - 1, m));
                if (q > even + PIECE) q = 0;
            }
            p.len[0] = ok ? len : 0;
            p.tot[0] = tot;
            p.first[0] = p.part[0] = 0;
            p.first[1] = total;
            p.part[1] = q ? div_of(n + q - 1, q) * groups : 0;
            *p.cut = q;
        }
        __syncthreads();
        return;
    }
    for (int b = threadIdx.x; b < C.B; b += THREADS) {
        const int len = C.len[b];
        const bool ok = len >= 0 && len <= C.cap - T;
        if (!ok && report) atomicOr(err, SI_DEVERR_CACHE);
        p.len[b] = ok ? len : 0;
        p.tot[b] = ok ? len + T : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        // out[b]: sum of value(n tiles) * groups over the sequences before b
        auto scan = [&](int* out, auto value) {
            int base = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < C.B; b0 += 32) {
                const int b = b0 + lane;
                const int mine = b < C.B ? value(tiles_of<K>(p.tot[b])) * groups : 0;
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (b < C.B) out[b] = base + incl - mine;
                base += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            if (lane == 0) out[C.B] = base;
            return base;
        };
        const int total = scan(p.first, [](int n) { return n; });
        int q = 0;
        if (PIECE > 0 && C.B * groups <= ctas && (LEAST > 1 || total > ctas)) {
            // the least number of tiles a part, from the even share up, that needs no more than ctas parts
            const int even = max(LEAST, div_of(total + ctas - 1, ctas));
            // Four lanes try each number: 8 sequences on tcgen05 take 1.2 us more where all lanes try one number after the
            // other, and few rows a key 1 us more where a lane each tries them all over.
            static_assert(PIECE < 8, "eight numbers are tried");
            int parts = 0;
            for (int b = lane & 3; b < C.B; b += 4) parts += div_of(tiles_of<K>(p.tot[b]) + even + (lane >> 2) - 1, even + (lane >> 2));
            parts += __shfl_xor_sync(0xFFFFFFFFu, parts, 1);
            parts += __shfl_xor_sync(0xFFFFFFFFu, parts, 2);
            const unsigned fits = __ballot_sync(0xFFFFFFFFu, lane >> 2 <= PIECE && parts * groups <= ctas);
            if (fits) q = even + ((__ffs(fits) - 1) >> 2);
        }
        if (q) scan(p.part, [q](int n) { return div_of(n + q - 1, q); });
        if (lane == 0) *p.cut = q;
    }
    __syncthreads();
}

// Which tiles a CTA has, and which CTAs a list has. All in 32 bits: this runs
// for every row that is joined.
template <int K>
struct DealOf {
    const Plan& p;
    int B, q, end;
    unsigned base, rem;  // shares across lists: rem CTAs of base + 1 tiles, then base each

    __device__ __forceinline__ DealOf(const Plan& plan, int seqs, int ctas, int least) : p(plan), B(seqs) {
        q = *plan.cut;
        end = plan.first[seqs];
        base = rem = 0;
        if (q) return;
        const unsigned n = max(1u, min((unsigned)ctas, (unsigned)end / (unsigned)least));
        base = (unsigned)end / n;
        rem = (unsigned)end - base * n;
    }
    __device__ __forceinline__ int start(int cta) const { return min(end, (int)(cta * base + min((unsigned)cta, rem))); }
    __device__ __forceinline__ int owner(int x) const {
        const unsigned longer = rem * (base + 1);
        return (int)((unsigned)x < longer ? (unsigned)x / (base + 1) : rem + ((unsigned)x - longer) / base);
    }
    // first tile of part k of m of a list of n
    static __device__ __forceinline__ int part_start(int n, int m, int k) {
        const int each = div_of(n, m);
        return k * each + min(k, n - each * m);
    }
    __device__ __forceinline__ void range(int cta, int& x0, int& x1) const {
        if (!q) {
            x0 = start(cta), x1 = start(cta + 1);
            return;
        }
        x0 = x1 = 0;
        if (cta >= p.part[B]) return;
        int lo = 0, hi = B - 1;  // last b with part[b] <= cta
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.part[mid] <= cta) lo = mid;
            else hi = mid - 1;
        }
        const int n = tiles_of<K>(p.tot[lo]), m = div_of(n + q - 1, q);
        const int group = div_of(cta - p.part[lo], m), k = cta - p.part[lo] - group * m;
        x0 = p.first[lo] + group * n + part_start(n, m, k);
        x1 = p.first[lo] + group * n + part_start(n, m, k + 1);
    }
    // The CTAs of a list, and whether the first of them has another list before it.
    __device__ __forceinline__ void ctas_of(int b, int group, int& first, int& last, bool& second) const {
        const int n = tiles_of<K>(p.tot[b]);
        if (q) {
            const int m = div_of(n + q - 1, q);
            first = p.part[b] + group * m;
            last = first + m - 1;
            second = false;
            return;
        }
        const int y0 = p.first[b] + group * n;
        first = owner(y0);
        last = owner(y0 + n - 1);
        second = start(first) < y0;
    }
};
using Deal = DealOf<KT>;

// A position in the flat order of tiles.
struct At {
    int b, group, tile, ntile;
};

template <int K = KT>
__device__ __forceinline__ At locate(const Plan& p, int B, int x) {
    int lo = 0, hi = B - 1;  // last b with first[b] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    At a;
    a.b = lo;
    a.ntile = tiles_of<K>(p.tot[lo]);
    const int in = x - p.first[lo];
    a.group = div_of(in, a.ntile);
    a.tile = in - a.group * a.ntile;
    return a;
}

template <int K = KT>
__device__ __forceinline__ void step(const Plan& p, int B, int groups, At& a) {
    if (++a.tile < a.ntile) return;
    a.tile = 0;
    if (++a.group < groups) return;
    a.group = 0;
    if (++a.b < B) a.ntile = tiles_of<K>(p.tot[a.b]);
}

// Ancestor word of node t (mask NULL: a chain).
__device__ __forceinline__ unsigned long long word_of(const unsigned long long* mask, int T, int b, int t) {
    return mask ? mask[(long long)b * T + t] : (t >= 63 ? ~0ull : (2ull << t) - 1);
}

constexpr int kNoSlot = INT_MIN;

// Nodes of sequence b that any of its nodes sees (all lanes of a warp).
__device__ __forceinline__ unsigned long long seen_nodes(const unsigned long long* mask, int T, int b, int lane) {
    unsigned long long mine = lane < T ? word_of(mask, T, b, lane) : 0;
    if (lane + 32 < T) mine |= word_of(mask, T, b, lane + 32);
    return (unsigned long long)__reduce_or_sync(0xFFFFFFFFu, (unsigned)(mine >> 32)) << 32 |
           __reduce_or_sync(0xFFFFFFFFu, (unsigned)mine);
}

// Slot of list entry i, or kNoSlot where nothing is to be read. The value is not
// looked at here: it is used a tile later, so the load's latency is hidden.
__device__ __forceinline__ int slot_of(const int32_t* list, int i, int len, int tot, unsigned long long seen) {
    const bool on = i < len || (i < tot && (seen >> ((i - len) & 63) & 1));
    if (!on) return kNoSlot;
    return list ? list[i] : i;
}

// A slot outside the pool is reported and not read.
__device__ __forceinline__ bool slot_ok(int slot, int n_slots, unsigned* err) {
    if ((unsigned)slot < (unsigned)n_slots) return true;
    if (slot != kNoSlot) atomicOr(err, SI_DEVERR_CACHE);
    return false;
}

// Floats of one partial: RB rows of output, then their maxima and sums.
constexpr int part_floats(int rb, int dp) { return rb * (dp + 2); }

// Query rows a CTA of the tensor-memory kernel takes: two blocks of 128 in one CTA an SM copy a tile once, one
// block leaves room for two CTAs, which copy it twice (64 lists of up to 8192 keys of 128 elements, two blocks /
// one: 132 rows 61 / 71 us, 256 rows 71 / 79; 8 lists of 2000, 256 rows 21.1 / 20.7).
inline int wide_rows(int R) { return R <= 128 ? 128 : 256; }

// For it and the narrow kernel, the tiles a part of a list has at least and what a piece of a list costs beside its
// tiles, in tiles: 128 lists of up to 300 keys, 32 rows, take 18 us, 30 with the shares always across the lists.
constexpr int kWideLeast = 4, kWidePiece = 6;
constexpr int kNarrowLeast = 1, kNarrowPiece = 4;

// Who copies what: a warp copies sixteen keys of every tile, lane i < 16
// holding the slot of its key i.
template <int DP>
struct Copy {
    static constexpr int UNITS = DP / 8;            // 16-byte units of a row
    static constexpr int AT_ONCE = 32 / UNITS;      // rows one sweep of a warp copies
    static constexpr int SWEEPS = 16 / AT_ONCE;
    // row (of the warp's sixteen) that this lane copies in sweep j
    static __device__ __forceinline__ int row(int lane, int j) { return (lane / UNITS) * SWEEPS + j; }
    // Slots of the rows this lane copies, from the lanes that hold them. All at once, ahead of the copies:
    // a shuffle between two copies would put its latency between them.
    static __device__ __forceinline__ void slots(int held, int lane, int (&slot)[SWEEPS]) {
#pragma unroll
        for (int j = 0; j < SWEEPS; ++j) slot[j] = __shfl_sync(0xFFFFFFFFu, held, row(lane, j));
    }
};

// The copying side of a CTA's walk over its tiles: where the next tile's rows
// are. What depends on the list alone is worked out when the list changes. E: an
// element of the pools, two bytes or an e4m3 code.
template <class E, int K = KT>
struct SourceOf {
    At at;
    int x, x1;                 // flat index of the next tile, and of the first one that is not ours
    const int32_t* list;
    const E* k;
    const E* v;
    const uint8_t* k_scale;    // where E is a code
    const uint8_t* v_scale;
    const float* acc;
    int len, tot;
    unsigned long long seen;   // nodes that any row sees (all of them where the caller says so)

    __device__ __forceinline__ void start(const Plan& p, int B, int first, int end) {
        at = locate<K>(p, B, first);
        x = first, x1 = end;
    }
    __device__ __forceinline__ void enter(const KvView& C, const Plan& p, int row_blocks) {
        const int h = at.group / row_blocks;
        list = C.table ? C.table + at.b * C.tb + h * C.th : nullptr;
        k = static_cast<const E*>(C.k) + at.b * C.kb + h * C.kh;
        v = static_cast<const E*>(C.v) + at.b * C.vb + h * C.vh;
        if (sizeof(E) == 1) {
            k_scale = C.k_scale + at.b * C.kcb + h * C.kch;
            v_scale = C.v_scale + at.b * C.vcb + h * C.vch;
        }
        acc = C.acc + at.b * C.ab + h * C.ah;
        len = p.len[at.b], tot = p.tot[at.b];
    }
    // True where the next tile is of another list.
    __device__ __forceinline__ bool next(const Plan& p, int B, int groups) {
        ++x;
        if (++at.tile < at.ntile) return false;
        at.tile = at.ntile - 1;
        step<K>(p, B, groups, at);
        return true;
    }
};
using Source = SourceOf<uint16_t>;

inline cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, void** args, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace
}  // namespace si
