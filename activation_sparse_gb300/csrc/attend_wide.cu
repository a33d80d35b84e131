// attend_wide.cu -- tree attention for many rows a key (wide trees, shared
// heads) on the 5th-generation tensor cores.
//
// One or two blocks of 128 query rows of one list meet tiles of 64 keys, each
// with products of its own:
//   S = Q K^T   tcgen05.mma M = 128, N = 64, K = D    (accumulator in TMEM)
//   P = exp(scale (S - m))                            (one thread a row)
//   O += P V    tcgen05.mma M = 128, N = D, K = 64    (P and the accumulator in TMEM)
// There are two S, and P is written over the half of its S that has been
// read, so the softmax of a tile waits for nothing but its own S: with one S
// and P in shared memory every tile was a chain of waits (softmax, product,
// product), 1.1 us a tile with all work taken out. The value tile serves as
// it lies, [key][d], as an operand with d contiguous.
// The reference m of a row moves only when the maximum outgrows it by a
// factor of 2^8 (fp16: 2^4, see Weights): weights up to 256 are as exact in 16
// bits as weights up to 1, and the sums are in 32 bits, so the output is
// rescaled a few times a list instead of once a tile.
//
// Four warps a block do its softmax and output (TMEM lanes 32 w ..), one warp
// issues the matrix instructions, four copy keys and values through the slot
// table (16-byte asynchronous copies into the 128-byte swizzle the tensor
// cores read; the TMA's four-row gather moves as much an instruction but takes
// its operands from uniform registers, some twenty instructions a gather
// where a copy takes four, and was no faster). More than 128 rows go through
// one CTA an SM with two blocks, which copies a tile once; with one block two
// CTAs share the SM. 8 trees of 64 nodes x 32 heads over up to 8192 keys of 8
// heads of 128: 71 us with two blocks, 550 TFLOP/s (79 with one block and every
// tile copied twice); the tensor pipe is 33 % busy, what bounds it is the
// softmax's instructions and the waits between the roles. 64 keys take 1.7 us;
// a list costs some 6 us beside (queries in, rows out).
// P is rounded once to the cache's type: in two terms of it, as the kernel for
// few rows takes its weights, the output's error against 64 bits would be the
// output's own rounding alone (fp16 0.00021 instead of 0.00028), but the
// second terms' instructions lie in the chain that bounds this kernel (72 / 80 us
// above; 6 trees of 16 nodes, 9001 keys 27.5 / 28.6).
// Over a cache of e4m3 codes the copying warps copy the codes as they are, tiles
// ahead, and turn what they copied themselves into elements of the type of q,
// scale and all (exactly, see si_kv_create_e4m3): the rest of the kernel does
// not know. That work is on the way of every tile: the trees above take 81 us
// (bf16 90), of which the products wait for keys 13 %; the copying warps are
// busy nine tenths of a tile's time, with some 400 instructions that the caches
// of instructions cannot hold next to the softmax's. Eight copying warps instead
// of four: 3 us more and 3 less; a tile's codes held in registers instead of shared
// memory: 1 more and 2 less with two blocks, but 60 instead of 50 us with one (T = 16).
// Every write to shared memory is an ordinary one; the issuing warp's proxy
// fence, after the barrier that announces it, lets the tensor cores see it. All
// waits are bounded; TMEM is always released.
#include <type_traits>

#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kBlock = 128;        // query rows of one product: a TMEM lane each
constexpr int kCopyWarps = 4, kCopyThreads = 32 * kCopyWarps;

// NB row blocks a CTA meet every key tile it copies. E4M3: a cache of codes, which are copied as they are (a key or a
// value tile each of kRaw places) and then become a ring slot's elements.
template <int DP, int NB, bool E4M3>
struct WideCfg {
    static constexpr int kRows = kBlock * NB;
    static constexpr int kSoftmaxWarps = 4 * NB;
    static constexpr int kMmaWarp = kSoftmaxWarps, kCopyWarp = kMmaWarp + 1;
    static constexpr int kThreads = 32 * (kCopyWarp + kCopyWarps);
    static constexpr int kCtas = NB == 1 ? 2 : 1;              // an SM
    static constexpr int kMaxSlots = E4M3 ? (NB == 1 ? 3 : 8) : NB == 1 ? 5 : 9;  // ring slots: a key or a value tile each
    static constexpr int kTile = KT * DP * 2;
    static constexpr int kRaw = E4M3 ? 3 : 0;
    static constexpr int kScaleTiles = 4;                      // whose scales are kept
    static constexpr int kRawBytes = kRaw * (kTile / 2) + (E4M3 ? kCopyWarps * kScaleTiles * 32 * 4 : 0);
    static constexpr int kQ = kBlock * DP * 2;                 // of one block
    static constexpr int kOffRing = NB * kQ;
    static constexpr int kColP = KT / 2, kColO = 2 * KT;       // TMEM columns of a block: two S (P in the second half), O
    static constexpr int kCols = kColO + DP;
    static constexpr int kTmemCols = NB * kCols <= 256 ? 256 : 512;
    static constexpr int kBars = 2 * kMaxSlots + 7 * NB;
    static constexpr int fixed(int B) { return (kBars + 1) * 8 + (kMaxSlots + 1) * 8 + 16 + Plan::words(B) * 4; }
    static constexpr int smem(int B, int slots) { return kOffRing + slots * kTile + kRawBytes + fixed(B); }
    static constexpr int kSmemLimit = NB == 1 ? 113 * 1024 : 227 * 1024;  // of the SM's 228 KB, 1 KB a CTA is the system's
};

// 128-byte swizzled tile of rows of 64 elements: byte offset of 16-byte unit
// c (0..7) of row r.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Shared-memory matrix descriptor, 128-byte swizzle: start address >> 4 (bits
// 0-13), leading offset >> 4 (16-29), stride offset >> 4 (32-45), version 1
// (46-47), swizzle mode 2 (61-63). Stride: 1024 bytes between groups of eight
// 128-byte rows. Leading: between sub-tiles of 64 elements where the rows are
// the reduced dimension (the value tile), unused otherwise.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lead) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The products are issued by one lane of a warp that runs the surrounding
// code as a whole: what they take then lies in uniform registers. (A branch for
// the one lane costs some ninety cycles an instruction in moves, where a
// product takes 32 to 64.)
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}

// The same with A in TMEM: a row a lane, two elements a column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                          uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}

// One lane of the warp: 1 there, 0 elsewhere.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}

// 32 fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Bounded wait that an earlier failure does not cut short.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = cycles();
    while (!mbar_try_wait(bar, parity)) {
        if (cycles() - t0 > kDrainLimitCycles) return;
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace

// a * b in fp32 of two fp16
__device__ __forceinline__ float product(uint32_t a, uint32_t b, bool high) {
    float d;
    if (high) asm("{\n\t.reg .b16 x, y, s, t;\n\tmov.b32 {x, y}, %1;\n\tmov.b32 {s, t}, %2;\n\tfma.rn.f32.f16 %0, y, s, 0f00000000;\n\t}" : "=f"(d) : "r"(a), "r"(b));
    else asm("{\n\t.reg .b16 x, y, s, t;\n\tmov.b32 {x, y}, %1;\n\tmov.b32 {s, t}, %2;\n\tfma.rn.f32.f16 %0, x, s, 0f00000000;\n\t}" : "=f"(d) : "r"(a), "r"(b));
    return d;
}

// Sixteen codes times their scale as sixteen elements of the type, exactly. IN_HALF: the scale is an fp16 number (all of
// an fp16 cache's are), which the product takes as it is.
template <bool FP16, bool IN_HALF>
__device__ __forceinline__ void elements16(uint4 codes, float scale, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t e[8];
    const __half2 scale2 = __float2half2_rn(scale);
    const uint32_t scale_w = *reinterpret_cast<const uint32_t*>(&scale2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        halves4(w[i], h[0], h[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __half2 x = *reinterpret_cast<const __half2*>(&h[j]);
            if (FP16) {
                const __half2 y = __hmul2(x, scale2);
                e[2 * i + j] = *reinterpret_cast<const uint32_t*>(&y);
            } else if (IN_HALF) {
                e[2 * i + j] = pack<false>(product(h[j], scale_w, false), product(h[j], scale_w, true));
            } else {
                const float2 f = __half22float2(x);
                e[2 * i + j] = pack<false>(f.x * scale, f.y * scale);
            }
        }
    }
    lo = make_uint4(e[0], e[1], e[2], e[3]), hi = make_uint4(e[4], e[5], e[6], e[7]);
}

// The copying warps over a cache of codes: every lane copies 16 bytes of some of its warp's keys, several tiles ahead, and
// turns what it copied itself into elements.
template <int DP, int NB, bool FP16>
__device__ __forceinline__ void copy_codes(const AttendParams& P, const Plan& plan, int row_blocks, int x0, int x1, int slots,
                                           uint8_t* ring, uint64_t* full, uint64_t* empty, uint16_t* odd) {
    using Cfg = WideCfg<DP, NB, true>;
    constexpr int RAW = Cfg::kRaw;
    constexpr int WK = KT / kCopyWarps;  // sixteen keys a warp has of a tile
    using Cp = Copy8<DP, WK>;
    const KvView& C = P.c;
    const int T = P.T, D = C.D, groups = C.Hkv * row_blocks;
    const int warp = (threadIdx.x >> 5) - Cfg::kCopyWarp, lane = threadIdx.x & 31, unit = lane % Cp::UNITS;
    const int own0 = warp * WK, of_v = lane / WK & 1;  // lane i % WK has key i: its key's scale or, of the next WK lanes, its value's
    const bool unit_on = unit * 16 < D, whole_rows = D == DP;
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks, v_step = (int)C.vs;
    uint8_t* const sub_tile = ring + (unit >> 2) * (KT * 128);  // 64 elements are four units of codes
    uint8_t* const raw = ring + slots * Cfg::kTile + (warp * 32 + lane) * 16;  // [place][row of the lane][thread]
    float* const scale_s = reinterpret_cast<float*>(ring + slots * Cfg::kTile + RAW * (Cfg::kTile / 2)) + warp * Cfg::kScaleTiles * 32;
    const uint32_t raw_addr = smem_u32(raw);
    constexpr int kPlace = Cfg::kTile / 2, kRow = kCopyThreads * 16;
    SourceOf<uint8_t> src;
    src.start(plan, C.B, x0, x1);
    int held = kNoSlot, seen_b = -1;
    auto fetch = [&]() {
        const int i0 = src.at.tile * KT;
        if (i0 + KT > src.len && seen_b != src.at.b) {
            src.seen = seen_nodes(P.mask, T, src.at.b, lane);
            seen_b = src.at.b;
        }
        held = slot_of(src.list, i0 + own0 + lane % WK, src.len, src.tot, src.seen);
    };
    int slot[Cp::SWEEPS];
    int in = 0, in_tile = 0, byte = -1;  // place of the next copies; a scale on its way (-1: none)
    bool all = false;                   // whether they leave nothing out
    const uint8_t* v_from = nullptr;
    bool on = false;                    // whether the values of the tile whose keys went last are still to come
    auto copy = [&](const uint8_t* from, int step_) {
        if (all) {
            from += unit * 16;
#pragma unroll
            for (int j = 0; j < Cp::SWEEPS; ++j) cp16(raw_addr + in * kPlace + j * kRow, from + (long long)slot[j] * step_);
        } else {
#pragma unroll
            for (int j = 0; j < Cp::SWEEPS; ++j) {
                const bool there = slot[j] >= 0 && unit_on;
                cp16(raw_addr + in * kPlace + j * kRow, there ? from + (long long)slot[j] * step_ + unit * 16 : from, there);
            }
        }
        if (++in == RAW) in = 0;
    };
    // the next key or value tile's copies, in turn
    auto issue = [&]() {
        if (on) {
            copy(v_from, v_step);
            on = false;
            cp_commit();
            return;
        }
        if (byte >= 0) {  // the scales of the tile before have had a tile's time to arrive
            scale_s[in_tile * 32 + lane] = scale_of(byte, C.e_lo, C.e_hi);
            if (++in_tile == Cfg::kScaleTiles) in_tile = 0;
            byte = -1;
        }
        if (src.x < x1) {
            const bool ok = slot_ok(held, n_slots, P.err);
            const bool cached = src.at.tile * KT + KT <= src.len;
            const int mine = ok ? held : cached ? 0 : -1;  // a bad slot has been reported; slot 0 is read
            all = cached && whole_rows;
            Cp::slots(mine, lane, slot);
            byte = 127;
            if (mine >= 0) byte = (of_v ? src.v_scale : src.k_scale)[mine >> C.block_shift];
            copy(src.k, k_step);
            v_from = src.v;
            on = true;
            if (src.next(plan, C.B, groups) && src.x < x1) src.enter(C, plan, row_blocks);
            if (src.x < x1) fetch();
        }
        cp_commit();
    };
    int at = 0, fill = 0;               // ring slot of the next group and how often the ring has been round
    auto take = [&]() {
        if (fill > 0) mbar_wait(&empty[at], (uint32_t)((fill - 1) & 1), P.err, kSiteAttend | kSiteEmpty);
        __syncwarp();
        const int mine = at;
        if (++at == slots) at = 0, ++fill;
        return mine;
    };
    // The loops below are short on purpose: the code of all roles together does not fit the instruction caches next to the
    // warps, and straight code runs at the pace at which it is fetched.
    src.enter(C, plan, row_blocks);
    fetch();
#pragma unroll 1
    for (int i = 0; i < RAW - 1; ++i) issue();
    At a = locate(plan, C.B, x0);
    int out = 0, out_tile = 0;          // place of the next tile that becomes elements
    float scale = 1.0f;
    bool in_half = true, cached = true;
    int i0 = 0, len = 0;
#pragma unroll 1
    for (int half = 0; half < 2 * (x1 - x0); ++half) {
        const bool is_v = half & 1;
        cp_wait<RAW - 2>();
        issue();
        __syncwarp();
        if (!is_v) {
            i0 = a.tile * KT, len = plan.len[a.b];
            cached = i0 + KT <= len;
            step(plan, C.B, groups, a);
            scale = scale_s[out_tile * 32 + lane];  // written when the next tile's keys went out, at the latest just now
            if (++out_tile == Cfg::kScaleTiles) out_tile = 0;
            // 2^-24 .. 2^15, 0 or NaN; a cache of bf16 with other scales among the warp's takes the longer way
            in_half = FP16 || __all_sync(0xFFFFFFFFu, !(scale > 32768.0f) && !(scale < 5.9604644775390625e-8f && scale > 0.0f));
        }
        uint8_t* const from = raw + out * kPlace;
        if (++out == RAW) out = 0;
        const int to = take();
        if (is_v && !cached) {
            // New nodes' value rows that are NaN leave the tile (0 * NaN is NaN) and are reported, so that the rows that
            // see them get them back at the end. A lane looks at what it copied itself.
            unsigned bad = 0;
            const int node = i0 + own0 + lane % WK - len;
            if (of_v && node >= 0 && node < T && scale != scale) bad |= 1u << lane % WK, scale = 0.0f;
#pragma unroll 1
            for (int j = 0; j < Cp::SWEEPS; ++j) {
                const int r = Cp::row(lane, j), of = i0 + own0 + r - len;
                if (of < 0 || of >= T) continue;
                for (int i = 0; i < 16; ++i)
                    if (code_nan(from[j * kRow + i])) from[j * kRow + i] = 0, bad |= 1u << r;
            }
            bad = __reduce_or_sync(0xFFFFFFFFu, bad);
            if (lane == 0) odd[to * 4 + own0 / 16] = (uint16_t)bad;
        }
        uint8_t* const tile = sub_tile + to * Cfg::kTile;
#pragma unroll 1
        for (int j = 0; j < Cp::SWEEPS; ++j) {
            const int r = Cp::row(lane, j);
            const float by = __shfl_sync(0xFFFFFFFFu, scale, (is_v ? WK : 0) + r);
            const uint4 codes = *reinterpret_cast<const uint4*>(from + j * kRow);
            uint4 lo, hi;
            if (in_half) elements16<FP16, true>(codes, by, lo, hi);
            else elements16<FP16, false>(codes, by, lo, hi);
            *reinterpret_cast<uint4*>(tile + sw128(own0 + r, 2 * (unit & 3))) = lo;
            *reinterpret_cast<uint4*>(tile + sw128(own0 + r, 2 * (unit & 3) + 1)) = hi;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[to]);  // one arrival a warp
    }
    cp_wait<0>();
}

template <int DP, int NB, bool FP16, bool E4M3>
__global__ void __launch_bounds__(WideCfg<DP, NB, E4M3>::kThreads, WideCfg<DP, NB, E4M3>::kCtas)
    k_tree_attention_wide(const __grid_constant__ AttendParams P, int row_blocks, int slots) {
    using Cfg = WideCfg<DP, NB, E4M3>;
    constexpr int kThreads = Cfg::kThreads, kMaxSlots = Cfg::kMaxSlots;
    using Cp = Copy<DP>;
    using Wt = Weights<FP16, true>;
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle needs tiles on 1024-byte boundaries
    uint8_t* const q_s = smem;
    uint8_t* const ring = smem + Cfg::kOffRing;
    uint64_t* const full = reinterpret_cast<uint64_t*>(ring + slots * Cfg::kTile + Cfg::kRawBytes);
    uint64_t* const empty = full + kMaxSlots;
    uint64_t* const q_full = empty + kMaxSlots;  // [block] this list's queries are in shared memory
    uint64_t* const s_full = q_full + NB;        // [block][2] S of a tile is in TMEM
    // [block][2] P of a tile is in TMEM, and O includes the tile (its S and P are free). Two barriers of each, for
    // even and odd tiles: the S of a tile is out before the last tile's product, which waits for the slowest warp and
    // the other block, so a quick warp is done with its P while that product is still to come. One barrier would
    // then be waited for two phases ahead, which its parity cannot tell from none.
    uint64_t* const p_full = s_full + 2 * NB;
    uint64_t* const o_done = p_full + 2 * NB;
    uint16_t* const odd = reinterpret_cast<uint16_t*>(full + Cfg::kBars + 1);  // [slot][4]: keys of a value tile that are not finite
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(odd + kMaxSlots * 4);
    const Plan plan(reinterpret_cast<int*>(tmem_slot + 4), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = P.T, G = P.G, R = T * G, D = C.D;
    const int groups = C.Hkv * row_blocks;

    if (smem_u32(smem) & 1023u) {  // never seen: dynamic shared memory starts on such a boundary
        if (tid == 0) atomicOr(P.err, SI_DEVERR_COUNT);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < kMaxSlots; ++s) {
            mbar_init(&full[s], E4M3 ? kCopyWarps : kCopyThreads);
            mbar_init(&empty[s], 1);
        }
        for (int k = 0; k < NB; ++k) {
            mbar_init(&q_full[k], kBlock);
            mbar_init(&s_full[2 * k], 1);
            mbar_init(&s_full[2 * k + 1], 1);
            mbar_init(&p_full[2 * k], kBlock);
            mbar_init(&p_full[2 * k + 1], kBlock);
            mbar_init(&o_done[2 * k], 1);
            mbar_init(&o_done[2 * k + 1], 1);
        }
        fence_mbar_init();
    }
    if (warp == Cfg::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(Cfg::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    grid_dependency_wait();
    // After the wait: the join reads the lengths before its own. And by the warp that has the tensor memory: a later
    // grid that takes tensor memory and then waits for this one may only start where this one has its own.
    if (warp == Cfg::kMmaWarp) grid_launch_dependents();
    make_plan<kThreads, kWideLeast, kWidePiece>(C, T, groups, gridDim.x, plan, P.err, blockIdx.x == 0);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Deal deal(plan, C.B, gridDim.x, kWideLeast);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);

    if (x0 >= x1) {
        // more CTAs than tiles: nothing to do
    } else if (E4M3 && warp >= Cfg::kCopyWarp) {
        copy_codes<DP, NB, FP16>(P, plan, row_blocks, x0, x1, slots, ring, full, empty, odd);
    } else if (!E4M3 && warp >= Cfg::kCopyWarp) {
        // ---------------------------------------------------------- copies
        const int own0 = (warp - Cfg::kCopyWarp) * 16, unit = lane % Cp::UNITS;
        const bool unit_on = unit * 8 < D, whole_rows = D == DP;
        const int n_slots = (int)C.n_slots, k_step = (int)C.ks, v_step = (int)C.vs;
        const uint32_t ring_addr = smem_u32(ring) + (uint32_t)(unit >> 3) * (KT * 128);  // this lane's sub-tile
        Source src;
        src.start(plan, C.B, x0, x1);
        int held = kNoSlot, seen_b = -1;
        auto fetch = [&]() {
            const int i0 = src.at.tile * KT;
            if (i0 + KT > src.len && seen_b != src.at.b) {
                src.seen = seen_nodes(P.mask, T, src.at.b, lane);
                seen_b = src.at.b;
            }
            held = slot_of(src.list, i0 + own0 + (lane & 15), src.len, src.tot, src.seen);
        };
        // The barrier hears of this thread's copies when they land. The thread that issues the products
        // makes them visible to the tensor cores: a proxy fence here would wait for every copy in flight.
        auto arrive_landed = [&](int slot_at) {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[slot_at])) : "memory");
        };
        // New nodes' value rows that are not finite leave the tile (0 * NaN is NaN) and are
        // reported, so that the rows that see them get them back at the end.
        auto clean = [&](int slot_at, int i0, int len) {
            uint8_t* tile = ring + slot_at * Cfg::kTile + (unit >> 3) * (KT * 128);
            unsigned bad = 0;
#pragma unroll 1
            for (int j = 0; j < Cp::SWEEPS; ++j) {
                const int r = Cp::row(lane, j), node = i0 + own0 + r - len;
                if (node < 0 || node >= T) continue;
                uint16_t* e = reinterpret_cast<uint16_t*>(tile + sw128(own0 + r, unit & 7));
                for (int i = 0; i < 8; ++i)
                    if (not_finite<FP16>(e[i])) e[i] = 0, bad |= 1u << r;
            }
            bad = __reduce_or_sync(0xFFFFFFFFu, bad);
            if (lane == 0) odd[slot_at * 4 + own0 / 16] = (uint16_t)bad;
        };
        int at = 0, fill = 0;               // ring slot of the next group and how often the ring has been round
        auto take = [&]() {
            if (fill > 0) mbar_wait(&empty[at], (uint32_t)((fill - 1) & 1), P.err, kSiteAttend | kSiteEmpty);
            __syncwarp();
            const int mine = at;
            if (++at == slots) at = 0, ++fill;
            return mine;
        };
        src.enter(C, plan, row_blocks);
        fetch();
        while (src.x < x1) {
            const int i0 = src.at.tile * KT, len = src.len;
            const bool cached = i0 + KT <= len, ok = slot_ok(held, n_slots, P.err);
            int slot[Cp::SWEEPS];
            // cached keys: nothing to leave out (a slot outside the pool has been reported; slot 0 is read)
            Cp::slots(ok ? held : cached ? 0 : -1, lane, slot);
            const uint16_t *kp = src.k + unit * 8, *vp = src.v + unit * 8;
            auto copy = [&](uint32_t dst, const uint16_t* from, const uint16_t* nowhere, int step_) {
                if (cached && whole_rows) {
#pragma unroll
                    for (int j = 0; j < Cp::SWEEPS; ++j)
                        cp16(dst + sw128(own0 + Cp::row(lane, j), unit & 7), from + (long long)slot[j] * step_);
                } else {
#pragma unroll
                    for (int j = 0; j < Cp::SWEEPS; ++j) {
                        const bool on = slot[j] >= 0 && unit_on;
                        cp16(dst + sw128(own0 + Cp::row(lane, j), unit & 7),
                             on ? from + (long long)slot[j] * step_ : nowhere, on);
                    }
                }
            };
            const int k_at = take();
            copy(ring_addr + k_at * Cfg::kTile, kp, src.k, k_step);
            arrive_landed(k_at);
            const uint16_t* v_nowhere = src.v;
            if (src.next(plan, C.B, groups) && src.x < x1) src.enter(C, plan, row_blocks);
            if (src.x < x1) fetch();
            const int v_at = take();
            copy(ring_addr + v_at * Cfg::kTile, vp, v_nowhere, v_step);
            if (!cached) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                clean(v_at, i0, len);
                mbar_arrive(&full[v_at]);
            } else {
                arrive_landed(v_at);
            }
        }
        // No copy is in flight when the CTA ends, even after a wait that ran out.
        asm volatile("cp.async.wait_all;" ::: "memory");
        const int groups_in = 2 * (x1 - x0);
        for (int s = 0; s < slots && s < groups_in; ++s)
            mbar_drain(&full[s], (uint32_t)((groups_in - s + slots - 1) / slots - 1) & 1u);
    } else if (warp == Cfg::kMmaWarp) {
        // ------------------------------------------------- matrix products
        {
            const uint32_t leader = elect_lane();
            const int count = __reduce_max_sync(0xFFFFFFFFu, x1 - x0);  // uniform, and known to be
            constexpr uint32_t kType = FP16 ? 0u : (1u << 7) | (1u << 10);
            constexpr uint32_t kCommon = (1u << 4) | kType | ((uint32_t)(kBlock >> 4) << 24);
            constexpr uint32_t kDescS = kCommon | ((uint32_t)(KT >> 3) << 17);
            constexpr uint32_t kDescO = kCommon | (1u << 16) | ((uint32_t)(DP >> 3) << 17);  // V: d contiguous
            const uint32_t q_addr = smem_u32(q_s);
            At a = locate(plan, C.B, x0);
            int at = 0, round = 0, lists = 0;
            bool fresh = false;              // the tile whose product with V is pending starts its list's O
            int v_at = 0, v_round = 0;
            auto take = [&](int& slot_at, int& slot_round) {
                slot_at = at, slot_round = round;
                if (++at == slots) at = 0, ++round;
            };
            auto pv = [&](int n) {
                mbar_wait(&full[v_at], (uint32_t)(v_round & 1), P.err, kSiteAttend | kSiteFull);
                const uint64_t v_desc = desc128(smem_u32(ring + v_at * Cfg::kTile), KT * 128);
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    mbar_wait(&p_full[2 * k + (n & 1)], (uint32_t)((n >> 1) & 1), P.err, kSiteAttend | kSiteAccum);
                    if (k == 0) fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t block = tmem + k * Cfg::kCols, p_col = block + (n & 1) * KT + Cfg::kColP;
#pragma unroll
                    for (int i = 0; i < KT / 16; ++i)
                        tc_mma_ta(block + Cfg::kColO, p_col + i * 8, v_desc + (i * 16 * 128 >> 4), kDescO,
                                  !fresh || i > 0, leader);
                    tc_commit(&o_done[2 * k + (n & 1)], leader);
                }
                tc_commit(&empty[v_at], leader);
            };
            for (int n = 0; n < count; ++n) {
                const bool first = n == 0 || a.tile == 0;
                if (first && n > 0) pv(n - 1);  // the softmax warps load the next list's queries once they have the last one's O
                int k_at, k_round;
                take(k_at, k_round);
                mbar_wait(&full[k_at], (uint32_t)(k_round & 1), P.err, kSiteAttend | kSiteFull);
                const uint64_t k_desc = desc128(smem_u32(ring + k_at * Cfg::kTile), 16);
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    if (first) mbar_wait(&q_full[k], (uint32_t)(lists & 1), P.err, kSiteAttend | kSiteFull);
                    // the S this tile takes was tile n - 2's (where n - 1's product is out already, that one's phase)
                    if (n > 1 || (first && n > 0)) {
                        const int done = first ? n - 1 : n - 2;
                        mbar_wait(&o_done[2 * k + (done & 1)], (uint32_t)((done >> 1) & 1), P.err, kSiteAttend | kSiteAccum);
                    }
                    if (k == 0 || first) fence_proxy_async_smem();
                    tc_fence_after();
                    const uint64_t q_desc = desc128(q_addr + k * Cfg::kQ, 16);
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i)
                        tc_mma(tmem + k * Cfg::kCols + (n & 1) * KT, q_desc + ((i >> 2) * (kBlock * 128) + (i & 3) * 32 >> 4),
                               k_desc + ((i >> 2) * (KT * 128) + (i & 3) * 32 >> 4), kDescS, i > 0, leader);
                    tc_commit(&s_full[2 * k + (n & 1)], leader);
                }
                tc_commit(&empty[k_at], leader);
                if (first) ++lists;
                if (n > 0 && !first) pv(n - 1);
                take(v_at, v_round);
                fresh = first;
                step(plan, C.B, groups, a);
            }
            pv(count - 1);
        }
        __syncwarp();
    } else {
        // --------------------------------------------- softmax and output
        const float c2 = P.scale * kLog2e;
        const int block = warp >> 2, quarter = warp & 3;
        const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16) + block * Cfg::kCols, t_o = t_s + Cfg::kColO;
        const int r = warp * 32 + lane;  // this thread's row of the blocks
        uint8_t* const my_q = q_s + block * Cfg::kQ;
        At a = locate(plan, C.B, x0);
        int n = 0, segment = 0, v_at = 0, v_round = 0;  // ring position of the value tile of tile n
        auto advance = [&]() {
            if (++v_at == slots) v_at = 0, ++v_round;
        };
        auto wait_o = [&](int tile) {  // O of this block has the tile
            mbar_wait(&o_done[2 * block + (tile & 1)], (uint32_t)((tile >> 1) & 1), P.err, kSiteAttend | kSiteAccum);
        };
        for (int x = x0; x < x1; ++segment) {
            const int b = a.b, h = a.group / row_blocks, rb = a.group % row_blocks;
            const int len = plan.len[b], tot = plan.tot[b];
            const int seg_end = min(x1, x + a.ntile - a.tile);
            const bool whole = a.tile == 0 && seg_end - x == a.ntile;
            const int row = rb * Cfg::kRows + r;
            const int t = row / G, g = row - t * G;
            const bool real = row < R;
            {
                // Queries: whole lines at a time (a row a lane would touch 32 lines with every load); all loads ahead
                // of the stores, which they could not pass.
                const long long off = real ? b * P.qb + t * P.qt + (long long)(h * G + g) * P.qh : -1;
                constexpr int UNITS = DP / 8, AT_ONCE = 32 / UNITS, LOADS = 32 / AT_ONCE;
                const int u = lane % UNITS;
#pragma unroll
                for (int j0 = 0; j0 < LOADS; j0 += 8) {
                    uint4 val[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const long long from = __shfl_sync(0xFFFFFFFFu, off, (j0 + j) * AT_ONCE + lane / UNITS);
                        val[j] = make_uint4(0, 0, 0, 0);
                        if (from >= 0 && u * 8 < D)
                            val[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q) + from + u * 8);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(my_q + (u >> 3) * (kBlock * 128) +
                                                  sw128(quarter * 32 + (j0 + j) * AT_ONCE + lane / UNITS, u & 7)) = val[j];
                }
                mbar_arrive(&q_full[block]);
            }
            const unsigned long long word = real && tot > 0 ? word_of(P.mask, T, b, t) : 0;
            float ref = -INFINITY, sum = 0.0f;
            unsigned long long odd_nodes = 0;  // new nodes whose values were taken out and that this row sees
            const int n_first = n;
            for (; x < seg_end; ++x, ++n, ++a.tile) {
                advance();  // past the key tile
                mbar_wait(&s_full[2 * block + (n & 1)], (uint32_t)((n >> 1) & 1), P.err, kSiteAttend | kSiteAccum);
                __syncwarp();
                tc_fence_after();
                const uint32_t t_tile = t_s + (n & 1) * KT;
                // which of the 64 keys this row sees
                const int i0 = a.tile * KT;
                unsigned long long vis = ~0ull;
                if (i0 + KT > len) {  // the tile meets the new nodes or the list's end
                    const int cut = len - i0;  // keys before it are cached ones; < 64
                    vis = cut > 0 ? (1ull << cut) - 1 : 0;
                    const unsigned long long nodes = T >= 64 ? word : word & ((1ull << T) - 1);
                    if (cut >= 0) vis |= nodes << cut;
                    else if (cut > -64) vis |= nodes >> -cut;
                    mbar_wait(&full[v_at], (uint32_t)(v_round & 1), P.err, kSiteAttend | kSiteFull);
                    const unsigned long long bad = *reinterpret_cast<const unsigned long long*>(odd + v_at * 4) & vis;
                    if (bad) odd_nodes |= cut >= 0 ? bad >> cut : bad << -cut;
                    __syncwarp();
                }
                // the scores are read twice, 32 at a time: registers for all 64 would cost the second CTA
                uint32_t s[32];
                float top = -INFINITY;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    tmem_ld32(t_tile + half * 32, s);
                    tmem_ld_wait();
                    const unsigned in = (unsigned)(vis >> (half * 32));
                    if (__any_sync(0xFFFFFFFFu, in != 0xFFFFFFFFu)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(in >> i & 1)) s[i] = 0xFF800000u;  // -inf
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) top = max3(top, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                }
                float keep = 1.0f;
                if (ref == -INFINITY) {
                    ref = top;  // nothing seen so far, O's row is 0
                } else if ((top - ref) * c2 > (float)Wt::kLazy) {
                    keep = ex2((ref - top) * c2);
                    ref = top;
                    sum *= keep;
                }
                if (__any_sync(0xFFFFFFFFu, keep != 1.0f) && n > n_first) {
                    wait_o(n - 1);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DP; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(t_o + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                        tmem_st16(t_o + c, o);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                const float shift = ref == -INFINITY ? 0.0f : ref;
                const uint64_t shift2 = both(-shift, -shift), scale2 = both(c2, c2), up2 = both(Wt::kUp, Wt::kUp);
                uint64_t sum2 = 0;
#pragma unroll
                for (int half = 1; half >= 0; --half) {  // the second half is still in registers
                    if (half == 0) {
                        tmem_ld32(t_tile, s);
                        tmem_ld_wait();
                        const unsigned in = (unsigned)vis;
                        if (__any_sync(0xFFFFFFFFu, in != 0xFFFFFFFFu)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(in >> i & 1)) s[i] = 0xFF800000u;
                        }
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float p0, p1;
                        split(fma2(add2(both(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), shift2), scale2, up2),
                              p0, p1);
                        p0 = ex2(p0), p1 = ex2(p1);
                        sum2 = add2(sum2, both(p0, p1));
                        w[i] = pack<FP16>(p0, p1);  // rounded once, see above
                    }
                    tmem_st16(t_tile + Cfg::kColP + half * 16, w);
                }
                tmem_st_wait();
                tc_fence_before();
                {
                    float s0, s1;
                    split(sum2, s0, s1);
                    sum += s0 + s1;
                }
                mbar_arrive(&p_full[2 * block + (n & 1)]);
                advance();  // past the value tile
            }
            if (a.tile == a.ntile) {
                a.tile = a.ntile - 1;
                step(plan, C.B, groups, a);
            }
            // the list's O, or this CTA's part of it
            wait_o(n - 1);
            __syncwarp();
            tc_fence_after();
            const bool empty_row = word == 0 || sum == 0.0f;
            const float inv = !whole ? 1.0f : empty_row ? 0.0f : 1.0f / sum;
            const long long at = ((long long)b * T + t) * P.Hq + h * G + g;
            float* part = P.part + ((long long)blockIdx.x * 2 + (segment ? 1 : 0)) * part_floats(Cfg::kRows, DP);
            const int32_t* list = C.table ? C.table + b * C.tb + h * C.th : nullptr;
            uint8_t* const stage = my_q + quarter * 4096;  // Q has been read; a warp's rows of its first half are its own 4 KB
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                tmem_ld32(t_o + c, o);
                tmem_ld_wait();
                for (unsigned long long left = odd_nodes; left; left &= left - 1) {
                    const int node = __ffsll((long long)left) - 1;
                    const long long slot = list ? list[len + node] : len + node;
                    if (E4M3) {
                        const uint8_t* src = static_cast<const uint8_t*>(C.v) + b * C.vb + h * C.vh + slot * C.vs;
                        const bool row = C.v_scale[b * C.vcb + h * C.vch + (slot >> C.block_shift)] == kScaleNaN;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < D && (row || code_nan(src[c + i]))) o[i] = __float_as_uint(NAN);
                    } else {
                        const uint16_t* src = static_cast<const uint16_t*>(C.v) + b * C.vb + h * C.vh + slot * C.vs;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < D && not_finite<FP16>(src[c + i]))
                                o[i] = __float_as_uint(__uint_as_float(o[i]) + widen<FP16>(src[c + i]));
                    }
                }
                // 32 columns of the warp's 32 rows through shared memory, so that a store covers whole lines
                __syncwarp();
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = empty_row ? 0u
                                             : pack<FP16>(__uint_as_float(o[i + 2 * e]) * inv,
                                                          __uint_as_float(o[i + 2 * e + 1]) * inv);
                        *reinterpret_cast<uint4*>(stage + sw128(lane, i / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                    const int u = lane & 3;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int rr = j * 8 + (lane >> 2);
                        const long long to = __shfl_sync(0xFFFFFFFFu, real ? at : -1ll, rr);
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + sw128(rr, u));
                        if (to >= 0 && c + u * 8 < D)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + to * D + c + u * 8) = v;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(stage + sw128(lane, i / 4)) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    __syncwarp();
                    const int u = lane & 7;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int rr = j * 4 + (lane >> 3);
                        if (rb * Cfg::kRows + warp * 32 + rr < R)
                            *reinterpret_cast<uint4*>(part + (warp * 32 + rr) * DP + c + u * 4) =
                                *reinterpret_cast<const uint4*>(stage + sw128(rr, u));
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (real) {
                if (!whole) {
                    part[Cfg::kRows * DP + r] = ref;
                    part[Cfg::kRows * DP + Cfg::kRows + r] = sum;
                } else if (P.lse) {
                    P.lse[at] = empty_row ? -INFINITY : lse_of(ref, P.scale, sum * Wt::kDown);
                }
            }
        }
    }
    __syncthreads();
    if (warp == Cfg::kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Cfg::kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------ host

namespace {

template <int DP, int NB, bool FP16, bool E4M3>
cudaError_t launch_wide(const AttendParams& P, int row_blocks, int parts, cudaStream_t st) {
    using Cfg = WideCfg<DP, NB, E4M3>;
    const auto kern = k_tree_attention_wide<DP, NB, FP16, E4M3>;
    const cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    int slots = Cfg::kMaxSlots;
    while (slots > 3 && Cfg::smem(P.c.B, slots) > Cfg::kSmemLimit) --slots;
    void* args[3] = {const_cast<AttendParams*>(&P), &row_blocks, &slots};
    return launch(reinterpret_cast<const void*>(kern), dim3(parts, 1, 1), Cfg::kThreads, Cfg::smem(P.c.B, slots), args, st);
}

template <int DP, bool FP16, bool E4M3>
cudaError_t launch_rows(const AttendParams& P, int rows, int row_blocks, int parts, cudaStream_t st) {
    return rows == kBlock ? launch_wide<DP, 1, FP16, E4M3>(P, row_blocks, parts, st)
                          : launch_wide<DP, 2, FP16, E4M3>(P, row_blocks, parts, st);
}

template <bool FP16, bool E4M3>
cudaError_t launch_heads(const AttendParams& P, int rows, int row_blocks, int parts, cudaStream_t st) {
    return P.c.D <= 64 ? launch_rows<64, FP16, E4M3>(P, rows, row_blocks, parts, st)
                       : launch_rows<128, FP16, E4M3>(P, rows, row_blocks, parts, st);
}

}  // namespace

cudaError_t launch_tree_attention_wide(const AttendParams& P, int* row_blocks, int* parts, cudaStream_t st) {
    const int rows = wide_rows(P.T * P.G);
    *row_blocks = (P.T * P.G + rows - 1) / rows;
    *parts = sm_count() * (rows == kBlock ? 2 : 1);
    if (*parts < 1) return cudaErrorInvalidDevice;
    if (P.c.e4m3)
        return P.c.fp16 ? launch_heads<true, true>(P, rows, *row_blocks, *parts, st)
                        : launch_heads<false, true>(P, rows, *row_blocks, *parts, st);
    return P.c.fp16 ? launch_heads<true, false>(P, rows, *row_blocks, *parts, st)
                    : launch_heads<false, false>(P, rows, *row_blocks, *parts, st);
}

}  // namespace si
