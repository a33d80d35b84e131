// attend8.cu -- tree attention over a cache of e4m3 codes: the kernel for few
// rows a key. Lists are cut into tiles and dealt to CTAs as for the cache in 16
// bits (attend.cu). Where several CTAs have parts of a list, the last of them to
// be done joins the parts, in their order: the result does not depend on which
// one that is. The counters that say which one it is lie in the handle's scratch.
// The launches take kCounterSets sets of them in turn and clear the next one's: what
// a launch leaves in its own (two that ran at the same time, against the rules, or a
// length that changed under one) does not outlive the call after it.
//
// A warp takes 32 keys of a tile (sixteen of heads above 128 elements) and keeps
// its own softmax state. The products have the keys on the long side, so that up to eight query rows
// (one token's heads, mostly) fill the short one:
//   S^T (16 keys x 8 rows)  = K (16 x D) Q^T        mma m16n8k16
//   O^T (D x 8 rows)      += V^T (D x 16 keys) P^T
// Codes become fp16 in registers, two an instruction and exactly, on their way
// from shared memory to the product; the scales stay out of it. A key's scale
// multiplies its scores; a value's goes into the weight's exponent. What comes
// out goes into the product as two fp16 terms, so it is taken relative to a power
// of two of its row's own: the largest weight times scale that the row has met,
// which the output is rescaled by when it grows, as it is by the softmax's maximum.
// (A unit for all rows, from the scales alone, lost the keys that a row weighs beside
// a large scale that it does not. The rows' own cost 5 % at sixteen rows a key, 34.5 /
// 36.5 us for sixteen sequences of up to 4097, and 1 % up to eight.) Warps and parts
// are joined likewise: a part whose weights are below fp32's range beside another's
// may have scales that make up for it.
// Queries go in as fp16: bf16 rows times the power of two that brings their largest
// element below 2^15, so that what lies up to 2^29 below it is exact.
//
// Bound by memory where lists are long: one token of 32 heads over 131071 keys
// of 8 heads of 128 takes 52.5 us, 5.2 TB/s, 0.78 of what a plain copy reaches;
// the tiles themselves go by at 6.5 TB/s, 4 us pass before the first one is
// there and 5 at the end (slowest CTA, parts out, join). 1000 keys, heads of
// 64: 9.3 us, latency alone (lengths, slots, keys, parts out, parts in). With
// sixteen keys a warp and four CTAs an SM the long list took 75 us, most of it
// because the join was a launch of its own, whose blocks left the register file
// in pieces: the next call's last CTA did not fit beside the others and ran
// after them. Sixteen sequences of up to 4097 keys, mixed order: 26 us; the parts
// are whole tiles of 128 keys, nine or ten where an even share is seven and a half
// (shares that run across the lists' ends: 28 us; a list's end costs some 3).
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps

// fp16 weights, and a maximum that may be outgrown by 2^kLazy before anything is rescaled.
using Wt = Weights<true, true>;

// Two sixteens of keys a warp / one, the rest alike: 131071 keys, heads of 128, 51.8 / 66.9 us, sixteen sequences of up to
// 4097 25.8 / 30.9; heads of 256, 4 cache heads 63.2 / 70.2, sixteen sequences 55.1 / 39.9 (two leave one CTA an SM).
template <int DP, int NT>
struct Cfg8 {
    static constexpr int kRows = 8 * NT;                      // query rows of a block
    static constexpr int kMT = DP <= 128 ? 2 : 1;             // sixteens of keys a warp has of a tile
    static constexpr int kWarpKeys = 16 * kMT;
    static constexpr int kKeys = 4 * kWarpKeys;               // of a tile
    static constexpr int kTile = kKeys * DP;                  // bytes of a K or V tile
    static constexpr int kOffScale = 2 * kTile;               // in a stage: k's scale and the exponent of v's, of its keys
    static constexpr int kStage = 2 * kTile + kKeys * 8;
    static constexpr int kStages = DP == 64 ? 4 : 3;
    static constexpr int kCtas = DP == 64 ? 3 : 2;            // an SM
    static constexpr int kQRow = DP * 2 + 32;                 // bytes: eight rows' 32-byte pieces lie in different banks
    static constexpr int kJoinRow = DP + 4;                   // floats: likewise
    static constexpr bool kQInRegs = DP * NT <= 256;
    static constexpr int kOffQ = kStages * kStage;            // queries; the join of the warps takes their place
    static constexpr int kJoin = (NT == 1 ? 12 : 8) * kJoinRow * 4;  // three warps' rows of up to four, or one's of eight
    static constexpr int kUnion = kJoin > kRows * kQRow ? kJoin : kRows * kQRow;
    static constexpr int kOffFactor = kOffQ + kUnion;         // what a query row was divided by
    static constexpr int kOffState = kOffFactor + kRows * 4;  // [warp][row] {maximum, sum, base}
    static constexpr int kOffLast = kOffState + 4 * kRows * 16;  // [2] lists that this CTA joins
    static constexpr int kOffCounters = kOffLast + 2 * 24;
    static constexpr int kOffPlan = kOffLast + 2 * 32;
    static constexpr int smem(int B) { return kOffPlan + Plan::words(B) * 4; }
};

constexpr unsigned kCounterSets = 4;  // a power of two: the launches are counted modulo 2^32

// A list whose parts this CTA joins.
struct LastOf {
    int on, b, group, first, last, behind;
};
static_assert(sizeof(LastOf) == 24);

// The transposed 8 x 8 matrix of 16-bit elements that the warp's registers hold.
__device__ __forceinline__ uint32_t transposed(uint32_t w) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// over the eight lanes with the same lane % 4
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 16);
}

__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Where the parts of lists lie: for each of a CTA's two pieces [CTA][row][DP] outputs, then [CTA][row] {maximum, sum}, then
// [CTA][row] bases (all three in 16 bytes: 2 us more where lists have sixty parts), with as many rows as a block can have in this call. A list's parts are neighbours, but for the first one where
// another list comes before it in its CTA.
template <int DP, int RB>
struct Parts {
    float* const at;
    const int rows, ctas;
    __device__ __forceinline__ Parts(const AttendParams& P) : at(P.part), rows(min(RB, P.T * P.G)), ctas(gridDim.x) {}
    __device__ __forceinline__ float* out(int cta, int piece) const { return at + (long long)(piece * ctas + cta) * rows * DP; }
    __device__ __forceinline__ float2* state(int cta, int piece) const {
        return reinterpret_cast<float2*>(at + 2ll * ctas * rows * DP) + (piece * ctas + cta) * rows;
    }
    __device__ __forceinline__ float* base(int cta, int piece) const {
        return at + 2ll * ctas * rows * (DP + 2) + (piece * ctas + cta) * rows;
    }
};

// Joins a list's parts: the CTA's ring is empty and takes them, as many at once as fit.
template <int DP, int RB, int BYTES>
__device__ void join_parts(const AttendParams& P, const Plan& plan, int row_blocks, const LastOf l, uint8_t* smem) {
    constexpr int CHUNK = 64, QUADS = DP / 4, ITEMS = RB * QUADS / kThreads > 0 ? RB * QUADS / kThreads : 1;
    constexpr int kOffRows = (CHUNK + 4) * RB * 4;
    float* const weight_s = reinterpret_cast<float*>(smem);                    // [part of a chunk][row]
    float4* const state_s = reinterpret_cast<float4*>(weight_s + CHUNK * RB);  // [row] maximum, sum, base, what the rows so far are multiplied by
    float4* const rows_s = reinterpret_cast<float4*>(smem + kOffRows);         // [part of a chunk][row][DP]
    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = P.G, R = P.T * G, D = C.D;
    const int h = l.group / row_blocks, row0 = l.group % row_blocks * RB, rows = min(RB, R - row0);
    const int chunk = min(CHUNK, (BYTES - kOffRows) / (rows * DP * 4)), quads = rows * QUADS;
    const float c2 = P.scale * kLog2e;
    const Parts<DP, RB> parts(P);
    auto piece_of = [&](int c) { return c == l.first && l.behind ? 1 : 0; };
    __syncthreads();
    if (tid < RB) state_s[tid] = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
    float4 acc[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c0 = l.first; c0 <= l.last; c0 += chunk) {
        const int n = min(chunk, l.last - c0 + 1);
        __syncthreads();
        float2 st[2];
        float bs[2];
        auto load_state = [&](int r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                st[i] = make_float2(-INFINITY, 0.0f), bs[i] = 0.0f;
                const int c = c0 + lane + 32 * i;
                if (r < rows && lane + 32 * i < n) {
                    st[i] = __ldcg(parts.state(c, piece_of(c)) + r);
                    bs[i] = __ldcg(parts.base(c, piece_of(c)) + r);
                }
            }
        };
        load_state(warp);  // ahead of the copies, which it would queue behind
        // a thread copies what it will read: the quads tid, tid + kThreads, ... of every part
        const uint32_t to = smem_u32(rows_s);
        for (int q = tid; q < quads; q += kThreads) {
            const float4* from = reinterpret_cast<const float4*>(parts.out(c0, 0)) + q;
            const float4* from0 = reinterpret_cast<const float4*>(parts.out(c0, piece_of(c0))) + q;
#pragma unroll 8
            for (int c = 0; c < n; ++c) cp16(to + (c * quads + q) * 16, c ? from + (long long)c * (parts.rows * QUADS) : from0);
        }
        cp_commit();
        for (int r = warp; r < rows; r += 4) {
            if (r != warp) load_state(r);
            const float4 old = state_s[r];
            const float top = fmaxf(warp_max(fmaxf(st[0].x, st[1].x)), old.x), shift = shift_of(top);
            // The rows are brought to the largest base, beside the maximum: what a part's weights lose the scales may make up for.
            const float d[2] = {(st[0].x - shift) * c2, (st[1].x - shift) * c2}, d_old = (old.x - shift) * c2;
            const float base = shift_of(fmaxf(warp_max(fmaxf(d[0] + bs[0], d[1] + bs[1])), d_old + old.z));
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (lane + 32 * i < n) weight_s[(lane + 32 * i) * RB + r] = ex2(d[i] + (bs[i] - base));
                sum += ex2(d[i]) * st[i].y;
            }
            sum = warp_sum(sum);
            __syncwarp();
            if (lane == 0) state_s[r] = make_float4(top, old.y * ex2(d_old) + sum, base, ex2(d_old + (old.z - base)));
        }
        cp_wait<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int item = tid + i * kThreads, r = item / QUADS;
            if (item >= quads) continue;
            const float keep = state_s[r].w;
            acc[i].x *= keep, acc[i].y *= keep, acc[i].z *= keep, acc[i].w *= keep;
#pragma unroll 4
            for (int c = 0; c < n; ++c) {
                const float4 v = rows_s[c * quads + item];
                const float w = weight_s[c * RB + r];
                acc[i].x += w * v.x, acc[i].y += w * v.y, acc[i].z += w * v.z, acc[i].w += w * v.w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = tid + i * kThreads, r = item / QUADS, q = item % QUADS;
        if (item >= quads || q * 4 >= D) continue;
        const float4 st = state_s[r];
        const int t = div_of(row0 + r, G), g = row0 + r - t * G;
        const bool empty = plan.tot[l.b] == 0 || word_of(P.mask, P.T, l.b, t) == 0 || st.y == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / st.y, power = ex2(st.z) * Wt::kDown;
        const long long at = ((long long)l.b * P.T + t) * P.Hq + h * G + g;
        uint2 w = make_uint2(0, 0);
        const float4 a = make_float4(acc[i].x * inv * power, acc[i].y * inv * power, acc[i].z * inv * power, acc[i].w * inv * power);
        if (!empty) w = C.fp16 ? make_uint2(pack<true>(a.x, a.y), pack<true>(a.z, a.w)) : make_uint2(pack<false>(a.x, a.y), pack<false>(a.z, a.w));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + at * D + q * 4) = w;
        if (P.lse && q == 0) P.lse[at] = empty ? -INFINITY : lse_of(st.x, P.scale, st.y);
    }
}

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, Cfg8<DP, NT>::kCtas)
    k_tree_attention8(const __grid_constant__ AttendParams P, int row_blocks) {
    using Cfg = Cfg8<DP, NT>;
    using Cp = Copy8<DP, Cfg::kWarpKeys>;
    constexpr int RB = Cfg::kRows, KD = DP / 16, UNITS = Cp::UNITS, S = Cfg::kStages, MT = Cfg::kMT;
    constexpr int WK = Cfg::kWarpKeys, KEYS = Cfg::kKeys;

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + Cfg::kOffQ;
    float* const factor_s = reinterpret_cast<float*>(smem + Cfg::kOffFactor);
    float4* const state_s = reinterpret_cast<float4*>(smem + Cfg::kOffState);
    LastOf* const last_s = reinterpret_cast<LastOf*>(smem + Cfg::kOffLast);
    unsigned* const counters_s = reinterpret_cast<unsigned*>(smem + Cfg::kOffCounters);  // place of this launch's set
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;   // keys g, g + 8 of sixteen; rows 2c, 2c + 1 of each eight
    const int T = P.T, G = P.G, R = T * G, D = C.D;
    const int groups = C.Hkv * row_blocks;

    if (tid < 2) last_s[tid].on = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    if (tid == 32) {  // while the plan's lengths are on their way: how many launches this CTA has been in
        const unsigned n = __ldcg(P.done + blockIdx.x);
        atomicAdd(P.done + blockIdx.x, 1u);
        *counters_s = (1 + n % kCounterSets) * gridDim.x;
        P.done[(1 + (n + 1) % kCounterSets) * gridDim.x + blockIdx.x] = 0;
    }
    make_plan<kThreads, kNarrowLeast, kNarrowPiece, KEYS>(C, T, groups, gridDim.x, plan, P.err, blockIdx.x == 0);
    const DealOf<KEYS> deal(plan, C.B, gridDim.x, kNarrowLeast);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);
    if (x0 >= x1) return;

    const float c2 = P.scale * kLog2e;
    const int unit = lane % UNITS;
    const bool unit_on = unit * 16 < D, whole_rows = D == DP;
    const int own0 = warp * WK;  // this warp's keys of a tile
    const Cp cp(lane, own0);
    const Load8<DP> ld(lane, own0);
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks, v_step = (int)C.vs;

    // producer state: lane i holds the slot of key own0 + i (of sixteen: i % 16) of the tile to be issued next
    SourceOf<uint8_t, KEYS> src;
    At a = locate<KEYS>(plan, C.B, x0);
    src.at = a, src.x = x0, src.x1 = x1;
    const uint32_t ring = smem_u32(smem);
    int stage_in = 0, held = kNoSlot, seen_b = -1;
    // stages that wait for their scales, and this lane's key's: the older one first
    int pend[2] = {-1, -1}, pend_k[2] = {0, 0}, pend_v[2] = {0, 0};
    auto fetch = [&]() {
        const int i0 = src.at.tile * KEYS;
        if (i0 + KEYS > src.len && seen_b != src.at.b) {  // the tile meets the new nodes
            src.seen = seen_nodes(P.mask, T, src.at.b, lane);
            seen_b = src.at.b;
        }
        held = slot_of(src.list, i0 + own0 + lane % WK, src.len, src.tot, src.seen);
    };
    auto issue = [&]() {
        // The scales of the tile before last have had the time to arrive. A key that is not there (byte -1) is
        // below all.
        if (pend[0] >= 0) {
            float2* to = reinterpret_cast<float2*>(smem + pend[0] * Cfg::kStage + Cfg::kOffScale);
            if (WK == 32 || lane < WK)
                to[own0 + lane] = pend_k[0] < 0 ? make_float2(0.0f, -127.0f)
                                                : make_float2(scale_of(pend_k[0], C.e_lo, C.e_hi), exponent_of(pend_v[0], C.e_lo, C.e_hi));
        }
        pend[0] = pend[1], pend_k[0] = pend_k[1], pend_v[0] = pend_v[1], pend[1] = -1;
        if (src.x < x1) {
            int slot[Cp::SWEEPS];
            const uint8_t *kp = src.k + unit * 16, *vp = src.v + unit * 16;
            const bool ok = slot_ok(held, n_slots, P.err);
            const bool cached = src.at.tile * KEYS + KEYS <= src.len;
            // cached keys: nothing to leave out (a slot outside the pool has been reported; slot 0 is read)
            const int mine = ok ? held : cached ? 0 : -1;
            Cp::slots(mine, lane, slot);
            const uint32_t dst = ring + stage_in * Cfg::kStage;
            if (whole_rows && cached) {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const uint32_t at = dst + cp.place(j);
                    cp16(at, kp + (long long)slot[j] * k_step);
                    cp16(at + Cfg::kTile, vp + (long long)slot[j] * v_step);
                }
            } else {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const bool on = slot[j] >= 0 && unit_on;
                    const long long from = on ? slot[j] : 0;
                    const uint32_t at = dst + cp.place(j);
                    cp16(at, on ? kp + from * k_step : src.k, on);
                    cp16(at + Cfg::kTile, on ? vp + from * v_step : src.v, on);
                }
            }
            pend_k[1] = -1;
            if (mine >= 0) pend_k[1] = src.k_scale[mine >> C.block_shift], pend_v[1] = src.v_scale[mine >> C.block_shift];
            pend[1] = stage_in;
            if (++stage_in == S) stage_in = 0;
            if (src.next(plan, C.B, groups) && src.x < x1) src.enter(C, plan, row_blocks);
            if (src.x < x1) fetch();
        }
        cp_commit();
    };
    // Query rows of a list's block into shared memory (rows past R are zero), in two steps.
    constexpr int Q_AT_ONCE = 32 / (DP / 8);                             // rows a warp takes at once
    constexpr int Q_SWEEPS = (RB + 4 * Q_AT_ONCE - 1) / (4 * Q_AT_ONCE);
    uint4 queries[Q_SWEEPS];
    auto load_queries = [&](const At& at) {
        const int b = at.b, h = at.group / row_blocks, rb = at.group % row_blocks;
#pragma unroll
        for (int i = 0; i < Q_SWEEPS; ++i) {
            const int r = (i * 4 + warp) * Q_AT_ONCE + lane / (DP / 8), row = rb * RB + r, t = div_of(row, G);
            const bool on = r < RB && row < R;
            const uint16_t* from = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)(h * G + row - t * G) * P.qh;
            queries[i] = query_load<DP>(on ? from : nullptr, D, lane);
        }
    };
    auto store_queries = [&]() {
#pragma unroll
        for (int i = 0; i < Q_SWEEPS; ++i) {
            const int r = (i * 4 + warp) * Q_AT_ONCE + lane / (DP / 8);
            float down;
            const uint4 val = query_half<DP>(queries[i], C.fp16, down);
            if (r < RB) {
                *reinterpret_cast<uint4*>(q_s + r * Cfg::kQRow + lane % (DP / 8) * 16) = val;
                if (lane % (DP / 8) == 0) factor_s[r] = down;
            }
        }
    };
    // The first slots, the second tile's with the first's where they are of one list, and the first queries go out
    // together: each is a trip to memory of its own.
    src.enter(C, plan, row_blocks);
    fetch();
    const int first_slot = held;
    const bool two = x0 + 1 < x1 && a.tile + 1 < a.ntile;
    if (two) {
        ++src.at.tile;
        fetch();
        --src.at.tile;
    }
    const int second_slot = held;
    held = first_slot;
    load_queries(a);
    issue();
    if (two) held = second_slot;
#pragma unroll 1
    for (int s = 1; s < S - 1; ++s) issue();
    store_queries();

    int segment = 0, stage_out = 0;
    for (int x = x0; x < x1; ++segment) {
        // one list, or the part of it that this CTA has
        const int b = a.b, h = a.group / row_blocks, rb = a.group % row_blocks;
        const int len = plan.len[b], tot = plan.tot[b];
        const int seg_end = min(x1, x + a.ntile - a.tile);
        const bool whole = a.tile == 0 && seg_end - x == a.ntile;

        if (segment > 0) {
            __syncthreads();  // the previous list's joins and reads of q_s are over
            store_queries();
        }
        unsigned long long word[NT][2];
        float ref[NT][2], sum[NT][2], qdown[NT][2];
        float o[KD][NT][4];
        // o is over 2^base of its row too: log2 of the largest weight (over ref's) times its value's scale, kLazy below it at most.
        float base[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = rb * RB + n * 8 + 2 * c + e;
                word[n][e] = row < R && tot > 0 ? word_of(P.mask, T, b, div_of(row, G)) : 0;
                ref[n][e] = -INFINITY, base[n][e] = sum[n][e] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < KD; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
        __syncthreads();
        // Of sixteen elements the product's places 2c, 2c + 1, 2c + 8, 2c + 9 are elements 4c .. 4c + 3, on both sides.
        auto query = [&](int n, int u) { return *reinterpret_cast<const uint2*>(q_s + (n * 8 + g) * Cfg::kQRow + u * 32 + c * 8); };
        uint2 qf[Cfg::kQInRegs ? NT : 1][Cfg::kQInRegs ? KD : 1];
        if (Cfg::kQInRegs) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < KD; ++u) qf[Cfg::kQInRegs ? n : 0][Cfg::kQInRegs ? u : 0] = query(n, u);
        }
        bool steep = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float down = factor_s[n * 8 + 2 * c + e];
                steep |= down > kSteep;
                qdown[n][e] = fminf(down, kSteep);
            }
        steep = __any_sync(0xFFFFFFFFu, steep);

        for (; x < seg_end; ++x, ++a.tile) {
            cp_wait<S - 2>();
            uint8_t* const stage = smem + stage_out * Cfg::kStage;
            if (++stage_out == S) stage_out = 0;
            const int i0 = a.tile * KEYS + own0;
            const bool edge = i0 + WK > len;  // these keys meet the new nodes or the list's end
            unsigned odd = 0;                 // keys with codes of NaN
            if (edge) {
                // A node's value row may hold NaN that only its descendants may see, and 0 * NaN is NaN: such codes
                // leave the product here (each lane looks at what it copied itself) and come back below for the rows
                // that see them.
#pragma unroll 1
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const int key = Cp::row(lane, j), node = i0 + key - len;
                    if (node < 0 || node >= T) continue;
                    uint8_t* e = stage + Cfg::kTile + tile8_at<DP>(own0 + key, unit);
                    for (int i = 0; i < 16; ++i)
                        if (code_nan(e[i])) e[i] = 0, odd |= 1u << key;
                }
                odd = __reduce_or_sync(0xFFFFFFFFu, odd);
            }
            __syncwarp();  // the tile before has been read by every lane
            issue();
            __syncwarp();
            const uint32_t k_s = smem_u32(stage), v_s = k_s + Cfg::kTile;
            const float2* sc_s = reinterpret_cast<const float2*>(stage + Cfg::kOffScale) + own0;
            constexpr int CHAINS = MT * NT <= 2 ? 2 : 1;  // of products, for each sixteen keys and eight rows
            float s[MT][NT][4], s_odd[CHAINS == 2 ? MT : 1][CHAINS == 2 ? NT : 1][4] = {};
            float2 sc[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                sc[m][0] = sc_s[m * 16 + g], sc[m][1] = sc_s[m * 16 + g + 8];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.0f;
            }
#pragma unroll
            for (int u = 0; u < KD; u += 2) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t r[4];
                    ldsm4(r, k_s + ld.place(u, m));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t a0, a1, a2, a3;
                        halves4(r[2 * i], a0, a2);
                        halves4(r[2 * i + 1], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 q = Cfg::kQInRegs ? qf[Cfg::kQInRegs ? n : 0][Cfg::kQInRegs ? u + i : 0] : query(n, u + i);
                            mma16(CHAINS == 2 && i == 1 ? s_odd[CHAINS == 2 ? m : 0][CHAINS == 2 ? n : 0] : s[m][n], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
                }
            }
            // s[m][n][0..1]: key g with rows 2c, 2c + 1; s[m][n][2..3]: key g + 8
            float high = -127.0f;  // the largest exponent of values
#pragma unroll
            for (int m = 0; m < MT; ++m) high = fmaxf(high, fmaxf(sc[m][0].y, sc[m][1].y));  // NaN is passed over
            bool grows = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (CHAINS == 2) s[m][n][e] += s_odd[CHAINS == 2 ? m : 0][CHAINS == 2 ? n : 0][e];
                        s[m][n][e] = s[m][n][e] * qdown[n][e & 1] * sc[m][e >> 1].x;
                    }
                if (steep) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float rest = rest_of(factor_s[n * 8 + 2 * c + (e & 1)]);
#pragma unroll
                        for (int m = 0; m < MT; ++m) s[m][n][e] *= rest;
                    }
                }
                if (edge) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = i0 + m * 16 + g + (e & 2) * 4 - len;
                            const bool sees = j < 0 || (j < T && (word[n][e & 1] >> (j & 63) & 1));
                            if (!sees) s[m][n][e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
                    for (int m = 1; m < MT; ++m) top = fmaxf(top, fmaxf(s[m][n][e], s[m][n][e + 2]));
                    // The difference is taken before the scale: scores of the type's lowest value differ by 0 from
                    // their maximum, where a fused s * c2 - ref * c2 would be off by the product's rounding.
                    // A weight times its scale is at most the largest of both.
                    grows |= (top - ref[n][e]) * c2 + fmaxf(high - base[n][e], 0.0f) > (float)Wt::kLazy;
                }
            }
            if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float keep[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float old = ref[n][e];
                        float top = old, most = -INFINITY;
#pragma unroll
                        for (int m = 0; m < MT; ++m) top = fmaxf(top, fmaxf(s[m][n][e], s[m][n][e + 2]));
                        ref[n][e] = top = column_max(top);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = e; i < 4; i += 2)  // a scale of NaN is passed over: it makes the row NaN by itself
                                most = fmaxf(most, fmaf(s[m][n][i] - shift_of(top), c2, sc[m][i >> 1].y));
                        const float fall = top == old ? 0.0f : (old - top) * c2;  // of what there is, in powers of two
                        const float next = fmaxf(fmaxf(column_max(most), base[n][e] + fall), -126.0f);
                        sum[n][e] *= ex2(fall);
                        keep[e] = ex2(fall + (base[n][e] - next));
                        base[n][e] = next;
                    }
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
                        o[i][n][0] *= keep[0], o[i][n][2] *= keep[0];
                        o[i][n][1] *= keep[1], o[i][n][3] *= keep[1];
                    }
                }
            }
            uint32_t ph[MT][NT][2], pl[MT][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float shift[2] = {shift_of(ref[n][0]), shift_of(ref[n][1])};
                const float below[2] = {base[n][0] - Wt::kUp, base[n][1] - Wt::kUp};
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = ex2(fmaf(s[m][n][e] - shift[e & 1], c2, Wt::kUp));
                        sum[n][e & 1] += p;
                        w[e] = ex2(fmaf(s[m][n][e] - shift[e & 1], c2, sc[m][e >> 1].y - below[e & 1]));
                    }
                    if (edge) {  // whatever scale a key has that the row does not see
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (s[m][n][e] == -INFINITY) w[e] = 0.0f;
                    }
                    // The product takes fp16: a weight goes in as two terms, the second what the first one's rounding left.
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t hi = pack<true>(w[2 * i], w[2 * i + 1]);
                        const uint32_t lo = pack<true>(w[2 * i] - widen<true>((uint16_t)hi), w[2 * i + 1] - widen<true>((uint16_t)(hi >> 16)));
                        ph[m][n][i] = transposed(hi), pl[m][n][i] = transposed(lo);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < KD; u += 2) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t r[4];
                    ldsm4t(r, v_s + ld.place(u, m));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // a register holds two keys' codes of elements 2g, 2g + 1: rows g and g + 8 of the product
                        uint32_t a0, a1, a2, a3;
                        halves4(__byte_perm(r[2 * i], 0, 0x3120), a0, a1);
                        halves4(__byte_perm(r[2 * i + 1], 0, 0x3120), a2, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16(o[u + i][n], a0, a1, a2, a3, ph[m][n][0], ph[m][n][1]);
                            mma16(o[u + i][n], a0, a1, a2, a3, pl[m][n][0], pl[m][n][1]);
                        }
                    }
                }
            }
            if (odd) {
                // the codes taken out above: NaN, so their weight does not matter
                const int32_t* list = C.table ? C.table + b * C.tb + h * C.th : nullptr;
                for (unsigned left = odd; left; left &= left - 1) {
                    const int key = __ffs(left) - 1, node = i0 + key - len;
                    const long long slot = list ? list[len + node] : len + node;
                    if (slot < 0 || slot >= C.n_slots) continue;
                    const uint8_t* row = static_cast<const uint8_t*>(C.v) + b * C.vb + h * C.vh + slot * C.vs;
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = i * 16 + 2 * g + (e >> 1);
                            if (d >= D || !code_nan(row[d])) continue;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (word[n][e & 1] >> node & 1) o[i][n][e] = NAN;
                        }
                    }
                }
            }
        }
        if (a.tile == a.ntile) {
            a.tile = a.ntile - 1;
            step<KEYS>(plan, C.B, groups, a);
        }
        if (x < x1) load_queries(a);  // of the next list: they come while this one is finished

        // Join the warps: maxima, sums and bases, then output rows in warp order, through the place of this list's queries,
        // which are no longer needed: in the ring the next list's copies are in flight.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[n][e] = column_sum(sum[n][e]);
                if (g == 0) state_s[warp * RB + n * 8 + 2 * c + e] = make_float4(ref[n][e], sum[n][e], base[n][e], 0.0f);
            }
        __syncthreads();
        if (tid < RB) {  // a thread a row: what the row has, and what each warp's output is multiplied by
            float4 it[4];
            float top = -INFINITY, all = 0.0f, most = -INFINITY, d[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                it[w] = state_s[w * RB + tid];
                top = fmaxf(top, it[w].x);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                d[w] = (it[w].x - shift_of(top)) * c2;
                all += it[w].y * ex2(d[w]);
                most = fmaxf(most, d[w] + it[w].z);
            }
            most = shift_of(most);
#pragma unroll
            for (int w = 0; w < 4; ++w) state_s[w * RB + tid].w = ex2(d[w] + (it[w].z - most));
            *reinterpret_cast<float2*>(state_s + tid) = make_float2(top, all * Wt::kDown);
            state_s[tid].z = most;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = state_s[warp * RB + n * 8 + 2 * c + e].w;
#pragma unroll
                for (int i = 0; i < KD; ++i) o[i][n][e] *= f, o[i][n][e + 2] *= f;
            }
        // (All at once where the rows are few, or the ring is idle: after the CTA's last tile.)
        float* const join_s = reinterpret_cast<float*>(x < x1 ? q_s : smem);
        const int at_once = x == x1 || (NT == 1 && R <= 4) ? 3 : 1;
        const int area = (NT == 1 && R <= 4 ? 4 : 8) * Cfg::kJoinRow;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll 1
            for (int w = 1; w < 4; w += at_once) {
                if (n + w > 1) __syncthreads();
                float* const place = join_s + 2 * c * Cfg::kJoinRow + 2 * g;
                const bool rows_on = NT > 1 || 2 * c < R;  // rows past R are left out
                if (warp >= w && warp < w + at_once && rows_on) {
#pragma unroll
                    for (int i = 0; i < KD; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float2*>(place + (warp - w) * area + e * Cfg::kJoinRow + i * 16) =
                                make_float2(o[i][n][e], o[i][n][e + 2]);
                }
                __syncthreads();
                if (warp == 0 && rows_on) {
#pragma unroll 1
                    for (int k = 0; k < at_once; ++k)
#pragma unroll
                        for (int i = 0; i < KD; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 v = *reinterpret_cast<const float2*>(place + k * area + e * Cfg::kJoinRow + i * 16);
                                o[i][n][e] += v.x, o[i][n][e + 2] += v.y;
                            }
                }
            }
        if (warp != 0) continue;
        if (whole) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = rb * RB + n * 8 + 2 * c + e;
                    if (row >= R) continue;
                    const float4 it = state_s[n * 8 + 2 * c + e];
                    const bool empty = word[n][e] == 0 || it.y == 0.0f;
                    const float inv = empty ? 0.0f : 1.0f / it.y, power = ex2(it.z) * Wt::kDown;
                    const int t = div_of(row, G), gq = row - t * G;
                    const long long at = ((long long)b * T + t) * P.Hq + h * G + gq;
                    uint16_t* dst = static_cast<uint16_t*>(P.out) + at * D + 2 * g;
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
                        const float p = o[i][n][e] * inv * power, q = o[i][n][e + 2] * inv * power;
                        if (i * 16 < D)
                            *reinterpret_cast<uint32_t*>(dst + i * 16) = empty ? 0u : C.fp16 ? pack<true>(p, q) : pack<false>(p, q);
                    }
                    if (P.lse && g == 0) P.lse[at] = empty ? -INFINITY : lse_of(it.x, P.scale, it.y);
                }
        } else {
            const int piece = segment ? 1 : 0;
            const Parts<DP, RB> parts(P);
            float* part = parts.out(blockIdx.x, piece);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * c + e;
                    if (rb * RB + r >= R) continue;
#pragma unroll
                    for (int i = 0; i < KD; ++i)
                        if (i * 16 < D)
                            *reinterpret_cast<float2*>(part + r * DP + i * 16 + 2 * g) = make_float2(o[i][n][e], o[i][n][e + 2]);
                    if (g == 0) {
                        const float4 it = state_s[r];
                        parts.state(blockIdx.x, piece)[r] = make_float2(it.x, it.y);
                        parts.base(blockIdx.x, piece)[r] = it.z;
                    }
                }
            __threadfence();
            __syncwarp();
            if (lane == 0) {
                int first, last;
                bool behind;
                deal.ctas_of(b, rb + h * row_blocks, first, last, behind);
                unsigned* const there = P.done + *counters_s + first;
                if (atomicAdd(there, 1u) == (unsigned)(last - first)) {
                    *there = 0;
                    last_s[piece] = LastOf{1, b, rb + h * row_blocks, first, last, behind};
                }
            }
        }
    }
    cp_wait<0>();
    __syncthreads();
    if (!last_s[0].on && !last_s[1].on) return;
    __threadfence();
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        if (last_s[i].on) join_parts<DP, RB, Cfg::kOffQ>(P, plan, row_blocks, last_s[i], smem);
}

template <int DP, int NT>
cudaError_t launch_attend(const AttendParams& P, cudaStream_t st) {
    using Cfg = Cfg8<DP, NT>;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const int R = P.T * P.G;
    int row_blocks = (R + Cfg::kRows - 1) / Cfg::kRows;
    const int parts = sms * Cfg::kCtas;
    const auto kern = k_tree_attention8<DP, NT>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    void* args[2] = {const_cast<AttendParams*>(&P), &row_blocks};
    return launch(reinterpret_cast<const void*>(kern), dim3(parts, 1, 1), kThreads, Cfg::smem(P.c.B), args, st);
}

template <int NT>
cudaError_t launch_heads(const AttendParams& P, cudaStream_t st) {
    if (P.c.D <= 64) return launch_attend<64, NT>(P, st);
    return P.c.D <= 128 ? launch_attend<128, NT>(P, st) : launch_attend<256, NT>(P, st);
}

constexpr int kMostCtas = 3;  // an SM, of any of the kernels

}  // namespace

int attend8_counters() {
    const int sms = sm_count();
    return sms < 1 ? 0 : (1 + kCounterSets) * kMostCtas * sms;
}

long long attend8_partial_floats(int D) {
    const long long ctas = (long long)sm_count() * (D <= 64 ? Cfg8<64, 2>::kCtas : D <= 128 ? Cfg8<128, 2>::kCtas : Cfg8<256, 2>::kCtas);
    return ctas * 2 * 16 * ((D <= 64 ? 64 : D <= 128 ? 128 : 256) + 3);
}

// Blocks of eight rows where a key meets no more, else of sixteen. Four rows in blocks of eight / sixteen: 131071 keys 51.8 /
// 63.0 us, sixteen sequences 25.8 / 31.6.
cudaError_t launch_tree_attention8(const AttendParams& P, cudaStream_t st) {
    return P.T * P.G <= 8 ? launch_heads<1>(P, st) : launch_heads<2>(P, st);
}

}  // namespace si
