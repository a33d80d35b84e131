// attend8.cu -- tree attention over a cache of e4m3 codes: the kernel for few
// rows a key. Lists, tiles and the join of several CTAs' parts are those of the
// cache in 16 bits (attend.cu).
//
// A warp takes sixteen keys of every tile and keeps its own softmax state. The
// products have the keys on the long side, so that up to eight query rows
// (one token's heads, mostly) fill the short one:
//   S^T (16 keys x 8 rows) = K (16 x D) Q^T        mma m16n8k16
//   O^T (D x 8 rows)      += V^T (D x 16 keys) P^T
// Codes become fp16 in registers, two an instruction and exactly, on their way
// from shared memory to the product; the scales stay out of it. A key's scale
// multiplies its scores; a value's goes into the weight, relative to the largest
// that the warp has met so far, which the output is rescaled by when it grows,
// as it is by the softmax's maximum. Queries go in as fp16: bf16 rows times the
// power of two that brings their largest element below 2^15, so that what lies
// up to 2^29 below it is exact.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps of sixteen keys of a tile
constexpr int kKeys = 16;

// fp16 weights, and a maximum that may be outgrown by 2^kLazy before anything is rescaled.
using Wt = Weights<true, true>;

template <int DP, int NT>
struct Cfg8 {
    static constexpr int kRows = 8 * NT;                      // query rows of a block
    static constexpr int kTile = KT * DP;                     // bytes of a K or V tile
    static constexpr int kOffScale = 2 * kTile;               // in a stage: {k, v} scales of its keys
    static constexpr int kStage = 2 * kTile + KT * 8;
    static constexpr int kStages = 3;
    static constexpr int kCtas = DP > 128 || (DP == 128 && NT == 2) ? 2 : NT == 1 ? 4 : 3;  // an SM
    static constexpr int kQRow = DP * 2 + 32;                 // bytes: eight rows' 32-byte pieces lie in different banks
    static constexpr int kJoinRow = DP + 4;                   // floats: likewise
    static constexpr bool kQInRegs = DP * NT <= 256;
    static constexpr int kOffQ = kStages * kStage;            // queries; the join of the warps takes their place
    static constexpr int kUnion = kRows * kJoinRow * 4;       // >= kRows * kQRow
    static constexpr int kOffFactor = kOffQ + kUnion;         // what a query row was divided by
    static constexpr int kOffState = kOffFactor + kRows * 4;  // [warp][row] {maximum, sum}
    static constexpr int kOffPlan = kOffState + 4 * kRows * 8;
    static constexpr int smem(int B) { return kOffPlan + Plan::words(B) * 4; }
    static_assert(kRows * kQRow <= kUnion, "the queries fit the join's place");
};

// The transposed 8 x 8 matrix of 16-bit elements that the warp's registers hold.
__device__ __forceinline__ uint32_t transposed(uint32_t w) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
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

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, Cfg8<DP, NT>::kCtas)
    k_tree_attention8(const __grid_constant__ AttendParams P, int row_blocks) {
    using Cfg = Cfg8<DP, NT>;
    using Cp = Copy8<DP>;
    constexpr int RB = Cfg::kRows, KD = DP / 16, UNITS = Cp::UNITS, S = Cfg::kStages;

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + Cfg::kOffQ;
    float* const join_s = reinterpret_cast<float*>(q_s);
    float* const factor_s = reinterpret_cast<float*>(smem + Cfg::kOffFactor);
    float2* const state_s = reinterpret_cast<float2*>(smem + Cfg::kOffState);
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;   // keys g, g + 8; rows 2c, 2c + 1 of each eight
    const int T = P.T, G = P.G, R = T * G, D = C.D;
    const int groups = C.Hkv * row_blocks;

    grid_dependency_wait();
    grid_launch_dependents();  // after the wait: the join reads the lengths before its own
    make_plan<kThreads, kNarrowLeast, kNarrowPiece>(C, T, groups, gridDim.x, plan, P.err, blockIdx.x == 0);
    const Deal deal(plan, C.B, gridDim.x, kNarrowLeast);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);
    if (x0 >= x1) return;

    const float c2 = P.scale * kLog2e;
    const int unit = lane % UNITS;
    const bool unit_on = unit * 16 < D, whole_rows = D == DP;
    const int own0 = warp * kKeys;  // this warp's keys of a tile
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks, v_step = (int)C.vs;

    // producer state: lanes i and i + 16 hold the slot of key own0 + i of the tile to be issued next
    SourceOf<uint8_t> src;
    src.start(plan, C.B, x0, x1);
    const uint32_t ring = smem_u32(smem);
    int stage_in = 0, held = kNoSlot, seen_b = -1;
    int pend = -1, pend_byte = 0;   // the stage that waits for its scales, and this lane's (lanes below 16: k's)
    auto fetch = [&]() {
        const int i0 = src.at.tile * KT;
        if (i0 + KT > src.len && seen_b != src.at.b) {  // the tile meets the new nodes
            src.seen = seen_nodes(P.mask, T, src.at.b, lane);
            seen_b = src.at.b;
        }
        held = slot_of(src.list, i0 + own0 + (lane & 15), src.len, src.tot, src.seen);
    };
    auto issue = [&]() {
        // The scales of the tile before have had a tile's time to arrive. A key that is not there has 0 (byte -1).
        if (pend >= 0) {
            float* to = reinterpret_cast<float*>(smem + pend * Cfg::kStage + Cfg::kOffScale);
            to[(own0 + (lane & 15)) * 2 + (lane >> 4)] = pend_byte < 0 ? 0.0f : scale_of(pend_byte, C.e_lo, C.e_hi);
            pend = -1;
        }
        if (src.x < x1) {
            int slot[Cp::SWEEPS];
            const uint8_t *kp = src.k + unit * 16, *vp = src.v + unit * 16;
            const bool ok = slot_ok(held, n_slots, P.err);
            const bool cached = src.at.tile * KT + KT <= src.len;
            // cached keys: nothing to leave out (a slot outside the pool has been reported; slot 0 is read)
            const int mine = ok ? held : cached ? 0 : -1;
            Cp::slots(mine, lane, slot);
            const uint32_t dst = ring + stage_in * Cfg::kStage;
            if (whole_rows && cached) {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const uint32_t at = dst + tile8_at<DP>(own0 + Cp::row(lane, j), unit);
                    cp16(at, kp + (long long)slot[j] * k_step);
                    cp16(at + Cfg::kTile, vp + (long long)slot[j] * v_step);
                }
            } else {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const bool on = slot[j] >= 0 && unit_on;
                    const long long from = on ? slot[j] : 0;
                    const uint32_t at = dst + tile8_at<DP>(own0 + Cp::row(lane, j), unit);
                    cp16(at, on ? kp + from * k_step : src.k, on);
                    cp16(at + Cfg::kTile, on ? vp + from * v_step : src.v, on);
                }
            }
            pend_byte = mine < 0 ? -1 : (lane < 16 ? src.k_scale : src.v_scale)[mine >> C.block_shift];
            pend = stage_in;
            if (++stage_in == S) stage_in = 0;
            if (src.next(plan, C.B, groups) && src.x < x1) src.enter(C, plan, row_blocks);
            if (src.x < x1) fetch();
        }
        cp_commit();
    };
    src.enter(C, plan, row_blocks);
    fetch();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) issue();

    At a = locate(plan, C.B, x0);
    int segment = 0, stage_out = 0;
    for (int x = x0; x < x1; ++segment) {
        // one list, or the part of it that this CTA has
        const int b = a.b, h = a.group / row_blocks, rb = a.group % row_blocks;
        const int len = plan.len[b], tot = plan.tot[b];
        const int seg_end = min(x1, x + a.ntile - a.tile);
        const bool whole = a.tile == 0 && seg_end - x == a.ntile;

        // query rows of this block into shared memory (rows past R are zero)
        __syncthreads();  // the previous list's joins and reads of q_s are over
        {
            constexpr int AT_ONCE = 32 / (DP / 8);  // rows a warp takes at once
#pragma unroll
            for (int r0 = 0; r0 < RB; r0 += 4 * AT_ONCE) {
                const int r = r0 + warp * AT_ONCE + lane / (DP / 8), row = rb * RB + r, t = row / G;
                const bool on = r < RB && row < R;
                const uint16_t* from = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)(h * G + row - t * G) * P.qh;
                float down;
                const uint4 val = query_unit<DP>(on ? from : nullptr, D, C.fp16, lane, down);
                if (r < RB) {
                    *reinterpret_cast<uint4*>(q_s + r * Cfg::kQRow + lane % (DP / 8) * 16) = val;
                    if (lane % (DP / 8) == 0) factor_s[r] = down;
                }
            }
        }
        unsigned long long word[NT][2];
        float ref[NT][2], sum[NT][2], qdown[NT][2];
        float o[KD][NT][4];
        float unit_v = 0.0f, unit_inv = 1.0f;  // the largest scale of values so far
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = rb * RB + n * 8 + 2 * c + e;
                word[n][e] = row < R && tot > 0 ? word_of(P.mask, T, b, row / G) : 0;
                ref[n][e] = -INFINITY, sum[n][e] = 0.0f;
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
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) qdown[n][e] = factor_s[n * 8 + 2 * c + e];

        for (; x < seg_end; ++x, ++a.tile) {
            cp_wait<S - 2>();
            uint8_t* const stage = smem + stage_out * Cfg::kStage;
            if (++stage_out == S) stage_out = 0;
            const int i0 = a.tile * KT + own0;
            const bool edge = i0 + kKeys > len;  // these keys meet the new nodes or the list's end
            unsigned odd = 0;                    // keys (of the sixteen) with codes of NaN
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
            __syncwarp();
            issue();
            const uint32_t k_s = smem_u32(stage), v_s = k_s + Cfg::kTile;
            const float2* sc = reinterpret_cast<const float2*>(stage + Cfg::kOffScale) + own0;
            const float2 sc0 = sc[g], sc1 = sc[g + 8];
            // rows of an ldmatrix: keys 0-7, 8-15 of a unit, then of the next unit
            const int ld_key = own0 + (lane & 15), ld_unit = lane >> 4;
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
            for (int u = 0; u < KD; u += 2) {
                uint32_t r[4];
                ldsm4(r, k_s + tile8_at<DP>(ld_key, u + ld_unit));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t a0, a1, a2, a3;
                    halves4(r[2 * i], a0, a2);
                    halves4(r[2 * i + 1], a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 q = Cfg::kQInRegs ? qf[Cfg::kQInRegs ? n : 0][Cfg::kQInRegs ? u + i : 0] : query(n, u + i);
                        mma16(s[n], a0, a1, a2, a3, q.x, q.y);
                    }
                }
            }
            // s[n][0..1]: key g with rows 2c, 2c + 1; s[n][2..3]: key g + 8
            bool grows = fmaxf(sc0.y, sc1.y) > unit_v;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = s[n][e] * qdown[n][e & 1] * (e < 2 ? sc0.x : sc1.x);
                    if (edge) {
                        const int j = i0 + g + (e & 2) * 4 - len;
                        const bool sees = j < 0 || (j < T && (word[n][e & 1] >> (j & 63) & 1));
                        if (!sees) s[n][e] = -INFINITY;
                    }
                    // The difference is taken before the scale: scores of the type's lowest value differ by 0 from
                    // their maximum, where a fused s * c2 - ref * c2 would be off by the product's rounding.
                    grows |= (s[n][e] - ref[n][e & 1]) * c2 > (float)Wt::kLazy;
                }
            if (__any_sync(0xFFFFFFFFu, grows)) {
                const float most = column_max(fmaxf(unit_v, fmaxf(sc0.y, sc1.y)));  // NaN is passed over
                const float fall = unit_v * (most > 0.0f ? power_inverse(most) : 1.0f);
                if (most > 0.0f) unit_v = most, unit_inv = power_inverse(most);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float keep[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float top = column_max(fmaxf(ref[n][e], fmaxf(s[n][e], s[n][e + 2])));
                        keep[e] = top == ref[n][e] ? 1.0f : ex2((ref[n][e] - top) * c2);
                        ref[n][e] = top;
                        sum[n][e] *= keep[e];
                        keep[e] *= fall;
                    }
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
                        o[i][n][0] *= keep[0], o[i][n][2] *= keep[0];
                        o[i][n][1] *= keep[1], o[i][n][3] *= keep[1];
                    }
                }
            }
            const float v0 = sc0.y * unit_inv, v1 = sc1.y * unit_inv;
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float shift = ref[n][e & 1] == -INFINITY ? 0.0f : ref[n][e & 1];
                    const float p = ex2(fmaf(s[n][e] - shift, c2, Wt::kUp));
                    sum[n][e & 1] += p;
                    w[e] = p * (e < 2 ? v0 : v1);
                    if (edge && s[n][e] == -INFINITY) w[e] = 0.0f;  // whatever scale a key has that the row does not see
                }
                // The product takes fp16: a weight goes in as two terms, the second what the first one's rounding left.
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = pack<true>(w[2 * i], w[2 * i + 1]);
                    const uint32_t lo = pack<true>(w[2 * i] - widen<true>((uint16_t)hi), w[2 * i + 1] - widen<true>((uint16_t)(hi >> 16)));
                    ph[n][i] = transposed(hi), pl[n][i] = transposed(lo);
                }
            }
#pragma unroll
            for (int u = 0; u < KD; u += 2) {
                uint32_t r[4];
                ldsm4t(r, v_s + tile8_at<DP>(ld_key, u + ld_unit));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // a register holds two keys' codes of elements 2g, 2g + 1: rows g and g + 8 of the product
                    uint32_t a0, a1, a2, a3;
                    halves4(__byte_perm(r[2 * i], 0, 0x3120), a0, a1);
                    halves4(__byte_perm(r[2 * i + 1], 0, 0x3120), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16(o[u + i][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                        mma16(o[u + i][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
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
            step(plan, C.B, groups, a);
        }

        // Join the warps: maxima and sums, then output rows in warp order, through the place of this list's queries,
        // which are no longer needed. (The ring's stages are not touched: the next list's copies are in flight.)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[n][e] = column_sum(sum[n][e]);
                if (g == 0) state_s[warp * RB + n * 8 + 2 * c + e] = make_float2(ref[n][e], sum[n][e]);
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY, all = 0.0f;
                float2 st[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    st[w] = state_s[w * RB + n * 8 + 2 * c + e];
                    top = fmaxf(top, st[w].x);
                }
                const float sh = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int w = 0; w < 4; ++w) all += st[w].y * ex2((st[w].x - sh) * c2);
                const float f = ex2((ref[n][e] - sh) * c2) * Wt::kDown;
#pragma unroll
                for (int i = 0; i < KD; ++i) {
                    o[i][n][e] = o[i][n][e] * f * unit_v;
                    o[i][n][e + 2] = o[i][n][e + 2] * f * unit_v;
                }
                ref[n][e] = top;
                sum[n][e] = all * Wt::kDown;
            }
        for (int w = 1; w < 4; ++w) {
            if (w > 1) __syncthreads();
            if (warp == w) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < KD; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float2*>(join_s + (n * 8 + 2 * c + e) * Cfg::kJoinRow + i * 16 + 2 * g) =
                                make_float2(o[i][n][e], o[i][n][e + 2]);
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < KD; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 v = *reinterpret_cast<const float2*>(join_s + (n * 8 + 2 * c + e) * Cfg::kJoinRow + i * 16 + 2 * g);
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
                    const bool empty = word[n][e] == 0 || sum[n][e] == 0.0f;
                    const float inv = empty ? 0.0f : 1.0f / sum[n][e];
                    const int t = row / G, gq = row - t * G;
                    const long long at = ((long long)b * T + t) * P.Hq + h * G + gq;
                    uint16_t* dst = static_cast<uint16_t*>(P.out) + at * D + 2 * g;
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
                        const float p = o[i][n][e] * inv, q = o[i][n][e + 2] * inv;
                        if (i * 16 < D)
                            *reinterpret_cast<uint32_t*>(dst + i * 16) = empty ? 0u : C.fp16 ? pack<true>(p, q) : pack<false>(p, q);
                    }
                    if (P.lse && g == 0) P.lse[at] = empty ? -INFINITY : lse_of(ref[n][e], P.scale, sum[n][e]);
                }
        } else {
            // the join takes fp16 caches' rows and sums times 2^15, see Weights
            const float up = C.fp16 ? 1.0f / Weights<true, false>::kDown : 1.0f;
            float* part = P.part + ((long long)blockIdx.x * 2 + (segment ? 1 : 0)) * part_floats(RB, DP);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * c + e;
#pragma unroll
                    for (int i = 0; i < KD; ++i)
                        *reinterpret_cast<float2*>(part + r * DP + i * 16 + 2 * g) = make_float2(o[i][n][e] * up, o[i][n][e + 2] * up);
                    if (g == 0) {
                        part[RB * DP + r] = ref[n][e];
                        part[RB * DP + RB + r] = sum[n][e] * up;
                    }
                }
        }
    }
    cp_wait<0>();
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
    e = launch(reinterpret_cast<const void*>(kern), dim3(parts, 1, 1), kThreads, Cfg::smem(P.c.B), args, st);
    if (e != cudaSuccess) return e;
    return launch_tree_attention_join(P, Cfg::kRows, row_blocks, parts, st);
}

template <int NT>
cudaError_t launch_heads(const AttendParams& P, cudaStream_t st) {
    if (P.c.D <= 64) return launch_attend<64, NT>(P, st);
    return P.c.D <= 128 ? launch_attend<128, NT>(P, st) : launch_attend<256, NT>(P, st);
}

}  // namespace

cudaError_t launch_tree_attention8(const AttendParams& P, cudaStream_t st) {
    return P.T * P.G <= 8 ? launch_heads<1>(P, st) : launch_heads<2>(P, st);
}

}  // namespace si
