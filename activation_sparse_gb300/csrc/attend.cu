// attend.cu -- attention of a tree of new tokens over a key/value cache: the
// kernel for few rows a key, and the join of what several CTAs have of a list.
//
// A list of keys (one sequence, one cache head) is cut into tiles of 64; the
// tiles of all lists are dealt out evenly to the CTAs of one resident grid, so
// a long context of one sequence and a batch of ragged ones load every SM
// alike. A CTA walks its tiles with the keys and values of the next ones in
// flight (16-byte asynchronous copies, gathered through the slot table), and
// keeps the running maximum and sum of the softmax and the output rows in
// registers. A list that ends up in one CTA is finished there; the others
// leave partial rows that a second kernel joins in a fixed order, so results
// do not depend on timing.
//
// Bound by memory: one token of 32 heads over 131071 keys of 8 heads of 128
// takes 91 us, 6.0 TB/s, 0.88 of what a plain copy reaches. Short lists are
// bound by latency (1000 keys, heads of 64: 9.5 us with the join).
#include "attend.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps

// ------------------------------------------------------------- attention

template <int DP>
struct AttendCfg {
    static constexpr int kTile = KT * DP * 2;             // bytes of a K or V tile
    static constexpr int kStages = 3;
    static constexpr int kCtas = DP <= 128 ? 2 : 1;       // an SM
    static constexpr int kRows = DP <= 128 ? 16 : 32;     // query rows a block has at most
    static constexpr int kQBytes = kRows * DP * 2;
    static constexpr int kOffQ = kStages * 2 * kTile;
    static constexpr int kOffPlan = kOffQ + kQBytes;
    static constexpr int kOffOdd = kOffPlan;              // new nodes whose value row is not finite (a word)
    static constexpr int smem(int B) { return kOffPlan + 16 + Plan::words(B) * 4; }
};

template <int THREADS>
__device__ __forceinline__ void group_sync(int id) {
    if (THREADS == 32) __syncwarp();
    else named_bar_sync(id, THREADS);
}

// MW row warps x KW key warps = 4: a block of RB = 16 * MW rows; each key
// warp takes KT / KW keys of every tile with its own softmax state, joined at
// the end of a list.
template <int DP, int MW, bool FP16>
__global__ void __launch_bounds__(kThreads, AttendCfg<DP>::kCtas)
    k_tree_attention(const __grid_constant__ AttendParams P, int row_blocks) {
    using Cfg = AttendCfg<DP>;
    using Cp = Copy<DP>;
    constexpr int KW = 4 / MW;
    constexpr int RB = 16 * MW;
    constexpr int WK = KT / KW;          // keys of a tile per warp
    constexpr int NS = WK / 8;           // n8 score tiles
    constexpr int KD = DP / 16;          // k steps over D
    constexpr int UNITS = Cp::UNITS;
    constexpr int S = Cfg::kStages;
    constexpr bool TWO = MW == 1;        // terms of a weight
    using Wt = Weights<FP16, false>;
    static_assert(WK == 16 * MW, "a group's warps copy sixteen keys each");

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const tiles = smem;
    uint8_t* const q_s = smem + Cfg::kOffQ;
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan + 16), P.c.B);
    unsigned long long* odd_s = reinterpret_cast<unsigned long long*>(smem + Cfg::kOffOdd);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mw = warp % MW, kw = warp / MW;
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
    const bool unit_on = unit * 8 < D;
    const int own0 = kw * WK + mw * 16;  // this warp copies keys own0 .. own0 + 15 of a tile
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks, v_step = (int)C.vs;

    // producer state: lane i < 16 holds the slot of key own0 + i of the tile to be issued next
    Source src;
    src.start(plan, C.B, x0, x1);
    const bool whole_rows = D == DP;
    const uint32_t ring = smem_u32(tiles);
    uint32_t stage_in = ring;
    int held = kNoSlot, seen_b = -1;
    auto fetch = [&]() {
        const int i0 = src.at.tile * KT;
        if (i0 + KT > src.len && seen_b != src.at.b) {  // the tile meets the new nodes
            src.seen = seen_nodes(P.mask, T, src.at.b, lane);
            seen_b = src.at.b;
        }
        held = slot_of(src.list, i0 + own0 + (lane & 15), src.len, src.tot, src.seen);
    };
    auto issue = [&]() {
        if (src.x < x1) {
            int slot[Cp::SWEEPS];
            const uint16_t *kp = src.k + unit * 8, *vp = src.v + unit * 8;
            const bool ok = slot_ok(held, n_slots, P.err);
            if (whole_rows && src.at.tile * KT + KT <= src.len) {
                // cached keys: nothing to leave out (a slot outside the pool has been reported; slot 0 is read)
                Cp::slots(ok ? held : 0, lane, slot);
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const uint32_t at = stage_in + tile_at<DP>(own0 + Cp::row(lane, j), unit);
                    cp16(at, kp + (long long)slot[j] * k_step);
                    cp16(at + Cfg::kTile, vp + (long long)slot[j] * v_step);
                }
            } else {
                Cp::slots(ok ? held : -1, lane, slot);
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const bool on = slot[j] >= 0 && unit_on;
                    const long long from = on ? slot[j] : 0;
                    const uint32_t at = stage_in + tile_at<DP>(own0 + Cp::row(lane, j), unit);
                    cp16(at, on ? kp + from * k_step : src.k, on);
                    cp16(at + Cfg::kTile, on ? vp + from * v_step : src.v, on);
                }
            }
            stage_in = stage_in + 2 * Cfg::kTile == ring + S * 2 * Cfg::kTile ? ring : stage_in + 2 * Cfg::kTile;
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
        if (tid == 0) *odd_s = 0;
        for (int i = tid; i < RB * UNITS; i += kThreads) {
            const int r = i / UNITS, u = i % UNITS, row = rb * RB + r;
            uint4 val = make_uint4(0, 0, 0, 0);
            if (row < R && u * 8 < D) {
                const int t = row / G, g = row - t * G;
                val = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt +
                                                      (long long)(h * G + g) * P.qh + u * 8);
            }
            *reinterpret_cast<uint4*>(q_s + tile_at<DP>(r, u)) = val;
        }
        unsigned long long word[2] = {0, 0};
        int row[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            row[e] = rb * RB + mw * 16 + e * 8 + (lane >> 2);
            if (row[e] < R && tot > 0) word[e] = word_of(P.mask, T, b, row[e] / G);
        }
        float o[DP / 8][4];
        float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        __syncthreads();
        uint32_t qf[DP <= 128 ? KD : 1][4];
        const uint32_t q_addr = smem_u32(q_s);
        if (DP <= 128) {
#pragma unroll
            for (int k = 0; k < KD; ++k)
                ldsm4(qf[DP <= 128 ? k : 0], q_addr + tile_at<DP>(mw * 16 + (lane & 15), 2 * k + (lane >> 4)));
        }

        for (; x < seg_end; ++x, ++a.tile) {
            cp_wait<S - 2>();
            uint8_t* const stage = tiles + stage_out * 2 * Cfg::kTile;
            if (++stage_out == S) stage_out = 0;
            const bool meets_new = a.tile * KT + KT > len;
            if (meets_new) {
                // A node's value row may hold infinities or NaN that only its descendants may
                // see, and 0 * NaN is NaN: such elements leave the product here (each lane
                // looks at what it copied itself) and come back below for the rows that see them.
#pragma unroll 1
                for (int j = 0; j < Cp::SWEEPS; ++j) {
                    const int key = own0 + Cp::row(lane, j), node = a.tile * KT + key - len;
                    if (node < 0 || node >= T) continue;
                    uint16_t* e = reinterpret_cast<uint16_t*>(stage + Cfg::kTile + tile_at<DP>(key, unit));
                    bool odd = false;
                    for (int i = 0; i < 8; ++i)
                        if (not_finite<FP16>(e[i])) e[i] = 0, odd = true;
                    if (odd) atomicOr(odd_s, 1ull << node);
                }
            }
            group_sync<32 * MW>(1 + kw);
            issue();
            const uint32_t k_s = smem_u32(stage);
            const uint32_t v_s = k_s + Cfg::kTile;
            const int key0 = kw * WK;
            float s[NS][4];
#pragma unroll
            for (int n = 0; n < NS; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < KD; ++k) {
                uint32_t qk[4];
                if (DP > 128) ldsm4(qk, q_addr + tile_at<DP>(mw * 16 + (lane & 15), 2 * k + (lane >> 4)));
                const uint32_t(&qa)[4] = DP <= 128 ? qf[DP <= 128 ? k : 0] : qk;
#pragma unroll
                for (int n = 0; n < NS; n += 2) {
                    // keys n*8 .. +15: matrices (keys 0-7, d 0-7), (keys 0-7, d 8-15), (keys 8-15, ...)
                    uint32_t kf[4];
                    ldsm4(kf, k_s + tile_at<DP>(key0 + n * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                    mma<FP16>(s[n], qa, kf[0], kf[1]);
                    mma<FP16>(s[n + 1], qa, kf[2], kf[3]);
                }
            }
            const int i0 = a.tile * KT + key0;
            if (i0 + WK > len) {  // the tile meets the new nodes or the list's end
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = i0 + n * 8 + (lane & 3) * 2 + (e & 1) - len;
                        const bool sees = j < 0 || (j < T && (word[e >> 1] >> (j & 63) & 1));
                        if (!sees) s[n][e] = -INFINITY;
                    }
            }
            float top[2] = {mx[0], mx[1]};
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                top[0] = fmaxf(top[0], fmaxf(s[n][0], s[n][1]));
                top[1] = fmaxf(top[1], fmaxf(s[n][2], s[n][3]));
            }
            float shift[2], keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 2));
                // The difference is taken before the scale: scores of the type's lowest value
                // differ by 0 from their maximum, where a fused s * c2 - top * c2 would be off by the
                // product's rounding, which at that size is a number of any size.
                shift[e] = top[e] == -INFINITY ? 0.0f : top[e];  // a row that has seen nothing yet
                keep[e] = ex2((mx[e] - shift[e]) * c2);
                mx[e] = top[e];
                sum[e] *= keep[e];
            }
            // a new maximum is rare after the first tiles: the output rows are rescaled only then
            if (__any_sync(0xFFFFFFFFu, keep[0] != 1.0f || keep[1] != 1.0f)) {
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    o[i][0] *= keep[0];
                    o[i][1] *= keep[0];
                    o[i][2] *= keep[1];
                    o[i][3] *= keep[1];
                }
            }
#pragma unroll
            for (int n = 0; n < NS; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = ex2(fmaf(s[n][e] - shift[e >> 1], c2, Wt::kUp));
                    sum[e >> 1] += s[n][e];
                }
            }
#pragma unroll
            for (int n = 0; n < NS; n += 2) {
                // The matrix product takes both sides in one type. With up to 16 rows a key, bound by memory, a weight
                // goes in as two terms of it, the second what the first one's rounding left: good to U^2 for a rounding
                // of U. (One term / two: 8 sequences of 8192 keys, 8 heads of 128, 16 rows 60.7 / 61.3 us; with more rows
                // the products bound it, 4 of 8192, 4 heads of 256, 64 rows 79 / 94, and one rounding is left.)
                uint32_t pf[4], pr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = s[n + (e >> 1)][(e & 1) * 2], b = s[n + (e >> 1)][(e & 1) * 2 + 1];
                    pf[e] = pack<FP16>(a, b);
                    if (TWO) pr[e] = pack<FP16>(a - widen<FP16>((uint16_t)pf[e]), b - widen<FP16>((uint16_t)(pf[e] >> 16)));
                }
#pragma unroll
                for (int i = 0; i < DP / 8; i += 2) {
                    uint32_t vf[4];
                    ldsm4t(vf, v_s + tile_at<DP>(key0 + n * 8 + (lane & 15), i + (lane >> 4)));
                    mma<FP16>(o[i], pf, vf[0], vf[1]);
                    mma<FP16>(o[i + 1], pf, vf[2], vf[3]);
                    if (TWO) mma<FP16>(o[i], pr, vf[0], vf[1]);
                    if (TWO) mma<FP16>(o[i + 1], pr, vf[2], vf[3]);
                }
            }
            if (meets_new && *odd_s) {
                // the value elements taken out above: not finite, so their weight does not matter
                const int32_t* list = C.table ? C.table + b * C.tb + h * C.th : nullptr;
                for (int key = 0; key < WK; ++key) {
                    const int node = i0 + key - len;
                    if (node < 0 || node >= T || !(*odd_s >> node & 1)) continue;
                    const long long slot = list ? list[len + node] : len + node;
                    if (slot < 0 || slot >= C.n_slots) continue;
                    const uint16_t* src = static_cast<const uint16_t*>(C.v) + b * C.vb + h * C.vh + slot * C.vs;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        const int d = i * 8 + (lane & 3) * 2;
                        if (d >= D) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint16_t w = src[d + (e & 1)];
                            if (not_finite<FP16>(w) && (word[e >> 1] >> node & 1)) o[i][e] += widen<FP16>(w);
                        }
                    }
                }
            }
        }
        if (a.tile == a.ntile) {
            a.tile = a.ntile - 1;
            step(plan, C.B, groups, a);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
            sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
        }

        // Join the key warps: maxima and sums, then output rows in key-warp order, through the place of this list's
        // queries, which are no longer needed. (The ring's stages are not touched: the next list's copies are in flight.)
        if (KW > 1) {
            __syncthreads();
            float* ms = reinterpret_cast<float*>(q_s);  // [KW][RB][2]
            if ((lane & 3) == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mw * 16 + e * 8 + (lane >> 2);
                    ms[(kw * RB + r) * 2] = mx[e];
                    ms[(kw * RB + r) * 2 + 1] = sum[e];
                }
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mw * 16 + e * 8 + (lane >> 2);
                float top = -INFINITY, all = 0.0f;
                for (int w = 0; w < KW; ++w) top = fmaxf(top, ms[(w * RB + r) * 2]);
                const float sh = top == -INFINITY ? 0.0f : top;
                for (int w = 0; w < KW; ++w) all += ms[(w * RB + r) * 2 + 1] * ex2((ms[(w * RB + r) * 2] - sh) * c2);
                const float f = ex2((mx[e] - sh) * c2);
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) o[i][2 * e] *= f, o[i][2 * e + 1] *= f;
                mx[e] = top;
                sum[e] = all;
            }
            float* acc = reinterpret_cast<float*>(q_s);
            constexpr int kHalf = Cfg::kQBytes / 4 / RB;  // columns that fit at once
            constexpr int COLS = kHalf < DP ? kHalf : DP;
            for (int col = 0; col < DP; col += COLS) {
                for (int w = 1; w < KW; ++w) {
                    __syncthreads();
                    if (kw == w) {
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) {
                            const int cc = i * 8 + (lane & 3) * 2 - col;
                            if (cc < 0 || cc >= COLS) continue;
                            const int r = mw * 16 + (lane >> 2);
                            *reinterpret_cast<float2*>(acc + r * COLS + cc) = make_float2(o[i][0], o[i][1]);
                            *reinterpret_cast<float2*>(acc + (r + 8) * COLS + cc) = make_float2(o[i][2], o[i][3]);
                        }
                    }
                    __syncthreads();
                    if (kw == 0) {
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) {
                            const int cc = i * 8 + (lane & 3) * 2 - col;
                            if (cc < 0 || cc >= COLS) continue;
                            const int r = mw * 16 + (lane >> 2);
                            const float2 u0 = *reinterpret_cast<const float2*>(acc + r * COLS + cc);
                            const float2 u1 = *reinterpret_cast<const float2*>(acc + (r + 8) * COLS + cc);
                            o[i][0] += u0.x, o[i][1] += u0.y, o[i][2] += u1.x, o[i][3] += u1.y;
                        }
                    }
                }
            }
        }
        if (kw == 0) {
            if (whole) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (row[e] >= R) continue;
                    const bool empty = word[e] == 0 || sum[e] == 0.0f;
                    const float inv = empty ? 0.0f : 1.0f / sum[e];
                    const int t = row[e] / G, g = row[e] - t * G;
                    const long long at = ((long long)b * T + t) * P.Hq + h * G + g;
                    uint16_t* dst = static_cast<uint16_t*>(P.out) + at * D;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        const int d = i * 8 + (lane & 3) * 2;
                        if (d < D)
                            *reinterpret_cast<uint32_t*>(dst + d) =
                                empty ? 0u : pack<FP16>(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
                    }
                    if (P.lse && (lane & 3) == 0)
                        P.lse[at] = empty ? -INFINITY : lse_of(mx[e], P.scale, sum[e] * Wt::kDown);
                }
            } else {
                float* part = P.part + ((long long)blockIdx.x * 2 + (segment ? 1 : 0)) * part_floats(RB, DP);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mw * 16 + e * 8 + (lane >> 2);
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
                        *reinterpret_cast<float2*>(part + r * DP + i * 8 + (lane & 3) * 2) =
                            make_float2(o[i][2 * e], o[i][2 * e + 1]);
                    if ((lane & 3) == 0) {
                        part[RB * DP + r] = mx[e];
                        part[RB * DP + RB + r] = sum[e];
                    }
                }
            }
        }
    }
    cp_wait<0>();
}

// Joins the partial rows of the lists that more than one CTA worked on. A row
// belongs to JW warps of one block: warp w takes parts w, w + JW, ..., and
// the warps' sums are added in their order, so the result does not depend on
// timing. JW = 8 or 1.
constexpr int kJoinWarps = 8;

template <int DP, int RB, int JW, bool FP16>
__global__ void __launch_bounds__(kJoinWarps * 32)
    k_tree_attention_join(const __grid_constant__ AttendParams P, int row_blocks, int parts) {
    constexpr int E = DP / 32;  // columns a lane
    constexpr int ROWS = kJoinWarps / JW;  // rows a block
    __shared__ float acc_s[JW > 1 ? JW : 1][DP];
    __shared__ float sum_s[kJoinWarps], top_s[kJoinWarps];
    extern __shared__ __align__(128) uint8_t smem[];
    const KvView& C = P.c;
    const Plan plan(reinterpret_cast<int*>(smem), P.c.B);
    const int T = P.T, G = P.G, R = T * G, D = C.D;
    const int groups = C.Hkv * row_blocks;
    // The first kernel lets this one start once everything before it is complete, and does not change the
    // lengths: the plan is made under its last tiles.
    constexpr int LEAST = RB >= 128 ? kWideLeast : kNarrowLeast, PIECE = RB >= 128 ? kWidePiece : kNarrowPiece;
    make_plan<kJoinWarps * 32, LEAST, PIECE>(C, T, groups, parts, plan, P.err, false);
    grid_launch_dependents();
    grid_dependency_wait();
    const Deal deal(plan, C.B, parts, LEAST);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row_sets = (min(R, RB) + ROWS - 1) / ROWS;
    const int list_id = blockIdx.x / row_sets;
    const int b = list_id / groups, group = list_id % groups;
    const int r = blockIdx.x % row_sets * ROWS + warp / JW;
    const int h = group / row_blocks, row = group % row_blocks * RB + r;
    int first, last;
    bool behind;  // only the first part can follow another list in its CTA
    deal.ctas_of(b, group, first, last, behind);
    if (first == last) return;  // finished by its CTA
    const bool on = row < R && r < RB;
    const float c2 = P.scale * kLog2e;
    const int w = warp % JW;
    auto part_of = [&](int c) {
        return P.part + ((long long)c * 2 + (c == first && behind)) * part_floats(RB, DP);
    };
    // Four parts at a time, maxima, sums and rows together: one trip to memory each.
    float top = -INFINITY, sum = 0.0f, acc[E] = {};
    auto shift_of = [](float m) { return m == -INFINITY ? 0.0f : m; };
    if (on) {
        for (int c0 = first + w; c0 <= last; c0 += 4 * JW) {
            float m[4], l[4], o[4][E];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * JW;
                m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[i][e] = 0.0f;
                if (c <= last) {
                    const float* p = part_of(c);
                    m[i] = p[RB * DP + r];
                    l[i] = p[RB * DP + RB + r];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[i][e] = p[r * DP + e * 32 + lane];
                }
            }
            const float high = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
            const float shift = shift_of(high), keep = ex2((top - shift) * c2);
            top = high;
            sum *= keep;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= keep;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = ex2((m[i] - shift) * c2);
                sum += f * l[i];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += f * o[i][e];
            }
        }
    }
    if (JW > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc_s[JW > 1 ? w : 0][e * 32 + lane] = acc[e];
        if (lane == 0) top_s[w] = top, sum_s[w] = sum;
        __syncthreads();
        if (w > 0) return;
        for (int i = 1; i < JW; ++i) top = fmaxf(top, top_s[i]);
        const float shift = shift_of(top);
        sum = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < JW; ++i) {
            const float f = ex2((top_s[i] - shift) * c2);
            sum += f * sum_s[i];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += f * acc_s[JW > 1 ? i : 0][e * 32 + lane];
        }
    }
    if (!on) return;
    const int t = row / G, g = row - t * G;
    const bool empty = plan.tot[b] == 0 || word_of(P.mask, T, b, t) == 0 || sum == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / sum;
    const long long at = ((long long)b * T + t) * P.Hq + h * G + g;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = e * 32 + lane;
        if (d >= D) continue;
        const float v = empty ? 0.0f : acc[e] * inv;
        uint16_t bits;
        if (FP16) {
            const __half hv = __float2half_rn(v);
            bits = *reinterpret_cast<const uint16_t*>(&hv);
        } else {
            const __nv_bfloat16 hv = __float2bfloat16_rn(v);
            bits = *reinterpret_cast<const uint16_t*>(&hv);
        }
        static_cast<uint16_t*>(P.out)[at * D + d] = bits;
    }
    if (P.lse && lane == 0) P.lse[at] = empty ? -INFINITY : lse_of(top, P.scale, sum * Weights<FP16, (RB >= 128)>::kDown);
}

// ------------------------------------------------------------------ host

int per_sm(int dp) { return dp <= 128 ? 2 : 1; }
int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Row warps of heads of more than 128 elements; more rows than 32 go in further row blocks. Four sequences of
// up to 8192 keys, 4 heads of 256, one / two: 16 rows 28.6 / 30.1 us, 20 rows 45 / 31, 64 rows 84 / 54.
int row_warps(int R) { return R <= 16 ? 1 : 2; }

// Up to 16 rows a key: the tiles above, bound by memory. More rows: 128-row
// tiles on the tensor memory path, whose cost a key hardly depends on the
// rows (it is not built for heads of more than 128 elements). 8 sequences of up
// to 8192 keys, 8 heads of 128, here / there: 16 rows 42.8 / 39.8 us, 20 rows 63
// / 40, 64 rows 114 / 43; one of 30000 keys, heads of 64: 16 rows 20.0 / 23.3 us,
// 20 rows 30 / 24.
bool many_rows(int D, int R) { return R > 16 && D <= 128; }

template <int DP, int RB, bool FP16>
cudaError_t launch_join(const AttendParams& P, int row_blocks, int parts, cudaStream_t st) {
    void* args[3] = {const_cast<AttendParams*>(&P), &row_blocks, &parts};
    const long long lists = (long long)P.c.B * P.c.Hkv * row_blocks;
    const int rows = P.T * P.G < RB ? P.T * P.G : RB;
    // A block a row (eight warps share its parts) where lists have eight parts and the rows fit the GPU twice
    // over; else a warp a row. The whole call by the one / the other: 8 lists of 131071 keys, 4 rows 94 / 97 us; 12
    // of up to 9001, 128 rows 23.7 / 27.3; 128 of 8192, 4 rows 70.0 / 69.7; 256 of 4096, 4 rows 98 / 93; 32 of 1000,
    // 256 rows 41 / 18; 64 of 8192, 256 rows 134 / 70.
    const bool many = parts >= 8 * lists && lists * rows <= 16ll * sm_count();  // parts of a list: about parts / lists
    const int per_block = many ? 1 : kJoinWarps;
    const long long blocks = lists * ((rows + per_block - 1) / per_block);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const void* join = many ? reinterpret_cast<const void*>(&k_tree_attention_join<DP, RB, kJoinWarps, FP16>)
                            : reinterpret_cast<const void*>(&k_tree_attention_join<DP, RB, 1, FP16>);
    return launch(join, dim3((unsigned)blocks, 1, 1), kJoinWarps * 32, Plan::words(P.c.B) * 4, args, st);
}

template <int DP, int MW, bool FP16>
cudaError_t launch_attend(const AttendParams& P, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const int R = P.T * P.G;
    int row_blocks = (R + 16 * MW - 1) / (16 * MW);
    int parts = sms * per_sm(DP);
    const auto kern = k_tree_attention<DP, MW, FP16>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    void* args[2] = {const_cast<AttendParams*>(&P), &row_blocks};
    e = launch(reinterpret_cast<const void*>(kern), dim3(parts, 1, 1), kThreads, AttendCfg<DP>::smem(P.c.B), args, st);
    if (e != cudaSuccess) return e;
    return launch_join<DP, 16 * MW, FP16>(P, row_blocks, parts, st);
}

template <bool FP16>
cudaError_t launch_attend_type(const AttendParams& P, cudaStream_t st) {
    const int R = P.T * P.G;
    switch (padded(P.c.D)) {
        case 64: return launch_attend<64, 1, FP16>(P, st);
        case 128: return launch_attend<128, 1, FP16>(P, st);
        default: return row_warps(R) == 1 ? launch_attend<256, 1, FP16>(P, st) : launch_attend<256, 2, FP16>(P, st);
    }
}

template <int DP, int RB>
cudaError_t launch_wide_join(const AttendParams& P, int row_blocks, int parts, cudaStream_t st) {
    return P.c.fp16 ? launch_join<DP, RB, true>(P, row_blocks, parts, st) : launch_join<DP, RB, false>(P, row_blocks, parts, st);
}

cudaError_t launch_wide(const AttendParams& P, cudaStream_t st) {
    int row_blocks = 0, parts = 0;
    const cudaError_t e = launch_tree_attention_wide(P, &row_blocks, &parts, st);
    if (e != cudaSuccess) return e;
    if (wide_rows(P.T * P.G) == 128)
        return P.c.D <= 64 ? launch_wide_join<64, 128>(P, row_blocks, parts, st)
                           : launch_wide_join<128, 128>(P, row_blocks, parts, st);
    return P.c.D <= 64 ? launch_wide_join<64, 256>(P, row_blocks, parts, st)
                       : launch_wide_join<128, 256>(P, row_blocks, parts, st);
}

}  // namespace

// Partial rows of every CTA (two pieces of lists each), for as many rows as a call can have: 40 MB for heads of 128.
long long attend_partial_floats(int D) {
    const int dp = padded(D);
    if (many_rows(D, INT_MAX)) return 2ll * sm_count() * 2 * part_floats(128, dp);  // two CTAs an SM, or one with twice the rows
    return 2ll * sm_count() * per_sm(dp) * part_floats(16 * row_warps(INT_MAX), dp);
}

bool attend_counts_fit(const AttendParams& P) {
    constexpr long long kMost = INT_MAX - (1 << 20);  // room for a grid and a tile beside them
    const int R = P.T * P.G;
    const int rows = many_rows(P.c.D, R) ? wide_rows(R) : 16 * (padded(P.c.D) > 128 ? row_warps(R) : 1);
    const long long lists = (long long)P.c.B * P.c.Hkv * ((R + rows - 1) / rows);
    const long long tiles = (long long)P.c.cap / KT + 1;
    return P.c.cap <= kMost && lists <= kMost / tiles && lists <= kMost / rows;
}

cudaError_t launch_tree_attention(const AttendParams& P, cudaStream_t st) {
    if (many_rows(P.c.D, P.T * P.G)) return launch_wide(P, st);
    return P.c.fp16 ? launch_attend_type<true>(P, st) : launch_attend_type<false>(P, st);
}

}  // namespace si
