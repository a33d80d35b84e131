// weigh8.cu -- the attention weight that each key of a cache of e4m3 codes received.
#include <type_traits>

#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps
constexpr int kRows = 64;      // kept in shared memory at once

template <int DP>
struct Cfg8 {
    static constexpr int kMT = DP <= 128 ? 2 : 1;             // sixteens of keys a warp has of a tile
    static constexpr int kWarpKeys = 16 * kMT;
    static constexpr int kKeys = 4 * kWarpKeys;               // of a tile
    static constexpr int kTile = kKeys * DP;
    static constexpr int kOffKey = kTile;                     // in a stage: slots, old weights, scales of its keys
    static constexpr int kStage = kTile + kKeys * 12;
    static constexpr int kStages = 2;
    static constexpr int kCtas = DP <= 128 ? 4 : 2;           // an SM
    static constexpr int kQRow = DP * 2 + 32;
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffRow = kOffQ + kRows * kQRow;     // per row: ancestor word, lse, factor, node; the nodes' number
    static constexpr int kOffPlan = kOffRow + kRows * (8 + 4 + 4 + 4) + 16;
    static constexpr int smem(int B) { return kOffPlan + Plan::words(B) * 4; }
};

// acc_out[slot] = acc[slot] + sum over counted rows of exp(scale * scale_k * q.code - lse).
// As over a cache in 16 bits: keys are the long side of the product and rows
// the short one, a thread sums its keys' weights over the rows in registers,
// and a key belongs to one warp, which also copies it, its scale and its old
// weight. A tile's codes become fp16 once, in registers, for all of the rows.
// 8 sequences of up to 16384 keys, 8 heads of 128, four nodes of 32 heads: 31 us,
// 2.6 TB/s, 0.39 of what a plain copy reaches (36 us over 16 bits). Bound by latency:
// a warp has some 690 instructions for its 32 keys and sixteen rows, most of them in
// chains (codes in, products, exponentials), and the 16 warps that fit an SM fill 40 %
// of the issue slots. Two stages and four CTAs an SM / three and three: 32.1 / 35.5
// us; sixteen keys a warp, four stages and four CTAs: 36.8.
// More than 64 counted rows are staged anew, in blocks of 64, for every tile: 64
// rows (16 nodes) of the sequences above take 62 us, 128 173 and 252 315.
template <int DP>
__global__ void __launch_bounds__(kThreads, Cfg8<DP>::kCtas) k_kv_accumulate8(const __grid_constant__ AttendParams P) {
    using Cfg = Cfg8<DP>;
    using Cp = Copy8<DP, Cfg::kWarpKeys>;
    constexpr int KD = DP / 16, UNITS = Cp::UNITS, S = Cfg::kStages, MT = Cfg::kMT, WK = Cfg::kWarpKeys, KEYS = Cfg::kKeys;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + Cfg::kOffQ;
    unsigned long long* const word_s = reinterpret_cast<unsigned long long*>(smem + Cfg::kOffRow);
    float* const lse_s = reinterpret_cast<float*>(word_s + kRows);
    float* const factor_s = lse_s + kRows;
    int* const node_s = reinterpret_cast<int*>(factor_s + kRows);  // counted nodes, ascending; then their number
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;  // keys g, g + 8 of sixteen; rows 2c, 2c + 1 of each eight
    const int T = P.T, G = P.G, D = C.D;

    grid_launch_dependents();
    grid_dependency_wait();
    make_plan<kThreads, 1, 0, KEYS>(C, T, C.Hkv, gridDim.x, plan, P.err, blockIdx.x == 0);
    const DealOf<KEYS> deal(plan, C.B, gridDim.x, 1);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);
    if (x0 >= x1) return;
    const int unit = lane % UNITS, own0 = warp * WK;
    const bool unit_on = unit * 16 < D, whole_rows = D == DP;
    const Cp cp(lane, own0);
    const Load8<DP> ld(lane, own0);
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks;

    SourceOf<uint8_t, KEYS> src;
    At a = locate<KEYS>(plan, C.B, x0);
    src.at = a, src.x = x0, src.x1 = x1;
    const uint32_t ring = smem_u32(smem);
    int stage_in = 0, held = kNoSlot;  // lane i: the slot of the warp's key i (of sixteen: i % 16) of the tile to be issued next
    int pend[S - 1], pend_byte[S - 1];  // stages that wait for their scales, and this lane's: the oldest first
#pragma unroll
    for (int i = 0; i < S - 1; ++i) pend[i] = -1, pend_byte[i] = 0;
    auto fetch = [&]() {
        held = slot_of(src.list, src.at.tile * KEYS + own0 + lane % WK, src.tot, src.tot, 0);
    };
    auto issue = [&]() {
        // The scales of the tile that is read next, which have had the time of S - 1 tiles to arrive.
        if (pend[0] >= 0 && (WK == 32 || lane < WK))
            reinterpret_cast<float*>(smem + pend[0] * Cfg::kStage + Cfg::kOffKey + KEYS * 8)[own0 + lane] =
                scale_of(pend_byte[0], C.e_lo, C.e_hi);
#pragma unroll
        for (int i = 0; i + 1 < S - 1; ++i) pend[i] = pend[i + 1], pend_byte[i] = pend_byte[i + 1];
        pend[S - 2] = -1;
        if (src.x < x1) {
            const uint8_t* kp = src.k + unit * 16;
            const uint32_t dst = ring + stage_in * Cfg::kStage;
            const bool ok = slot_ok(held, n_slots, P.err);
            const int mine = ok ? held : 0;  // keys past the end are read from slot 0 and not counted
            int slot[Cp::SWEEPS];
            Cp::slots(mine, lane, slot);
            if (whole_rows) {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + cp.place(j), kp + (long long)slot[j] * k_step);
            } else {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + cp.place(j),
                         unit_on ? kp + (long long)slot[j] * k_step : src.k, unit_on);
            }
            if (WK == 32 || lane < WK) {
                int* at = reinterpret_cast<int*>(smem + stage_in * Cfg::kStage + Cfg::kOffKey) + own0 + lane;
                *at = ok ? held : -1;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(at + KEYS)),
                             "l"(src.acc + mine), "r"(ok ? 4 : 0)
                             : "memory");
                pend_byte[S - 2] = src.k_scale[mine >> C.block_shift];
            }
            pend[S - 2] = stage_in;
            if (++stage_in == S) stage_in = 0;
            if (src.next(plan, C.B, C.Hkv) && src.x < x1) src.enter(C, plan, 1);
            if (src.x < x1) fetch();
        }
        cp_commit();
    };
    // The first slots, and the second tile's where they are of the same list, go out together.
    src.enter(C, plan, 1);
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
    issue();
    if (two) held = second_slot;
#pragma unroll 1
    for (int s = 1; s < S - 1; ++s) issue();

    int have_b = -1, have_h = -1, have_block = -1, n_rows = 0, stage_out = 0;
    bool steep = false;  // of the rows that are staged
    for (int x = x0; x < x1; ++x, step<KEYS>(plan, C.B, C.Hkv, a)) {
        const int b = a.b, h = a.group, len = plan.len[b], tot = plan.tot[b];  // tot = 0: nothing counts
        if (have_b != b) {
            // counted nodes of this sequence
            __syncthreads();
            if (warp == 0) {
                const unsigned long long want = P.rows ? P.rows[b] : ~0ull;
                int n = 0;
                for (int t0 = 0; t0 < T; t0 += 32) {
                    const int t = t0 + lane;
                    const bool on = t < T && (want >> (t & 63) & 1) && word_of(P.mask, T, b, t) != 0 && tot > 0;
                    const unsigned who = __ballot_sync(0xFFFFFFFFu, on);
                    if (on) node_s[n + __popc(who & lanemask_lt())] = t;
                    n += __popc(who);
                }
                if (lane == 0) node_s[kRows] = n;
            }
            __syncthreads();
            n_rows = node_s[kRows] * G;
            have_b = b;
            have_h = -1;
        }
        // queries r0 .. r0 + nr - 1 of those that count
        auto stage_rows = [&](int r0, int nr) {
            if (have_h == h && have_block == r0) return;
            __syncthreads();
            const int padded = (nr + 15) & ~15;
            constexpr int AT_ONCE = 32 / (DP / 8);
            bool far = false;
            for (int base = warp * AT_ONCE; base < padded; base += 4 * AT_ONCE) {
                const int r = base + lane / (DP / 8), u = lane % (DP / 8);
                const bool on = r < nr;
                const int nth = div_of(r0 + r, G), t = on ? node_s[nth] : 0, gq = r0 + r - nth * G;
                const uint16_t* from = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)(h * G + gq) * P.qh;
                float down;
                const uint4 val = query_half<DP>(query_load<DP>(on ? from : nullptr, D, lane), C.fp16, down);
                if (r < padded) {
                    *reinterpret_cast<uint4*>(q_s + r * Cfg::kQRow + u * 16) = val;
                    if (u == 0) {
                        float lse = INFINITY;  // a padding row: exp(-inf) = 0
                        if (on) lse = P.lse[((long long)b * T + t) * P.Hq + h * G + gq];
                        // a row that saw nothing gives nothing
                        lse_s[r] = lse == -INFINITY ? INFINITY : lse;
                        word_s[r] = on ? word_of(P.mask, T, b, t) : 0;
                        factor_s[r] = down;
                        far |= down > kSteep;
                    }
                }
            }
            have_h = h;
            have_block = r0;
            steep = __syncthreads_or(far);
        };
        if (n_rows > 0) stage_rows(0, min(kRows, n_rows));
        cp_wait<S - 2>();
        __syncwarp();  // the tile before has been read by every lane
        issue();
        __syncwarp();
        uint8_t* const stage = smem + stage_out * Cfg::kStage;
        if (++stage_out == S) stage_out = 0;
        const uint32_t k_s = smem_u32(stage);
        uint32_t kf[MT][KD][4];
        const float* key_s = reinterpret_cast<const float*>(stage + Cfg::kOffKey);  // slots, old weights, scales
        float sk[MT][2], w[MT][2];  // of keys g and g + 8
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            sk[m][0] = key_s[2 * KEYS + own0 + m * 16 + g], sk[m][1] = key_s[2 * KEYS + own0 + m * 16 + g + 8];
            w[m][0] = w[m][1] = 0.0f;
#pragma unroll
            for (int u = 0; u < KD; u += 2) {
                uint32_t r[4];
                ldsm4(r, k_s + ld.place(u, m));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    halves4(r[2 * i], kf[m][u + i][0], kf[m][u + i][2]);
                    halves4(r[2 * i + 1], kf[m][u + i][1], kf[m][u + i][3]);
                }
            }
        }
        const int i0 = a.tile * KEYS + own0;
        const bool edge = i0 + WK > len;
        for (int r0 = 0; r0 < n_rows; r0 += kRows) {
            const int nr = min(kRows, n_rows - r0);
            if (n_rows > kRows) stage_rows(r0, nr);
            // 16 rows at a time, or the last 8: several chains of products
            auto rows = [&](int n, auto tiles) {
                constexpr int NT = decltype(tiles)::value, CHAINS = NT == 1 ? 2 : 1;
                float s[CHAINS][MT][NT][4] = {};
                const uint8_t* q_at = q_s + (n + g) * Cfg::kQRow + c * 8;
#pragma unroll
                for (int u = 0; u < KD; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint2 q = *reinterpret_cast<const uint2*>(q_at + t * 8 * Cfg::kQRow + u * 32);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            mma16(s[u % CHAINS][m][t], kf[m][u][0], kf[m][u][1], kf[m][u][2], kf[m][u][3], q.x, q.y);
                    }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int r = n + t * 8 + c * 2;
                    const float2 lse = *reinterpret_cast<const float2*>(lse_s + r), whole = *reinterpret_cast<const float2*>(factor_s + r);
                    const float2 down = make_float2(fminf(whole.x, kSteep), fminf(whole.y, kSteep));
                    // The difference is taken before the base's factor, and of the rounded product, as lse was: scores of
                    // the type's lowest value then differ from lse by 0.
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            uint64_t z2 = both(s[0][m][t][e], s[0][m][t][e + 1]);
                            if (CHAINS == 2) z2 = add2(z2, both(s[CHAINS - 1][m][t][e], s[CHAINS - 1][m][t][e + 1]));
                            z2 = mul2(mul2(z2, both(down.x, down.y)), both(sk[m][e >> 1], sk[m][e >> 1]));
                            split(z2, p[e], p[e + 1]);
                        }
                        if (steep) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[e] *= rest_of(factor_s[r + (e & 1)]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = __fadd_rn(__fmul_rn(p[e], P.scale), e & 1 ? -lse.y : -lse.x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = ex2(p[e] * kLog2e);
                        if (n + NT * 8 > nr) {  // a padding row's zeros meet what a key holds, and 0 * NaN is NaN
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (r + (e & 1) >= nr) p[e] = 0.0f;
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = i0 + m * 16 + g + (e >> 1) * 8 - len;
                                if (!(j < 0 || (j < T && (word_s[r + (e & 1)] >> (j & 63) & 1)))) p[e] = 0.0f;
                            }
                        }
                        w[m][0] += p[0] + p[1], w[m][1] += p[2] + p[3];
                    }
                }
            };
            int n = 0;
            for (; n + 8 < nr; n += 16) rows(n, std::integral_constant<int, 2>());
            if (n < nr) rows(n, std::integral_constant<int, 1>());
        }
        float* out = P.acc_out + b * C.ab + h * C.ah;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[m][e] += __shfl_xor_sync(0xFFFFFFFFu, w[m][e], 1);
                w[m][e] += __shfl_xor_sync(0xFFFFFFFFu, w[m][e], 2);
            }
        // the four lanes that have a key's sum share the keys out
        if (c < 2 * MT) {
            const float sum = MT == 1 ? (c & 1 ? w[0][1] : w[0][0])
                                      : c & 2 ? (c & 1 ? w[MT - 1][1] : w[MT - 1][0]) : (c & 1 ? w[0][1] : w[0][0]);
            const int key = own0 + (c >> 1) * 16 + (c & 1) * 8 + g, slot = reinterpret_cast<const int*>(key_s)[key];
            if (slot >= 0) out[slot] = key_s[KEYS + key] + sum;
        }
    }
    cp_wait<0>();
}

template <int DP>
cudaError_t launch_weigh(const AttendParams& P, cudaStream_t st) {
    using Cfg = Cfg8<DP>;
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const auto kern = k_kv_accumulate8<DP>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    void* args[1] = {const_cast<AttendParams*>(&P)};
    return launch(reinterpret_cast<const void*>(kern), dim3(sms * Cfg::kCtas, 1, 1), kThreads, Cfg::smem(P.c.B), args, st);
}

}  // namespace

cudaError_t launch_kv_accumulate8(const AttendParams& P, cudaStream_t st) {
    if (P.c.D <= 64) return launch_weigh<64>(P, st);
    return P.c.D <= 128 ? launch_weigh<128>(P, st) : launch_weigh<256>(P, st);
}

}  // namespace si
