// weigh8.cu -- the attention weight that each key of a cache of e4m3 codes received.
#include "attend.cuh"
#include "kv8.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps of sixteen keys of a tile
constexpr int kKeys = 16;
constexpr int kRows = 64;      // kept in shared memory at once

template <int DP>
struct Cfg8 {
    static constexpr int kTile = KT * DP;
    static constexpr int kOffKey = kTile;                     // in a stage: slots, old weights, scales of its keys
    static constexpr int kStage = kTile + KT * 12;
    static constexpr int kStages = 4;
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
template <int DP>
__global__ void __launch_bounds__(kThreads, Cfg8<DP>::kCtas) k_kv_accumulate8(const __grid_constant__ AttendParams P) {
    using Cfg = Cfg8<DP>;
    using Cp = Copy8<DP>;
    constexpr int KD = DP / 16, UNITS = Cp::UNITS, S = Cfg::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + Cfg::kOffQ;
    unsigned long long* const word_s = reinterpret_cast<unsigned long long*>(smem + Cfg::kOffRow);
    float* const lse_s = reinterpret_cast<float*>(word_s + kRows);
    float* const factor_s = lse_s + kRows;
    int* const node_s = reinterpret_cast<int*>(factor_s + kRows);  // counted nodes, ascending; then their number
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;  // keys g, g + 8; rows 2c, 2c + 1 of each eight
    const int T = P.T, G = P.G, D = C.D;

    grid_launch_dependents();
    grid_dependency_wait();
    make_plan<kThreads, 1, 0>(C, T, C.Hkv, gridDim.x, plan, P.err, blockIdx.x == 0);
    const Deal deal(plan, C.B, gridDim.x, 1);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);
    if (x0 >= x1) return;
    const int unit = lane % UNITS, own0 = warp * kKeys;
    const bool unit_on = unit * 16 < D, whole_rows = D == DP;
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks;

    SourceOf<uint8_t> src;
    src.start(plan, C.B, x0, x1);
    const uint32_t ring = smem_u32(smem);
    int stage_in = 0, held = kNoSlot;  // lanes i and i + 16: the slot of the warp's key i of the tile to be issued next
    int pend = -1, pend_byte = 0;      // the stage that waits for its scales, and this lane's
    auto fetch = [&]() {
        held = slot_of(src.list, src.at.tile * KT + own0 + (lane & 15), src.tot, src.tot, 0);
    };
    auto issue = [&]() {
        if (pend >= 0) {  // the scales of the tile before have had a tile's time to arrive
            if (lane < 16)
                reinterpret_cast<float*>(smem + pend * Cfg::kStage + Cfg::kOffKey + KT * 8)[own0 + lane] =
                    scale_of(pend_byte, C.e_lo, C.e_hi);
            pend = -1;
        }
        if (src.x < x1) {
            const uint8_t* kp = src.k + unit * 16;
            const uint32_t dst = ring + stage_in * Cfg::kStage;
            const bool ok = slot_ok(held, n_slots, P.err);
            if (lane < 16) {
                int* at = reinterpret_cast<int*>(smem + stage_in * Cfg::kStage + Cfg::kOffKey) + own0 + lane;
                *at = ok ? held : -1;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(at + KT)),
                             "l"(src.acc + (ok ? held : 0)), "r"(ok ? 4 : 0)
                             : "memory");
                pend_byte = src.k_scale[(ok ? held : 0) >> C.block_shift];
            }
            pend = stage_in;
            int slot[Cp::SWEEPS];
            Cp::slots(ok ? held : 0, lane, slot);  // keys past the end are read from slot 0 and not counted
            if (whole_rows) {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + tile8_at<DP>(own0 + Cp::row(lane, j), unit), kp + (long long)slot[j] * k_step);
            } else {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + tile8_at<DP>(own0 + Cp::row(lane, j), unit),
                         unit_on ? kp + (long long)slot[j] * k_step : src.k, unit_on);
            }
            if (++stage_in == S) stage_in = 0;
            if (src.next(plan, C.B, C.Hkv) && src.x < x1) src.enter(C, plan, 1);
            if (src.x < x1) fetch();
        }
        cp_commit();
    };
    src.enter(C, plan, 1);
    fetch();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) issue();

    At a = locate(plan, C.B, x0);
    int have_b = -1, have_h = -1, have_block = -1, n_rows = 0, stage_out = 0;
    for (int x = x0; x < x1; ++x, step(plan, C.B, C.Hkv, a)) {
        cp_wait<S - 2>();
        __syncwarp();
        issue();
        const int b = a.b, h = a.group, len = plan.len[b], tot = plan.tot[b];  // tot = 0: nothing counts
        uint8_t* const stage = smem + stage_out * Cfg::kStage;
        if (++stage_out == S) stage_out = 0;
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
        const uint32_t k_s = smem_u32(stage);
        uint32_t kf[KD][4];
        const float* key_s = reinterpret_cast<const float*>(stage + Cfg::kOffKey);  // slots, old weights, scales
        const float sk0 = key_s[2 * KT + own0 + g], sk1 = key_s[2 * KT + own0 + g + 8];
#pragma unroll
        for (int u = 0; u < KD; u += 2) {
            uint32_t r[4];
            ldsm4(r, k_s + tile8_at<DP>(own0 + (lane & 15), u + (lane >> 4)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                halves4(r[2 * i], kf[u + i][0], kf[u + i][2]);
                halves4(r[2 * i + 1], kf[u + i][1], kf[u + i][3]);
            }
        }
        float w[2] = {0.0f, 0.0f};  // keys g and g + 8
        const int i0 = a.tile * KT + own0;
        const bool edge = i0 + kKeys > len;
        for (int r0 = 0; r0 < n_rows; r0 += kRows) {
            const int nr = min(kRows, n_rows - r0);
            if (have_h != h || have_block != r0) {
                __syncthreads();
                const int padded = (nr + 7) & ~7;
                constexpr int AT_ONCE = 32 / (DP / 8);
                for (int base = warp * AT_ONCE; base < padded; base += 4 * AT_ONCE) {
                    const int r = base + lane / (DP / 8), u = lane % (DP / 8);
                    const bool on = r < nr;
                    const int t = on ? node_s[(r0 + r) / G] : 0, gq = (r0 + r) % G;
                    const uint16_t* from = static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt + (long long)(h * G + gq) * P.qh;
                    float down;
                    const uint4 val = query_unit<DP>(on ? from : nullptr, D, C.fp16, lane, down);
                    if (r < padded) {
                        *reinterpret_cast<uint4*>(q_s + r * Cfg::kQRow + u * 16) = val;
                        if (u == 0) {
                            float lse = INFINITY;  // a padding row: exp(-inf) = 0
                            if (on) lse = P.lse[((long long)b * T + t) * P.Hq + h * G + gq];
                            // a row that saw nothing gives nothing
                            lse_s[r] = lse == -INFINITY ? INFINITY : lse;
                            word_s[r] = on ? word_of(P.mask, T, b, t) : 0;
                            factor_s[r] = down;
                        }
                    }
                }
                have_h = h;
                have_block = r0;
                __syncthreads();
            }
            for (int n = 0; n < nr; n += 8) {
                float s[4] = {};
                const uint8_t* q_at = q_s + (n + g) * Cfg::kQRow + c * 8;
#pragma unroll
                for (int u = 0; u < KD; ++u) {
                    const uint2 q = *reinterpret_cast<const uint2*>(q_at + u * 32);
                    mma16(s, kf[u][0], kf[u][1], kf[u][2], kf[u][3], q.x, q.y);
                }
                const int r = n + c * 2;
                const float2 lse = *reinterpret_cast<const float2*>(lse_s + r), down = *reinterpret_cast<const float2*>(factor_s + r);
                // The difference is taken before the base's factor, and of the rounded product, as lse was: scores of
                // the type's lowest value then differ from lse by 0.
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = s[e] * (e & 1 ? down.y : down.x) * (e < 2 ? sk0 : sk1);
                    float p = ex2(__fadd_rn(__fmul_rn(z, P.scale), e & 1 ? -lse.y : -lse.x) * kLog2e);
                    // a padding row's zeros meet what a key holds, and 0 * NaN is NaN
                    if (n + 8 > nr && r + (e & 1) >= nr) p = 0.0f;
                    if (edge) {
                        const int j = i0 + g + (e >> 1) * 8 - len;
                        if (!(j < 0 || (j < T && (word_s[r + (e & 1)] >> (j & 63) & 1)))) p = 0.0f;
                    }
                    w[e >> 1] += p;
                }
            }
        }
        float* out = P.acc_out + b * C.ab + h * C.ah;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w[e] += __shfl_xor_sync(0xFFFFFFFFu, w[e], 1);
            w[e] += __shfl_xor_sync(0xFFFFFFFFu, w[e], 2);
            const int key = own0 + g + e * 8, slot = reinterpret_cast<const int*>(key_s)[key];
            if (c == 0 && slot >= 0) out[slot] = key_s[KT + key] + w[e];
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
