// weigh.cu -- the attention weight that each cached key received.
#include "attend.cuh"

namespace si {

namespace {

constexpr int kThreads = 128;  // four warps

int per_sm(int dp) { return dp <= 128 ? 3 : 1; }
int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Rows kept in shared memory at once.
constexpr int kWeighRows = 64;

template <int DP>
struct WeighCfg {
    static constexpr int kTile = KT * DP * 2;
    static constexpr int kStages = DP <= 128 ? 3 : 4;
    static constexpr int kOffQ = kStages * kTile;
    static constexpr int kOffRow = kOffQ + kWeighRows * DP * 2;      // per row: ancestor word, lse; the counted nodes
    static constexpr int kOffKey = kOffRow + kWeighRows * (8 + 4 + 4) + 16;  // per stage and key: slot, acc
    static constexpr int kOffPlan = kOffKey + kStages * KT * 8;
    static constexpr int smem(int B) { return kOffPlan + Plan::words(B) * 4; }
};

// acc_out[slot] = acc[slot] + sum over counted rows of exp(scale * q.k - lse).
// Keys are the m side of the matrix product and rows the n side, so that a
// thread sums its keys' weights over the rows in registers. Reads K once; a
// key belongs to one warp, which also copies it and its old weight, so warps
// only meet when the list (and with it the queries) changes. 8 sequences of up
// to 16384 keys, 8 heads of 128, four nodes of 32 heads: 36 us, 4.4 TB/s, 0.65
// of what a plain copy reaches; bound by issue (47 % of the slots with the 12
// warps that fit an SM; 42 us with eight). Above 64 counted rows a key the
// queries take turns in shared memory, a block of 64 after another for every
// tile (the same lists: 64 rows 62 us, 128 rows 210).
template <int DP, bool FP16>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 3 : 1) k_kv_accumulate(const __grid_constant__ AttendParams P) {
    using Cfg = WeighCfg<DP>;
    using Cp = Copy<DP>;
    constexpr int KD = DP / 16;
    constexpr int UNITS = Cp::UNITS;
    constexpr int S = Cfg::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + Cfg::kOffQ;
    unsigned long long* word_s = reinterpret_cast<unsigned long long*>(smem + Cfg::kOffRow);
    float* lse_s = reinterpret_cast<float*>(word_s + kWeighRows);
    int* node_s = reinterpret_cast<int*>(lse_s + kWeighRows);  // counted nodes, ascending; then their number
    int* slot_s = reinterpret_cast<int*>(smem + Cfg::kOffKey);  // [stage][key]
    float* old_s = reinterpret_cast<float*>(slot_s + S * KT);
    const Plan plan(reinterpret_cast<int*>(smem + Cfg::kOffPlan), P.c.B);

    const KvView& C = P.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = P.T, G = P.G, D = C.D;

    grid_launch_dependents();
    grid_dependency_wait();
    make_plan<kThreads, 1, 0>(C, T, C.Hkv, gridDim.x, plan, P.err, blockIdx.x == 0);
    const Deal deal(plan, C.B, gridDim.x, 1);
    int x0, x1;
    deal.range(blockIdx.x, x0, x1);
    if (x0 >= x1) return;
    const int unit = lane % UNITS;
    const bool unit_on = unit * 8 < D;
    const int n_slots = (int)C.n_slots, k_step = (int)C.ks;

    Source src;
    src.start(plan, C.B, x0, x1);
    const bool whole_rows = D == DP;
    const uint32_t ring = smem_u32(smem);
    int stage_in = 0, held = kNoSlot;  // lane i < 16: the slot of the warp's key i of the tile to be issued next
    auto fetch = [&]() {
        held = slot_of(src.list, src.at.tile * KT + warp * 16 + (lane & 15), src.tot, src.tot, 0);
    };
    auto issue = [&]() {
        if (src.x < x1) {
            const uint16_t* kp = src.k + unit * 8;
            const uint32_t dst = ring + stage_in * Cfg::kTile;
            const bool ok = slot_ok(held, n_slots, P.err);
            if (lane < 16) {
                const int at = stage_in * KT + warp * 16 + lane;
                slot_s[at] = ok ? held : -1;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(old_s + at)),
                             "l"(src.acc + (ok ? held : 0)), "r"(ok ? 4 : 0)
                             : "memory");
            }
            int slot[Cp::SWEEPS];
            Cp::slots(ok ? held : 0, lane, slot);  // keys past the end are read from slot 0 and not counted
            if (whole_rows) {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + tile_at<DP>(warp * 16 + Cp::row(lane, j), unit), kp + (long long)slot[j] * k_step);
            } else {
#pragma unroll
                for (int j = 0; j < Cp::SWEEPS; ++j)
                    cp16(dst + tile_at<DP>(warp * 16 + Cp::row(lane, j), unit),
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
    int have_b = -1, have_h = -1, have_block = -1, out_h = -1, n_rows = 0, stage_out = 0;
    float* out = nullptr;
    for (int x = x0; x < x1; ++x, step(plan, C.B, C.Hkv, a)) {
        cp_wait<S - 2>();
        __syncwarp();
        issue();
        const int b = a.b, h = a.group, len = plan.len[b], tot = plan.tot[b];  // tot = 0: nothing counts
        const int stage = stage_out;
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
                if (lane == 0) node_s[64] = n;
            }
            __syncthreads();
            n_rows = node_s[64] * G;
            have_b = b;
            have_h = out_h = -1;
        }
        if (out_h != h) {
            out = P.acc_out + b * C.ab + h * C.ah;
            out_h = h;
        }
        const uint32_t k_s = ring + stage * Cfg::kTile, q_addr = smem_u32(q_s);
        uint32_t kf[DP <= 128 ? KD : 1][4];
        if (DP <= 128) {
#pragma unroll
            for (int k = 0; k < KD; ++k)
                ldsm4(kf[DP <= 128 ? k : 0], k_s + tile_at<DP>(warp * 16 + (lane & 15), 2 * k + (lane >> 4)));
        }
        float w[2] = {0.0f, 0.0f};  // keys lane/4 and lane/4 + 8 of the warp's sixteen
        const int i0 = a.tile * KT + warp * 16 + (lane >> 2);
        for (int r0 = 0; r0 < n_rows; r0 += kWeighRows) {
            const int nr = min(kWeighRows, n_rows - r0);
            if (have_h != h || have_block != r0) {
                __syncthreads();
                const int padded = (nr + 15) & ~15;
                for (int i = tid; i < padded * UNITS; i += kThreads) {
                    const int r = i / UNITS, u = i % UNITS;
                    uint4 val = make_uint4(0, 0, 0, 0);
                    if (r < nr && u * 8 < D) {
                        const int t = node_s[(r0 + r) / G], g = (r0 + r) % G;
                        val = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q) + b * P.qb + t * P.qt +
                                                              (long long)(h * G + g) * P.qh + u * 8);
                    }
                    *reinterpret_cast<uint4*>(q_s + tile_at<DP>(r, u)) = val;
                }
                for (int r = tid; r < padded; r += kThreads) {
                    float lse = INFINITY;  // a padding row: exp(-inf) = 0
                    unsigned long long word = 0;
                    if (r < nr) {
                        const int t = node_s[(r0 + r) / G], g = (r0 + r) % G;
                        lse = P.lse[((long long)b * T + t) * P.Hq + h * G + g];
                        word = word_of(P.mask, T, b, t);
                    }
                    // a row that saw nothing gives nothing
                    lse_s[r] = lse == -INFINITY ? INFINITY : lse;
                    word_s[r] = word;
                }
                have_h = h;
                have_block = r0;
                __syncthreads();
            }
            const bool edge = a.tile * KT + warp * 16 + 16 > len;
            for (int n = 0; n < nr; n += 16) {  // two chains of products
                float s[2][4] = {};
#pragma unroll
                for (int k = 0; k < KD; k += 2) {
                    // rows n .. n+7 and n+8 .. n+15, d 32 wide: two k steps
                    uint32_t qa[4], qb[4];
                    ldsm4(qa, q_addr + tile_at<DP>(n + (lane & 7), 2 * k + (lane >> 3)));
                    ldsm4(qb, q_addr + tile_at<DP>(n + 8 + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t kx[4];
                        if (DP > 128) ldsm4(kx, k_s + tile_at<DP>(warp * 16 + (lane & 15), 2 * (k + kk) + (lane >> 4)));
                        const uint32_t(&ka)[4] = DP > 128 ? kx : kf[DP <= 128 ? k + kk : 0];
                        mma<FP16>(s[0], ka, qa[2 * kk], qa[2 * kk + 1]);
                        mma<FP16>(s[1], ka, qb[2 * kk], qb[2 * kk + 1]);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = n + c * 8 + (lane & 3) * 2;
                    const float2 lse = *reinterpret_cast<const float2*>(lse_s + r);
                    // The difference is taken before the base's factor, and of the rounded product, as lse was: scores of
                    // the type's lowest value then differ from lse by 0, where s * (scale * log2 e) would be off by a
                    // rounding of that size, and its power of two 0 or infinite.
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = ex2(__fadd_rn(__fmul_rn(s[c][e], P.scale), e & 1 ? -lse.y : -lse.x) * kLog2e);
                        // a padding row's zeros meet what a key holds, and 0 * infinity is NaN
                        if (n + 16 > nr && r + (e & 1) >= nr) p = 0.0f;
                        if (edge) {
                            const int j = i0 + (e >> 1) * 8 - len;
                            if (!(j < 0 || (j < T && (word_s[r + (e & 1)] >> (j & 63) & 1)))) p = 0.0f;
                        }
                        w[e >> 1] += p;
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w[e] += __shfl_xor_sync(0xFFFFFFFFu, w[e], 1);
            w[e] += __shfl_xor_sync(0xFFFFFFFFu, w[e], 2);
            const int key = stage * KT + warp * 16 + (lane >> 2) + e * 8;
            const int slot = slot_s[key];
            if ((lane & 3) == 0 && slot >= 0) out[slot] = old_s[key] + w[e];
        }
    }
    cp_wait<0>();
}

template <int DP, bool FP16>
cudaError_t launch_weigh(const AttendParams& P, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    const auto kern = k_kv_accumulate<DP, FP16>;
    cudaError_t e = allow_max_smem(kern);
    if (e != cudaSuccess) return e;
    void* args[1] = {const_cast<AttendParams*>(&P)};
    return launch(reinterpret_cast<const void*>(kern), dim3(sms * per_sm(DP), 1, 1), kThreads,
                  WeighCfg<DP>::smem(P.c.B), args, st);
}

template <bool FP16>
cudaError_t launch_weigh_type(const AttendParams& P, cudaStream_t st) {
    switch (padded(P.c.D)) {
        case 64: return launch_weigh<64, FP16>(P, st);
        case 128: return launch_weigh<128, FP16>(P, st);
        default: return launch_weigh<256, FP16>(P, st);
    }
}

}  // namespace

cudaError_t launch_kv_accumulate(const AttendParams& P, cudaStream_t st) {
    return P.c.fp16 ? launch_weigh_type<true>(P, st) : launch_weigh_type<false>(P, st);
}

}  // namespace si
