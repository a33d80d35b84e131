// logprobs.cu -- log probabilities, entropy and best alternatives of rows of logits.
#include <climits>

#include "attend.cuh"

namespace si {

namespace {

constexpr int kThreads = 256;

template <int DTYPE>
__device__ __forceinline__ float logit(const void* row, long long i) {
    if (DTYPE == SI_FP32) return static_cast<const float*>(row)[i];
    return widen<DTYPE == SI_FP16>(static_cast<const uint16_t*>(row)[i]);
}

// Larger logit <=> larger key, -0 and +0 alike, every NaN the same and above all; then the lower id.
__device__ __forceinline__ unsigned long long order_of(float x, int id) {
    const uint32_t key = x != x ? 0xFFFFFFFFu : value_key(x);
    return (unsigned long long)key << 32 | (uint32_t)~id;
}

template <class T, class F>
__device__ T block_reduce(T v, F f, T* shared) {
    __syncthreads();
    shared[threadIdx.x] = v;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) shared[threadIdx.x] = f(shared[threadIdx.x], shared[threadIdx.x + o]);
        __syncthreads();
    }
    return shared[0];
}

// A block a row: the maximum, the sums, the tokens, then the largest logits one after another.
template <int DTYPE>
__global__ void __launch_bounds__(kThreads) k_token_logprobs(const __grid_constant__ LogprobsParams P) {
    __shared__ float shared[kThreads];
    __shared__ unsigned long long best_s[kThreads];
    grid_launch_dependents();
    grid_dependency_wait();
    const long long n = blockIdx.x;
    const void* row = static_cast<const uint8_t*>(P.x) + n * P.stride * (DTYPE == SI_FP32 ? 4 : 2);
    const int tid = threadIdx.x;
    auto add = [](float a, float b) { return a + b; };
    float top = -INFINITY;
    for (long long i = tid; i < P.V; i += kThreads) top = fmaxf(top, logit<DTYPE>(row, i));
    top = block_reduce(top, [](float a, float b) { return fmaxf(a, b); }, shared);
    float s = 0.0f, u = 0.0f;  // sums of exp(z) and of z exp(z), z = (x - top) / temperature
    for (long long i = tid; i < P.V; i += kThreads) {
        const float x = logit<DTYPE>(row, i);
        const float z = x == top ? top == INFINITY ? NAN : 0.0f : (x - top) * P.inv_t;
        const float p = top == -INFINITY && x == x ? 0.0f : expf(z);
        s += p;
        if (p != 0.0f) u += p * z;
    }
    s = block_reduce(s, add, shared);
    u = block_reduce(u, add, shared);
    const bool none = top == -INFINITY && s == 0.0f;
    const float rest = logf(s);
    auto logp_of = [&](float x) { return none ? -INFINITY : x == top && s == s ? -rest : (x - top) * P.inv_t - rest; };
    if (tid == 0 && P.entropy) P.entropy[n] = none ? 0.0f : rest - u / s;
    for (int m = tid; m < P.M; m += kThreads) {
        const int id = P.targets[n * P.M + m];
        P.logp[n * P.M + m] = id >= 0 && id < P.V ? logp_of(logit<DTYPE>(row, id)) : -INFINITY;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < P.K; ++k) {
        unsigned long long best = 0;
        for (long long i = tid; i < P.V; i += kThreads) {
            const unsigned long long o = order_of(logit<DTYPE>(row, i), (int)i);
            if (o < last || k == 0) best = max(best, o);
        }
        last = block_reduce(best, [](unsigned long long a, unsigned long long b) { return max(a, b); }, best_s);
        const int id = (int)~(uint32_t)last;
        if (tid == 0) {
            P.top_ids[n * P.K + k] = id;
            P.top_logp[n * P.K + k] = logp_of(logit<DTYPE>(row, id));
        }
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobsParams& P, cudaStream_t st) {
    void* args[1] = {const_cast<LogprobsParams*>(&P)};
    const void* fn = P.dtype == SI_FP32   ? reinterpret_cast<const void*>(&k_token_logprobs<SI_FP32>)
                     : P.dtype == SI_FP16 ? reinterpret_cast<const void*>(&k_token_logprobs<SI_FP16>)
                                          : reinterpret_cast<const void*>(&k_token_logprobs<SI_BF16>);
    return launch(fn, dim3(P.N, 1, 1), kThreads, 0, args, st);
}

}  // namespace si
