// kv.h -- launcher interface of the key/value cache between its C ABI
// (kv_api.cu) and its kernels (kv.cu, attend.cu, attend_wide.cu, weigh.cu; append8.cu,
// attend8.cu, weigh8.cu for a cache in 8 bits; logprobs.cu).
// Not installed; not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace si {

// One layer of a cache, as the kernels see it. Strides in elements.
struct KvView {
    const void* k;
    const void* v;
    long long kb, kh, ks;     // sequence, head, slot
    long long vb, vh, vs;
    const int32_t* table;     // nullptr: entry i is slot i
    long long tb, th;
    const int32_t* len;       // [B]
    float* acc;
    long long ab, ah;
    long long n_slots;
    int B, Hkv, D, cap, fp16;
    // A cache of e4m3 codes: fp16 is then the type of q and out alone, and slot s has the scale byte s >> block_shift
    // of its head, taken within [e_lo, e_hi].
    int e4m3, block_shift, e_lo, e_hi;
    uint8_t* k_scale;
    uint8_t* v_scale;
    long long kcb, kch, vcb, vch;  // sequence, head
};

constexpr int kRopeMaxPairs = 128;
// Turns per position of each pair, 0.64 fixed point (wraps modulo one turn).
struct RopeTable {
    unsigned long long turn[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];
    int n_pairs, n_axes, interleaved;
};

struct KvAppendParams {
    KvView c;
    int T, Hq;
    const void *q, *k, *v;
    long long qb, qt, qh, kb, kt, kh, vb, vt, vh;  // sequence, token, head
    const int32_t* pos;       // [B][T][n_axes]
    void* q_out;              // [B][T][Hq][D]
    unsigned* err;
};
cudaError_t launch_kv_append(const KvAppendParams& P, const RopeTable& R, cudaStream_t st);
// append8.cu: the same into a cache of e4m3 codes
cudaError_t launch_kv_append8(const KvAppendParams& P, const RopeTable& R, cudaStream_t st);

constexpr int kEvictMaxCap = 196608;
struct KvEvictParams {
    int32_t* table;           // [L][B][Hkv][cap], strides below
    long long tl, tb, th;
    int32_t* len;             // [L][B]
    const float* acc;
    long long al, ab, ah;
    int32_t* table_out;       // in place, or its own buffer with its own strides
    long long ol, ob, oh;
    int32_t* len_out;
    const int32_t* path;      // [B][T] or nullptr
    const int32_t* n_path;    // [B] or nullptr
    long long n_slots;
    int L, B, Hkv, cap, T, budget, sinks, recent;
    int in_place;
    unsigned* ticket;         // zero between launches; then L * B words for the new lengths
    unsigned* err;
};
cudaError_t launch_kv_evict(const KvEvictParams& P, cudaStream_t st);

struct AttendParams {
    KvView c;
    int T, Hq, G;
    const void* q;
    long long qb, qt, qh;
    const unsigned long long* mask;   // [B][T] or nullptr (chain)
    const unsigned long long* rows;   // accumulate: counted nodes [B] or nullptr (all)
    float scale;
    void* out;                // attention
    float* lse;               // attention: written (may be null); accumulate: read
    float* acc_out;           // accumulate (the cache's strides)
    float* part;              // attention: partial rows
    unsigned* done;           // attention over codes: launches by CTA, then sets of counters of a list's parts by its first CTA; zero at first
    unsigned* err;
};
// Scratch floats that launch_tree_attention needs at most for heads of D elements (0: cannot query the device).
long long attend_partial_floats(int D);
// Whether the kernels' 32-bit counts hold every tile of 64 keys of every list's row blocks, and the join's blocks.
bool attend_counts_fit(const AttendParams& P);
cudaError_t launch_tree_attention(const AttendParams& P, cudaStream_t st);  // of either kind of cache
// attend_wide.cu: the first of the two kernels for many rows; says how it cut the work for the join.
cudaError_t launch_tree_attention_wide(const AttendParams& P, int* row_blocks, int* parts, cudaStream_t st);
cudaError_t launch_kv_accumulate(const AttendParams& P, cudaStream_t st);
// attend8.cu, weigh8.cu: attention of few rows a key, and weights, over a cache of e4m3 codes
cudaError_t launch_tree_attention8(const AttendParams& P, cudaStream_t st);
long long attend8_partial_floats(int D);
int attend8_counters();
cudaError_t launch_kv_accumulate8(const AttendParams& P, cudaStream_t st);

// logprobs.cu
struct LogprobsParams {
    const void* x;            // [N][V], row n at element n * stride
    long long stride;
    int dtype, N, V, M, K;
    float inv_t;              // 1 / temperature
    const int32_t* targets;   // [N][M] or nullptr
    float* logp;              // [N][M]
    float* entropy;           // [N] or nullptr
    float* top_logp;          // [N][K] or nullptr
    int32_t* top_ids;
};
cudaError_t launch_token_logprobs(const LogprobsParams& P, cudaStream_t st);

// api.cu: the device error word of the current device (allocated on first use)
int device_error_word(unsigned** out);

// api.cu: sets the message si_last_error_string() returns on this thread
void set_error_message(const char* msg);

}  // namespace si
