// kv_api.cu -- the C ABI of the key/value cache (declared in include/si.h):
// handles, argument validation and launches. The kernels are in kv.cu (append,
// evict), attend.cu and attend_wide.cu (tree attention), and weigh.cu (weights).
#include <cmath>
#include <cstring>
#include <new>
#include <string>

#include "../../include/si.h"
#include "kv.h"
#include <nvtx3/nvToolsExt.h>

namespace {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

int fail(int code, const char* msg) {
    si::set_error_message(msg);
    return code;
}

int cuda_fail(cudaError_t e, const char* what) {
    si::set_error_message((std::string(what) + ": " + cudaGetErrorString(e)).c_str());
    return e == cudaErrorMemoryAllocation ? SI_ERR_OOM : SI_ERR_CUDA;
}

bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &s) != cudaSuccess) return false;
    return s != cudaStreamCaptureStatusNone;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of an array of these extents. What stands at a dimension of one element is not looked at (tensors from
// elsewhere may hold anything there) and taken as 0.
struct Strides {
    long long at[4] = {};
    template <int N>
    Strides(const long long* s, const long long (&extents)[N]) {
        for (int i = 0; i < N; ++i) at[i] = extents[i] == 1 ? 0 : s[i];
    }
    bool whole_units() const {
        for (long long s : at)
            if (s < 0 || s % 8) return false;
        return true;
    }
};

}  // namespace

#define SI_TRACE(name) NvtxRange si_trace_range_(name)

struct si_rope {
    si::RopeTable t;
};

struct si_kv {
    si_kv_desc d;
    int device = -1;          // of the scratch, set with its first allocation
    float* part = nullptr;    // partial attention rows
    unsigned* ticket = nullptr;  // eviction: a ticket and L * B lengths
};

namespace {

// The scratch belongs to one device; calls with another current device are refused.
int on_device(si_kv* kv) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (kv->device < 0) kv->device = dev;
    if (kv->device != dev) return fail(SI_ERR_INVALID_ARG, "the cache handle belongs to another device");
    return SI_OK;
}

// The attention's scratch, for whatever this handle's calls may need: made once and kept, because a captured graph
// holds its address.
int make_part(si_kv* kv, cudaStream_t st) {
    if (kv->part) return SI_OK;
    const long long need = si::attend_partial_floats(kv->d.D);
    if (need <= 0) return fail(SI_ERR_CUDA, "cannot query the device for the attention grid");
    if (capturing(st)) return fail(SI_ERR_INVALID_ARG, "attention scratch must be made; call once before capture");
    const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&kv->part), (size_t)need * sizeof(float));
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        kv->part = nullptr;
        return fail(SI_ERR_OOM, "cudaMalloc failed for the attention scratch");
    }
    return SI_OK;
}

si::KvView view_of(const si_kv_desc& d, int layer) {
    si::KvView c = {};
    c.k = static_cast<const uint16_t*>(d.k) + layer * d.k_stride[0];
    c.v = static_cast<const uint16_t*>(d.v) + layer * d.v_stride[0];
    c.kb = d.k_stride[1], c.kh = d.k_stride[2], c.ks = d.k_stride[3];
    c.vb = d.v_stride[1], c.vh = d.v_stride[2], c.vs = d.v_stride[3];
    c.table = d.table ? d.table + layer * d.table_stride[0] : nullptr;
    c.tb = d.table_stride[1], c.th = d.table_stride[2];
    c.len = d.len + (long long)layer * d.B;
    c.acc = d.acc ? d.acc + layer * d.acc_stride[0] : nullptr;
    c.ab = d.acc_stride[1], c.ah = d.acc_stride[2];
    c.n_slots = d.n_slots;
    c.B = d.B, c.Hkv = d.Hkv, c.D = d.D, c.cap = d.cap;
    c.fp16 = d.dtype == SI_FP16;
    return c;
}

// radians / (2 pi) modulo one turn, in steps of 2^-64 (rounded): the product
// with an integer position then wraps to the exact fraction of a turn. The
// product of the double's 53-bit mantissa with 1 / (2 pi) to 192 bits is taken in
// integers, so every machine gets the same table.
unsigned long long turn_of(double radians) {
    static const unsigned long long inv_2pi[3] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull,
                                                  0x36D8A5664F10E410ull};
    int e = 0;
    const double m = std::frexp(std::fabs(radians), &e);
    const unsigned long long mant = (unsigned long long)std::ldexp(m, 53);  // |radians| = mant * 2^(e - 53)
    unsigned long long w[4];  // mant * inv_2pi, 192 fraction bits, most significant word first
    unsigned __int128 carry = 0;
    for (int i = 2; i >= 0; --i) {
        carry += (unsigned __int128)mant * inv_2pi[i];
        w[i + 1] = (unsigned long long)carry;
        carry >>= 64;
    }
    w[0] = (unsigned long long)carry;
    // bits of weight 2^-1 .. 2^-64 of w * 2^(e - 53): the word that ends 128 - (e - 53) bits above w's end
    const int shift = 128 - (e - 53) - 1;  // one bit lower, for the rounding
    if (shift >= 256) return 0;
    const int words = shift / 64, bits = shift % 64;
    auto at = [&](int k) { return k >= 0 && k < 4 ? w[3 - k] : 0ull; };
    unsigned long long lo = at(words) >> bits, hi = at(words + 1) >> bits;
    if (bits) lo |= at(words + 1) << (64 - bits), hi |= at(words + 2) << (64 - bits);
    const unsigned long long turn = ((lo >> 1) | (hi << 63)) + (lo & 1u);
    return radians < 0 ? 0ull - turn : turn;
}

// What si_tree_attention and si_kv_accumulate check alike.
int check_rows(const si_kv* kv, int layer, int T, int Hq, const void* q, const long long* q_stride, float scale) {
    if (!kv || !q || !q_stride) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    if (layer < 0 || layer >= kv->d.L) return fail(SI_ERR_INVALID_ARG, "layer outside the cache");
    if (T < 1 || T > 64) return fail(SI_ERR_INVALID_ARG, "need 1 <= T <= 64");
    if (T > kv->d.cap) return fail(SI_ERR_INVALID_ARG, "T exceeds the cache's entries");
    if (Hq < 1 || Hq % kv->d.Hkv) return fail(SI_ERR_INVALID_ARG, "need Hq a multiple of Hkv");
    if (Hq / kv->d.Hkv > 256) return fail(SI_ERR_UNSUPPORTED, "more than 256 query heads per cache head");
    if (!aligned16(q) || !Strides(q_stride, {kv->d.B, T, Hq}).whole_units())
        return fail(SI_ERR_INVALID_ARG, "q must be 16-byte aligned with strides that are multiples of 8");
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(SI_ERR_INVALID_ARG, "need a finite scale > 0");
    return SI_OK;
}

si::AttendParams rows_of(const si_kv* kv, int layer, int T, int Hq, const void* q, const long long* q_stride,
                         const uint64_t* mask, float scale) {
    si::AttendParams P = {};
    P.c = view_of(kv->d, layer);
    P.T = T, P.Hq = Hq, P.G = Hq / kv->d.Hkv;
    P.q = q;
    const Strides qs(q_stride, {kv->d.B, T, Hq});
    P.qb = qs.at[0], P.qt = qs.at[1], P.qh = qs.at[2];
    P.mask = reinterpret_cast<const unsigned long long*>(mask);
    P.scale = scale;
    return P;
}

}  // namespace

extern "C" {

int si_kv_create(const si_kv_desc* desc, si_kv** out) {
    if (!desc || !out) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    *out = nullptr;
    const si_kv_desc& d = *desc;
    if (!d.k || !d.v || !d.len) return fail(SI_ERR_INVALID_ARG, "NULL pointer in the cache description");
    if (d.dtype != SI_BF16 && d.dtype != SI_FP16) return fail(SI_ERR_INVALID_ARG, "dtype must be SI_BF16 or SI_FP16");
    if (d.L < 1 || d.B < 1 || d.Hkv < 1 || d.cap < 1 || d.n_slots < 1)
        return fail(SI_ERR_INVALID_ARG, "need L, B, Hkv, cap, n_slots >= 1");
    if (d.D < 8 || d.D > 256 || d.D % 8) return fail(SI_ERR_INVALID_ARG, "need 8 <= D <= 256 and D % 8 == 0");
    if (d.B > 1024) return fail(SI_ERR_UNSUPPORTED, "more than 1024 sequences");
    if (d.Hkv > 1024) return fail(SI_ERR_UNSUPPORTED, "more than 1024 cache heads");
    if (d.n_slots > 0x7FFFFFFFLL) return fail(SI_ERR_INVALID_ARG, "slots are int32: n_slots is too large");
    const long long pool[4] = {d.L, d.B, d.Hkv, d.n_slots}, lists[3] = {d.L, d.B, d.Hkv};
    const Strides ks(d.k_stride, pool), vs(d.v_stride, pool), ts(d.table_stride, lists), as(d.acc_stride, lists);
    if (!aligned16(d.k) || !aligned16(d.v) || !ks.whole_units() || !vs.whole_units())
        return fail(SI_ERR_INVALID_ARG, "k and v must be 16-byte aligned with strides that are multiples of 8");
    if (ks.at[3] > 0x7FFFFFFFLL || vs.at[3] > 0x7FFFFFFFLL)
        return fail(SI_ERR_UNSUPPORTED, "a slot stride exceeds 2^31 - 1 elements");
    if (!d.table && d.cap > d.n_slots) return fail(SI_ERR_INVALID_ARG, "without a table cap must not exceed n_slots");
    for (int i = 0; i < 3; ++i)
        if (ts.at[i] < 0 || as.at[i] < 0) return fail(SI_ERR_INVALID_ARG, "negative stride");
    si_kv* kv = new (std::nothrow) si_kv;
    if (!kv) return fail(SI_ERR_OOM, "out of host memory");
    kv->d = d;
    std::memcpy(kv->d.k_stride, ks.at, sizeof d.k_stride);
    std::memcpy(kv->d.v_stride, vs.at, sizeof d.v_stride);
    std::memcpy(kv->d.table_stride, ts.at, sizeof d.table_stride);
    std::memcpy(kv->d.acc_stride, as.at, sizeof d.acc_stride);
    *out = kv;
    return SI_OK;
}

int si_kv_destroy(si_kv* kv) {
    SI_TRACE("si_kv_destroy");
    if (!kv) return SI_OK;
    cudaError_t e = cudaSuccess;
    if (kv->part || kv->ticket) e = cudaDeviceSynchronize();
    if (kv->part) cudaFree(kv->part);
    if (kv->ticket) cudaFree(kv->ticket);
    delete kv;
    return e == cudaSuccess ? SI_OK : cuda_fail(e, "cudaDeviceSynchronize");
}

int si_rope_create(int n_pairs, const double* inv_freq, const uint8_t* axis, int n_axes, int interleaved,
                   si_rope** out) {
    if (!inv_freq || !axis || !out) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    *out = nullptr;
    if (n_pairs < 8 || n_pairs > si::kRopeMaxPairs || n_pairs % 8)
        return fail(SI_ERR_INVALID_ARG, "need 8 <= n_pairs <= 128 and n_pairs % 8 == 0");
    if (n_axes < 1 || n_axes > 4) return fail(SI_ERR_INVALID_ARG, "need 1 <= n_axes <= 4");
    for (int i = 0; i < n_pairs; ++i) {
        if (!(std::fabs(inv_freq[i]) <= 1048576.0)) return fail(SI_ERR_INVALID_ARG, "need |inv_freq| <= 2^20");
        if (axis[i] >= n_axes) return fail(SI_ERR_INVALID_ARG, "axis index outside n_axes");
    }
    si_rope* r = new (std::nothrow) si_rope;
    if (!r) return fail(SI_ERR_OOM, "out of host memory");
    std::memset(&r->t, 0, sizeof r->t);
    r->t.n_pairs = n_pairs;
    r->t.n_axes = n_axes;
    r->t.interleaved = interleaved != 0;
    for (int i = 0; i < n_pairs; ++i) {
        r->t.turn[i] = turn_of(inv_freq[i]);
        r->t.axis[i] = axis[i];
    }
    *out = r;
    return SI_OK;
}

int si_rope_destroy(si_rope* rope) {
    delete rope;
    return SI_OK;
}

int si_kv_append(si_kv* kv, int layer, const si_rope* rope, int T, int Hq, const void* q, const long long* q_stride,
                 const void* k, const long long* k_stride, const void* v, const long long* v_stride,
                 const int32_t* pos, void* q_out, void* stream) {
    SI_TRACE("si_kv_append");
    if (!kv || !rope || !k || !k_stride || !v || !v_stride || !pos) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    if (Hq < 0 || (Hq > 0 && (!q || !q_stride || !q_out))) return fail(SI_ERR_INVALID_ARG, "q, q_stride and q_out go with Hq");
    const si_kv_desc& d = kv->d;
    if (layer < 0 || layer >= d.L) return fail(SI_ERR_INVALID_ARG, "layer outside the cache");
    if (T < 1 || T > d.cap) return fail(SI_ERR_INVALID_ARG, "need 1 <= T <= cap");
    if (2 * rope->t.n_pairs > d.D) return fail(SI_ERR_INVALID_ARG, "the rotary pairs exceed D");
    static const long long none[3] = {};
    const Strides qs(Hq > 0 ? q_stride : none, {d.B, T, Hq}), ks(k_stride, {d.B, T, d.Hkv}), vs(v_stride, {d.B, T, d.Hkv});
    if (!aligned16(k) || !aligned16(v) || !ks.whole_units() || !vs.whole_units() ||
        (Hq > 0 && (!aligned16(q) || !aligned16(q_out) || !qs.whole_units())))
        return fail(SI_ERR_INVALID_ARG, "q, k, v, q_out must be 16-byte aligned with strides that are multiples of 8");
    if ((long long)d.B * T > 0x7FFFFFFFLL) return fail(SI_ERR_UNSUPPORTED, "B * T exceeds 2^31 - 1");
    if (((long long)Hq + 2ll * d.Hkv) * (d.D / 8) > 0x7FFF0000LL)
        return fail(SI_ERR_UNSUPPORTED, "a token's heads exceed 32-bit counts");
    si::KvAppendParams P = {};
    P.c = view_of(d, layer);
    P.T = T, P.Hq = Hq;
    P.q = q, P.k = k, P.v = v;
    P.qb = qs.at[0], P.qt = qs.at[1], P.qh = qs.at[2];
    P.kb = ks.at[0], P.kt = ks.at[1], P.kh = ks.at[2];
    P.vb = vs.at[0], P.vt = vs.at[1], P.vh = vs.at[2];
    P.pos = pos;
    P.q_out = q_out;
    const int rc = si::device_error_word(&P.err);
    if (rc) return rc;
    const cudaError_t e = si::launch_kv_append(P, rope->t, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SI_OK : cuda_fail(e, "si_kv_append");
}

int si_tree_attention(si_kv* kv, int layer, int T, int Hq, const void* q, const long long* q_stride,
                      const uint64_t* mask, float scale, void* out, float* lse, void* stream) {
    SI_TRACE("si_tree_attention");
    int rc = check_rows(kv, layer, T, Hq, q, q_stride, scale);
    if (rc) return rc;
    if (!out) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    if (out == q) return fail(SI_ERR_INVALID_ARG, "out may not be q");
    if (!aligned16(out)) return fail(SI_ERR_INVALID_ARG, "out must be 16-byte aligned");
    si::AttendParams P = rows_of(kv, layer, T, Hq, q, q_stride, mask, scale);
    if (!si::attend_counts_fit(P)) return fail(SI_ERR_UNSUPPORTED, "lists, row blocks and entries exceed 32-bit counts");
    P.out = out;
    P.lse = lse;
    if ((rc = on_device(kv))) return rc;
    if ((rc = si::device_error_word(&P.err))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((rc = make_part(kv, st))) return rc;
    P.part = kv->part;
    const cudaError_t e = si::launch_tree_attention(P, st);
    return e == cudaSuccess ? SI_OK : cuda_fail(e, "si_tree_attention");
}

int si_kv_accumulate(si_kv* kv, int layer, int T, int Hq, const void* q, const long long* q_stride, const float* lse,
                     const uint64_t* mask, const uint64_t* rows, float scale, float* acc_out, void* stream) {
    SI_TRACE("si_kv_accumulate");
    int rc = check_rows(kv, layer, T, Hq, q, q_stride, scale);
    if (rc) return rc;
    if (!lse) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    if (!kv->d.acc) return fail(SI_ERR_INVALID_ARG, "the cache has no acc");
    si::AttendParams P = rows_of(kv, layer, T, Hq, q, q_stride, mask, scale);
    if (!si::attend_counts_fit(P)) return fail(SI_ERR_UNSUPPORTED, "lists, row blocks and entries exceed 32-bit counts");
    P.lse = const_cast<float*>(lse);
    P.rows = reinterpret_cast<const unsigned long long*>(rows);
    P.acc_out = acc_out ? acc_out : P.c.acc;
    if ((rc = si::device_error_word(&P.err))) return rc;
    const cudaError_t e = si::launch_kv_accumulate(P, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SI_OK : cuda_fail(e, "si_kv_accumulate");
}

int si_kv_evict(si_kv* kv, int layer, int T, const int32_t* path, const int32_t* n_path, int budget, int sinks,
                int recent, int32_t* table_out, int32_t* len_out, void* stream) {
    SI_TRACE("si_kv_evict");
    if (!kv) return fail(SI_ERR_INVALID_ARG, "NULL pointer");
    const si_kv_desc& d = kv->d;
    if (!d.table) return fail(SI_ERR_INVALID_ARG, "the cache has no table");
    if (layer < -1 || layer >= d.L) return fail(SI_ERR_INVALID_ARG, "layer outside the cache");
    if (T < 0 || T > d.cap) return fail(SI_ERR_INVALID_ARG, "need 0 <= T <= cap");
    if (path && (T > 64 || !n_path)) return fail(SI_ERR_INVALID_ARG, "a path needs T <= 64 and n_path");
    if (budget < 0 || sinks < 0 || recent < 0) return fail(SI_ERR_INVALID_ARG, "need budget, sinks, recent >= 0");
    if (budget > 0 && (long long)sinks + recent > budget) return fail(SI_ERR_INVALID_ARG, "need sinks + recent <= budget");
    if (budget > 0 && !d.acc) return fail(SI_ERR_INVALID_ARG, "the cache has no acc");
    if ((table_out == nullptr) != (len_out == nullptr))
        return fail(SI_ERR_INVALID_ARG, "table_out and len_out go together");
    if (d.cap > si::kEvictMaxCap) return fail(SI_ERR_UNSUPPORTED, "cap exceeds 196608");
    const int layers = layer < 0 ? d.L : 1, first = layer < 0 ? 0 : layer;
    if ((long long)layers * d.B * d.Hkv > 1000000) return fail(SI_ERR_UNSUPPORTED, "more than 1000000 lists");
    if (table_out) {
        // the lists' extents in memory must not meet
        const long long rows = (long long)d.L * d.B * d.Hkv;
        const int32_t* a0 = d.table;
        const int32_t* a1 = d.table + (d.L - 1) * d.table_stride[0] + (d.B - 1) * d.table_stride[1] +
                            (d.Hkv - 1) * d.table_stride[2] + d.cap;
        if (table_out < a1 && a0 < table_out + rows * d.cap) return fail(SI_ERR_INVALID_ARG, "table_out overlaps the table");
        if (len_out < d.len + (long long)d.L * d.B && d.len < len_out + (long long)d.L * d.B)
            return fail(SI_ERR_INVALID_ARG, "len_out overlaps len");
    }
    int rc = on_device(kv);
    if (rc) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!kv->ticket) {
        if (capturing(st)) return fail(SI_ERR_INVALID_ARG, "eviction scratch must be made; call once before capture");
        // the ticket, then a length per list of lists (the in-place form keeps the new lengths there)
        const size_t words = 1 + (size_t)d.L * d.B;
        cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&kv->ticket), words * sizeof(unsigned));
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            kv->ticket = nullptr;
            return fail(SI_ERR_OOM, "cudaMalloc failed for the eviction ticket");
        }
        e = cudaMemset(kv->ticket, 0, words * sizeof(unsigned));
        // the memset is on the legacy stream, `stream` may not wait for that one
        if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
        if (e != cudaSuccess) {
            cudaFree(kv->ticket);  // a ticket that may not be zero is not kept
            kv->ticket = nullptr;
            return cuda_fail(e, "cudaMemset");
        }
    }
    si::KvEvictParams P = {};
    P.table = d.table + first * d.table_stride[0];
    P.tl = d.table_stride[0], P.tb = d.table_stride[1], P.th = d.table_stride[2];
    P.len = d.len + (long long)first * d.B;
    P.acc = d.acc ? d.acc + first * d.acc_stride[0] : nullptr;
    P.al = d.acc_stride[0], P.ab = d.acc_stride[1], P.ah = d.acc_stride[2];
    P.in_place = table_out == nullptr;
    if (table_out) {
        P.oh = d.cap, P.ob = (long long)d.Hkv * d.cap, P.ol = (long long)d.B * d.Hkv * d.cap;
        P.table_out = table_out + first * P.ol;
        P.len_out = len_out + (long long)first * d.B;
    } else {
        P.table_out = P.table, P.ol = P.tl, P.ob = P.tb, P.oh = P.th;
        P.len_out = P.len;
    }
    P.path = path;
    P.n_path = n_path;
    P.n_slots = d.n_slots;
    P.L = layers, P.B = d.B, P.Hkv = d.Hkv, P.cap = d.cap;
    P.T = T, P.budget = budget, P.sinks = sinks, P.recent = recent;
    P.ticket = kv->ticket;
    if ((rc = si::device_error_word(&P.err))) return rc;
    const cudaError_t e = si::launch_kv_evict(P, st);
    return e == cudaSuccess ? SI_OK : cuda_fail(e, "si_kv_evict");
}

}  // extern "C"
