// Penalties for repeated tokens, biases and grammar masks on logits
// (q3tts_process_logits in q3tts.h).
//
// Bound by reading and writing the logits once, and below that by chains of
// dependent loads.  A CTA takes 8192 ids of a row.  It asks for everything at once:
// their logits (16 bytes a load), the history and biases, the mask's words.  It
// counts the history's ids among its own in shared memory, stores the logits through the mask, and then puts right the few ids that a
// history or a bias names, each from the logit as it came, so that it is rounded
// once.  Counts are whole numbers and an id's biases are added in their order, so
// the result does not depend on timing.
//
// Where there are more such CTAs than SMs, each with the same history to go
// through, a second kernel does that for a row at once, with a table of its ids
// in shared memory (256 x 151936 bf16 with 512 to 1024 tokens and a mask for each
// row: 61 us in one kernel, 41 in two, 24 for the bytes; 32 x 151936 fp32 with
// 1024 to 2048 tokens: 12.7 and 22; one row of 2048: 3.0).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "pdl.cuh"

namespace q3 {

namespace {

constexpr int P_SLICE = 8192, P_THREADS = 512, P_MAX_VOCAB = 262144;
constexpr int P_PLACES = 16384;                       // of the second kernel's table, at most; half of them are filled
constexpr uint32_t P_FREE = 0xffffffffu;              // the id of a place that is free
// a word of an id: times among the generated tokens, and
constexpr uint32_t P_SEEN = 1u << 29, P_DONE = 1u << 30, P_BIAS = 1u << 31, P_COUNT = P_SEEN - 1;

struct ProcessArgs {
    int V;
    const void* logits;
    int64_t ld;
    const int32_t *history, *n_history, *n_prompt;
    int cap;
    int64_t ldh;
    const float *rep, *pres, *freq;
    int n_bias;
    const int32_t *bias_off, *bias_ids;
    const float* bias;
    int n_masks;
    const uint32_t* mask;
    int64_t ldm;
    const int32_t* mask_row;
    void* out;
    int64_t ldo;
    int* err;
};

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// the logits of a 16-byte piece whose bit is not set become -inf
template <typename T> __device__ __forceinline__ uint4 masked(uint4 v, uint32_t bits);
template <> __device__ __forceinline__ uint4 masked<float>(uint4 v, uint32_t bits) {
    return make_uint4(bits & 1 ? v.x : 0xff800000u, bits & 2 ? v.y : 0xff800000u, bits & 4 ? v.z : 0xff800000u,
                      bits & 8 ? v.w : 0xff800000u);
}
__device__ __forceinline__ uint32_t masked2(uint32_t v, uint32_t bits) {
    const uint32_t keep = (bits & 1 ? 0xffffu : 0u) | (bits & 2 ? 0xffff0000u : 0u);
    return (v & keep) | (0xff80ff80u & ~keep);
}
template <> __device__ __forceinline__ uint4 masked<bf16>(uint4 v, uint32_t bits) {
    return make_uint4(masked2(v.x, bits), masked2(v.y, bits >> 2), masked2(v.z, bits >> 4), masked2(v.w, bits >> 6));
}

// A row's lists, cut to what is there.
struct ProcessRow {
    int nh, np, b0, b1;
    bool bad, none;              // something is out of range; nothing may be drawn
    const uint32_t* mask;
    __device__ __forceinline__ ProcessRow(const ProcessArgs& a, int r) : nh(0), np(0), b0(0), b1(0), bad(false), none(false), mask(nullptr) {
        if (a.history) {
            const int n = a.n_history[r];
            nh = min(max(n, 0), a.cap);
            bad |= nh != n;
            np = a.n_prompt ? min(max(a.n_prompt[r], 0), nh) : 0;
        }
        if (a.bias_off) {
            b0 = a.bias_off[r];
            b1 = a.bias_off[r + 1];
            if (b0 < 0 || b1 < b0 || b1 > a.n_bias) { bad = true; b0 = b1 = 0; }
        }
        if (a.mask) {
            const int m = a.mask_row ? a.mask_row[r] : r;
            if (m < -1 || m >= a.n_masks) { bad = none = true; }
            else if (m >= 0) mask = a.mask + m * a.ldm;
        }
    }
    __device__ __forceinline__ bool allowed(int i) const { return !none && (!mask || mask[i >> 5] >> (i & 31) & 1); }
};
// A logit after the penalties: what the word of its id says.
template <typename T> struct Penalties {
    float rep, pres, freq;
    __device__ __forceinline__ Penalties(const ProcessArgs& a, int r)
        : rep(a.rep ? a.rep[r] : 1.f), pres(a.pres ? a.pres[r] : 0.f), freq(a.freq ? a.freq[r] : 0.f) {}
    __device__ __forceinline__ float operator()(T x, uint32_t w) const {
        float v = to_f(x);
        if (w & (P_SEEN | P_COUNT)) v = v < 0.f ? v * rep : v / rep;
        if (w & P_COUNT) v -= fmaf(freq, (float)(w & P_COUNT), pres);
        return v;
    }
};
// the sum of an id's biases, in their order
__device__ __forceinline__ float bias_of(const ProcessArgs& a, int b0, int b1, int id) {
    float b = 0.f;
    for (int i = b0; i < b1; ++i)
        if (a.bias_ids[i] == id) b += a.bias[i];
    return b;
}

// NAMES: the ids that are named are put right too.
template <typename T, bool NAMES>
__global__ void __launch_bounds__(P_THREADS, NAMES ? 2 : 4) process_kernel(const ProcessArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = 16 / (int)sizeof(T), NV = P_SLICE / N / P_THREADS;   // logits of a piece, pieces of a thread
    extern __shared__ uint32_t words[];
    __shared__ int s_dup;
    const int r = blockIdx.y, lo = blockIdx.x * P_SLICE, hi = min(lo + P_SLICE, a.V), tid = threadIdx.x;
    const T* x = (const T*)a.logits + r * a.ld;
    T* out = (T*)a.out + r * a.ldo;
    const bool in_place = a.logits == a.out;
    // pieces: as the output is aligned, and loaded as such where the logits lie alike
    const int off = (int)(((uintptr_t)(out + lo) & 15) / sizeof(T)), head = min(off ? N - off : 0, hi - lo);
    const int pieces = (hi - lo - head) / N;
    const bool alike = (((uintptr_t)x ^ (uintptr_t)out) & 15) == 0;
    uint4 v[NV];
    if (!in_place && alike)
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (tid + j * P_THREADS < pieces) v[j] = ld16(x + lo + head + (tid + j * P_THREADS) * N);

    const ProcessRow row(a, r);
    const int nh = NAMES ? row.nh : 0, b0 = row.b0, b1 = NAMES ? row.b1 : row.b0, np = row.np;
    const bool tell = a.err && blockIdx.x == 0, none = row.none;
    const uint32_t* mask = row.mask;
    if (row.bad && tell && tid == 0) atomicOr(a.err, ERRB_BOUNDS);
    auto allowed = [&](int i) { return row.allowed(i); };
    const bool named = nh > 0 || b1 > b0, through = !in_place || mask || none;
    const int32_t* h = a.history + r * a.ldh;
    constexpr int NH = 4;        // ids of the history that a thread has in flight
    int first[NH], bias_id = -1;
    float bias = 0.f;
    auto ask = [&](int j0, int (&id)[NH]) {
#pragma unroll
        for (int k = 0; k < NH; ++k) id[k] = j0 + k * P_THREADS < nh ? h[j0 + k * P_THREADS] : -1;
    };
    // the logits of those in the slice, and whether they are allowed, also all asked for together
    T xs[NH];
    bool may[NH];
    auto look = [&](const int (&id)[NH]) {
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            may[k] = id[k] >= lo && id[k] < hi;
            if (may[k]) { xs[k] = x[id[k]]; may[k] = allowed(id[k]); }
        }
    };
    ask(tid, first);
    if (b0 + tid < b1) {
        bias_id = a.bias_ids[b0 + tid];
        bias = a.bias[b0 + tid];
    }
    T bias_x = from_f<T>(0.f);
    bool bias_may = false;
    uint32_t bits[NV];           // of the ids of each piece
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        bits[j] = none ? 0 : 0xffffffffu;
        const int i = lo + head + (tid + j * P_THREADS) * N;
        if (mask && tid + j * P_THREADS < pieces) {
            const uint32_t w0 = mask[i >> 5], w1 = (i & 31) > 32 - N ? mask[(i >> 5) + 1] : 0;
            bits[j] = __funnelshift_r(w0, w1, i & 31);
        }
    }
    if (named) {
        for (int i = tid; i < hi - lo; i += P_THREADS) words[i] = 0;
        if (tid == 0) s_dup = 0;
        __syncthreads();
        auto count = [&](int j0, const int (&id)[NH]) {
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                if (id[k] >= a.V && tell) atomicOr(a.err, ERRB_BOUNDS);
                if (id[k] < lo || id[k] >= hi) continue;
                if (j0 + k * P_THREADS < np) atomicOr(&words[id[k] - lo], P_SEEN);
                else atomicAdd(&words[id[k] - lo], 1u);
            }
        };
        look(first);
        if (bias_id >= lo && bias_id < hi) { bias_x = x[bias_id]; bias_may = allowed(bias_id); }
        count(tid, first);
        for (int j = tid + NH * P_THREADS; j < nh; j += NH * P_THREADS) {
            int id[NH];
            ask(j, id);
            count(j, id);
        }
        for (int j = b0 + tid; j < b1; j += P_THREADS) {
            const int id = j < b0 + P_THREADS ? bias_id : a.bias_ids[j];
            if ((id < 0 || id >= a.V) && tell) atomicOr(a.err, ERRB_BOUNDS);
            if (id >= lo && id < hi && atomicOr(&words[id - lo], P_BIAS) & P_BIAS) s_dup = 1;
        }
    }
    // ---- the slice through the mask
    if (through) {
        const int from = lo + head;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int p = tid + j * P_THREADS, i = from + p * N;
            if (p >= pieces) break;
            if (in_place) {
                if (!(bits[j] & ((1u << N) - 1))) *(uint4*)(out + i) = masked<T>(make_uint4(0, 0, 0, 0), 0);
                else
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (!(bits[j] >> e & 1)) out[i + e] = from_f<T>(-INFINITY);
                continue;
            }
            if (!alike) {
                alignas(16) T t[N];
#pragma unroll
                for (int e = 0; e < N; ++e) t[e] = x[i + e];
                v[j] = *(const uint4*)t;
            }
            *(uint4*)(out + i) = masked<T>(v[j], bits[j]);
        }
        for (int i = tid; i < hi - lo - pieces * N; i += P_THREADS) {     // in front of the pieces and behind them
            const int id = lo + (i < head ? i : i + pieces * N);
            if (!allowed(id)) out[id] = from_f<T>(-INFINITY);
            else if (!in_place) out[id] = x[id];
        }
    }
    if (!named || none) return;
    __syncthreads();
    // ---- the ids that are named
    const Penalties<T> adjusted(a, r);
    for (int j = b0 + tid; j < b1; j += P_THREADS) {
        const int id = j < b0 + P_THREADS ? bias_id : a.bias_ids[j];
        if (id < lo || id >= hi) continue;
        const uint32_t w = atomicOr(&words[id - lo], P_DONE);
        const bool mine = j < b0 + P_THREADS;
        if (w & P_DONE || !(mine ? bias_may : allowed(id))) continue;
        const float b = s_dup ? bias_of(a, b0, b1, id) : mine ? bias : a.bias[j];
        out[id] = from_f<T>(adjusted(mine ? bias_x : x[id], w) + b);
    }
    auto plain = [&](const int (&id)[NH]) {      // those of the history without a bias, each once
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            if (!may[k] || words[id[k] - lo] & P_BIAS) continue;
            const uint32_t w = atomicOr(&words[id[k] - lo], P_DONE);
            if (!(w & P_DONE)) out[id[k]] = from_f<T>(adjusted(xs[k], w));
        }
    };
    plain(first);
    for (int j = tid + NH * P_THREADS; j < nh; j += NH * P_THREADS) {
        int id[NH];
        ask(j, id);
        look(id);
        plain(id);
    }
}

// The ids that are named, a row a CTA, behind process_kernel: a table of them in shared memory (open addressing, places:
// at least twice as many as ids), or, where they are too many for it, a word for each id of a part of the vocabulary at
// a time.  Behind process_kernel (copied), whose CTAs let this one start when all that came before them is done, the
// table is filled while that one copies.  Every CTA waits for the copies before it ends, as what follows waits for this
// kernel alone.
template <typename T>
__global__ void __launch_bounds__(P_THREADS) process_names_kernel(const ProcessArgs a, int places, bool copied) {
    if (!copied) pdl_wait();
    extern __shared__ uint32_t words[];       // [places], then their ids
    __shared__ int s_dup;
    uint32_t* ids = words + places;
    const int r = blockIdx.x, tid = threadIdx.x;
    const T* x = (const T*)a.logits + r * a.ld;
    T* out = (T*)a.out + r * a.ldo;
    const ProcessRow row(a, r);
    const int nh = row.nh, np = row.np, b0 = row.b0, b1 = row.b1;
    const int32_t* h = a.history + r * a.ldh;
    if (!copied && row.bad && a.err && tid == 0) atomicOr(a.err, ERRB_BOUNDS);
    if (row.none || (nh == 0 && b1 == b0)) {
        pdl_wait();
        return;
    }
    const bool few = (int64_t)nh + (b1 - b0) <= places / 2;
    const int shift = 32 - (31 - __clz(places));
    // the word of an id of [from, to); with a table, that of its place, taken if need be
    auto word_of = [&](int id, int from) {
        if (!few) return id - from;
        for (uint32_t i = (uint32_t)id * 2654435769u >> shift;; i = (i + 1) & (places - 1)) {
            const uint32_t was = atomicCAS(&ids[i], P_FREE, (uint32_t)id);
            if (was == P_FREE || was == (uint32_t)id) return (int)i;
        }
    };
    const Penalties<T> adjusted(a, r);
    for (int from = 0; from < a.V; from += places) {
        const int to = few ? a.V : min(from + places, a.V);
        for (int i = tid; i < places; i += P_THREADS) {
            words[i] = 0;
            ids[i] = P_FREE;
        }
        if (tid == 0) s_dup = 0;
        __syncthreads();
        constexpr int NH = 4;                 // ids of the history that a thread has in flight, and keeps of the first ones
        int first[NH], place[NH];
        auto ask = [&](int j0, int (&id)[NH]) {
#pragma unroll
            for (int k = 0; k < NH; ++k) id[k] = j0 + k * P_THREADS < nh ? h[j0 + k * P_THREADS] : -1;
        };
        auto count = [&](int j0, const int (&id)[NH], int (&at)[NH]) {
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                if (id[k] >= a.V && a.err) atomicOr(a.err, ERRB_BOUNDS);
                at[k] = -1;
                if (id[k] < from || id[k] >= to) continue;
                at[k] = word_of(id[k], from);
                if (j0 + k * P_THREADS < np) atomicOr(&words[at[k]], P_SEEN);
                else atomicAdd(&words[at[k]], 1u);
            }
        };
        // their logits, and whether they are allowed, also all asked for together (in place, what process_kernel writes
        // meanwhile is at ids that are not)
        T xs[NH], bias_x = from_f<T>(0.f);
        bool may[NH], bias_may = false;
        auto look = [&](const int (&id)[NH]) {
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                may[k] = id[k] >= from && id[k] < to;
                if (may[k]) { xs[k] = x[id[k]]; may[k] = row.allowed(id[k]); }
            }
        };
        ask(tid, first);
        int bias_id = -1;
        float bias = 0.f;
        if (b0 + tid < b1) { bias_id = a.bias_ids[b0 + tid]; bias = a.bias[b0 + tid]; }
        look(first);
        if (bias_id >= from && bias_id < to) { bias_x = x[bias_id]; bias_may = row.allowed(bias_id); }
        count(tid, first, place);
        for (int j = tid + NH * P_THREADS; j < nh; j += NH * P_THREADS) {
            int id[NH], at[NH];
            ask(j, id);
            count(j, id, at);
        }
        for (int j = b0 + tid; j < b1; j += P_THREADS) {
            const int id = j < b0 + P_THREADS ? bias_id : a.bias_ids[j];
            if ((id < 0 || id >= a.V) && a.err) atomicOr(a.err, ERRB_BOUNDS);
            if (id >= from && id < to && atomicOr(&words[word_of(id, from)], P_BIAS) & P_BIAS) s_dup = 1;
        }
        __syncthreads();
        pdl_wait();                           // the copies are done
        pdl_trigger();
        for (int j = b0 + tid; j < b1; j += P_THREADS) {
            const bool mine = j < b0 + P_THREADS;
            const int id = mine ? bias_id : a.bias_ids[j];
            if (id < from || id >= to) continue;
            const uint32_t w = atomicOr(&words[word_of(id, from)], P_DONE);
            if (w & P_DONE || !(mine ? bias_may : row.allowed(id))) continue;
            const float b = s_dup ? bias_of(a, b0, b1, id) : mine ? bias : a.bias[j];
            out[id] = from_f<T>(adjusted(mine ? bias_x : x[id], w) + b);
        }
        auto plain = [&](const int (&id)[NH], const int (&at)[NH]) {      // those of the history without a bias, each once
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                if (!may[k] || words[at[k]] & P_BIAS) continue;
                const uint32_t w = atomicOr(&words[at[k]], P_DONE);
                if (!(w & P_DONE)) out[id[k]] = from_f<T>(adjusted(xs[k], w));
            }
        };
        plain(first, place);
        for (int j = tid + NH * P_THREADS; j < nh; j += NH * P_THREADS) {
            int id[NH], at[NH];
            ask(j, id);
#pragma unroll
            for (int k = 0; k < NH; ++k) at[k] = id[k] >= from && id[k] < to ? word_of(id[k], from) : -1;
            look(id);
            plain(id, at);
        }
        if (few) return;
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_t(int n, const ProcessArgs& a, cudaStream_t st) {
    const bool named = a.history || a.bias_off, through = a.mask || a.logits != a.out;
    if (!named && !through) return cudaSuccess;      // (in place, nothing to do)
    const dim3 grid((a.V + P_SLICE - 1) / P_SLICE, n);
    // In one kernel where its CTAs run beside each other, or where the history may be longer than a table takes (a CTA a
    // row would go through it for every part of the vocabulary).
    const bool one = named && ((int64_t)grid.x * n <= 4 * device_sm_count() || a.cap > P_PLACES / 2);
    if (one) return launch_pdl(process_kernel<T, true>, grid, P_THREADS, std::min(P_SLICE, a.V) * 4, st, a);
    cudaError_t e;
    if (through) {
        e = launch_pdl(process_kernel<T, false>, grid, P_THREADS, 0, st, a);
        if (e != cudaSuccess || !named) return e;
    }
    int places = 1024;
    while (places < P_PLACES && places < 2 * (a.cap + 512)) places *= 2;
    // a per-device attribute: set on every call (a host-side table lookup)
    e = cudaFuncSetAttribute(process_names_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, P_PLACES * 8);
    if (e != cudaSuccess) return e;
    return launch_pdl(process_names_kernel<T>, n, P_THREADS, places * 8, st, a, places, through);
}

}  // namespace
}  // namespace q3

using namespace q3;

extern "C" int q3tts_process_logits(int n, int vocab, const void* logits, int dtype, int64_t logits_stride,
                                    const int32_t* history, int history_cap, int64_t history_stride,
                                    const int32_t* n_history, const int32_t* n_prompt, const float* repetition,
                                    const float* presence, const float* frequency, int n_bias, const int32_t* bias_off,
                                    const int32_t* bias_ids, const float* bias, int n_masks, const uint32_t* mask,
                                    int64_t mask_stride, const int32_t* mask_row, void* out, int64_t out_stride,
                                    int32_t* err, void* stream) {
    if (n < 0 || n > 65535) return paged_fail(Q3_ERR_ARG, "n must be in 0..65535");
    if (vocab < 1 || vocab > P_MAX_VOCAB) return paged_fail(Q3_ERR_ARG, "vocab must be in 1..%d", P_MAX_VOCAB);
    if (dtype != Q3_F32 && dtype != Q3_BF16) return paged_fail(Q3_ERR_ARG, "dtype must be Q3_F32 or Q3_BF16");
    if (n == 0) return Q3_OK;
    if (!logits || !out) return paged_fail(Q3_ERR_ARG, "NULL logits or out");
    if (logits_stride == 0) logits_stride = vocab;
    if (out_stride == 0) out_stride = vocab;
    if (logits_stride < vocab || out_stride < vocab) return paged_fail(Q3_ERR_ARG, "a stride is less than vocab");
    if (logits == out && logits_stride != out_stride)
        return paged_fail(Q3_ERR_ARG, "in place, out_stride must be the logits'");
    if (!history && (n_history || n_prompt)) return paged_fail(Q3_ERR_ARG, "n_history or n_prompt without a history");
    if (history) {
        if (!n_history) return paged_fail(Q3_ERR_ARG, "n_history is NULL");
        if (history_cap < 0 || history_cap > 0x10000000) return paged_fail(Q3_ERR_ARG, "history_cap must be in 0..2^28");
        if (history_stride == 0) history_stride = history_cap;
        if (history_stride < history_cap) return paged_fail(Q3_ERR_ARG, "history_stride is less than history_cap");
    }
    if (!bias_off != !bias_ids || !bias_off != !bias)
        return paged_fail(Q3_ERR_ARG, "bias_off, bias_ids and bias: all or none");
    if (bias_off && n_bias < 0) return paged_fail(Q3_ERR_ARG, "negative n_bias");
    if (!mask && mask_row) return paged_fail(Q3_ERR_ARG, "mask_row without masks");
    const int mask_words = (vocab + 31) / 32;
    if (mask) {
        if (n_masks < 1) return paged_fail(Q3_ERR_ARG, "n_masks must be >= 1");
        if (!mask_row && n_masks < n) return paged_fail(Q3_ERR_ARG, "%d masks for %d rows: mask_row is needed", n_masks, n);
        if (mask_stride == 0) mask_stride = mask_words;
        if (mask_stride < mask_words) return paged_fail(Q3_ERR_ARG, "mask_stride is less than %d words", mask_words);
    }
    const ProcessArgs a = {vocab, logits, logits_stride, history, n_history, n_prompt, history_cap, history_stride,
                           repetition, presence, frequency, n_bias, bias_off, bias_ids, bias, n_masks, mask, mask_stride,
                           mask_row, out, out_stride, err};
    const cudaError_t e = dtype == Q3_BF16 ? launch_t<bf16>(n, a, (cudaStream_t)stream) : launch_t<float>(n, a, (cudaStream_t)stream);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "process: %s", cudaGetErrorString(e));
    return Q3_OK;
}
