// Penalties for repeated tokens, biases and grammar masks on logits
// (q3tts_process_logits in q3tts.h).
//
// Bound by reading and writing the logits once.  A CTA takes 8192 ids of a row:
// it has their logits on the way (16 bytes a load, all in flight together) while
// it counts the history's ids among them in shared memory and lists each once;
// it stores the logits through the mask, and then puts right the few ids that a
// history or a bias names, each from the logit as it came, so that it is rounded
// once.  Counts are whole numbers and an id's biases are added in their order, so
// the result does not depend on timing.
#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "pdl.cuh"

namespace q3 {

namespace {

constexpr int P_SLICE = 8192, P_THREADS = 512, P_MAX_VOCAB = 262144;
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

template <typename T>
__global__ void __launch_bounds__(P_THREADS) process_kernel(const ProcessArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = 16 / (int)sizeof(T), NV = P_SLICE / N / P_THREADS;   // logits of a piece, pieces of a thread
    extern __shared__ uint32_t words[];
    __shared__ int s_dup, s_count;
    const int r = blockIdx.y, lo = blockIdx.x * P_SLICE, hi = min(lo + P_SLICE, a.V), tid = threadIdx.x;
    uint16_t* list = (uint16_t*)(words + min(P_SLICE, a.V));     // ids of the slice that the history names
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

    const bool tell = a.err && blockIdx.x == 0;
    int nh = 0, np = 0;
    bool bad = false;
    if (a.history) {
        const int n = a.n_history[r];
        nh = min(max(n, 0), a.cap);
        bad |= nh != n;
        np = a.n_prompt ? min(max(a.n_prompt[r], 0), nh) : 0;
    }
    int b0 = 0, b1 = 0;
    if (a.bias_off) {
        b0 = a.bias_off[r];
        b1 = a.bias_off[r + 1];
        if (b0 < 0 || b1 < b0 || b1 > a.n_bias) { bad = true; b0 = b1 = 0; }
    }
    const uint32_t* mask = nullptr;
    bool none = false;        // nothing may be drawn
    if (a.mask) {
        const int m = a.mask_row ? a.mask_row[r] : r;
        if (m < -1 || m >= a.n_masks) { bad = none = true; }
        else if (m >= 0) mask = a.mask + m * a.ldm;
    }
    if (bad && tell && tid == 0) atomicOr(a.err, ERRB_BOUNDS);
    auto allowed = [&](int i) { return !none && (!mask || mask[i >> 5] >> (i & 31) & 1); };
    auto allowed_of = [&](int i) -> uint32_t {      // of the N ids from i on
        if (none) return 0;
        if (!mask) return 0xffffffffu;
        const uint32_t w0 = mask[i >> 5], w1 = (i & 31) > 32 - N ? mask[(i >> 5) + 1] : 0;
        return __funnelshift_r(w0, w1, i & 31);
    };
    const bool named = nh > 0 || b1 > b0;
    const int32_t* h = a.history + r * a.ldh;
    if (named) {
        for (int i = tid; i < hi - lo; i += P_THREADS) words[i] = 0;
        if (tid == 0) s_dup = s_count = 0;
        __syncthreads();
        for (int j = tid; j < nh; j += P_THREADS) {
            const int id = h[j];
            if (id >= a.V && tell) atomicOr(a.err, ERRB_BOUNDS);
            if (id < lo || id >= hi) continue;
            const uint32_t was = j < np ? atomicOr(&words[id - lo], P_SEEN) : atomicAdd(&words[id - lo], 1u);
            if (!(was & (P_SEEN | P_COUNT))) list[atomicAdd(&s_count, 1)] = (uint16_t)(id - lo);
        }
        for (int j = b0 + tid; j < b1; j += P_THREADS) {
            const int id = a.bias_ids[j];
            if ((id < 0 || id >= a.V) && tell) atomicOr(a.err, ERRB_BOUNDS);
            if (id >= lo && id < hi && atomicOr(&words[id - lo], P_BIAS) & P_BIAS) s_dup = 1;
        }
    }
    // ---- the slice through the mask
    if (!in_place || mask || none) {
        const int from = lo + head;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int p = tid + j * P_THREADS, i = from + p * N;
            if (p >= pieces) break;
            const uint32_t bits = allowed_of(i);
            if (in_place) {
                if (!(bits & ((1u << N) - 1))) *(uint4*)(out + i) = masked<T>(make_uint4(0, 0, 0, 0), 0);
                else
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (!(bits >> e & 1)) out[i + e] = from_f<T>(-INFINITY);
                continue;
            }
            if (!alike) {
                alignas(16) T t[N];
#pragma unroll
                for (int e = 0; e < N; ++e) t[e] = x[i + e];
                v[j] = *(const uint4*)t;
            }
            *(uint4*)(out + i) = masked<T>(v[j], bits);
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
    const float rep = a.rep ? a.rep[r] : 1.f, pres = a.pres ? a.pres[r] : 0.f, freq = a.freq ? a.freq[r] : 0.f;
    auto adjusted = [&](int id, uint32_t w) {
        float v = to_f(x[id]);
        if (w & (P_SEEN | P_COUNT)) v = v < 0.f ? v * rep : v / rep;
        if (w & P_COUNT) v -= fmaf(freq, (float)(w & P_COUNT), pres);
        return v;
    };
    for (int j = b0 + tid; j < b1; j += P_THREADS) {
        const int id = a.bias_ids[j];
        if (id < lo || id >= hi) continue;
        const uint32_t w = atomicOr(&words[id - lo], P_DONE);
        if (w & P_DONE || !allowed(id)) continue;
        float b = a.bias[j];
        if (s_dup) {
            b = 0.f;
            for (int i = b0; i < b1; ++i)
                if (a.bias_ids[i] == id) b += a.bias[i];
        }
        out[id] = from_f<T>(adjusted(id, w) + b);
    }
    for (int j = tid; j < s_count; j += P_THREADS) {
        const int id = lo + list[j];
        const uint32_t w = words[id - lo];
        if (!(w & P_BIAS) && allowed(id)) out[id] = from_f<T>(adjusted(id, w));
    }
}

template <typename T>
cudaError_t launch_t(int n, const ProcessArgs& a, cudaStream_t st) {
    const bool named = a.history || a.bias_off;
    if (!named && !a.mask && a.logits == a.out) return cudaSuccess;
    const int smem = named ? min(P_SLICE, a.V) * 6 : 0;
    // a per-device attribute: set on every call (a host-side table lookup)
    const cudaError_t e = cudaFuncSetAttribute(process_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SLICE * 6);
    if (e != cudaSuccess) return e;
    return launch_pdl(process_kernel<T>, dim3((a.V + P_SLICE - 1) / P_SLICE, n), P_THREADS, smem, st, a);
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
