// q3tts_sample_given: the draw from logits with temperature, top-k, top-p and
// min-p from one given uniform number a row (definition in q3tts.h).
#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "pdl.cuh"
#include "sampler.cuh"

namespace q3 {

namespace {

constexpr int GT = 512;                 // threads of a row
constexpr int GIVEN_MAX_VOCAB = 262144; // whole weights of a row stay below 2^58

__device__ __forceinline__ float lval(const float* p, int i) { return p[i]; }
__device__ __forceinline__ float lval(const bf16* p, int i) { return __bfloat162float(p[i]); }

// floor(e * 2^40) of 0 <= e <= 1, exactly
__device__ __forceinline__ unsigned long long weight_of(float e) {
    const uint32_t b = __float_as_uint(e);
    const int sh = (int)(b >> 23) - 127 - 23 + 40;
    const unsigned long long m = (b & 0x7FFFFFu) | 0x800000u;
    return (b >> 23) == 0 ? 0ull : sh >= 0 ? m << sh : sh > -24 ? m >> -sh : 0ull;
}

struct GivenSmem {
    unsigned long long hist[256];
    unsigned long long scan[GT];
    unsigned long long v;
    int i, n;
};

// block sum / scan over the GT threads (thread order), inclusive; total to all
__device__ unsigned long long scan_incl(GivenSmem& s, unsigned long long v, unsigned long long* total) {
    __syncthreads();
    s.scan[threadIdx.x] = v;
    __syncthreads();
    for (int o = 1; o < GT; o <<= 1) {
        const unsigned long long a = threadIdx.x >= o ? s.scan[threadIdx.x - o] : 0ull;
        __syncthreads();
        s.scan[threadIdx.x] += a;
        __syncthreads();
    }
    *total = s.scan[GT - 1];
    return s.scan[threadIdx.x];
}

template <typename T>
__global__ void __launch_bounds__(GT) given_plain_kernel(int V, const T* logits, int64_t ld, const float* u_,
                                                         const float* temp_, const int32_t* topk_, const float* topp_,
                                                         const float* minp_, int32_t* ids, float* logprob, int* err) {
    pdl_wait();
    pdl_trigger();
    __shared__ GivenSmem s;
    const int r = blockIdx.x, tid = threadIdx.x;
    const T* x = logits + r * ld;
    const float temp = temp_[r];
    const float div = temp > 0.f ? temp : 1.f;
    auto l_of = [&](int i) { const float v = __fdiv_rn(lval(x, i), div); return v == 0.f ? 0.f : v; };   // -0 is +0
    // the largest value and its lowest id, NaN and +inf
    unsigned long long best = 0;   // (order key, ~id)
    int bad = !(temp >= 0.f);
    for (int i = tid; i < V; i += GT) {
        const float v = l_of(i);
        bad |= isnan(v) || v == INFINITY;
        const unsigned long long k = ((unsigned long long)order_key(v) << 32) | (uint32_t)~i;
        best = k > best ? k : best;
    }
    s.scan[tid] = best;
    bad = __syncthreads_or(bad);
    for (int o = GT / 2; o; o >>= 1) {
        if (tid < o && s.scan[tid + o] > s.scan[tid]) s.scan[tid] = s.scan[tid + o];
        __syncthreads();
    }
    const int first = (int)~(uint32_t)s.scan[0];
    const float m = order_key_inv((uint32_t)(s.scan[0] >> 32));
    if (bad || m == -INFINITY) {
        if (tid == 0) {
            ids[r] = -1;
            if (logprob) logprob[r] = __uint_as_float(0x7fc00000u);
            if (err) atomicOr(err, ERRB_NAN);
        }
        return;
    }
    if (temp == 0.f) {
        if (tid == 0) { ids[r] = first; if (logprob) logprob[r] = 0.f; }
        return;
    }
    auto w_of = [&](float v) { return weight_of(spec_expf(__fsub_rn(v, m))); };
    // top-k: the k-th largest key, eight bits a pass
    uint32_t kth = 0;
    const int k = topk_[r];
    if (k > 0 && k < V) {
        uint32_t prefix = 0, mask = 0;
        unsigned long long kk = k;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) s.hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += GT) {
                const uint32_t key = order_key(l_of(i));
                if ((key & mask) == prefix) atomicAdd(&s.hist[(key >> shift) & 255u], 1ull);
            }
            unsigned long long tot;
            __syncthreads();
            const unsigned long long c = tid < 256 ? s.hist[255 - tid] : 0ull;
            const unsigned long long incl = scan_incl(s, c, &tot);
            if (incl - c < kk && kk <= incl) { s.i = 255 - tid; s.v = incl - c; }
            __syncthreads();
            prefix |= (uint32_t)s.i << shift;
            mask |= 255u << shift;
            kk -= s.v;
        }
        kth = prefix;
    }
    // top-p: the key at which the weight from the top reaches top_p * Z, and
    // how many ids of that key are kept
    const float top_p = topp_[r];
    uint32_t edge = kth;
    int ties = V;   // ids with key == edge that are kept
    if (!(top_p >= 1.f)) {
        unsigned long long z = 0, Z;
        for (int i = tid; i < V; i += GT) {
            const float v = l_of(i);
            if (order_key(v) >= kth) z += w_of(v);
        }
        scan_incl(s, z, &Z);
        const double limit = __dmul_rn((double)top_p, (double)Z);
        unsigned long long above = 0;
        uint32_t prefix = 0, mask = 0;
        bool found = true;
        for (int shift = 24; shift >= 0 && found; shift -= 8) {
            __syncthreads();
            if (tid < 256) s.hist[tid] = 0;
            if (tid == 0) s.i = -1;
            __syncthreads();
            for (int i = tid; i < V; i += GT) {
                const float v = l_of(i);
                const uint32_t key = order_key(v);
                if (key >= kth && (key & mask) == prefix) atomicAdd(&s.hist[(key >> shift) & 255u], w_of(v));
            }
            __syncthreads();
            unsigned long long tot;
            const unsigned long long c = tid < 256 ? s.hist[255 - tid] : 0ull;
            const unsigned long long incl = scan_incl(s, c, &tot);
            if (tid < 256 && (double)(above + incl - c) < limit && !((double)(above + incl) < limit)) {
                s.i = 255 - tid;
                s.v = incl - c;
            }
            __syncthreads();
            found = s.i >= 0;
            if (found) {
                prefix |= (uint32_t)s.i << shift;
                mask |= 255u << shift;
                above += s.v;
            }
        }
        if (found) {
            edge = prefix;
            const unsigned long long w = w_of(order_key_inv(prefix));
            long long n = (long long)((limit - (double)above) / (double)w);
            while (n > 0 && !((double)(above + (n - 1) * w) < limit)) --n;
            while ((double)(above + n * w) < limit) ++n;
            ties = (int)min(n, (long long)V);
        } else if (!(0.0 < limit)) {   // top_p <= 0 or NaN: the largest alone
            edge = order_key(m);
            ties = 1;
        }
    }
    // kept weight in id order; thread t holds ids [t per, t per + per)
    const float min_p = minp_[r];
    const bool only_first = !(min_p <= 1.f);
    const int per = (V + GT - 1) / GT;
    const int i0 = min(tid * per, V), i1 = min(i0 + per, V);
    unsigned long long tot;
    unsigned long long n_tie = 0;
    for (int i = i0; i < i1; ++i) n_tie += order_key(l_of(i)) == edge;
    const unsigned long long tie0 = scan_incl(s, n_tie, &tot) - n_tie;
    auto kept = [&](int i, unsigned long long& rank) -> unsigned long long {
        const float v = l_of(i);
        const uint32_t key = order_key(v);
        if (key < edge) return 0ull;
        if (key == edge && rank++ >= (unsigned long long)ties) return 0ull;
        const float e = spec_expf(__fsub_rn(v, m));
        if (i != first && (only_first || !(e >= min_p))) return 0ull;
        return weight_of(e);
    };
    unsigned long long sum = 0, rank = tie0, Z;
    for (int i = i0; i < i1; ++i) sum += kept(i, rank);
    const unsigned long long incl = scan_incl(s, sum, &Z);
    const float u = u_[r];
    unsigned long long target = u > 0.f ? (unsigned long long)__dmul_rn((double)u, (double)Z) : 0ull;
    target = min(target, Z - 1);
    if (incl - sum <= target && target < incl) {
        unsigned long long run = incl - sum;
        rank = tie0;
        for (int i = i0; i < i1; ++i) {
            run += kept(i, rank);
            if (run > target) {
                ids[r] = i;
                if (logprob) logprob[r] = (float)((double)__fsub_rn(l_of(i), m) - log((double)Z * 0x1p-40));
                break;
            }
        }
    }
}

}  // namespace

cudaError_t launch_sample_given(int n, int V, const void* logits, int dtype, int64_t ld, const float* u,
                                const float* temp, const int32_t* topk, const float* topp, const float* minp,
                                int32_t* ids, float* logprob, int* err, cudaStream_t st) {
    if (dtype == Q3_BF16)
        return launch_pdl(given_plain_kernel<bf16>, n, GT, 0, st, V, (const bf16*)logits, ld, u, temp, topk, topp,
                          minp, ids, logprob, err);
    return launch_pdl(given_plain_kernel<float>, n, GT, 0, st, V, (const float*)logits, ld, u, temp, topk, topp, minp,
                      ids, logprob, err);
}

}  // namespace q3

using namespace q3;

extern "C" int q3tts_sample_given(int n, int vocab, const void* logits, int dtype, int64_t logits_stride,
                                  const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                                  const float* min_p, int32_t* ids_out, float* logprob_out, int32_t* err,
                                  void* stream) {
    if (n < 0 || n > 65535) return paged_fail(Q3_ERR_ARG, "n must be in 0..65535");
    if (vocab < 1 || vocab > GIVEN_MAX_VOCAB) return paged_fail(Q3_ERR_ARG, "vocab must be in 1..%d", GIVEN_MAX_VOCAB);
    if (dtype != Q3_F32 && dtype != Q3_BF16) return paged_fail(Q3_ERR_ARG, "dtype must be Q3_F32 or Q3_BF16");
    if (n == 0) return Q3_OK;
    if (!logits || !u || !temperature || !top_k || !top_p || !min_p || !ids_out)
        return paged_fail(Q3_ERR_ARG, "NULL argument");
    if (logits_stride == 0) logits_stride = vocab;
    if (logits_stride < vocab) return paged_fail(Q3_ERR_ARG, "logits_stride is less than vocab");
    const cudaError_t e = launch_sample_given(n, vocab, logits, dtype, logits_stride, u, temperature, top_k, top_p,
                                              min_p, ids_out, logprob_out, err, (cudaStream_t)stream);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "draw: %s", cudaGetErrorString(e));
    return Q3_OK;
}
