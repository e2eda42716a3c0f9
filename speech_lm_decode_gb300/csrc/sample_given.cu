// q3tts_sample_given: the draw from logits with temperature, top-k, top-p and
// min-p from one given uniform number a row (definition in q3tts.h).
//
// A row belongs to a cluster of up to eight CTAs.  Each reads its slice of the
// logits once, keeps the quotients l in shared memory, and everything after
// that happens there; the CTAs exchange maxima, histograms and sums through
// distributed shared memory.  Kept weights are whole numbers (at most 2^40
// each), so no result depends on the order of a sum.
//   - k <= 128: the k-th largest of 512 group maxima bounds the k-th largest
//     value from below; the few values that reach it go to the first CTA, which
//     does the rest on that list.
//   - otherwise: one pass replaces l by e = exp(l - max), adds up the exact
//     weights and (top-p) a histogram of them, 16 bins an octave of e.  The
//     histogram says in which bins the top-p border lies; a second pass adds up
//     exactly what lies above them and lists what lies inside, and a radix
//     selection on the list finds the border (on the whole slices if the list
//     overflows or the histogram misjudged it).  Ids of a tie at the border are
//     kept from the lowest on: a second selection, on the ids.
//   - the draw: every warp has the kept weight of its run of ids, so only one
//     warp of one CTA scans its run.
// What bounds it: about 45 instructions a logit (division, exp, weight), not
// the 2 or 4 bytes read.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "pdl.cuh"
#include "sampler.cuh"

namespace q3 {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int GT = 512, GW = GT / 32;   // threads, warps of a CTA
constexpr int GIVEN_MAX_VOCAB = 262144; // whole weights of a row stay below 2^58
constexpr int MAX_CLUSTER = 8;
constexpr int LIST = 1024;              // entries of the candidate lists
constexpr int SMALL_K = 128;            // top-k that the list path takes
constexpr int GROUPS = 512;             // group maxima of a row
constexpr int BINS = 656;               // 41 octaves of 16 bins: e from 2^-41 to 1
constexpr uint32_t BIN0 = (127u - 40u) << 4;   // bits >> 19 of 2^-40

__device__ __forceinline__ float lval(const float* p, int i) { return p[i]; }
__device__ __forceinline__ float lval(const bf16* p, int i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void lval4(const float* p, float (&v)[4]) {
    const float4 a = __ldg((const float4*)p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void lval4(const bf16* p, float (&v)[4]) {
    const uint2 a = __ldg((const uint2*)p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// floor(e * 2^40) of 0 <= e <= 1, exactly
__device__ __forceinline__ u64 weight_of(float e) {
    const uint32_t b = __float_as_uint(e);
    return ((u64)((b & 0x7FFFFFu) | 0x800000u) << 17) >> min(127 - (int)(b >> 23), 63);
}
// the draws' exp of d <= 0 (spec_expf) with the rounding of the quotient done by
// adding 1.5 * 2^23 and the power of two added to the exponent: the same values
__device__ __forceinline__ float exp_of(float d) {
    const float c = fmaxf(d, -87.f);
    const float s = __fadd_rn(__fmul_rn(c, kInvLn2), 12582912.0f), n = __fsub_rn(s, 12582912.0f);
    const float r = __fsub_rn(__fsub_rn(c, __fmul_rn(n, kLn2Hi)), __fmul_rn(n, kLn2Lo));
    float p = 1.0f / 40320.0f;
    p = __fadd_rn(1.0f / 5040.0f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f / 720.0f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f / 120.0f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f / 24.0f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f / 6.0f, __fmul_rn(r, p));
    p = __fadd_rn(0.5f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f, __fmul_rn(r, p));
    p = __fadd_rn(1.0f, __fmul_rn(r, p));
    const float e = __uint_as_float(__float_as_uint(p) + ((__float_as_uint(s) - 0x4B400000u) << 23));
    return d < -86.0f ? 0.f : e;
}

// x / T rounded to nearest.  With y the rounded reciprocal of T, two residual
// corrections of x y give the rounded quotient (P. Markstein, IBM J. Res. Dev.
// 34, 1990) while nothing under- or overflows; other operands are divided.
struct Quotient {
    float T, y;
    bool fast;
    __device__ explicit Quotient(float t) : T(t), y(1.f / t), fast(t > 0x1p-32f && t < 0x1p32f) {}
    __device__ __forceinline__ bool in_range(float x) const {
        const float a = fabsf(x);
        return fast && ((a < 0x1p64f && (a > 0x1p-60f || a == 0.f)) || x == -INFINITY);
    }
    __device__ __forceinline__ float quick(float x) const {
        const float q0 = __fmul_rn(x, y);
        const float q1 = __fmaf_rn(__fmaf_rn(-q0, T, x), y, q0);
        const float q = __fadd_rn(__fmaf_rn(__fmaf_rn(-q1, T, x), y, q1), 0.f);   // -0 becomes +0
        return x == -INFINITY ? x : q;
    }
    __device__ __forceinline__ float operator()(float x) const {
        return in_range(x) ? quick(x) : __fadd_rn(__fdiv_rn(x, T), 0.f);
    }
};

struct GivenSmem {
    u64 hist64[2][256];          // radix passes, in turn
    u64 wsum[GW];                // kept weight of each warp's ids
    u64 red[GW + 1];
    u64 best;                    // largest (order key, ~id) of the slice
    u64 total, above;            // weight of the slice; of it above the bracket
    uint32_t hist[BINS];         // sums of mantissas, by e
    uint32_t maxima[GROUPS];     // first CTA: group maxima of the row
    alignas(16) uint32_t mine[GROUPS];   // a copy of them
    uint32_t lkey[LIST], skey[LIST];
    int lid[LIST], sid[LIST];
    int n_list, bad, pick;
    u64 pick64;
    int edge_bin;
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
    }
    return v;
}
// sum over the CTA, to every thread
__device__ u64 cta_sum64(GivenSmem& s, u64 v) {
    v = warp_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < GW; ++w) t += s.red[w];
    return t;
}
// inclusive scan over the CTA's threads
__device__ u64 cta_scan64(GivenSmem& s, u64 v) {
    const int warp = threadIdx.x >> 5;
    v = warp_scan64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) s.red[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < GW; ++w)
        if (w < warp) v += s.red[w];
    return v;
}

// One row's state that all its functions use.
template <typename T>
struct Row {
    GivenSmem& s;
    cg::cluster_group cl;
    float* e;            // the slice: l, then e
    const T* x;          // the row's logits
    Quotient q;
    int V, C, rank, slice, seg, base;   // base: id of the slice's first entry
    float m;             // largest l
    int first;           // its lowest id

    __device__ float l_of(int id) const { return q(lval(x, id)); }

    // Radix selection over (key, amount) pairs that each(f) walks on every CTA: the key at which the amounts from
    // the top, starting with `above`, reach the goal; reach(sum) says whether a sum does.  Returns whether there
    // is one; then *above is the amount above that key.  All threads of the cluster call it.
    template <class Each, class Reach>
    __device__ bool select(Each each, Reach reach, int bits, uint32_t* key, u64* above) {
        uint32_t prefix = 0, mask = 0;
        for (int shift = bits - 8, pass = 0; shift >= 0; shift -= 8, ++pass) {
            u64* h = s.hist64[pass & 1];
            if (threadIdx.x < 256) h[threadIdx.x] = 0;
            if (threadIdx.x == 0) s.pick = -1;
            __syncthreads();
            each([&](uint32_t k, u64 amount) {
                if ((k & mask) == prefix) atomicAdd(&h[(k >> shift) & 255u], amount);
            });
            cl.sync();
            u64 c = 0;
            if (threadIdx.x < 256)
                for (int r = 0; r < C; ++r) c += cl.map_shared_rank(h, r)[255 - threadIdx.x];
            const u64 incl = cta_scan64(s, c);
            if (threadIdx.x < 256 && !reach(*above + incl - c) && reach(*above + incl)) {
                s.pick = 255 - threadIdx.x;
                s.pick64 = incl - c;
            }
            __syncthreads();
            const int pick = s.pick;
            if (pick < 0) return false;   // the same on every CTA
            prefix |= (uint32_t)pick << shift;
            mask |= 255u << shift;
            *above += s.pick64;
            __syncthreads();
        }
        *key = prefix;
        return true;
    }
};

template <typename T>
__global__ void __launch_bounds__(GT, 2) sample_given_kernel(int V, int slice, const T* logits, int64_t ld,
                                                             const float* u_, const float* temp_, const int32_t* topk_,
                                                             const float* topp_, const float* minp_, int32_t* ids,
                                                             float* logprob, int* err) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) float e[];
    __shared__ __align__(16) GivenSmem s;
    // before the first access to another CTA's shared memory, all of the cluster's have started
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank();
    const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float temp = temp_[row], top_p = topp_[row], min_p = minp_[row];
    const int k = topk_[row];
    Row<T> R{s, cl, e, logits + row * ld, Quotient(temp > 0.f ? temp : 1.f), V, C, rank, slice, slice / GW,
             rank * slice, 0.f, 0};
    const int seg = R.seg, base = R.base, w0 = warp * seg;   // the warp's run of the slice

    // ---- quotients into shared memory; the largest, and maxima of groups of C lanes
    float mx = -INFINITY;
    int at = 0, bad = !(temp >= 0.f);
    {
        const T* x = R.x + base;
        const bool vec = ((uintptr_t)x & (4 * sizeof(T) - 1)) == 0;
#pragma unroll 4
        for (int i = w0 + lane * 4; i < w0 + seg; i += 128) {
            float v[4];
            if (vec && base + i + 3 < V) {
                lval4(x + i, v);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = base + i + j < V ? lval(x, i + j) : -INFINITY;
            }
            const bool quick = R.q.in_range(v[0]) && R.q.in_range(v[1]) && R.q.in_range(v[2]) && R.q.in_range(v[3]);
            if (quick) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = R.q.quick(v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = R.q(v[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= !(v[j] < INFINITY);
                if (v[j] > mx) { mx = v[j]; at = base + i + j; }
            }
            *(float4*)(e + i) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    {
        const uint32_t key = order_key(mx);
        u64 best = (u64)key << 32 | (uint32_t)~at;
        uint32_t gm = key;
        __syncwarp();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        for (int o = 1; o < C; o <<= 1) gm = max(gm, __shfl_xor_sync(0xffffffffu, gm, o));
        if ((lane & (C - 1)) == 0) cl.map_shared_rank(s.maxima, 0)[((rank * GW + warp) * 32 + lane) / C] = gm;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const u64 b = __shfl_xor_sync(0xffffffffu, best, o);
            best = b > best ? b : best;
        }
        if (lane == 0) s.red[warp] = best;
        if (tid == 0) s.n_list = 0;
        bad = __syncthreads_or(bad);
        if (tid == 0) {
            best = s.red[0];
            for (int w = 1; w < GW; ++w) best = s.red[w] > best ? s.red[w] : best;
            s.best = best;
            s.bad = bad;
        }
    }
    cl.sync();
    u64 best = 0;
    bad = 0;
    for (int r = 0; r < C; ++r) {
        const u64 b = *cl.map_shared_rank(&s.best, r);
        best = b > best ? b : best;
        bad |= *cl.map_shared_rank(&s.bad, r);
    }
    const float m = R.m = order_key_inv((uint32_t)(best >> 32));
    const int first = R.first = (int)~(uint32_t)best;
    const bool fails = bad || m == -INFINITY;
    // the largest alone: greedy, or nothing else passes top-p or min-p
    if (fails || temp == 0.f || !(top_p > 0.f) || !(min_p <= 1.f)) {
        if (rank == 0 && tid == 0) {
            ids[row] = fails ? -1 : first;
            if (logprob) logprob[row] = fails ? __uint_as_float(0x7fc00000u) : 0.f;
            if (fails && err) atomicOr(err, ERRB_NAN);
        }
        cl.sync();   // no CTA leaves while another reads its shared memory
        return;
    }
    const float u = u_[row];
    auto target_of = [&](u64 Z) {
        const u64 t = u > 0.f ? (u64)__dmul_rn((double)u, (double)Z) : 0ull;
        return min(t, Z - 1);
    };
    auto finish = [&](int id, float l, u64 Z) {
        ids[row] = id;
        if (logprob) logprob[row] = (float)((double)__fsub_rn(l, m) - log((double)Z * 0x1p-40));
    };

    // ---- small k: the list path
    const bool with_k = k > 0 && k < V;
    if (with_k && k <= SMALL_K) {
        s.mine[tid] = cl.map_shared_rank(s.maxima, 0)[tid];
        if (tid == 0) s.pick = 0;
        __syncthreads();
        {
            const uint32_t v = s.mine[tid];
            int ge = 0;
#pragma unroll 8
            for (int j = 0; j < GROUPS; j += 4) {
                const uint4 o = *(const uint4*)&s.mine[j];
                ge += (o.x >= v) + (o.y >= v) + (o.z >= v) + (o.w >= v);
            }
            if (ge >= k) atomicMax((unsigned*)&s.pick, v);
        }
        __syncthreads();
        const float tau = order_key_inv((uint32_t)s.pick);   // at least k values reach it
        GivenSmem* lead = cl.map_shared_rank(&s, 0);
        for (int i = w0 + lane * 4; i < w0 + seg; i += 128) {
            const float4 v = *(const float4*)(e + i);
            if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= tau) {
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (a[j] >= tau && base + i + j < V) {
                        const int n = atomicAdd(&lead->n_list, 1);
                        if (n < LIST) { lead->lkey[n] = order_key(a[j]); lead->lid[n] = base + i + j; }
                    }
            }
        }
        cl.sync();
        const int n = *cl.map_shared_rank(&s.n_list, 0);
        if (n <= LIST) {
            if (rank == 0) {
                // sorted by (l descending, id ascending)
                for (int i = tid; i < n; i += GT) {
                    const uint32_t a = s.lkey[i];
                    const int id = s.lid[i];
                    int r = 0;
                    for (int j = 0; j < n; ++j) r += s.lkey[j] > a || (s.lkey[j] == a && s.lid[j] < id);
                    s.skey[r] = a;
                    s.sid[r] = id;
                }
                __syncthreads();
                const uint32_t kth = s.skey[k - 1];
                // consecutive entries a thread: weights, those before them, what is kept
                constexpr int PER = LIST / GT;
                u64 w[PER], own = 0;
                float ex[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int i = tid * PER + j;
                    ex[j] = i < n && s.skey[i] >= kth ? exp_of(__fsub_rn(order_key_inv(s.skey[i]), m)) : -1.f;
                    w[j] = ex[j] >= 0.f ? weight_of(ex[j]) : 0ull;
                    own += w[j];
                }
                u64 before = cta_scan64(s, own) - own;
                const u64 Z = cta_sum64(s, own);
                const double limit = __dmul_rn((double)top_p, (double)Z);
                u64 kept = 0;
                u64* wk = reinterpret_cast<u64*>(e);   // the slice (2048 floats at least) is not needed any more
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int i = tid * PER + j;
                    const bool in = ex[j] >= 0.f && (i == 0 || ((top_p >= 1.f || (double)before < limit) && ex[j] >= min_p));
                    before += w[j];
                    if (!in) w[j] = 0;
                    kept += w[j];
                    if (i < n) wk[i] = w[j];
                }
                const u64 Zk = cta_sum64(s, kept);
                const u64 target = target_of(Zk);
                if (tid == 0) s.pick = 0x7fffffff;
                __syncthreads();
                // ids are few: the weight up to an id is summed for each of them
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int i = tid * PER + j;
                    if (i >= n || w[j] == 0) continue;
                    u64 upto = 0;
                    for (int o = 0; o < n && s.skey[o] >= kth; ++o)
                        if (s.sid[o] <= s.sid[i]) upto += wk[o];
                    if (upto > target) atomicMin(&s.pick, s.sid[i]);
                }
                __syncthreads();
                if (tid == 0) finish(s.pick, R.l_of(s.pick), Zk);
            }
            cl.sync();
            return;
        }
    }

    // ---- the k-th largest value
    float kth = -INFINITY;
    if (with_k) {
        uint32_t key = 0;
        u64 above = 0;
        R.select([&](auto f) {
            for (int i = w0 + lane; i < w0 + seg; i += 32)
                if (base + i < V) f(order_key(e[i]), 1ull);
        }, [&](u64 n) { return n >= (u64)k; }, 32, &key, &above);
        kth = order_key_inv(key);
    }

    // ---- e in place of l; weights, and their histogram where top-p needs it
    const bool with_p = top_p < 1.f;
    for (int i = tid; i < BINS; i += GT) s.hist[i] = 0;
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    u64 sum = 0, kept = 0;
    for (int i = w0 + lane * 4; i < w0 + seg; i += 128) {
        const float4 v = *(const float4*)(e + i);
        float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = a[j] >= kth ? exp_of(__fsub_rn(a[j], m)) : 0.f;
            const u64 w = weight_of(a[j]);
            sum += w;
            if (a[j] >= min_p) kept += w;
            if (with_p) {
                const uint32_t b = __float_as_uint(a[j]);
                // 16 bits of the mantissa: at most 2^15 logits a slice, so 32 bits hold their sum
                if (b >= BIN0 << 19) atomicAdd(&s.hist[(b >> 19) - BIN0], ((b & 0x7FFFFFu) | 0x800000u) >> 8);
            }
        }
        *(float4*)(e + i) = make_float4(a[0], a[1], a[2], a[3]);
    }
    float lo = 0.f;            // entries with e below it are not kept
    kept = warp_sum64(kept);
    if (lane == 0) s.wsum[warp] = kept;
    if (with_p) {
        sum = cta_sum64(s, sum);
        if (tid == 0) s.total = sum;
        cl.sync();
        u64 Z = 0;
        for (int r = 0; r < C; ++r) Z += *cl.map_shared_rank(&s.total, r);
        const double limit = __dmul_rn((double)top_p, (double)Z);
        // the bin in which the histogram, from the top, passes the limit
        {
            if (tid == 0) s.edge_bin = 0;
            u64 h2[2] = {0, 0};
            for (int j = 0; j < 2; ++j) {
                const int b = BINS - 1 - (tid * 2 + j);
                if (b >= 0) {
                    for (int r = 0; r < C; ++r) h2[j] += cl.map_shared_rank(s.hist, r)[b];
                    const int o = (b >> 4) - 15;   // of e's exponent: weights in units of 2^-40
                    h2[j] = o >= 0 ? h2[j] << o : h2[j] >> -o;
                }
            }
            const u64 incl = cta_scan64(s, h2[0] + h2[1]);
            const u64 all = cta_sum64(s, h2[0] + h2[1]);
            const double lim = (double)top_p * (double)all;
            u64 c = incl - h2[0] - h2[1];
            for (int j = 0; j < 2; ++j) {
                if ((double)c < lim && (double)(c + h2[j]) >= lim) s.edge_bin = BINS - 1 - (tid * 2 + j);
                c += h2[j];
            }
            __syncthreads();
        }
        float hi;
        uint32_t edge = 0;
        u64 above = 0;
        bool found = false;
        auto inside = [&](float v) { return v >= lo && v < hi; };
        auto each_inside = [&](auto f) {   // f(entry of the slice) for what lies in the bracket
            if (s.n_list <= LIST) {
                for (int i = tid; i < s.n_list; i += GT) f(s.lid[i]);
            } else {
                for (int i = w0 + lane; i < w0 + seg; i += 32)
                    if (base + i < V && inside(e[i])) f(i);
            }
        };
        for (int attempt = 0; attempt < 2 && !found; ++attempt) {
            const int b = s.edge_bin;
            lo = attempt || b <= 1 ? 0.f : __uint_as_float((uint32_t)(b - 1 + BIN0) << 19);
            hi = attempt ? 2.f : __uint_as_float((uint32_t)(b + 2 + BIN0) << 19);
            __syncthreads();
            if (tid == 0) s.n_list = 0;
            __syncthreads();
            sum = kept = 0;
            for (int i = w0 + lane * 4; i < w0 + seg; i += 128) {
                const float4 v = *(const float4*)(e + i);
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (a[j] >= hi) {
                        const u64 w = weight_of(a[j]);
                        sum += w;
                        if (a[j] >= min_p) kept += w;
                    } else if (a[j] >= lo && base + i + j < V) {
                        const int n = atomicAdd(&s.n_list, 1);
                        if (n < LIST) s.lid[n] = i + j;
                    }
                }
            }
            kept = warp_sum64(kept);
            if (lane == 0) s.wsum[warp] = kept;
            sum = cta_sum64(s, sum);
            if (tid == 0) s.above = sum;
            cl.sync();
            above = 0;
            for (int r = 0; r < C; ++r) above += *cl.map_shared_rank(&s.above, r);
            // (a border above the bracket: nothing to select)
            found = (double)above < limit && R.select([&](auto f) {
                each_inside([&](int i) { if (e[i] > 0.f) f(order_key(R.l_of(base + i)), weight_of(e[i])); });
            }, [&](u64 n) { return !((double)n < limit); }, 32, &edge, &above);
            if (found && !attempt) {
                // e is monotone in l up to rounding: the border has to lie clearly inside the bracket
                const float eb = exp_of(__fsub_rn(order_key_inv(edge), m));
                if (!((lo == 0.f || eb > lo * 1.0001f) && (hi == 2.f || eb < hi * 0.9999f))) found = false;
            }
            cl.sync();   // s.above and the histograms have been read
        }
        if (found) {
            // of the ids at the border, the lowest ones until the limit
            const u64 w = weight_of(exp_of(__fsub_rn(order_key_inv(edge), m)));
            long long n = (long long)((limit - (double)above) / (double)w);
            while (n > 0 && !((double)(above + (n - 1) * w) < limit)) --n;
            while ((double)(above + n * w) < limit) ++n;
            u64 ties = 0;
            each_inside([&](int i) { ties += order_key(R.l_of(base + i)) == edge; });
            ties = cta_sum64(s, ties);
            if (tid == 0) s.total = ties;
            cl.sync();
            u64 all = 0;
            for (int r = 0; r < C; ++r) all += *cl.map_shared_rank(&s.total, r);
            int cut = V;
            if (n < (long long)all) {
                uint32_t key = 0;
                u64 zero = 0;
                // the n-th smallest id is the n-th largest of 2^24 - 1 - id
                R.select([&](auto f) {
                    each_inside([&](int i) {
                        if (order_key(R.l_of(base + i)) == edge) f(0xFFFFFFu - (uint32_t)(base + i), 1ull);
                    });
                }, [&](u64 c) { return c >= (u64)n; }, 24, &key, &zero);
                cut = (int)(0xFFFFFFu - key);
            }
            each_inside([&](int i) {
                const uint32_t key = order_key(R.l_of(base + i));
                if (key > edge || (key == edge && base + i <= cut)) {
                    if (e[i] >= min_p) atomicAdd(&s.wsum[i / seg], weight_of(e[i]));
                } else {
                    e[i] = 0.f;
                }
            });
        } else {
            // rounding of the limit: everything is kept
            lo = 0.f;
            kept = 0;
            for (int i = w0 + lane; i < w0 + seg; i += 32) kept += e[i] >= min_p ? weight_of(e[i]) : 0ull;
            kept = warp_sum64(kept);
            __syncthreads();
            if (lane == 0) s.wsum[warp] = kept;
        }
    }
    cl.sync();

    // ---- the draw: the warp whose run of ids holds the target
    u64 Z = 0, before = 0, mine = 0;
    for (int r = 0; r < C; ++r)
        for (int w = 0; w < GW; ++w) {
            const u64 v = cl.map_shared_rank(s.wsum, r)[w];
            if (r < rank || (r == rank && w < warp)) before += v;
            if (r == rank && w == warp) mine = v;
            Z += v;
        }
    const u64 target = target_of(Z);
    if (before <= target && target < before + mine) {
        for (int i = w0 + lane * 4; ; i += 128) {
            const float4 v = *(const float4*)(e + i);
            const float a[4] = {v.x, v.y, v.z, v.w};
            u64 w[4], own = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = a[j] >= lo && a[j] >= min_p && a[j] > 0.f ? weight_of(a[j]) : 0ull;
                own += w[j];
            }
            const u64 incl = warp_scan64(own);
            const u64 all = __shfl_sync(0xffffffffu, incl, 31);
            if (target < before + all) {
                u64 run = before + incl - own;
                if (run <= target && target < run + own) {
                    int j = 0;
                    while (target >= run + w[j]) run += w[j++];
                    const int id = base + i + j;
                    finish(id, R.l_of(id), Z);
                }
                break;
            }
            before += all;
            if (i - lane * 4 + 128 >= w0 + seg) break;
        }
    }
    cl.sync();
}

template <typename T>
cudaError_t launch_t(int n, int V, const void* logits, int64_t ld, const float* u, const float* temp,
                     const int32_t* topk, const float* topp, const float* minp, int32_t* ids, float* logprob, int* err,
                     cudaStream_t st) {
    // CTAs of a row: enough for slices of at most 19456 logits (76 KB, two CTAs an SM); with few rows, more of them
    // as long as they fill the GPU twice at most and a slice has 4096 logits
    int C = 1;
    while (C < MAX_CLUSTER && ((V + C - 1) / C > 19456 || ((int64_t)n * C * 2 <= 2 * device_sm_count() && V / (2 * C) >= 4096)))
        C *= 2;
    const int slice = ((V + C - 1) / C + GW * 128 - 1) / (GW * 128) * (GW * 128);
    const int smem = slice * (int)sizeof(float);
    // a per-device attribute: set on every call (a host-side table lookup)
    cudaError_t e = cudaFuncSetAttribute(sample_given_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         GIVEN_MAX_VOCAB / MAX_CLUSTER * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n * C);
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_given_kernel<T>, V, slice, (const T*)logits, ld, u, temp, topk, topp, minp,
                              ids, logprob, err);
}

}  // namespace

cudaError_t launch_sample_given(int n, int V, const void* logits, int dtype, int64_t ld, const float* u,
                                const float* temp, const int32_t* topk, const float* topp, const float* minp,
                                int32_t* ids, float* logprob, int* err, cudaStream_t st) {
    return dtype == Q3_BF16 ? launch_t<bf16>(n, V, logits, ld, u, temp, topk, topp, minp, ids, logprob, err, st)
                            : launch_t<float>(n, V, logits, ld, u, temp, topk, topp, minp, ids, logprob, err, st);
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
