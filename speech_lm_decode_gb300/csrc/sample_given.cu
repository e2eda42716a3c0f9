// q3tts_sample_given: the draw from logits with temperature, top-k, top-p and
// min-p from one given uniform number a row (definition in q3tts.h).
//
// A row belongs to one CTA or to a cluster of up to eight, as many as run at
// once with all rows.  Where a CTA's slice fits (HELD) it is read once into
// shared memory and everything after that happens there; else each pass reads
// the row again, from L2 mostly, and forms e again.  Against clusters of eight
// that hold every slice, 256 rows of 151936 bf16 logits took 180 us instead of
// 309 (213 since the products of e are rounded by themselves again): the meetings
// of a cluster cost more than the passes over L2.  The CTAs of
// a row exchange maxima, histograms, lists and sums through distributed shared
// memory.  Kept weights are whole numbers (at most 2^40 each), so no result
// depends on the order of a sum.
//   - k <= 128: the k-th largest of 512 group maxima bounds the k-th largest
//     value from below; the few values that reach it go to the first CTA, which
//     does the rest on that list while the others leave.
//   - otherwise: one pass forms e = exp(l - max), adds up the exact weights and
//     (top-p) a histogram of them, 128 bins an octave of e.  The histogram says
//     in which bin the top-p border lies; a second pass adds up exactly what
//     lies above it and lists what lies inside, and entries of the list find
//     the weight in front of them.  A bin with more entries than a list holds is
//     searched by radix instead (and, of the ids that tie at the border, which
//     are kept).  A k above 128 is found the same way, by a histogram of max - l
//     and a list.
//   - the draw: every warp has the kept weight of its run of ids, so only one
//     run is scanned.
// What bounds it: the meetings of a row's CTAs and the latency of each step at
// small sizes (one row of 2048 logits, k 50: 10 us; 32 rows of 151936, k 50: 19
// us); at large ones about 87 instructions a logit (reading 8, quotient, exp and
// weights 29 in each of two passes, histogram 9, border 10), more than half of
// the time in the packed fp32 operations, and the 48 SMs of 152 that have one row
// of 256 where the others have two.
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
constexpr int MAX_SLICE = GIVEN_MAX_VOCAB / MAX_CLUSTER;   // that shared memory holds
constexpr int LIST = 1024;              // entries of a CTA's list
constexpr int MERGED = 1024;            // of the lists of a row together
constexpr int SMALL_K = 128;            // top-k that the list path takes
constexpr int GROUPS = 512;             // group maxima of a row
constexpr int BINS = 30 * 128;          // 128 bins an octave: e from 2^-29 to 2
constexpr int COARSE = BINS / 16;
constexpr uint32_t BIN0 = (127u - 29u) << 7;   // bits >> 16 of 2^-29

__device__ __forceinline__ float lval(const float* p, int i) { return p[i]; }
__device__ __forceinline__ float lval(const bf16* p, int i) { return __bfloat162float(p[i]); }
// four logits, as they lie in memory
__device__ __forceinline__ float4 lval4(const float* p) { return __ldg((const float4*)p); }
__device__ __forceinline__ uint2 lval4(const bf16* p) { return __ldg((const uint2*)p); }
__device__ __forceinline__ float4 four(const float4& a) { return a; }
__device__ __forceinline__ float4 four(const uint2& a) {
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xffff0000u));
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

// two fp32 values side by side: one instruction rounds both
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpk(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Products of exp_of2: with -0 as an addend that the compiler does not know (a kernel argument).  It fuses packed
// products and the sums that they enter, rounding modes or not, which it never does with scalar ones; an fma stays.
__device__ __forceinline__ f2 product2(f2 a, f2 b, f2 zeros) { return fma2(a, b, zeros); }
// exp_of of the two l - m.  Where that is below -86, exp_of is zero and this is
// not, but small enough (2^-124) for a weight of zero, which is all that counts.
__device__ __forceinline__ f2 exp_of2(f2 l, f2 minus_m, f2 zeros) {
    float d0, d1;
    unpk(add2(l, minus_m), d0, d1);
    const f2 c = pk(fmaxf(d0, -87.f), fmaxf(d1, -87.f));
    const f2 s = add2(product2(c, pk(kInvLn2, kInvLn2), zeros), pk(12582912.0f, 12582912.0f));
    const f2 n = add2(s, pk(-12582912.0f, -12582912.0f));
    // (n kLn2Hi is exact, kLn2Hi having 15 bits)
    const f2 r = add2(fma2(n, pk(-kLn2Hi, -kLn2Hi), c), product2(n, pk(-kLn2Lo, -kLn2Lo), zeros));
    auto both = [](float v) { return pk(v, v); };
    f2 p = both(1.0f / 40320.0f);
    p = add2(both(1.0f / 5040.0f), product2(r, p, zeros));
    p = add2(both(1.0f / 720.0f), product2(r, p, zeros));
    p = add2(both(1.0f / 120.0f), product2(r, p, zeros));
    p = add2(both(1.0f / 24.0f), product2(r, p, zeros));
    p = add2(both(1.0f / 6.0f), product2(r, p, zeros));
    p = add2(both(0.5f), product2(r, p, zeros));
    p = add2(both(1.0f), product2(r, p, zeros));
    p = add2(both(1.0f), product2(r, p, zeros));
    float p0, p1, s0, s1;
    unpk(p, p0, p1);
    unpk(s, s0, s1);
    return pk(__uint_as_float(__float_as_uint(p0) + (__float_as_uint(s0) << 23) - (0x4B400000u << 23)),
              __uint_as_float(__float_as_uint(p1) + (__float_as_uint(s1) << 23) - (0x4B400000u << 23)));
}

// A thread's sum of weights floor(2^40 e), two e at a time: 2^20 e is split into
// its whole part and the rest, 2^20 times the rest again, by additions to 2^23
// that round toward zero, so that the two parts stand in the low bits of floats
// and are added as integers (2^11 weights at most).
struct WeightSum {
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(f2 e) {
        const f2 up = pk(0x1p20f, 0x1p20f), two23 = pk(0x1p23f, 0x1p23f);
        f2 h, l;
        asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(h) : "l"(e), "l"(up), "l"(two23));
        const f2 rest = fma2(e, up, fma2(h, pk(-1.f, -1.f), two23));
        asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(l) : "l"(rest), "l"(up), "l"(two23));
        hi += (uint32_t)h + (uint32_t)(h >> 32);
        lo += (uint32_t)l + (uint32_t)(l >> 32);
    }
    // of n weights
    __device__ __forceinline__ u64 sum(int n) const {
        return ((u64)(hi - (uint32_t)n * 0x4B000000u) << 20) + (lo - (uint32_t)n * 0x4B000000u);
    }
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
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
    // Whether quotient2 serves a row whose largest logit is x and m its quotient: quotients far below m, which overflow
    // may have made NaN, have no weight, and those next to zero, which may be a step off, are lost beside m.
    __device__ bool row(float x, float m) const { return fast && fabsf(x) < 0x1p64f && fabsf(m) > 0x1p-30f && m > -0x1p20f; }
    __device__ __forceinline__ float operator()(float x) const {
        return in_range(x) ? quick(x) : __fadd_rn(__fdiv_rn(x, T), 0.f);
    }
};

struct Merged {              // the lists of all CTAs of a row: weights, order keys, ids
    u64 w[MERGED];
    uint32_t key[MERGED];
    int id[MERGED];
};

struct GivenSmem {
    u64 wsum[GW];                // kept weight of each warp's ids
    u64 red[GW + 1];
    u64 total, above, kept;      // weight of the slice; of it above the bin; kept
    union {                      // a histogram has been read by all CTAs when its bin's lists are merged
        struct {
            uint32_t hist[BINS];     // sums of mantissas by e, or counts by max - l, from the top
            uint32_t coarse[COARSE]; // of 16 bins each
        };
        Merged lists;                // (HELD)
    };
    union {                      // a radix selection follows where the lists have not done
        struct {
            uint32_t lkey[LIST];     // this CTA's list: order keys, ids, e
            int lid[LIST];
            float le[LIST];
        };
        uint32_t radix[2][3 * 256];  // passes in turn
    };
    uint32_t maxima[GROUPS];     // first CTA: group maxima of the row
    unsigned short between[LIST];  // merged entries among which the border is
    int n_between;
    u64 kept_to, cut_from;       // and their ends
    uint32_t best;               // largest order key of the slice
    int n_list, pick, cut;
    uint32_t edge;               // order key and id of the last entry that top-p keeps
    u64 pick64;
    double logz;
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

// *p of CTA r of the cluster (volatile: eight ranks' addresses are not kept in registers between the calls)
template <class P>
__device__ __forceinline__ P from_cta(const P* p, int r) {
    static_assert(sizeof(P) == 4 || sizeof(P) == 8, "");
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    if constexpr (sizeof(P) == 4) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
        return (P)v;
    } else {
        u64 v;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
        return (P)v;
    }
}
// *p of every CTA of the cluster, all loads in flight at once: f(rank, value)
template <class P, class F>
__device__ __forceinline__ void from_all(cg::cluster_group& cl, int C, P* p, F f) {
    P v[MAX_CLUSTER];
#pragma unroll
    for (int r = 0; r < MAX_CLUSTER; ++r)
        if (r < C) v[r] = from_cta(p, r);
#pragma unroll
    for (int r = 0; r < MAX_CLUSTER; ++r)
        if (r < C) f(r, v[r]);
}

// two quotients by t with the reciprocal y; by 1: the numbers themselves
__device__ __forceinline__ f2 quotient2(f2 x, float t, float y) {
    const f2 yy = pk(y, y), tt = pk(-t, -t);
    const f2 q0 = mul2(x, yy);
    const f2 q1 = fma2(fma2(q0, tt, x), yy, q0);
    return fma2(fma2(q1, tt, x), yy, q1);
}

// One row's state that all its functions use.  HELD: the slice is in shared
// memory, as logits first and then as e; otherwise it is read again each time
// (from L2, mostly) and e formed again.
template <typename T, bool HELD>
struct Row {
    GivenSmem& s;
    cg::cluster_group cl;
    float* e;            // HELD: the slice: logits, then e
    Merged& M;
    const T* x;          // the row's logits
    Quotient q;
    int V, C, rank, slice, seg, base;   // base: id of the slice's first entry
    float m;             // largest l
    float kth;           // entries below it have e = 0
    bool vec;            // the slice is aligned for loads of four
    bool quick;          // quotient2 serves the row, with (qt, qy); else its quotients are formed one by one in front of it
    float qt, qy;
    f2 zeros;            // two of -0 (product2)

    __device__ float l_of(int id) const { return q(lval(x, id)); }
    // four logits from the row; -inf behind its end
    __device__ __forceinline__ float4 fetch4(int i) const {
        if (vec && base + i + 3 < V) return four(lval4(x + base + i));
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = base + i + j < V ? lval(x, base + i + j) : -INFINITY;
        return make_float4(v[0], v[1], v[2], v[3]);
    }
    // f(i, four logits) for the entries [from, end) of the slice, by one warp, with NB loads in flight; Q: quotients
    // where quick is not set
    template <int NB, bool Q = false, class F>
    __device__ __forceinline__ void walk_row(int from, int end, F f) const {
        const int lane = threadIdx.x & 31;
        const int plain = vec && (!Q || quick) ? max(min(end, from + ((V - base - from) & ~127)), from) : from;   // in whole blocks up to here
        int i0 = from + lane * 4;
        for (; i0 < plain; i0 += 128 * NB) {
            decltype(lval4(x)) r[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i0 + 128 * j < plain) r[j] = lval4(x + base + i0 + 128 * j);
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i0 + 128 * j < plain) f(i0 + 128 * j, four(r[j]));
        }
#pragma unroll 1
        for (i0 = plain + lane * 4; i0 < end; i0 += 128) {
            float4 v = fetch4(i0);
            if (Q && !quick) v = slow4(v);
            f(i0, v);
        }
    }
    // the same over what shared memory holds (logits, later e), or over the row's logits
    template <int NB, bool Q = false, class F>
    __device__ __forceinline__ void walk(int from, int end, F f) const {
        if constexpr (HELD) {
#pragma unroll 2
            for (int i = from + (int)(threadIdx.x & 31) * 4; i < end; i += 128) f(i, *(const float4*)(e + i));
        } else {
            walk_row<NB, Q>(from, end, f);
        }
    }
    __device__ __forceinline__ float raw(int i) const {
        return HELD ? e[i] : base + i < V ? lval(x, base + i) : -INFINITY;
    }
    __device__ __forceinline__ float4 slow4(const float4& v) const { return make_float4(q(v.x), q(v.y), q(v.z), q(v.w)); }
    // e of four logits (quotients where quick is not set)
    __device__ __forceinline__ void e_of(const float4& v, float (&a)[4]) const {
        const f2 l0 = quotient2(pk(v.x, v.y), qt, qy), l1 = quotient2(pk(v.z, v.w), qt, qy);
        unpk(exp_of2(l0, pk(-m, -m), zeros), a[0], a[1]);
        unpk(exp_of2(l1, pk(-m, -m), zeros), a[2], a[3]);
        if (kth > -INFINITY) {
            float l[4];
            unpk(l0, l[0], l[1]);
            unpk(l1, l[2], l[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = l[j] >= kth ? a[j] : 0.f;
        }
    }
    // e of the slice, once it is formed
    __device__ __forceinline__ void e4(int i, float (&a)[4]) const {
        if constexpr (HELD) {
            const float4 v = *(const float4*)(e + i);
            a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
        } else {
            const float4 v = fetch4(i);
            e_of(quick ? v : slow4(v), a);
        }
    }
    __device__ __forceinline__ float e1(int i) const {
        if constexpr (HELD) return e[i];
        if (base + i >= V) return 0.f;
        const float l = l_of(base + i);
        return l >= kth ? exp_of(__fsub_rn(l, m)) : 0.f;
    }

    // Radix selection over (key, amount) pairs that each(f) walks on every CTA: the key at which the amounts from
    // the top, starting with `above`, reach the goal; reach(sum) says whether a sum does.  Returns whether there
    // is one; then *above is the amount above that key.  All threads of the cluster call it.  Amounts (up to
    // 2^41) are added in three parts of 14 bits, as 32-bit atomics are the native ones: 2^15 entries a slice fit.
    template <class Each, class Reach>
    __device__ bool select(Each each, Reach reach, int bits, uint32_t* key, u64* above) {
        uint32_t prefix = 0, mask = 0;
        for (int shift = bits - 8, pass = 0; shift >= 0; shift -= 8, ++pass) {
            uint32_t* h = s.radix[pass & 1];
            for (int i = threadIdx.x; i < 3 * 256; i += GT) h[i] = 0;
            if (threadIdx.x == 0) s.pick = -1;
            __syncthreads();
            each([&](uint32_t k, u64 amount) {
                if ((k & mask) == prefix) {
                    uint32_t* d = h + ((k >> shift) & 255u);
                    atomicAdd(d, (uint32_t)amount & 0x3FFFu);
                    if (amount >> 14) {
                        atomicAdd(d + 256, (uint32_t)(amount >> 14) & 0x3FFFu);
                        atomicAdd(d + 512, (uint32_t)(amount >> 28));
                    }
                }
            });
            cl.sync();
            u64 c = 0;
            if (threadIdx.x < 256) {
                uint32_t* d = &h[255 - threadIdx.x];
                from_all(cl, C, d, [&](int, uint32_t v) { c += v; });
                from_all(cl, C, d + 256, [&](int, uint32_t v) { c += (u64)v << 14; });
                from_all(cl, C, d + 512, [&](int, uint32_t v) { c += (u64)v << 28; });
            }
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

    // The bin of the cluster's histograms in which the running sum of weigh(entry, bin) passes the goal (into
    // s.edge_bin, -1: none) and the sum in front of it (s.pick64).  All threads of the cluster call it; its CTAs have
    // to get the same, as what they do next, and how often they meet, goes by it.
    // goal(): sets the goal, once the CTAs have met.
    template <class Weigh, class Reach, class Goal>
    __device__ void locate(Weigh weigh, Reach reach, Goal goal) {
        const int t = threadIdx.x;
        __syncthreads();
        if (t < COARSE) {
            uint32_t c = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) c += s.hist[t * 16 + ((i + t) & 15)];
            s.coarse[t] = c;
        }
        if (t == 0) { s.pick = -1; s.edge_bin = -1; s.pick64 = 0; }
        cl.sync();
        u64 c = 0;
        if (t < COARSE) from_all(cl, C, &s.coarse[t], [&](int, uint32_t v) { c += weigh(v, t * 16); });
        goal();
        u64 incl = cta_scan64(s, c);
        if (t < COARSE && !reach(incl - c) && reach(incl)) { s.pick = t; s.pick64 = incl - c; }
        if (t == COARSE - 1 && !reach(incl)) s.pick64 = incl;   // none: all of it lies in front, on every CTA alike
        __syncthreads();
        if (s.pick >= 0 && t < 32) {
            const int b = s.pick * 16 + (t & 15);
            c = 0;
            from_all(cl, C, &s.hist[b], [&](int, uint32_t v) { c += weigh(v, b); });
            if (t >= 16) c = 0;
            const u64 front = s.pick64;
            incl = warp_scan64(c) + front;
            __syncwarp();
            if (t < 16 && !reach(incl - c) && reach(incl)) { s.edge_bin = b; s.pick64 = incl - c; }
        }
        __syncthreads();
    }

    // Adds an entry to this CTA's list; one that finds no place is only counted.
    __device__ void push(uint32_t key, int id, float ev) {
        const int n = atomicAdd(&s.n_list, 1);
        if (n < LIST) { s.lkey[n] = key; s.lid[n] = id; s.le[n] = ev; }
    }
    // The lists of all CTAs, by rank, into the merged ones of each; *own: where this CTA's begins.  Returns their
    // length, or -1 if one of them overflowed or all are more than MERGED.  All threads of the cluster call it.
    __device__ int merge(int* own) {
        cl.sync();
        int total = 0, n[MAX_CLUSTER];
        *own = 0;
        from_all(cl, C, &s.n_list, [&](int r, int v) {
            if (r < rank) *own += v;
            total += v;
            n[r] = v;
        });
        if (total > MERGED) return -1;
        bool fits = true;
#pragma unroll
        for (int r = 0; r < MAX_CLUSTER; ++r)
            if (r < C) fits = fits && n[r] <= LIST;
        if (!fits) return -1;
        for (int i = threadIdx.x; i < total; i += GT) {
            int from = 0, at = i;
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER - 1; ++r)
                if (r < C - 1 && from == r && at >= n[r]) { at -= n[r]; ++from; }
            const GivenSmem* o = cl.map_shared_rank(&s, from);
            const uint32_t key = o->lkey[at];
            const int id = o->lid[at];
            const float ev = o->le[at];
            M.key[i] = key;
            M.id[i] = id;
            M.w[i] = weight_of(ev);
        }
        __syncthreads();
        return total;
    }
};

template <typename T, bool HELD>
__global__ void __launch_bounds__(GT, 2) sample_given_kernel(int V, int slice, int n, int ahead, const T* logits, int64_t ld,
                                                             const float* u_, const float* temp_, const int32_t* topk_,
                                                             const float* topp_, const float* minp_, int32_t* ids,
                                                             float* logprob, int* err, f2 zeros) {
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
    Merged& M = HELD ? s.lists : *reinterpret_cast<Merged*>(e);
    Row<T, HELD> R{s, cl, e, M, logits + row * ld, Quotient(temp > 0.f ? temp : 1.f), V, C, rank, slice, slice / GW,
                   rank * slice, 0.f, -INFINITY, false, true, 1.f, 1.f, zeros};
    R.vec = ((uintptr_t)(R.x + R.base) & (4 * sizeof(T) - 1)) == 0;
    const int seg = R.seg, base = R.base, w0 = warp * seg;   // the warp's run of the slice

    // ---- logits into shared memory; the largest (division is monotone: its quotient is the largest too), and maxima
    // of groups of C lanes
    float mx = -INFINITY;   // NaN once it has met one
    R.template walk_row<5>(w0, w0 + seg, [&](int i, const float4& v) {
        mx = max_nan(mx, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
        if constexpr (HELD) *(float4*)(e + i) = v;
    });
    // the slice of the row that takes this one's place on the GPU, into L2
    if (HELD && row + ahead < n) {
        const char* next = (const char*)(R.x + (int64_t)ahead * ld + base);
        const int bytes = min(slice, V - base) * (int)sizeof(T);
        for (int i = tid * 128; i < bytes; i += GT * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i));
    }
    {
        const uint32_t key = mx < INFINITY && temp >= 0.f ? order_key(mx) : 0xFFFFFFFFu;   // all ones: the row fails
        uint32_t gm = key;
        __syncwarp();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        for (int o = 1; o < C; o <<= 1) gm = max(gm, __shfl_xor_sync(0xffffffffu, gm, o));
        if ((lane & (C - 1)) == 0) cl.map_shared_rank(s.maxima, 0)[((rank * GW + warp) * 32 + lane) / C] = gm;
        gm = __reduce_max_sync(0xffffffffu, key);
        if (tid == 0) { s.n_list = 0; s.best = 0; }
        __syncthreads();
        if (lane == 0) atomicMax(&s.best, gm);
    }
    cl.sync();
    uint32_t best = 0;
    from_all(cl, C, &s.best, [&](int, uint32_t b) { best = max(best, b); });
    const float m = R.m = R.q(order_key_inv(best));
    bool bad = best == 0xFFFFFFFFu || !(m < INFINITY);
    if (temp == INFINITY) {     // -inf / inf is no number
        int none = 0;
        for (int i = w0 + lane; i < w0 + seg; i += 32) none |= base + i < V && R.raw(i) == -INFINITY;
        none = __syncthreads_or(none);
        if (tid == 0) s.pick = none;
        cl.sync();
        from_all(cl, C, &s.pick, [&](int, int v) { bad |= v != 0; });
        cl.sync();
    }
    const bool fails = bad || m == -INFINITY;
    // the largest alone (the lowest id on ties): greedy, or nothing else passes top-p or min-p
    if (fails || temp == 0.f || !(top_p > 0.f) || !(min_p <= 1.f)) {
        if (tid == 0) s.pick = 0x7fffffff;
        __syncthreads();
        if (!fails)
            R.template walk<4>(w0, w0 + seg, [&](int i, const float4& v) {
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (R.q(a[j]) == m) atomicMin(&s.pick, base + i + j);   // (m is finite, what lies past the end is not)
            });
        cl.sync();
        int first = 0x7fffffff;
        if (rank == 0) from_all(cl, C, &s.pick, [&](int, int v) { first = min(first, v); });
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

    // ---- small k: the list path (its list is the first CTA's alone)
    const bool with_k = k > 0 && k < V;
    if (with_k && k <= SMALL_K) {
        // the k-th largest group maximum, rounded down to 16 bits of its key: at least k logits reach it.  One step of
        // 2^-7 lower, and every logit with the same quotient as any of those does too (unless quotients are denormal).
        uint32_t* mine = s.hist;   // (not yet in use)
        mine[tid] = cl.map_shared_rank(s.maxima, 0)[tid];
        __syncthreads();
        if (warp == 0) {
            uint32_t v[GROUPS / 32], t = 0;
#pragma unroll
            for (int i = 0; i < GROUPS / 32; ++i) v[i] = mine[lane + 32 * i];
#pragma unroll 1
            for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
                const uint32_t c = t | bit;
                int n = 0;
#pragma unroll
                for (int i = 0; i < GROUPS / 32; ++i) n += v[i] >= c;
                if (__reduce_add_sync(0xffffffffu, n) >= k) t = c;
            }
            if (lane == 0) s.pick = (int)t;
        }
        __syncthreads();
        const uint32_t tk = (uint32_t)s.pick;
        float tau = tk < 0x00820000u ? -INFINITY : order_key_inv(tk - 0x10000u);
        if (!(fabsf(R.q(tau)) > 0x1p-100f)) tau = -INFINITY;
        GivenSmem* lead = cl.map_shared_rank(&s, 0);
        R.template walk<4>(w0, w0 + seg, [&](int i, const float4& v) {
            if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= tau) {
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (a[j] >= tau && base + i + j < V) {
                        const int n = atomicAdd(&lead->n_list, 1);
                        if (n < LIST) { lead->lkey[n] = order_key(R.q(a[j])); lead->lid[n] = base + i + j; }
                    }
            }
        });
        cl.sync();
        const int n = *cl.map_shared_rank(&s.n_list, 0);
        if (n <= GT) {
            cl.sync();       // from here on the first CTA works on its own memory alone
            if (rank == 0) {
                // sorted by (l descending, id ascending): eight threads count an entry's rank
                for (int i0 = 0; i0 < n; i0 += GT / 8) {
                    const int i = min(i0 + tid / 8, n - 1);
                    const uint32_t a = s.lkey[i];
                    const int id = s.lid[i];
                    int r = 0;
                    for (int j = tid & 7; j < n; j += 8) {
                        const uint32_t o = s.lkey[j];
                        r += o > a || (o == a && s.lid[j] < id);
                    }
                    r += __shfl_xor_sync(0xffffffffu, r, 1);
                    r += __shfl_xor_sync(0xffffffffu, r, 2);
                    r += __shfl_xor_sync(0xffffffffu, r, 4);
                    M.key[r] = a;
                    M.id[r] = id;
                }
                __syncthreads();
                const uint32_t kth = M.key[k - 1];
                // an entry a thread: its weight, the weight before it, whether it is kept
                const float ex = tid < n && M.key[tid] >= kth ? exp_of(__fsub_rn(order_key_inv(M.key[tid]), m)) : -1.f;
                const u64 w = ex >= 0.f ? weight_of(ex) : 0ull;
                const u64 before = cta_scan64(s, w) - w;
                const u64 Z = cta_sum64(s, w);
                const double limit = __dmul_rn((double)top_p, (double)Z);
                const bool in = ex >= 0.f && (tid == 0 || ((top_p >= 1.f || (double)before < limit) && ex >= min_p));
                const u64 kept = in ? w : 0ull;
                u64* wk = HELD ? reinterpret_cast<u64*>(e) : M.w;   // (2 GT floats at least, not needed any more)
                if (tid < n) wk[tid] = kept;
                const u64 Zk = cta_sum64(s, kept);
                const u64 target = target_of(Zk);
                if (tid == 0) { s.pick = 0x7fffffff; s.pick64 = 0; }
                if (tid == GT - 1) s.logz = log((double)Zk * 0x1p-40);
                __syncthreads();
                // the weight up to an id is summed for each of the few ids, by eight threads
                for (int i0 = 0; i0 < n && M.key[i0] >= kth; i0 += GT / 8) {
                    const int i = min(i0 + tid / 8, n - 1), id = M.id[i];
                    u64 upto = 0;
                    for (int o = tid & 7; o < n && M.key[o] >= kth; o += 8)
                        if (M.id[o] <= id) upto += wk[o];
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) upto += __shfl_xor_sync(0xffffffffu, upto, o);
                    // (id, place in the order)
                    if (M.key[i] >= kth && wk[i] && upto > target) atomicMin(&s.pick, id * GT + i);
                }
                __syncthreads();
                if (tid == 0) {
                    ids[row] = s.pick / GT;
                    if (logprob)
                        logprob[row] = (float)((double)__fsub_rn(order_key_inv(M.key[s.pick % GT]), m) - s.logz);
                }
            }
            return;
        }
        cl.sync();   // everyone knows that the list overflowed
    }

    // ---- the k-th largest value: a histogram of max - l says in which bin it lies, a list of that bin which it is
    if (with_k) {
        auto bin_of = [&](float l) { return min((int)__fmul_rn(__fsub_rn(m, l), 136.f), BINS - 1); };
        for (int i = tid; i < BINS; i += GT) s.hist[i] = 0;
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        R.template walk<4>(w0, w0 + seg, [&](int i, const float4& v) {
            const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (base + i + j < V) atomicAdd(&s.hist[bin_of(R.q(a[j]))], 1u);
        });
        R.locate([](uint32_t v, int) { return (u64)v; }, [&](u64 c) { return c >= (u64)k; }, [] {});
        const int b = s.edge_bin;
        u64 above = s.pick64;
        R.template walk<4>(w0, w0 + seg, [&](int i, const float4& v) {
            const float a[4] = {R.q(v.x), R.q(v.y), R.q(v.z), R.q(v.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (base + i + j < V && bin_of(a[j]) == b) R.push(order_key(a[j]), base + i + j, 0.f);
        });
        int own;
        const int n = R.merge(&own);
        if (n >= 0) {
            // the value with fewer than k above it and at least k down to it
            for (int i0 = 0; i0 < n; i0 += GT / 8) {
                const int i = min(i0 + tid / 8, n - 1);
                const uint32_t a = M.key[i];
                int gt = 0, ge = 0;
                for (int j = tid & 7; j < n; j += 8) {
                    const uint32_t o = M.key[j];
                    gt += o > a;
                    ge += o >= a;
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    gt += __shfl_xor_sync(0xffffffffu, gt, o);
                    ge += __shfl_xor_sync(0xffffffffu, ge, o);
                }
                if ((int)above + gt < k && (int)above + ge >= k) s.pick = (int)a;
            }
            __syncthreads();
            R.kth = order_key_inv((uint32_t)s.pick);
        } else {
            uint32_t key = 0;
            R.select([&](auto f) {
                for (int i = w0 + lane; i < w0 + seg; i += 32) {
                    const float l = R.q(R.raw(i));
                    if (base + i < V && bin_of(l) == b) f(order_key(l), 1ull);
                }
            }, [&](u64 c) { return c >= (u64)k; }, 32, &key, &above);
            R.kth = order_key_inv(key);
        }
        cl.sync();   // lists and histograms have been read
    }

    R.quick = R.q.row(order_key_inv(best), m) && (!with_k || fabsf(R.kth) > 0x1p-50f);
    if (R.quick) { R.qt = R.q.T; R.qy = R.q.y; }
    else if (HELD)
#pragma unroll 1
        for (int i = w0 + lane; i < w0 + seg; i += 32) e[i] = R.q(e[i]);
    // ---- e in place of the logits; weights, and their histogram where top-p needs it
    const bool with_p = top_p < 1.f;
    for (int i = tid; i < BINS; i += GT) s.hist[i] = 0;
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    u64 kept = 0;
    const int per = (seg - lane * 4 + 127) / 128 * 4;   // entries of a thread, four of every 128
    WeightSum ws;
    constexpr int SH = HELD ? 8 : 11;   // bits of the mantissa that the histogram leaves out
    if (with_p) {
        R.template walk<4, true>(w0, w0 + seg, [&](int i, const float4& v) {
            float a[4];
            R.e_of(v, a);
            if constexpr (HELD) *(float4*)(e + i) = make_float4(a[0], a[1], a[2], a[3]);
            ws.add(pk(a[0], a[1]));
            ws.add(pk(a[2], a[3]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = __float_as_uint(a[j]);
                // 16 bits of the mantissa (at most 2^15 logits in shared memory) or 13 (2^18): 32 bits hold their sum
                if (b >= BIN0 << 16)
                    atomicAdd(&s.hist[BINS - 1 + BIN0 - (b >> 16)], ((b & 0x7FFFFFu) + 0x800000u + (1u << (SH - 1))) >> SH);
            }
        });
        const u64 all = cta_sum64(s, ws.sum(per));
        if (tid == 0) s.total = all;
    } else {
        R.template walk<4, true>(w0, w0 + seg, [&](int i, const float4& v) {
            float a[4];
            R.e_of(v, a);
            if constexpr (HELD) *(float4*)(e + i) = make_float4(a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = a[j] >= min_p ? a[j] : 0.f;
            ws.add(pk(a[0], a[1]));
            ws.add(pk(a[2], a[3]));
        });
        kept = ws.sum(per);
    }
    // Kept are the entries with e >= min_p and e >= whole, and of those with lo <= e < whole the ones up to the last
    // one that top-p keeps (HELD: the others' e is zero).
    float lo = 0.f, whole = 0.f;
    uint32_t edge = 0;
    int cut = V;
    kept = warp_sum64(kept);
    if (lane == 0) s.wsum[warp] = kept;
    if (with_p) {
        double limit = 0.;
        // the bin in which the histogram, from the top, passes the limit (in units of 2^-40; nearly exact)
        auto weigh = [](uint32_t v, int i) {
            const int o = ((BINS - 1 - i) >> 7) - 12 + SH;   // of e's exponent
            return o >= 0 ? (u64)v << o : (u64)v >> -o;
        };
        R.locate(weigh, [&](u64 c) { return !((double)c < limit); }, [&] {
            u64 Z = 0;
            from_all(cl, C, &s.total, [&](int, u64 v) { Z += v; });
            limit = __dmul_rn((double)top_p, (double)Z);
        });
        // What lies above that bin is added up, what lies in it listed, and each listed entry finds the weight in
        // front of it (attempt 0, on the next bin if the border turns out to lie there); a bin with too many entries is
        // searched by radix (1).  e is monotone in l up to rounding only, so the border has to lie clearly inside the
        // bin; else its neighbours (2) or all entries (3) are searched.
        float hi;
        bool found = false;
        int edge_bin = s.edge_bin < 0 ? 0 : BINS - 1 - s.edge_bin, tries = 0, more = 0;
        u64 front = s.pick64;       // what the histogram says lies above the bin
        for (int attempt = 0; attempt < 4 && !found;) {
            const int wide = attempt == 2, b0 = edge_bin - wide, b1 = edge_bin + 1 + wide;
            lo = attempt == 3 || b0 <= 0 ? 0.f : __uint_as_float(((uint32_t)(b0 + BIN0) << 16) - more);
            hi = attempt == 3 ? 2.f : __uint_as_float(((uint32_t)(b1 + BIN0) << 16) + more);
            const float from = fmaxf(lo, 0x1p-40f);     // (below: no weight)
            auto inside = [&](float v) { return v >= from && v < hi; };
            auto clear = [&](float v) {    // of a border at e = v (exp_of is within 2^-20); the largest l always is
                return (lo == 0.f || v > lo * 1.000002f) && (hi > 1.f || v < hi * 0.999998f);
            };
            u64 above = 0;
            if (attempt != 1) {
                __syncthreads();
                if (tid == 0) s.n_list = 0;
                __syncthreads();
                WeightSum wa;
                R.template walk<4, true>(w0, w0 + seg, [&](int i, const float4& v) {
                    float a[4] = {v.x, v.y, v.z, v.w};
                    if constexpr (!HELD) R.e_of(v, a);
                    float top[4];
                    bool in[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        top[j] = a[j] >= hi ? a[j] : 0.f;
                        in[j] = a[j] >= from && a[j] < hi;
                    }
                    wa.add(pk(top[0], top[1]));
                    wa.add(pk(top[2], top[3]));
                    if (attempt == 0 && (in[0] || in[1] || in[2] || in[3])) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (in[j]) R.push(0u, base + i + j, a[j]);   // (its key: below)
                    }
                });
                const u64 sum = wa.sum(per);
                kept = sum;
                if (min_p > hi) {
                    kept = 0;
                    for (int i = w0 + lane; i < w0 + seg; i += 32) kept += R.e1(i) >= min_p ? weight_of(R.e1(i)) : 0ull;
                }
                kept = warp_sum64(kept);
                if (lane == 0) s.wsum[warp] = kept;
                above = cta_sum64(s, sum);
                if (tid == 0) s.above = above;
                above = 0;
                if (attempt == 0)
                    for (int i = tid; i < min(s.n_list, LIST); i += GT) s.lkey[i] = order_key(R.l_of(s.lid[i]));
            }
            int own = 0, n = -1;
            if (attempt == 0) n = R.merge(&own);
            else cl.sync();
            from_all(cl, C, &s.above, [&](int, u64 v) { above += v; });
            if (attempt == 0 && n < 0) { attempt = 1; cl.sync(); continue; }
            if (attempt == 0) {
                // A few threads add up what is in front of an entry of this CTA; the last entry kept is the border.  Of
                // many entries, every eighth comes first, and then only those between the last of them that is kept
                // and the first that is not.
                const int mine = s.n_list;
                auto order_of = [&](int i) { return (u64)M.key[i] << 32 | (uint32_t)~M.id[i]; };
                auto rank_entries = [&](int count, auto entry, auto use) {
                    const int per = count <= GT / 32 ? 32 : count <= GT / 16 ? 16 : 8;
                    for (int i0 = 0; i0 < count; i0 += GT / per) {
                        const int i = entry(min(i0 + tid / per, count - 1));
                        const u64 a = order_of(i);
                        u64 before = 0;
#pragma unroll 4
                        for (int j = tid & (per - 1); j < n; j += per)
                            if (order_of(j) > a) before += M.w[j];
                        for (int o = 1; o < per; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
                        if ((tid & (per - 1)) == 0) use(i, a, before + above);
                    }
                };
                if (tid == 0) { s.pick = 0; s.n_between = 0; s.kept_to = ~0ull; s.cut_from = 0; }   // pick 1: the border is here, 2: not clear of the bin's ends
                __syncthreads();
                auto test = [&](int i, u64 a, u64 before) {
                    if ((double)before < limit && !((double)(before + M.w[i]) < limit)) {      // one entry of the row
                        s.pick = clear(s.le[i - own]) || M.key[i] == order_key(m) ? 1 : 2;
                        s.edge = M.key[i];
                        s.cut = M.id[i];
                    }
                };
                if (mine <= GT / 8) {
                    rank_entries(mine, [&](int i) { return own + i; }, test);
                } else {
                    rank_entries((mine + 7) / 8, [&](int i) { return own + 8 * i; }, [&](int, u64 a, u64 before) {
                        if ((double)before < limit) atomicMin(&s.kept_to, a);
                        else atomicMax(&s.cut_from, a);
                    });
                    __syncthreads();
                    for (int i = tid; i < mine; i += GT) {
                        const u64 a = order_of(own + i);
                        if (a <= s.kept_to && a > s.cut_from) s.between[atomicAdd(&s.n_between, 1)] = own + i;
                    }
                    __syncthreads();
                    rank_entries(s.n_between, [&](int i) { return (int)s.between[i]; }, test);
                }
                cl.sync();
                int border = 0, at = 0;
                from_all(cl, C, &s.pick, [&](int r, int v) {
                    border |= v;
                    if (v) at = r;
                });
                edge = from_cta(&s.edge, at);
                cut = from_cta(&s.cut, at);
                found = border == 1;
                if (!found) {
                    cl.sync();      // lists and sums have been read
                    // unclear: once more with half a bin more on either side.  Elsewhere: next door or, where the
                    // histogram is still there, in the bin that it names now that the sum above this one is known.
                    if (border == 2 && more == 0) { more = 0x8000; continue; }
                    if (border == 2 || ++tries > 3) { attempt = 2; continue; }
                    const int step = !((double)above < limit) ? 1 : -1;
                    if constexpr (HELD) {
                        edge_bin = min(max(edge_bin + step, 0), BINS - 1);
                    } else {
                        const double goal = limit + ((double)front - (double)above);
                        R.locate(weigh, [&](u64 c) { return !((double)c < goal); }, [] {});
                        const int to = s.edge_bin < 0 ? 0 : BINS - 1 - s.edge_bin;
                        edge_bin = to != edge_bin ? to : min(max(to + step, 0), BINS - 1);
                        front = s.pick64;
                    }
                    continue;
                }
                // the warp's share of the kept ones
                kept = 0;
                for (int i = lane; i < mine; i += 32) {
                    const int at = M.id[own + i] - base;
                    if (at < w0 || at >= w0 + seg) continue;
                    const uint32_t key = M.key[own + i];
                    const bool keep = key > edge || (key == edge && M.id[own + i] <= cut);
                    if (HELD && !keep) e[at] = 0.f;
                    if (keep && s.le[i] >= min_p) kept += M.w[own + i];
                }
                kept = warp_sum64(kept);
                if (lane == 0) s.wsum[warp] += kept;
                whole = hi;
                break;
            }
            // by radix: the border's key, then, of the ids there, the lowest ones until the limit
            auto each_inside = [&](auto f) {     // a warp walks its own run: f(id, e)
                for (int i = w0 + lane * 4; i < w0 + seg; i += 128) {
                    float a[4];
                    R.e4(i, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (base + i + j < V && inside(a[j])) f(base + i + j, a[j]);
                }
            };
            edge = 0;
            found = (double)above < limit && R.select([&](auto f) {
                each_inside([&](int id, float a) { f(order_key(R.l_of(id)), weight_of(a)); });
            }, [&](u64 c) { return !((double)c < limit); }, 32, &edge, &above);
            const float eb = exp_of(__fsub_rn(order_key_inv(edge), m));
            if (found && !clear(eb) && edge != order_key(m)) found = false;
            if (!found) {
                cl.sync();
                ++attempt;
                continue;
            }
            const u64 w = weight_of(eb);
            long long n_tie = (long long)((limit - (double)above) / (double)w);
            while (n_tie > 0 && !((double)(above + (n_tie - 1) * w) < limit)) --n_tie;
            while ((double)(above + n_tie * w) < limit) ++n_tie;
            u64 ties = 0;
            each_inside([&](int id, float) { ties += order_key(R.l_of(id)) == edge; });
            ties = cta_sum64(s, ties);
            if (tid == 0) s.above = ties;
            cl.sync();
            u64 all = 0;
            from_all(cl, C, &s.above, [&](int, u64 v) { all += v; });
            cut = V;
            if (n_tie < (long long)all) {
                uint32_t key = 0;
                u64 zero = 0;
                // the n-th smallest id is the n-th largest of 2^24 - 1 - id
                R.select([&](auto f) {
                    each_inside([&](int id, float) {
                        if (order_key(R.l_of(id)) == edge) f(0xFFFFFFu - (uint32_t)id, 1ull);
                    });
                }, [&](u64 c) { return c >= (u64)n_tie; }, 24, &key, &zero);
                cut = (int)(0xFFFFFFu - key);
            }
            kept = 0;
            each_inside([&](int id, float a) {
                const uint32_t key = order_key(R.l_of(id));
                if (key > edge || (key == edge && id <= cut)) {
                    if (a >= min_p) kept += weight_of(a);
                } else if (HELD) {
                    e[id - base] = 0.f;
                }
            });
            kept = warp_sum64(kept);
            if (lane == 0) s.wsum[warp] += kept;
            whole = hi;
        }
        if (!found) {
            // rounding of the limit: everything is kept
            lo = whole = 0.f;
            kept = 0;
            for (int i = w0 + lane; i < w0 + seg; i += 32) kept += R.e1(i) >= min_p ? weight_of(R.e1(i)) : 0ull;
            kept = warp_sum64(kept);
            __syncthreads();
            if (lane == 0) s.wsum[warp] = kept;
        }
    }
    __syncthreads();

    // ---- the draw: the warp whose run of ids holds the target
    if (tid == 0) {
        u64 t = 0;
#pragma unroll
        for (int w = 0; w < GW; ++w) t += s.wsum[w];
        s.kept = t;
    }
    cl.sync();
    u64 Z = 0, before = 0;
    from_all(cl, C, &s.kept, [&](int r, u64 v) {
        if (r < rank) before += v;
        Z += v;
    });
    cl.sync();    // from here on a CTA works on its own memory alone
    const u64 target = target_of(Z);
    // weights of the kept ones among four entries
    auto kept4 = [&](int i, int end, u64 (&w)[4]) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        if (i < end) R.e4(i, a);
        u64 own = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bool in = a[j] >= lo && a[j] >= min_p && a[j] >= 0x1p-40f;
            if (!HELD && in && a[j] < whole) {
                const uint32_t key = order_key(R.l_of(base + i + j));
                in = key > edge || (key == edge && base + i + j <= cut);
            }
            w[j] = in ? weight_of(a[j]) : 0ull;
            own += w[j];
        }
        return own;
    };
    // the run of ids that holds the target, and the kept weight in front of it: one of the warps' runs
    int from = w0, end = w0 + seg;
    u64 mine = s.wsum[warp];
    if constexpr (HELD) {
        for (int w = 0; w < warp; ++w) before += s.wsum[w];
    } else {
        // and one of sixteen parts of that, which the warps add up again
        int w = 0;
        if (target < before) return;
        while (w < GW && target >= before + s.wsum[w]) before += s.wsum[w++];
        if (w == GW) return;
        const int part = (seg / 4 + GW - 1) / GW * 4;
        end = w * seg + min((warp + 1) * part, seg);
        from = min(w * seg + warp * part, end);
        mine = 0;
        for (int i = from + lane * 4; i < end; i += 128) {
            u64 w4[4];
            mine += kept4(i, end, w4);
        }
        mine = warp_sum64(mine);
        if (lane == 0) s.red[warp] = mine;
        __syncthreads();
        for (int v = 0; v < warp; ++v) before += s.red[v];
    }
    if (before <= target && target < before + mine) {
        for (int i = from + lane * 4; ; i += 128) {
            u64 w[4];
            const u64 own = kept4(i, end, w);
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
            if (i - lane * 4 + 128 >= end) break;
        }
    }
}

template <typename T, bool HELD>
cudaError_t launch_t(int C, int slice, int V, int n, const void* logits, int64_t ld, const float* u, const float* temp,
                     const int32_t* topk, const float* topp, const float* minp, int32_t* ids, float* logprob, int* err,
                     cudaStream_t st) {
    // a per-device attribute: set on every call (a host-side table lookup)
    cudaError_t e = cudaFuncSetAttribute(sample_given_kernel<T, HELD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         MAX_SLICE * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n * C);
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = HELD ? max(slice, 2 * GT) * sizeof(float) : sizeof(Merged);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const int ahead = max(1, 2 * device_sm_count() / C);   // rows that run at once, with two CTAs an SM
    return cudaLaunchKernelEx(&cfg, sample_given_kernel<T, HELD>, V, slice, n, ahead, (const T*)logits, ld, u, temp, topk,
                              topp, minp, ids, logprob, err, (f2)0x8000000080000000ull);
}

}  // namespace

cudaError_t launch_sample_given(int n, int V, const void* logits, int dtype, int64_t ld, const float* u,
                                const float* temp, const int32_t* topk, const float* topp, const float* minp,
                                int32_t* ids, float* logprob, int* err, cudaStream_t st) {
    // CTAs of a row: as long as all run at once (two an SM) and a slice has 4096 logits.  Slices of up to 19456 logits
    // (76 KB, two CTAs an SM) are held in shared memory, and larger ones where an SM has one CTA anyway.
    const int sms = device_sm_count();
    int C = 1;
    while (C < MAX_CLUSTER && (int64_t)n * C <= sms && V / (2 * C) >= 4096) C *= 2;
    const int slice = ((V + C - 1) / C + GW * 32 - 1) / (GW * 32) * (GW * 32);
    const bool held = slice <= 19456 || (slice <= MAX_SLICE && (int64_t)n * C <= sms);
    auto go = [&](auto f) { return f(C, slice, V, n, logits, ld, u, temp, topk, topp, minp, ids, logprob, err, st); };
    if (dtype == Q3_BF16) return held ? go(launch_t<bf16, true>) : go(launch_t<bf16, false>);
    return held ? go(launch_t<float, true>) : go(launch_t<float, false>);
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
