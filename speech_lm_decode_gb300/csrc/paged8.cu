// Paged cache of 8-bit codes: argument checks and C entry points (q3paged8.h),
// the append and the read kernel.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "paged8.h"
#include "pdl.cuh"

namespace q3 {

namespace {

// ------------------------------------------------------------------ append
// Bound by the bytes (14 KB a token with 16/8 heads in bf16) and, below that, by
// the chain lengths -> page -> entries -> scale -> codes of a warp.  A unit is the
// new tokens of one block and four heads, a head to a warp; the CTAs share the
// units evenly.  Nothing else writes a block's codes of a head, so its scale needs
// no exchange: the warp has the new entries in registers (that many of them are
// what limits the warps of an SM), takes their largest magnitude, and rounds them
// with the scale that follows.  Blocks of more than sixteen new tokens are gone
// through twice.  A lane has the partners of the rotation, so that it needs no
// exchange (with 16 contiguous bytes a lane and shuffles 65 us instead of 46).
// 9374 tokens of 32 prompts: bf16 45 us (134 MB: 3.0 TB/s), fp32 69.
constexpr int A8_WARPS = 4;
// Tokens that a warp keeps the entries of, pairs of them whose loads are in flight together, and CTAs of an SM: of calls
// whose sequences have one or two new tokens (a warp would form sixteen entries for one: 256 tokens 11.5 us instead
// of 7.3), and of others.
template <bool FEW> struct A8 { static constexpr int TOKENS = FEW ? 2 : 16, NB = FEW ? 1 : 4, CTAS = FEW ? 8 : 4; };

// A lane has eight values of a head: four from 4 i on and their partners of the rotation, 64 further on.
struct Raw16 { uint2 lo, hi; };
struct Raw32 { float4 lo, hi; };
__device__ __forceinline__ void fetch(const bf16* p, Raw16& r) { r = {*(const uint2*)p, *(const uint2*)(p + HD / 2)}; }
__device__ __forceinline__ void fetch(const float* p, Raw32& r) { r = {*(const float4*)p, *(const float4*)(p + HD / 2)}; }
__device__ __forceinline__ void expand(const Raw16& r, float (&v)[8]) { unpack_bf16x8(make_uint4(r.lo.x, r.lo.y, r.hi.x, r.hi.y), v); }
__device__ __forceinline__ void expand(const Raw32& r, float (&v)[8]) {
    v[0] = r.lo.x; v[1] = r.lo.y; v[2] = r.lo.z; v[3] = r.lo.w; v[4] = r.hi.x; v[5] = r.hi.y; v[6] = r.hi.z; v[7] = r.hi.w;
}
__device__ __forceinline__ uint32_t two(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
}
__device__ __forceinline__ void put(bf16* p, const float (&v)[8]) {
    *(uint2*)p = make_uint2(two(v[0], v[1]), two(v[2], v[3]));
    *(uint2*)(p + HD / 2) = make_uint2(two(v[4], v[5]), two(v[6], v[7]));
}
__device__ __forceinline__ void put(float* p, const float (&v)[8]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(p + HD / 2) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put_codes(uint8_t* p, const float (&v)[8], float f) {
    *(uint32_t*)p = codes_of(v[0] * f, v[1] * f) | codes_of(v[2] * f, v[3] * f) << 16;
    *(uint32_t*)(p + HD / 2) = codes_of(v[4] * f, v[5] * f) | codes_of(v[6] * f, v[7] * f) << 16;
}

// the byte of the least 2^e with amax <= 448 2^e = 1.75 2^(8 + e), held to what append writes
__device__ __forceinline__ int need_of(float amax) {
    const uint32_t u = __float_as_uint(amax);
    return min(max((int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u), E8_MIN), E8_MAX);
}

// A sequence's new tokens that are appended: rows row0 + (p - first) for positions p in [from, to).
struct A8Seq { int row0, first, from, to; };

__device__ __forceinline__ A8Seq a8_seq(const Paged8Append& a, int s, bool report) {
    A8Seq q;
    q.row0 = a.q_off[s];
    const int end = a.q_off[s + 1], ctx = a.ctx[s];
    // (the order matters: the difference is formed of offsets in range only, as that of any two may wrap around)
    bool bad = q.row0 < 0 || end < q.row0 || end > a.n_tokens || end - q.row0 > a.max_q;
    const int n = bad ? 0 : end - q.row0;
    if (n > 0 && (ctx < 0 || ctx > a.c.max_pages << a.c.page_shift)) bad = true;
    q.first = ctx - n;
    q.from = max(q.first, 0);
    q.to = bad || n == 0 ? q.from : min(ctx, a.rope_rows);
    if ((bad || (n > 0 && ctx > a.rope_rows)) && report && a.err) atomicOr(a.err, ERRB_BOUNDS);
    return q;
}

template <typename TA, bool FEW>
__global__ void __launch_bounds__(A8_WARPS * 32, A8<FEW>::CTAS) paged8_append_kernel(const Paged8Append a) {
    pdl_wait();
    pdl_trigger();
    constexpr int NB = A8<FEW>::NB, TOKENS = A8<FEW>::TOKENS;
    using Raw = std::conditional_t<sizeof(TA) == 2, Raw16, Raw32>;
    const PagedView& c = a.c;
    const int heads = c.nq + 2 * c.nkv, groups = (heads + A8_WARPS - 1) / A8_WARPS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, odd = lane >> 4, sub = lane & 15;
    const int B = 1 << a.block_shift, per_shift = c.page_shift - a.block_shift;
    auto blocks_of = [&](const A8Seq& q) {
        return q.to > q.from ? ((q.to - 1) >> a.block_shift) - (q.from >> a.block_shift) + 1 : 0;
    };

    // ---- this CTA's units
    __shared__ long long warp_sum_s[A8_WARPS];
    __shared__ int found_s;
    __shared__ long long found_start;
    const int per = (c.n_seqs + A8_WARPS * 32 - 1) / (A8_WARPS * 32);
    const int s0 = min((int)threadIdx.x * per, c.n_seqs), s1 = min(s0 + per, c.n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) mine += (long long)groups * blocks_of(a8_seq(a, s, blockIdx.x == 0));
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum_s[warp] = incl;
    __syncthreads();
    long long W = 0, before = 0;
#pragma unroll
    for (int w = 0; w < A8_WARPS; ++w) {
        if (w < warp) before += warp_sum_s[w];
        W += warp_sum_s[w];
    }
    const long long u0 = W * blockIdx.x / gridDim.x, u1 = W * (blockIdx.x + 1) / gridDim.x;
    if (u0 >= u1) return;
    long long start = before + incl - mine;
    if (start <= u0 && u0 < start + mine) {
        int s = s0;
        for (;; ++s) {
            const long long n = (long long)groups * blocks_of(a8_seq(a, s, false));
            if (u0 < start + n) break;
            start += n;
        }
        found_s = s;
        found_start = u0 - start;
    }
    __syncthreads();
    int s = found_s;
    long long rel = found_start;
    A8Seq q = a8_seq(a, s, false);
    int nb = blocks_of(q);
    for (long long u = u0; u < u1; ++u, ++rel) {
        while (rel >= (long long)groups * nb) {
            rel -= (long long)groups * nb;
            q = a8_seq(a, ++s, false);
            nb = blocks_of(q);
        }
        const int b = (int)(rel / groups), h = (int)(rel - (long long)b * groups) * A8_WARPS + warp;
        if (h >= heads) continue;
        const int block0 = ((q.from >> a.block_shift) + b) << a.block_shift;     // the block's first position
        const int p0 = max(q.from, block0), p1 = min(q.to, block0 + B);          // its new ones
        const int page = c.table[(int64_t)s * c.max_pages + (block0 >> c.page_shift)];
        if ((unsigned)page >= (unsigned)c.n_pages) {
            if (lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
            continue;
        }
        const int slot0 = block0 & ((1 << c.page_shift) - 1);
        const TA* src = (const TA*)a.qkv + ((int64_t)q.row0 - q.first) * a.ldq + (int64_t)h * HD + sub * 4;   // of position 0
        const bool is_q = h < c.nq, is_v = h >= c.nq + c.nkv;
        const float* w = is_q ? a.qn : a.kn;
        float wn[8];
        if (!is_v && w) {
            const float4 lo = *(const float4*)(w + sub * 4), hi = *(const float4*)(w + HD / 2 + sub * 4);
            wn[0] = lo.x; wn[1] = lo.y; wn[2] = lo.z; wn[3] = lo.w; wn[4] = hi.x; wn[5] = hi.y; wn[6] = hi.z; wn[7] = hi.w;
        }
        // use(i, p, x) of the tokens at positions t0 .. t0 + 7, two at a time: the lane's is p, its values x
        auto batch = [&](int t0, auto use) {
            Raw raw[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) fetch(src + min(t0 + 2 * i + odd, p1 - 1) * a.ldq, raw[i]);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int p = min(t0 + 2 * i + odd, p1 - 1);       // (past the last one: that one again)
                float x[8];
                expand(raw[i], x);
                if (!is_v) {
                    const float4* cs = (const float4*)(a.rope + (int64_t)p * (HD / 2) + sub * 4);
                    const float4 c01 = cs[0], c23 = cs[1];
                    if (w) {
                        float ss = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        const float r = rsqrtf(fmaf(ss, 1.0f / HD, a.eps));   // within 2^-22
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= r * wn[j];
                    }
                    const float co[4] = {c01.x, c01.z, c23.x, c23.z}, si[4] = {c01.y, c01.w, c23.y, c23.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float lo = x[j], hi = x[j + 4];
                        x[j] = fmaf(lo, co[j], -hi * si[j]);
                        x[j + 4] = fmaf(hi, co[j], lo * si[j]);
                    }
                }
                use(i, p, x);
            }
        };
        if (is_q) {
            TA* dst = (TA*)a.q_out + ((int64_t)q.row0 - q.first) * a.ldo + (int64_t)h * HD + sub * 4;
            for (int t0 = p0; t0 < p1; t0 += 2 * NB)
                batch(t0, [&](int i, int p, const float (&x)[8]) {
                    if (t0 + 2 * i + odd < p1) put(dst + p * a.ldo, x);
                });
            continue;
        }
        const int hk = h - c.nq - (is_v ? c.nkv : 0);
        uint8_t* sc = (is_v ? a.vs : a.ks) + (((int64_t)page * c.nkv + hk) << per_shift) + (slot0 >> a.block_shift);
        uint8_t* codes = (uint8_t*)(is_v ? c.v : c.k) + page * c.page_stride + hk * c.head_stride + slot0 * c.token_stride;
        const bool once = p1 - p0 <= TOKENS;
        float y[TOKENS / 2][8], amax = 0.f;
        auto form = [&](int t0) {      // entries of the tokens at positions t0 .. t0 + 15
#pragma unroll
            for (int z = 0; z < TOKENS / 2 / NB; ++z)
                if (t0 + 2 * NB * z < p1)
                    batch(t0 + 2 * NB * z, [&](int i, int, const float (&x)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = fmaf(x[j], 0.f, x[j]);      // infinities become NaN, which the maximum passes over
                            amax = fmaxf(amax, fabsf(v));
                            y[z * NB + i][j] = v;
                        }
                    });
        };
        for (int t0 = p0; t0 < p1; t0 += TOKENS) form(t0);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        int e = need_of(amax);
        if (p0 > block0) {       // older positions
            const int was = *sc;
            if (was < e) {
                // below 2^-20 of the new scale nothing is left of a code; from there on f16 has every value above 2^-11 exactly
                const int d = min(e - was, 20);
                const __half2 f = __float2half2_rn(__uint_as_float((uint32_t)(127 - d) << 23));
                for (int t = 0; t < p0 - block0; ++t) {
                    uint32_t* at = (uint32_t*)(codes + t * c.token_stride) + lane;
                    uint32_t lo, hi;
                    half4_of(*at, lo, hi);
                    const float2 x = __half22float2(__hmul2(*(const __half2*)&lo, f)), z = __half22float2(__hmul2(*(const __half2*)&hi, f));
                    *at = codes_of(x.x, x.y) | codes_of(z.x, z.y) << 16;
                }
            } else {
                e = was;
            }
        }
        const float f = e8m0(e >= 254 ? 0 : 254 - e);      // (a block of scale NaN stays one)
        for (int t0 = p0; t0 < p1; t0 += TOKENS) {
            if (!once) form(t0);
#pragma unroll
            for (int i = 0; i < TOKENS / 2; ++i) {
                const int p = t0 + 2 * i + odd;
                if (p < p1) put_codes(codes + (p - block0) * c.token_stride + sub * 4, y[i], f);
            }
        }
        if (lane == 0) *sc = (uint8_t)e;
    }
}

// ------------------------------------------------------------------ read
// Bound by the bytes: one in and two (four) out a code.  A thread takes sixteen codes at a time (four of its pieces in
// flight together, a CTA for each 1024 of a page, were no faster: 14.4 us instead of 12.6 for the 309 pages of 32
// positions that 9374 tokens lie in, 58 MB).
template <typename TO>
__global__ void __launch_bounds__(256) paged8_read_kernel(PagedView c, int block_shift, const uint8_t* ks, const uint8_t* vs,
                                                          int n, const int32_t* __restrict__ pages, TO* k_out, TO* v_out,
                                                          int* err) {
    pdl_wait();
    pdl_trigger();
    const int64_t rows = (int64_t)n * c.nkv << c.page_shift;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * 16; i += (int64_t)gridDim.x * 256) {
        const bool is_v = i >= rows * 8;
        TO* out = is_v ? v_out : k_out;
        if (!out) continue;
        const int64_t r = is_v ? i - rows * 8 : i;
        const int piece = (int)(r & 7);
        const int64_t row = r >> 3, ph = row >> c.page_shift;
        const int slot = (int)(row & ((1 << c.page_shift) - 1)), h = (int)(ph % c.nkv), page = pages[ph / c.nkv];
        if ((unsigned)page >= (unsigned)c.n_pages) {
            if (err) atomicOr(err, ERRB_BOUNDS);
            continue;
        }
        const uint8_t* src = (const uint8_t*)(is_v ? c.v : c.k) + page * c.page_stride + h * c.head_stride + slot * c.token_stride;
        const uint4 w = *(const uint4*)(src + piece * 16);
        const float f = e8m0((is_v ? vs : ks)[(((int64_t)page * c.nkv + h) << (c.page_shift - block_shift)) + (slot >> block_shift)]);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[4];
            float4_of(words[j], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * j + e] = x[e] * f;
        }
        TO* dst = out + row * HD + piece * 16;
        if constexpr (sizeof(TO) == 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *(uint4*)(dst + 8 * j) = make_uint4(two(v[8 * j], v[8 * j + 1]), two(v[8 * j + 2], v[8 * j + 3]),
                                                    two(v[8 * j + 4], v[8 * j + 5]), two(v[8 * j + 6], v[8 * j + 7]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) *(float4*)(dst + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
    }
}

// ------------------------------------------------------------------ C entry points
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

int view8_of(const q3paged8_cache* c8, PagedView* v, int* block_shift, bool pools) {
    if (!c8) return paged_fail(Q3_ERR_ARG, "cache is NULL");
    const q3paged_cache* c = &c8->cache;
    if (c->kv_dtype != Q3_E4M3) return paged_fail(Q3_ERR_ARG, "kv_dtype must be Q3_E4M3");
    // the other fields follow q3paged.h's rules for bf16 pages (strides are checked here, as they count bytes)
    q3paged_cache plain = *c;
    plain.kv_dtype = Q3_BF16;
    const int r = paged_view(&plain, v, false);
    if (r) return r;
    if (c8->scale_block < 16 || c8->scale_block > c->page_size || (c8->scale_block & (c8->scale_block - 1)))
        return paged_fail(Q3_ERR_ARG, "scale_block must be a power of two in 16..page_size");
    *block_shift = 0;
    while ((1 << *block_shift) < c8->scale_block) ++*block_shift;
    if (!pools) return Q3_OK;
    if (!v->k || !v->v || !v->table || !c8->k_scale || !c8->v_scale)
        return paged_fail(Q3_ERR_ARG, "NULL pages, scales or page table");
    for (int64_t s : {v->token_stride, v->head_stride, v->page_stride})
        if (s < HD || s % 16 || s >= (int64_t)1 << 40)
            return paged_fail(Q3_ERR_ARG, "strides must be at least 128 bytes, below 2^40, in multiples of 16");
    if (v->token_stride * c->page_size > 0x7fffffff)
        return paged_fail(Q3_ERR_ARG, "the positions of a page must lie within 2^31 bytes");
    if (!aligned16(v->k) || !aligned16(v->v)) return paged_fail(Q3_ERR_ARG, "pages must start on 16-byte boundaries");
    return Q3_OK;
}

}  // namespace
}  // namespace q3

using namespace q3;

extern "C" {

int q3paged8_append(const q3paged8_cache* cache, int n_tokens, int max_q, const void* qkv, int64_t qkv_stride,
                    const int32_t* q_off, const int32_t* ctx_len, const float* q_norm, const float* k_norm, float eps,
                    const float* rope_cs, int rope_rows, void* q_out, int64_t q_stride, int32_t* err, void* stream) {
    Paged8Append a{};
    int r = view8_of(cache, &a.c, &a.block_shift, true);
    if (r) return r;
    const int act = cache->cache.act_dtype;
    if (n_tokens < 0 || max_q < 0) return paged_fail(Q3_ERR_ARG, "negative n_tokens or max_q");
    if (n_tokens == 0 || max_q == 0) return Q3_OK;
    if ((r = paged_rows("qkv", qkv, &qkv_stride, (a.c.nq + 2 * a.c.nkv) * HD, act))) return r;
    if ((r = paged_rows("q_out", q_out, &q_stride, a.c.nq * HD, act))) return r;
    if (!q_off || !ctx_len || !rope_cs) return paged_fail(Q3_ERR_ARG, "NULL q_off, ctx_len or rope_cs");
    if (!q_norm != !k_norm) return paged_fail(Q3_ERR_ARG, "q_norm and k_norm: both or neither");
    if (!aligned16(rope_cs) || !aligned16(q_norm) || !aligned16(k_norm))
        return paged_fail(Q3_ERR_ARG, "rope_cs and the norm weights must start on 16-byte boundaries");
    if (rope_rows < 1) return paged_fail(Q3_ERR_ARG, "rope_rows must be >= 1");
    if (!(eps >= 0.f) || std::isinf(eps)) return paged_fail(Q3_ERR_ARG, "eps must be finite and >= 0");
    a.ks = cache->k_scale;
    a.vs = cache->v_scale;
    a.n_tokens = n_tokens;
    a.max_q = max_q < n_tokens ? max_q : n_tokens;
    a.qkv = qkv;
    a.ldq = qkv_stride;
    a.q_off = q_off;
    a.ctx = ctx_len;
    a.qn = q_norm;
    a.kn = k_norm;
    a.eps = eps;
    a.rope = (const float2*)rope_cs;
    a.rope_rows = rope_rows;
    a.q_out = q_out;
    a.ldo = q_stride;
    a.err = err;
    // no more CTAs than units: the blocks that n_tokens tokens can touch, four heads each
    const int groups = (a.c.nq + 2 * a.c.nkv + A8_WARPS - 1) / A8_WARPS;
    const int64_t units = groups * std::min<int64_t>(n_tokens, (n_tokens >> a.block_shift) + 2LL * a.c.n_seqs);
    const bool few = a.max_q <= 2;
    const unsigned grid = (unsigned)std::min<int64_t>(units, (few ? A8<true>::CTAS : A8<false>::CTAS) * device_sm_count());
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, A8_WARPS * 32, 0, (cudaStream_t)stream, a); };
    const cudaError_t e = act == Q3_BF16 ? few ? go(paged8_append_kernel<bf16, true>) : go(paged8_append_kernel<bf16, false>)
                                         : few ? go(paged8_append_kernel<float, true>) : go(paged8_append_kernel<float, false>);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "append: %s", cudaGetErrorString(e));
    return Q3_OK;
}

size_t q3paged8_workspace_bytes(const q3paged8_cache* cache) {
    PagedView v;
    int shift;
    if (view8_of(cache, &v, &shift, false)) return 0;
    return paged_workspace_bytes();
}

int q3paged8_attention(const q3paged8_cache* cache, int n_tokens, int max_q, const void* q, int64_t q_stride,
                       const int32_t* q_off, const int32_t* ctx_len, float scale, void* out, int64_t out_stride,
                       void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
    Paged8Attn a{};
    int r = view8_of(cache, &a.c, &a.block_shift, true);
    if (r) return r;
    if (n_tokens < 0 || max_q < 0) return paged_fail(Q3_ERR_ARG, "negative n_tokens or max_q");
    if (n_tokens == 0 || max_q == 0) return Q3_OK;
    if ((r = paged_attn_args(&a, &cache->cache, n_tokens, max_q, q, q_stride, q_off, ctx_len, scale, out, out_stride,
                             workspace, workspace_bytes, err)))
        return r;
    a.ks = cache->k_scale;
    a.vs = cache->v_scale;
    const cudaError_t e = paged8_decode_takes(a) ? launch_paged8_decode(a, (cudaStream_t)stream)
                                                 : launch_paged8_chunk(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "attention: %s", cudaGetErrorString(e));
    return Q3_OK;
}

int q3paged8_read(const q3paged8_cache* cache, int n, const int32_t* pages, int out_dtype, void* k_out, void* v_out,
                  int32_t* err, void* stream) {
    PagedView v;
    int shift;
    const int r = view8_of(cache, &v, &shift, true);
    if (r) return r;
    if (n < 0) return paged_fail(Q3_ERR_ARG, "negative n");
    if (out_dtype != Q3_F32 && out_dtype != Q3_BF16) return paged_fail(Q3_ERR_ARG, "out_dtype must be Q3_F32 or Q3_BF16");
    if (!aligned16(k_out) || !aligned16(v_out)) return paged_fail(Q3_ERR_ARG, "k_out and v_out must start on 16-byte boundaries");
    if (n == 0 || (!k_out && !v_out)) return Q3_OK;
    if (!pages) return paged_fail(Q3_ERR_ARG, "pages is NULL");
    const int64_t threads = ((int64_t)n * v.nkv << v.page_shift) * 16;
    const unsigned grid = (unsigned)std::min<int64_t>((threads + 255) / 256, (int64_t)device_sm_count() * 8);
    const uint8_t *ks = cache->k_scale, *vs = cache->v_scale;
    const cudaError_t e = out_dtype == Q3_BF16
        ? launch_pdl(paged8_read_kernel<bf16>, grid, 256, 0, (cudaStream_t)stream, v, shift, ks, vs, n, pages, (bf16*)k_out, (bf16*)v_out, err)
        : launch_pdl(paged8_read_kernel<float>, grid, 256, 0, (cudaStream_t)stream, v, shift, ks, vs, n, pages, (float*)k_out, (float*)v_out, err);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "read: %s", cudaGetErrorString(e));
    return Q3_OK;
}

}  // extern "C"
