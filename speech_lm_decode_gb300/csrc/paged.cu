// Paged-cache operators: argument checks and C entry points (q3paged.h), and
// the append kernel.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "pdl.cuh"

namespace q3 {

namespace {
thread_local char g_reason[256] = "";
}

int paged_fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_reason, sizeof g_reason, fmt, ap);
    va_end(ap);
    return code;
}

namespace {

// ------------------------------------------------------------------ append
// Bound by the bytes moved (18 KB in and out a token with 16/8 heads in bf16)
// and, below that, by the chain position -> page -> stores of a warp.  A warp
// takes NL 16-byte loads of one token, all in flight together; a head is 16
// lanes of 8 bf16 or 32 lanes of 4 fp32 values, so a load brings two heads or
// one, and the rotation's pair (j, j + 64) lies half a head's lanes apart.
// With few tokens a warp takes one load, so that the heads of a token run
// beside each other (256 tokens, fp32: 3.1 us; one: 2.0 us); from 1024 on eight
// (9374 tokens of 32 prompts, bf16: 42 us, 4.0 TB/s; with 8-byte lanes and four
// heads a warp 55 us, with four loads 43 us).
constexpr int APPEND_WARPS = 4;

// 16 bytes of activations as fp32 values
__device__ __forceinline__ void expand(const uint4& r, float (&v)[8]) { unpack_bf16x8(r, v); }
__device__ __forceinline__ void expand(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint32_t two(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
}
__device__ __forceinline__ void put(bf16* p, const float (&v)[8]) {
    *(uint4*)p = make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7]));
}
__device__ __forceinline__ void put(bf16* p, const float (&v)[4]) { *(uint2*)p = make_uint2(two(v[0], v[1]), two(v[2], v[3])); }
__device__ __forceinline__ void put(float* p, const float (&v)[4]) { *(float4*)p = make_float4(v[0], v[1], v[2], v[3]); }

template <typename TA, typename TK, int NL>
__global__ void __launch_bounds__(APPEND_WARPS * 32, 8)
paged_append_kernel(PagedView c, int n_tokens, const TA* qkv, int64_t ldq, const int32_t* __restrict__ tok_seq,
                    const int32_t* __restrict__ tok_pos, const float* __restrict__ qn, const float* __restrict__ kn,
                    float eps, const float2* __restrict__ rope, int rope_rows, TA* q_out, int64_t ldo, int* err) {
    pdl_wait();
    pdl_trigger();
    constexpr int VL = 16 / (int)sizeof(TA), LPH = HD / VL, HPL = 32 / LPH;   // values of a lane, lanes of a head, heads of a load
    const int heads = c.nq + 2 * c.nkv, groups = (heads + NL * HPL - 1) / (NL * HPL);
    const int lane = threadIdx.x & 31, sub = lane & (LPH - 1);
    const int64_t item = (int64_t)blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5);
    const int64_t m = item / groups;
    const int h0 = (int)(item - m * groups) * NL * HPL + lane / LPH;
    if (m >= n_tokens) return;
    const TA* row = qkv + m * ldq;
    uint4 raw[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i)
        raw[i] = h0 + i * HPL < heads ? *(const uint4*)(row + (h0 + i * HPL) * HD + sub * VL) : make_uint4(0, 0, 0, 0);
    const int pos = tok_pos[m], seq = tok_seq[m];
    if (pos < 0) return;
    const int pi = pos >> c.page_shift;
    int page = -1;
    if (seq >= 0 && seq < c.n_seqs && pi < c.max_pages && pos < rope_rows) page = c.table[(int64_t)seq * c.max_pages + pi];
    if (page < 0 || page >= c.n_pages) {
        if (lane == 0 && err) atomicOr(err, ERRB_BOUNDS);
        return;
    }
    // cosine and sine of this lane's pairs; the lower half of a head subtracts, the upper adds
    float co[VL], si[VL];
    {
        const float4* cs = (const float4*)(rope + (int64_t)pos * (HD / 2) + (sub & (LPH / 2 - 1)) * VL);
        const float sign = sub < LPH / 2 ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < VL; j += 2) {
            const float4 f = cs[j / 2];
            co[j] = f.x; si[j] = sign * f.y; co[j + 1] = f.z; si[j + 1] = sign * f.w;
        }
    }
    const int64_t base = page * c.page_stride + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.token_stride + sub * VL;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int h = h0 + i * HPL;
        float x[VL], y[VL];
        expand(raw[i], x);
        if (qn) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VL; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(fmaf(ss, 1.0f / HD, eps));   // within 2^-22
            if (h < c.nq + c.nkv) {
                const float4* w = (const float4*)((h < c.nq ? qn : kn) + sub * VL);
#pragma unroll
                for (int j = 0; j < VL; j += 4) {
                    const float4 f = w[j / 4];
                    x[j] *= r * f.x; x[j + 1] *= r * f.y; x[j + 2] *= r * f.z; x[j + 3] *= r * f.w;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < VL; ++j) y[j] = fmaf(x[j], co[j], __shfl_xor_sync(0xffffffffu, x[j], LPH / 2) * si[j]);
        if (h < c.nq) put(q_out + m * ldo + h * HD + sub * VL, y);
        else if (h < c.nq + c.nkv) put((TK*)c.k + base + (h - c.nq) * c.head_stride, y);
        else if (h < heads) put((TK*)c.v + base + (h - c.nq - c.nkv) * c.head_stride, x);
    }
}

template <typename TA, typename TK, int NL>
cudaError_t append_t(const PagedView& c, int n_tokens, const void* qkv, int64_t ldq, const int32_t* seq,
                     const int32_t* pos, const float* qn, const float* kn, float eps, const float* rope, int rope_rows,
                     void* q_out, int64_t ldo, int* err, cudaStream_t st) {
    constexpr int per = NL * (sizeof(TA) == 2 ? 2 : 1);   // heads of a warp
    const int groups = (c.nq + 2 * c.nkv + per - 1) / per;
    const int64_t blocks = ((int64_t)n_tokens * groups + APPEND_WARPS - 1) / APPEND_WARPS;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(paged_append_kernel<TA, TK, NL>, (unsigned)blocks, APPEND_WARPS * 32, 0, st, c, n_tokens,
                      (const TA*)qkv, ldq, seq, pos, qn, kn, eps, (const float2*)rope, rope_rows, (TA*)q_out, ldo, err);
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& c, int act, int kv, int n_tokens, const void* qkv, int64_t qkv_stride,
                                const int32_t* tok_seq, const int32_t* tok_pos, const float* q_norm,
                                const float* k_norm, float eps, const float* rope_cs, int rope_rows, void* q_out,
                                int64_t q_stride, int* err, cudaStream_t st) {
    if (n_tokens <= 0) return cudaSuccess;
    auto go = [&](auto f) { return f(c, n_tokens, qkv, qkv_stride, tok_seq, tok_pos, q_norm, k_norm, eps, rope_cs,
                                     rope_rows, q_out, q_stride, err, st); };
    const bool many = n_tokens >= 1024;
    if (act == Q3_BF16) return many ? go(append_t<bf16, bf16, 8>) : go(append_t<bf16, bf16, 1>);
    if (kv == Q3_BF16) return many ? go(append_t<float, bf16, 8>) : go(append_t<float, bf16, 1>);
    return many ? go(append_t<float, float, 8>) : go(append_t<float, float, 1>);
}

namespace {
__global__ void paged_lengths_kernel(const int* __restrict__ pos, int n, int* __restrict__ ctx) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) ctx[i] = max(pos[i] + 1, 0);
}
}  // namespace

cudaError_t launch_paged_lengths(const int* pos, int n, int* ctx, cudaStream_t st) {
    return launch_pdl(paged_lengths_kernel, (n + 127) / 128, 128, 0, st, pos, n, ctx);
}

// ------------------------------------------------------------------ C entry points
namespace {

int esize(int dtype) { return dtype == Q3_BF16 ? 2 : 4; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// the cache as kernels see it; pools: the page pointers and strides are checked too
int view_of(const q3paged_cache* c, PagedView* v, bool pools) {
    if (!c) return paged_fail(Q3_ERR_ARG, "cache is NULL");
    if (c->head_dim != HD) return paged_fail(Q3_ERR_ARG, "head_dim must be 128");
    if (c->n_kv_heads < 1 || c->n_kv_heads > 256 || c->n_q_heads < c->n_kv_heads || c->n_q_heads % c->n_kv_heads ||
        c->n_q_heads / c->n_kv_heads > PAGED_MAX_GROUP)
        return paged_fail(Q3_ERR_ARG, "n_kv_heads must be 1..256 and n_q_heads a multiple of it, at most 16 times");
    if ((c->act_dtype != Q3_F32 && c->act_dtype != Q3_BF16) || (c->kv_dtype != Q3_F32 && c->kv_dtype != Q3_BF16))
        return paged_fail(Q3_ERR_ARG, "act_dtype and kv_dtype must be Q3_F32 or Q3_BF16");
    if (c->act_dtype == Q3_BF16 && c->kv_dtype == Q3_F32)
        return paged_fail(Q3_ERR_ARG, "fp32 pages go with fp32 activations");
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return paged_fail(Q3_ERR_ARG, "page_size must be a power of two in 16..1024");
    if (c->n_pages < 1 || c->n_seqs < 1 || c->max_pages < 1 || (int64_t)c->max_pages * c->page_size > 0x7fffff00)
        return paged_fail(Q3_ERR_ARG, "n_pages, n_seqs and max_pages must be >= 1 (positions below 2^31)");
    if (c->inject_timeout < 0) return paged_fail(Q3_ERR_ARG, "inject_timeout must be >= 0");
    v->nq = c->n_q_heads;
    v->nkv = c->n_kv_heads;
    v->G = v->nq / v->nkv;
    v->page_shift = 0;
    while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
    v->n_pages = c->n_pages;
    v->n_seqs = c->n_seqs;
    v->max_pages = c->max_pages;
    v->token_stride = c->token_stride ? c->token_stride : HD;
    v->head_stride = c->head_stride ? c->head_stride : (int64_t)c->page_size * HD;
    v->page_stride = c->page_stride ? c->page_stride : (int64_t)c->n_kv_heads * c->page_size * HD;
    v->k = c->k_pages;
    v->v = c->v_pages;
    v->table = c->page_table;
    if (!pools) return Q3_OK;
    if (!v->k || !v->v || !v->table) return paged_fail(Q3_ERR_ARG, "NULL pages or page table");
    const int e = esize(c->kv_dtype);
    for (int64_t s : {v->token_stride, v->head_stride, v->page_stride})
        if (s < HD || s * e % 16 || s * e >= (int64_t)1 << 40)
            return paged_fail(Q3_ERR_ARG, "strides must be at least 128 elements, below 2^40 bytes, in multiples of 16 bytes");
    if (!aligned16(v->k) || !aligned16(v->v)) return paged_fail(Q3_ERR_ARG, "pages must start on 16-byte boundaries");
    return Q3_OK;
}

// rows of activations: pointer, stride (0: packed) and alignment
int rows_ok(const char* what, const void* p, int64_t* stride, int width, int dtype) {
    if (!p) return paged_fail(Q3_ERR_ARG, "%s is NULL", what);
    if (*stride == 0) *stride = width;
    if (*stride < width || *stride * esize(dtype) % 16 || !aligned16(p))
        return paged_fail(Q3_ERR_ARG, "%s: rows of %d values must start on 16-byte boundaries", what, width);
    return Q3_OK;
}

}  // namespace
}  // namespace q3

using namespace q3;

extern "C" {

const char* q3paged_last_error(void) { return g_reason; }

int q3paged_append(const q3paged_cache* cache, int n_tokens, const void* qkv, int64_t qkv_stride,
                   const int32_t* tok_seq, const int32_t* tok_pos, const float* q_norm, const float* k_norm, float eps,
                   const float* rope_cs, int rope_rows, void* q_out, int64_t q_stride, int32_t* err, void* stream) {
    PagedView v;
    int r = view_of(cache, &v, true);
    if (r) return r;
    if (n_tokens < 0) return paged_fail(Q3_ERR_ARG, "negative n_tokens");
    if (n_tokens == 0) return Q3_OK;
    if ((r = rows_ok("qkv", qkv, &qkv_stride, (v.nq + 2 * v.nkv) * HD, cache->act_dtype))) return r;
    if ((r = rows_ok("q_out", q_out, &q_stride, v.nq * HD, cache->act_dtype))) return r;
    if (!tok_seq || !tok_pos || !rope_cs) return paged_fail(Q3_ERR_ARG, "NULL tok_seq, tok_pos or rope_cs");
    if (!q_norm != !k_norm) return paged_fail(Q3_ERR_ARG, "q_norm and k_norm: both or neither");
    if (!aligned16(rope_cs) || !aligned16(q_norm) || !aligned16(k_norm))
        return paged_fail(Q3_ERR_ARG, "rope_cs and the norm weights must start on 16-byte boundaries");
    if (rope_rows < 1) return paged_fail(Q3_ERR_ARG, "rope_rows must be >= 1");
    if (!(eps >= 0.f) || std::isinf(eps)) return paged_fail(Q3_ERR_ARG, "eps must be finite and >= 0");
    const cudaError_t e = launch_paged_append(v, cache->act_dtype, cache->kv_dtype, n_tokens, qkv, qkv_stride, tok_seq,
                                              tok_pos, q_norm, k_norm, eps, rope_cs, rope_rows, q_out, q_stride, err,
                                              (cudaStream_t)stream);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "append: %s", cudaGetErrorString(e));
    return Q3_OK;
}

size_t q3paged_workspace_bytes(const q3paged_cache* cache) {
    PagedView v;
    if (view_of(cache, &v, false)) return 0;
    return paged_workspace_bytes();
}

int q3paged_attention(const q3paged_cache* cache, int n_tokens, int max_q, const void* q, int64_t q_stride,
                      const int32_t* q_off, const int32_t* ctx_len, float scale, void* out, int64_t out_stride,
                      void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
    PagedAttn a{};
    int r = view_of(cache, &a.c, true);
    if (r) return r;
    if (n_tokens < 0 || max_q < 0) return paged_fail(Q3_ERR_ARG, "negative n_tokens or max_q");
    if (n_tokens == 0 || max_q == 0) return Q3_OK;
    if ((r = rows_ok("q", q, &q_stride, a.c.nq * HD, cache->act_dtype))) return r;
    if ((r = rows_ok("out", out, &out_stride, a.c.nq * HD, cache->act_dtype))) return r;
    if (!q_off || !ctx_len) return paged_fail(Q3_ERR_ARG, "NULL q_off or ctx_len");
    if (!(scale > 0.f) || std::isinf(scale)) return paged_fail(Q3_ERR_ARG, "scale must be finite and > 0");
    if (!workspace || ((uintptr_t)workspace & 255)) return paged_fail(Q3_ERR_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < paged_workspace_bytes())
        return paged_fail(Q3_ERR_CAPACITY, "workspace of %zu bytes: %zu are needed", workspace_bytes,
                          paged_workspace_bytes());
    a.act = cache->act_dtype;
    a.kv = cache->kv_dtype;
    a.inject = cache->inject_timeout;
    a.n_tokens = n_tokens;
    a.max_q = max_q < n_tokens ? max_q : n_tokens;
    a.q = q;
    a.q_stride = q_stride;
    a.q_off = q_off;
    a.ctx = ctx_len;
    a.scale = scale;
    a.out = out;
    a.out_stride = out_stride;
    a.ws = workspace;
    a.err = err;
    const cudaError_t e = launch_paged_attention(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return paged_fail(Q3_ERR_CUDA, "attention: %s", cudaGetErrorString(e));
    return Q3_OK;
}

}  // extern "C"
