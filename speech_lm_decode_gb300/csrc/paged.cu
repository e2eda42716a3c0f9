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
// A warp takes HPW heads of one token (q, k, then v heads).  Lane l holds the
// four values 4l..4l+3 of a head, so the rotation's pair (j, j+64) lies in
// lanes l and l ^ 16, and every load and store of a head is one 512-byte (fp32)
// or 256-byte (bf16) access of the warp.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = *(const float4*)p;
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&v)[4]) {
    const uint2 a = *(const uint2*)p;
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *(uint2*)p = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
}

constexpr int APPEND_WARPS = 4;

template <typename TA, typename TK, int HPW>
__global__ void __launch_bounds__(APPEND_WARPS * 32)
paged_append_kernel(PagedView c, int n_tokens, const TA* qkv, int64_t ldq, const int32_t* __restrict__ tok_seq,
                    const int32_t* __restrict__ tok_pos, const float* __restrict__ qn, const float* __restrict__ kn,
                    float eps, const float2* __restrict__ rope, int rope_rows, TA* q_out, int64_t ldo, int* err) {
    pdl_wait();
    pdl_trigger();
    const int heads = c.nq + 2 * c.nkv, groups = (heads + HPW - 1) / HPW;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5);
    const int64_t m = item / groups;
    const int h0 = (int)(item - m * groups) * HPW;
    if (m >= n_tokens) return;
    const int pos = tok_pos[m], seq = tok_seq[m];
    if (pos < 0) return;
    const int pi = pos >> c.page_shift;
    int page = -1;
    if (seq >= 0 && seq < c.n_seqs && pi < c.max_pages && pos < rope_rows) page = c.table[(int64_t)seq * c.max_pages + pi];
    if (page < 0 || page >= c.n_pages) {
        if (lane == 0 && err) atomicOr(err, ERRB_BOUNDS);
        return;
    }
    const TA* row = qkv + m * ldq;
    float x[HPW][4];
#pragma unroll
    for (int i = 0; i < HPW; ++i)
        if (h0 + i < heads) load4(row + (h0 + i) * HD + lane * 4, x[i]);
    // cosine and sine of this lane's four pairs
    const float4* cs = (const float4*)(rope + (int64_t)pos * (HD / 2) + (lane & 15) * 4);
    const float4 c01 = cs[0], c23 = cs[1];
    const float co[4] = {c01.x, c01.z, c23.x, c23.z}, si[4] = {c01.y, c01.w, c23.y, c23.w};
    const int64_t base = page * c.page_stride + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.token_stride + lane * 4;
#pragma unroll
    for (int i = 0; i < HPW; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        if (h >= c.nq + c.nkv) {
            store4((TK*)c.v + base + (h - c.nq - c.nkv) * c.head_stride, x[i]);
            continue;
        }
        const bool is_q = h < c.nq;
        const float* wn = is_q ? qn : kn;
        if (wn) {
            const float ss = warp_sum(x[i][0] * x[i][0] + x[i][1] * x[i][1] + x[i][2] * x[i][2] + x[i][3] * x[i][3]);
            const float r = 1.0f / sqrtf(ss / (float)HD + eps);
            float w[4];
            load4(wn + lane * 4, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = x[i][j] * r * w[j];
        }
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, x[i][j], 16);
            y[j] = lane < 16 ? x[i][j] * co[j] - other * si[j] : x[i][j] * co[j] + other * si[j];
        }
        if (is_q) store4(q_out + m * ldo + h * HD + lane * 4, y);
        else store4((TK*)c.k + base + (h - c.nq) * c.head_stride, y);
    }
}

template <typename TA, typename TK, int HPW>
cudaError_t append_t(const PagedView& c, int n_tokens, const void* qkv, int64_t ldq, const int32_t* seq,
                     const int32_t* pos, const float* qn, const float* kn, float eps, const float* rope, int rope_rows,
                     void* q_out, int64_t ldo, int* err, cudaStream_t st) {
    const int groups = (c.nq + 2 * c.nkv + HPW - 1) / HPW;
    const int64_t blocks = ((int64_t)n_tokens * groups + APPEND_WARPS - 1) / APPEND_WARPS;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(paged_append_kernel<TA, TK, HPW>, (unsigned)blocks, APPEND_WARPS * 32, 0, st, c, n_tokens,
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
    if (act == Q3_BF16) return go(append_t<bf16, bf16, 4>);
    if (kv == Q3_BF16) return go(append_t<float, bf16, 4>);
    return go(append_t<float, float, 4>);
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
