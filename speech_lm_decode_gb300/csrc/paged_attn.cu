// Attention of new tokens over a paged cache (q3paged.h).
#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_sched.cuh"
#include "pdl.cuh"

namespace q3 {

namespace {

// One warp for each (token, q head): lane l holds values 4l..4l+3, the keys
// are walked one at a time with a running maximum and sum.
template <typename T> __device__ __forceinline__ float4 ld4(const T* p);
template <> __device__ __forceinline__ float4 ld4<float>(const float* p) { return *(const float4*)p; }
template <> __device__ __forceinline__ float4 ld4<bf16>(const bf16* p) {
    const uint2 a = *(const uint2*)p;
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xffff0000u));
}

template <typename TA, typename TK>
__global__ void __launch_bounds__(128) paged_plain_kernel(PagedAttn a) {
    pdl_wait();
    pdl_trigger();
    const PagedView& c = a.c;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int m = (int)(item / c.nq), h = (int)(item % c.nq);
    if (m >= a.n_tokens) return;
    int lo = 0, hi = c.n_seqs;   // the last sequence whose rows start at or before m
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.q_off[mid] <= m) lo = mid; else hi = mid;
    }
    const int s = lo, end = a.q_off[s + 1];
    if (m >= end) return;
    int ctx = a.ctx[s];
    const int cap = c.max_pages << c.page_shift;
    if (ctx > cap || end - a.q_off[s] > a.max_q || end > a.n_tokens) {
        if (lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
        ctx = min(ctx, cap);
    }
    const int n = ctx - (end - m) + 1;   // visible keys
    const float4 q = ld4((const TA*)a.q + m * a.q_stride + h * HD + lane * 4);
    float mx = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < n; ++j) {
        int page = c.table[(int64_t)s * c.max_pages + (j >> c.page_shift)];
        if (page < 0 || page >= c.n_pages) {
            if (lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
            continue;
        }
        const int64_t off = page * c.page_stride + (h / c.G) * c.head_stride +
                            (int64_t)(j & ((1 << c.page_shift) - 1)) * c.token_stride + lane * 4;
        const float4 k = ld4((const TK*)c.k + off), v = ld4((const TK*)c.v + off);
        const float sc = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * a.scale;
        const float nm = fmaxf(mx, sc), f = expf(mx - nm), p = expf(sc - nm);
        l = l * f + p;
        o.x = o.x * f + p * v.x; o.y = o.y * f + p * v.y; o.z = o.z * f + p * v.z; o.w = o.w * f + p * v.w;
        mx = nm;
    }
    const float r = l > 0.f ? 1.f / l : 0.f;
    TA* dst = (TA*)a.out + m * a.out_stride + h * HD + lane * 4;
    dst[0] = from_f<TA>(o.x * r); dst[1] = from_f<TA>(o.y * r); dst[2] = from_f<TA>(o.z * r); dst[3] = from_f<TA>(o.w * r);
}

}  // namespace

size_t paged_workspace_bytes() { return PAGED_COUNTER_BYTES + max(paged_decode_ws(), paged_chunk_ws()); }

cudaError_t launch_paged_attention(const PagedAttn& a, cudaStream_t st) {
    if (paged_decode_takes(a)) return launch_paged_decode(a, st);
    if (a.kv == Q3_BF16) return launch_paged_chunk(a, st);
    const int64_t blocks = ((int64_t)a.n_tokens * a.c.nq + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (a.act == Q3_BF16) return launch_pdl(paged_plain_kernel<bf16, bf16>, (unsigned)blocks, 128, 0, st, a);
    if (a.kv == Q3_BF16) return launch_pdl(paged_plain_kernel<float, bf16>, (unsigned)blocks, 128, 0, st, a);
    return launch_pdl(paged_plain_kernel<float, float>, (unsigned)blocks, 128, 0, st, a);
}

}  // namespace q3
