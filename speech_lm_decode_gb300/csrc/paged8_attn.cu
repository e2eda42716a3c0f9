// Attention over a paged cache of 8-bit codes: a warp for each query row of a
// head, its keys one after the other.
#include "kernels.h"
#include "paged8.h"
#include "paged_sched.cuh"
#include "pdl.cuh"

namespace q3 {
namespace {

template <typename TA>
__global__ void __launch_bounds__(128) paged8_row_kernel(const Paged8Attn a) {
    pdl_wait();
    pdl_trigger();
    const PagedView& c = a.c;
    const int lane = threadIdx.x & 31, s = blockIdx.y;
    const PagedSeq q = paged_seq(a, s, blockIdx.x == 0 && threadIdx.x == 0);
    for (int it = blockIdx.x * 4 + (threadIdx.x >> 5); it < q.n_new * c.nq; it += gridDim.x * 4) {
        const int tok = it / c.nq, h = it - tok * c.nq, hk = h / c.G;
        const int lim = min(q.ctx - q.n_new + tok + 1, q.ctx);
        float x[4], o[4] = {}, m = -INFINITY, l = 0.f;
        const TA* src = (const TA*)a.q + (int64_t)(q.row0 + tok) * a.q_stride + h * HD + lane * 4;
        for (int j = 0; j < 4; ++j) x[j] = to_f(src[j]) * a.scale;
        for (int key = 0; key < lim; ++key) {
            const int page = c.table[(int64_t)s * c.max_pages + (key >> c.page_shift)], slot = key & ((1 << c.page_shift) - 1);
            if ((unsigned)page >= (unsigned)c.n_pages) {
                if (a.err) atomicOr(a.err, ERRB_BOUNDS);
                continue;
            }
            const int64_t at = page * c.page_stride + hk * c.head_stride + slot * c.token_stride + lane * 4;
            const int64_t sc = (((int64_t)page * c.nkv + hk) << (c.page_shift - a.block_shift)) + (slot >> a.block_shift);
            const uint32_t kw = *(const uint32_t*)((const uint8_t*)c.k + at), vw = *(const uint32_t*)((const uint8_t*)c.v + at);
            float k[4], v[4];
            float4_of(kw, k);
            float4_of(vw, v);
            const float score = warp_sum(x[0] * k[0] + x[1] * k[1] + x[2] * k[2] + x[3] * k[3]) * e8m0(a.ks[sc]);
            const float nm = fmaxf(m, score), f = expf(m - nm), p = expf(score - nm), fv = e8m0(a.vs[sc]);
            m = nm;
            l = l * f + p;
            for (int j = 0; j < 4; ++j) o[j] = o[j] * f + p * (v[j] * fv);
        }
        TA* dst = (TA*)a.out + (int64_t)(q.row0 + tok) * a.out_stride + h * HD + lane * 4;
        for (int j = 0; j < 4; ++j) dst[j] = from_f<TA>(l != 0.f ? o[j] / l : 0.f);
    }
}

}  // namespace

cudaError_t launch_paged8_attention(const Paged8Attn& a, cudaStream_t st) {
    if (paged8_decode_takes(a)) return launch_paged8_decode(a, st);
    const dim3 grid((unsigned)min((int64_t)a.max_q * a.c.nq / 4 + 1, (int64_t)1024), a.c.n_seqs);
    return a.act == Q3_BF16 ? launch_pdl(paged8_row_kernel<bf16>, grid, 128, 0, st, a)
                            : launch_pdl(paged8_row_kernel<float>, grid, 128, 0, st, a);
}

}  // namespace q3
