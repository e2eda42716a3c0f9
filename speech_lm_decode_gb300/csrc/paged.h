// Shared by the paged-cache operators (q3paged.h): the cache as kernels see it
// and the launchers behind the C entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "q3paged.h"

namespace q3 {

constexpr int PAGED_MAX_GROUP = 16;   // q heads of one kv head

struct PagedView {
    int nq, nkv, G;              // G = nq / nkv
    int page_shift, n_pages, n_seqs, max_pages;
    int64_t page_stride, head_stride, token_stride;
    void *k, *v;
    const int32_t* table;
};

// One attention call (validated arguments).
struct PagedAttn {
    PagedView c;
    int act, kv, n_tokens, max_q;
    int inject;                  // test only: the tile whose wait counts as run out (q3paged_cache)
    const void* q;
    int64_t q_stride;
    const int32_t *q_off, *ctx;
    float scale;
    void* out;
    int64_t out_stride;
    void* ws;
    int* err;
};

cudaError_t launch_paged_append(const PagedView& c, int act, int kv, int n_tokens, const void* qkv, int64_t qkv_stride,
                                const int32_t* tok_seq, const int32_t* tok_pos, const float* q_norm,
                                const float* k_norm, float eps, const float* rope_cs, int rope_rows, void* q_out,
                                int64_t q_stride, int* err, cudaStream_t st);
cudaError_t launch_paged_attention(const PagedAttn& a, cudaStream_t st);
size_t paged_workspace_bytes();
// ctx[b] = pos[b] + 1 for a step's rows (pos < 0, a finished row: 0)
cudaError_t launch_paged_lengths(const int* pos, int n, int* ctx, cudaStream_t st);
// few query rows over bf16 pages (paged_decode.cu)
bool paged_decode_takes(const PagedAttn& a);
cudaError_t launch_paged_decode(const PagedAttn& a, cudaStream_t st);
size_t paged_decode_ws();
// many query rows over bf16 pages (paged_chunk.cu)
cudaError_t launch_paged_chunk(const PagedAttn& a, cudaStream_t st);
size_t paged_chunk_ws();

// argument checks (paged.cu).  The cache as kernels see it; pools: the page pointers and strides are checked too.
int paged_view(const q3paged_cache* c, PagedView* v, bool pools);
// rows of activations: pointer, stride (0: packed) and alignment
int paged_rows(const char* what, const void* p, int64_t* stride, int width, int dtype);
// an attention call's other arguments into a, whose view is there already
int paged_attn_args(PagedAttn* a, const q3paged_cache* cache, int n_tokens, int max_q, const void* q, int64_t q_stride,
                    const int32_t* q_off, const int32_t* ctx_len, float scale, void* out, int64_t out_stride,
                    void* workspace, size_t workspace_bytes, int32_t* err);

// text of the calling thread's last error (q3paged_last_error)
int paged_fail(int code, const char* fmt, ...);

}  // namespace q3
