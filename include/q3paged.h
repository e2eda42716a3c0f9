/*
 * q3paged.h -- C ABI of the paged-cache operators of the GB300 (sm_103a)
 * library: appending keys and values to a paged cache (with the per-head norms
 * and the rotation on the way) and attention of new tokens over that cache.
 *
 * The talker's own cache is one slab of max_batch x max_ctx positions; a
 * serving program whose requests differ in length keeps its positions in pages
 * instead, and a table says which page holds which positions of a sequence.
 * The arithmetic is the talker's (ncnn discussion 6798, section 2: QK-RMSNorm,
 * rotate-half RoPE, grouped-query attention, causal softmax).  A q3tts handle
 * created with kv_page_size > 0 runs its talker through these two operators.
 *
 * Conventions
 *  - Return value: Q3_OK or a Q3_ERR_* code of q3tts.h; q3paged_last_error()
 *    has a one-line reason for the calling thread.  Arguments are checked on
 *    the host before anything is queued.
 *  - Calls only queue kernels on the stream that they are given (NULL: the
 *    legacy default stream): nothing is synchronised or copied to the host, so
 *    they can be captured into a CUDA graph and replayed with new lengths,
 *    positions, tables and values in the same arrays.
 *  - What the host cannot see (page ids, positions, lengths) is checked on the
 *    device: an entry out of range is never followed (attention: the keys of
 *    such a page do not count, as if they were masked); it sets bit
 *    Q3PAGED_ERR_BOUNDS of *err, and a device wait that gave up sets
 *    Q3PAGED_ERR_TIMEOUT.  Bits are only ever set; the caller clears them.
 *  - All pointers are device memory, borrowed for the duration of the work.
 *    Rows of qkv, q, q_out and out start on 16-byte boundaries, and so do the
 *    rows of a page (pointers and strides are checked).
 *  - The stream belongs to the current device, and so does the memory.
 */
#ifndef Q3PAGED_H
#define Q3PAGED_H

#include "q3tts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bits of the device error word */
#define Q3PAGED_ERR_BOUNDS   2
#define Q3PAGED_ERR_TIMEOUT  4

/* leading bytes of the workspace that are zero before its first use */
#define Q3PAGED_COUNTER_BYTES  4096

/* A paged cache.  Position p of sequence s is slot p % page_size of page
 * page_table[s][p / page_size]; pages may be shared between sequences that
 * only read them.  Strides are in elements; 0 selects the packed layout
 * [n_pages][n_kv_heads][page_size][128]. */
typedef struct {
    int n_q_heads;          /* a multiple of n_kv_heads, at most 16 times as many       */
    int n_kv_heads;         /* q head h reads kv head h / (n_q_heads / n_kv_heads)      */
    int head_dim;           /* 128                                                      */
    int act_dtype;          /* Q3_F32 or Q3_BF16: qkv, q and the outputs                */
    int kv_dtype;           /* Q3_F32 (with fp32 activations only) or Q3_BF16: pages    */
    int page_size;          /* positions of a page: a power of two, 16..1024            */
    int n_pages;            /* pages of the pools                                       */
    int n_seqs;             /* rows of page_table                                       */
    int max_pages;          /* entries of a row of page_table                           */
    int64_t page_stride;    /* elements from one page to the next                       */
    int64_t head_stride;    /* ... from one kv head of a page to the next               */
    int64_t token_stride;   /* ... from one position of a head to the next              */
    void* k_pages;
    void* v_pages;
    const int32_t* page_table;   /* [n_seqs][max_pages]; entries past a sequence's
                                    last page are not read                            */
    int inject_timeout;     /* test only (0 = off).  Attention of chunks over bf16 pages:
                               the wait of each CTA for a place for its n-th tile of
                               keys or values counts as run out: the call ends early
                               with Q3PAGED_ERR_TIMEOUT, its outputs are not determined */
} q3paged_cache;

/* Appends n_tokens tokens, in any order:
 *   qkv        [n_tokens][(nq + 2 nkv) * 128] activations, row stride qkv_stride
 *              elements (0: packed): q heads, k heads, v heads
 *   tok_seq    [n_tokens] sequence of each token
 *   tok_pos    [n_tokens] its position; < 0: the token is skipped (its row of
 *              q_out is left as it is)
 *   q_norm, k_norm  [128] f32 RMSNorm weights of every q and of every k head
 *              (x / sqrt(mean x^2 + eps) * w), or both NULL: no norm
 *   rope_cs    [rope_rows][64][2] f32: cosine and sine by which the pair
 *              (j, j + 64) of a head is turned at a position
 *   q_out      [n_tokens][nq * 128] activations, row stride q_stride (0:
 *              packed): normed and turned queries; may be the q columns of qkv
 * Keys (normed and turned) and values are rounded to the cache's type and
 * stored at their positions.  A (sequence, position) pair appears at most once
 * in a call (twice: which token's values stay is not determined).  err may be
 * NULL.  Errors: Q3_ERR_ARG, Q3_ERR_CUDA. */
int q3paged_append(const q3paged_cache* c, int n_tokens, const void* qkv, int64_t qkv_stride, const int32_t* tok_seq,
                   const int32_t* tok_pos, const float* q_norm, const float* k_norm, float eps, const float* rope_cs,
                   int rope_rows, void* q_out, int64_t q_stride, int32_t* err, void* stream);

/* Bytes of workspace that q3paged_attention wants: the same for every valid
 * cache (0: invalid cache).  The caller clears its first Q3PAGED_COUNTER_BYTES
 * bytes once; every call leaves it ready for the next, which may be for another
 * cache.  Calls that may run at the same time (other streams, graphs replayed
 * side by side) need one workspace each. */
size_t q3paged_workspace_bytes(const q3paged_cache* c);

/* Causal attention of new tokens over the cache, which holds them already:
 *   q          [n_tokens][nq * 128] activations, row stride q_stride (0: packed)
 *   q_off      [n_seqs + 1]: rows q_off[s] .. q_off[s+1]-1 of q are the newest
 *              tokens of sequence s, in order (none: the sequence is skipped);
 *              starts at 0, does not decrease
 *   ctx_len    [n_seqs]: positions of sequence s, its new tokens included
 *   max_q      upper bound of the new tokens of any one sequence (it chooses
 *              the kernel; a sequence with more sets Q3PAGED_ERR_BOUNDS)
 *   scale      factor of the scores, > 0 (1/sqrt(128) for the talker)
 *   out        [n_tokens][nq * 128] activations, row stride out_stride (0:
 *              packed); may be q itself (with its stride)
 * Token i of sequence s stands at position ctx_len[s] - n_s + i and sees the
 * positions up to its own; one that sees nothing (a negative position) gets
 * zeros.  Rows from q_off[n_seqs] on are left as they are, and so are those of
 * a sequence that is skipped for its offsets.  Softmax and sums are fp32, of
 * scaled scores below 2^127.  bf16 activations: the weights enter the second
 * product with 8 bits (chunks) or 17 (few rows: new tokens times the q heads of
 * a kv head up to 16).  fp32 activations over bf16 pages: q enters with its 24
 * bits, the weights with 17 (chunks) or 24 (few rows: up to 8).  Values of keys below ctx_len must be finite; what
 * pages hold beyond it does not matter.  err may be NULL.  Errors: Q3_ERR_ARG,
 * Q3_ERR_CAPACITY (workspace too small), Q3_ERR_CUDA. */
int q3paged_attention(const q3paged_cache* c, int n_tokens, int max_q, const void* q, int64_t q_stride,
                      const int32_t* q_off, const int32_t* ctx_len, float scale, void* out, int64_t out_stride,
                      void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

/* Reason of the calling thread's last error in this header's functions or in
 * q3tts_sample_given. */
const char* q3paged_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* Q3PAGED_H */
