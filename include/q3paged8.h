/*
 * q3paged8.h -- C ABI of the operators over a paged cache whose keys and values
 * are held in 8 bits, of the GB300 (sm_103a) library: appending to it,
 * attention of new tokens over it, reading its values back.
 *
 * A key or value is a number of the type e4m3 (4 exponent bits, 3 mantissa
 * bits, up to 448, no infinities; code 0x7f and 0xff: NaN) times the scale of
 * its block.  A block is scale_block positions of one kv head in one page, for
 * keys and for values apart; its scale is a power of two, held as one byte in
 * the type e8m0 (2^(byte - 127); 255: NaN).  Steps of e4m3 are relative to the
 * value, so a finer scale would gain nothing, and with powers of two a block's
 * codes keep their values when its scale grows (but for those that fall below
 * 2^-6 of the new one, which are rounded once more).
 *
 * Conventions are those of q3paged.h: checks on the host before anything is
 * queued, Q3_OK or a Q3_ERR_* code with q3paged_last_error()'s reason, kernels
 * queued on the given stream alone (nothing is synchronised, so that calls can
 * be captured into a CUDA graph), what the host cannot see checked on the device
 * (Q3PAGED_ERR_BOUNDS, Q3PAGED_ERR_TIMEOUT in *err).
 */
#ifndef Q3PAGED8_H
#define Q3PAGED8_H

#include "q3paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kv_dtype of the cache's description: codes of one byte */
#define Q3_E4M3  2

typedef struct {
    q3paged_cache cache;    /* kv_dtype Q3_E4M3, act_dtype Q3_F32 or Q3_BF16; pages are bytes
                               (strides in multiples of 16; page_size * token_stride below 2^31) */
    int scale_block;        /* positions of a block: a power of two, 16..page_size           */
    uint8_t* k_scale;       /* [n_pages][n_kv_heads][page_size / scale_block], packed        */
    uint8_t* v_scale;
} q3paged8_cache;

/* Appends the newest tokens of every sequence.
 *   qkv        [n_tokens][(nq + 2 nkv) * 128] activations, row stride qkv_stride
 *              elements (0: packed): q heads, k heads, v heads
 *   q_off      [n_seqs + 1]: rows q_off[s] .. q_off[s+1]-1 of qkv are the newest
 *              tokens of sequence s, in order; starts at 0, does not decrease
 *   ctx_len    [n_seqs]: positions of sequence s, its new tokens included:
 *              token i of n_s stands at position ctx_len[s] - n_s + i
 *   max_q      upper bound of the new tokens of any one sequence
 *   q_norm, k_norm, eps, rope_cs, rope_rows, q_out, q_stride
 *              as in q3paged_append
 * (the arguments of q3paged8_attention, which follows it).  Keys (normed and
 * turned) and values are rounded to the nearest code, ties to even.  A block's
 * scale becomes the least 2^e, e in -100..119, with which the largest finite
 * magnitude among its new entries is at most 448 2^e, and no less than it was if
 * the block holds older positions of the sequence (what lies there before its
 * first position does not count); the older entries of a block whose scale grows
 * are rounded to it.  What is larger than 448 2^119 becomes that, what is not
 * finite NaN.  Positions past the context are left as they are.
 * A sequence whose offsets or lengths are out of range (n_s above max_q, ctx_len
 * above the table) is skipped and reported; so is a token at a negative position
 * (not reported: padding), past the rotation's table, or on a page out of range
 * (reported).  The row of q_out of a token that is skipped is left as it is, and
 * so are rows from q_off[n_seqs] on.  Pages that sequences share are not
 * appended to; where two sequences of a call append to one block, its values are
 * not determined.  err may be NULL.  Errors: Q3_ERR_ARG, Q3_ERR_CUDA. */
int q3paged8_append(const q3paged8_cache* c, int n_tokens, int max_q, const void* qkv, int64_t qkv_stride,
                    const int32_t* q_off, const int32_t* ctx_len, const float* q_norm, const float* k_norm, float eps,
                    const float* rope_cs, int rope_rows, void* q_out, int64_t q_stride, int32_t* err, void* stream);

/* Bytes of workspace that q3paged8_attention wants; the rules are those of
 * q3paged_workspace_bytes, and one workspace serves both kinds of cache. */
size_t q3paged8_workspace_bytes(const q3paged8_cache* c);

/* Causal attention of new tokens over the cache, which holds them already: the
 * arguments and rules of q3paged_attention.  Sums are fp32.  q enters the
 * products with 22 bits relative to the row's largest value (bf16: exact), the
 * weights with 11 bits (bf16 activations) or 22 (fp32).  Few rows (new tokens times
 * the q heads of a kv head up to 16): the scales may be any.  More rows: codes are
 * taken relative to the largest scale among the keys that a row sees, those of a
 * block whose scale is less than 2^-15 of it lose bits from the smallest on.
 * Values of keys below ctx_len must not be NaN codes or scales; what pages hold
 * beyond it does not matter. */
int q3paged8_attention(const q3paged8_cache* c, int n_tokens, int max_q, const void* q, int64_t q_stride,
                       const int32_t* q_off, const int32_t* ctx_len, float scale, void* out, int64_t out_stride,
                       void* workspace, size_t workspace_bytes, int32_t* err, void* stream);

/* The values that n pages stand for:
 *   pages      [n] int32 page ids, any order, repeats allowed
 *   out_dtype  Q3_F32 or Q3_BF16 (exact in either within their ranges: a code has
 *              four bits)
 *   k_out, v_out  [n][n_kv_heads][page_size][128], packed, from 16-byte
 *              boundaries; either may be NULL
 * A page id out of range is reported and its part of the outputs left as it is.
 * err may be NULL.  Errors: Q3_ERR_ARG, Q3_ERR_CUDA. */
int q3paged8_read(const q3paged8_cache* c, int n, const int32_t* pages, int out_dtype, void* k_out, void* v_out,
                  int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* Q3PAGED8_H */
