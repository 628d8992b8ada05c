/*
 * coli_mla.h — C ABI of latent attention on MI355X (gfx950): the attention
 * that stands before the routed-expert MoE layer of a block (coli_moe.h).
 *
 * Keys and values of every head come from one latent vector a token:
 *
 *   c_t  = RMSNorm(a_t) * g                        (rank values, cached)
 *   r_t  = rotate(p_t, position)                   (64 values, cached, shared by the heads)
 *   k_th = [W^K_h c_t | r_t],  v_th = W^V_h c_t    (expanded form, prompts)
 *   s    = scale * <q, k>,  out = softmax(s) v
 *
 * and, because W^K and W^V do not depend on the token, equally (absorbed
 * form, single tokens)
 *
 *   s    = scale * (<W^K_h' q_nope, c_t> + <q_pe, r_t>),  out = W^V_h (softmax(s) c)
 *
 * so that decoding reads the cached latents once for all heads.
 *
 * Conventions are coli_moe.h's: device pointers, caller's workspace (zero
 * filled once before its first use), calls that enqueue and return, 0 or a
 * negative COLI_E* code with coli_moe_last_error(), and device-side
 * conditions (a slot, page id or length outside the cache, row offsets that do
 * not ascend or leave their rows) as sticky bits of the workspace's status
 * word, read and cleared by coli_moe_status().  Outputs after a non-zero status are unspecified;
 * no access leaves the arrays whose sizes the call was given.  Calls that
 * overlap in time need a workspace each.
 *
 * Arithmetic: inputs of 16 bits, products and sums in binary32, softmax
 * statistics in binary32, results rounded once to 16 bits.  The weights of a
 * softmax are rounded to 16 bits before their product with the values (over
 * an E4M3 cache, weight times the token's scale is, relative to the largest such
 * product that the query sees, whatever the scales).  In binary16 a weight below
 * 2^-19 of the row's largest has fewer than eleven bits, one below 2^-30 none.
 * Results do not depend on timing: no sum runs through an atomic.
 */
#ifndef COLI_MLA_H
#define COLI_MLA_H

#include "coli_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* coli_mla_dims.kv_format: one cached token is a row of
 *   COLI_KV_PLAIN  rank + 64 values of dtype: latent, rotated key
 *   COLI_KV_E4M3   rank E4M3 codes (OCP, bytes), then 64 values of dtype;
 *                  latent = code * kv_scale[slot] (binary32, amax / 448) */
#define COLI_KV_PLAIN 0
#define COLI_KV_E4M3 1

/* coli_mla_dims.rope_style: the two members of a rotated pair i < 32 */
#define COLI_ROPE_PAIRS 0  /* elements 2i and 2i + 1 */
#define COLI_ROPE_HALVES 1 /* elements i and i + 32 */

#define COLI_MLA_ROPE 64   /* rotated values a head */

typedef struct coli_mla_dims {
    int32_t n_heads;     /* 1..256 */
    int32_t rank;        /* latent width: 256 or 512 */
    int32_t nope;        /* unrotated width of a head's queries and keys, */
    int32_t v_dim;       /* and of its values: (128, 128) or (192, 256) */
    int32_t page_size;   /* tokens a page of the cache: 1..65536 */
    int32_t dtype;       /* COLI_BF16 or COLI_FP16 */
    int32_t kv_format;   /* COLI_KV_PLAIN or COLI_KV_E4M3 */
    int32_t rope_style;  /* COLI_ROPE_PAIRS or COLI_ROPE_HALVES */
    float norm_eps;      /* >= 0, finite */
    float softmax_scale; /* > 0, finite */
} coli_mla_dims;

/* Most query rows of one sequence in one decode call (n_q * n_heads), most
 * sequences, and most cached tokens (batch * max_kv). */
#define COLI_MLA_MAX_ROWS 16384
#define COLI_MLA_MAX_BATCH 4096
#define COLI_MLA_MAX_TOKENS (1ll << 36)
/* Longest sequence (max_kv), and most rows of queries, keys or expansions. */
#define COLI_MLA_MAX_LENGTH 0x7fffff00
/* Largest token stride of prefill's keys and values, in elements. */
#define COLI_MLA_MAX_STRIDE (1 << 23)

/* Bytes of one cached token (0 when dims are invalid). */
size_t coli_mla_row_bytes(const coli_mla_dims *dims);

/* Workspace for append, expand and prefill calls (batch = 0) and decode
 * calls of up to `batch` sequences with n_q new tokens each and up to max_kv
 * cached tokens.  0 when an argument is invalid. */
size_t coli_mla_workspace_bytes(const coli_mla_dims *dims, int32_t batch, int32_t n_q, int32_t max_kv);

/*
 * Norm, rotation and the write into the paged cache, for n_tokens tokens.
 *   kv_a       device [n_tokens, rank + 64] of dtype: latent before its norm, key before its rotation
 *   norm_w     device [rank] of dtype, or NULL: the latent is stored as it is
 *   positions  device int32 [n_tokens], any value
 *   slots      device int64 [n_tokens]: page * page_size + offset; negative = padding, not stored.
 *              Slots are distinct (two tokens of one slot race).
 *   inv_freq   device f64 [32]: angle of pair i = position * inv_freq[i], reduced in 64 bits
 *   q_pe       device [n_tokens, n_heads, 64] of dtype at the strides given (elements; multiples of 8), last
 *              dimension contiguous; may be NULL with n_heads' queries rotated elsewhere
 *   q_pe_out   the rotated queries, at strides of its own; may be q_pe itself
 *   pages      device [n_pages, page_size, row]; kv_scale device f32 [n_pages * page_size] (E4M3 only)
 * E4M3: scale = amax / 448 over the normed latent, codes = latent / scale rounded to nearest even; an all-zero
 * latent gets scale 0 and codes 0.
 */
int coli_mla_append(const coli_mla_dims *dims, int32_t n_tokens, const void *kv_a, const void *norm_w,
                    const int32_t *positions, const int64_t *slots, const double *inv_freq, const void *q_pe,
                    int64_t q_token_stride, int64_t q_head_stride, void *q_pe_out, int64_t out_token_stride,
                    int64_t out_head_stride, void *pages, float *kv_scale, int32_t n_pages, void *ws,
                    size_t ws_bytes, void *stream);

/*
 * Per-head products: out[t, h, :] = w[h] x[t, h, :] (queries into the latent
 * space, attention outputs out of it).
 *   x    device [n_tokens, n_heads, n_in] of dtype at the strides given (elements; multiples of 8)
 *   w    device [n_heads, n_out, n_in]; out device [n_tokens, n_heads, n_out]
 * n_in a multiple of 64 up to 1024, n_out a multiple of 64 up to 4096.
 */
int coli_mla_project(int32_t dtype, int32_t n_tokens, int32_t n_heads, int32_t n_in, int32_t n_out, const void *x,
                     int64_t x_token_stride, int64_t x_head_stride, const void *w, void *out, void *stream);

/*
 * Absorbed attention of n_q new tokens a sequence over the paged latents.
 * The new tokens are the last n_q of the sequence's kv_lens[b] cached ones:
 * query j sees tokens 0 .. kv_lens[b] - n_q + j.  A query that sees none gets
 * zeros and lse = -inf.
 *   q_lat  device [batch * n_q, n_heads, rank], q_pe device [batch * n_q, n_heads, 64], of dtype
 *   table  device int32 [batch, table_width]: page ids, in the sequence's order
 *   kv_lens device int32 [batch]; max_kv: host bound of them
 *   out    device [batch * n_q, n_heads, rank] of dtype: softmax(s) c
 *   lse    device f32 [batch * n_q, n_heads]: log of the sum of exp(s), or NULL
 */
int coli_mla_decode(const coli_mla_dims *dims, int32_t batch, int32_t n_q, const void *q_lat, const void *q_pe,
                    const void *pages, const float *kv_scale, int32_t n_pages, const int32_t *table,
                    int32_t table_width, const int32_t *kv_lens, int32_t max_kv, void *out, float *lse, void *ws,
                    size_t ws_bytes, void *stream);

/* Most query rows of a coli_mla_decode_shared call (batch * n_q * n_heads). */
#define COLI_MLA_MAX_SHARED_ROWS (1 << 20)

/* Workspace for coli_mla_decode_shared calls of up to these sizes.  0 when an
 * argument is invalid. */
size_t coli_mla_shared_workspace_bytes(const coli_mla_dims *dims, int32_t batch, int32_t n_q, int32_t prefix_len,
                                       int32_t max_kv);

/*
 * coli_mla_decode for sequences that begin with the same cached tokens:
 * sequence b is the prefix_len tokens of prefix_table, then kv_lens[b] tokens
 * of its own in its pages of table.  The prefix is read once for every 128
 * rows of all sequences, or by each sequence for itself where that is faster.
 * The n_q new tokens are the last of the whole sequence:
 * query j sees its first prefix_len + kv_lens[b] - n_q + 1 + j tokens (a
 * sequence of fewer own tokens than n_q has some of them in the prefix), and
 * one that sees none gets zeros and lse = -inf.
 *   prefix_table  device int32 [prefix_width]: page ids of the prefix, in order, prefix_width * page_size >=
 *                 prefix_len; may be NULL with prefix_len = 0
 *   prefix_len    host; 0 is coli_mla_decode
 *   max_kv        host bound of kv_lens; 0: no sequence has tokens of its own
 * Other arguments as for coli_mla_decode; batch * n_q * n_heads at most COLI_MLA_MAX_SHARED_ROWS.
 */
int coli_mla_decode_shared(const coli_mla_dims *dims, int32_t batch, int32_t n_q, const void *q_lat, const void *q_pe,
                           const void *pages, const float *kv_scale, int32_t n_pages, const int32_t *prefix_table,
                           int32_t prefix_width, int32_t prefix_len, const int32_t *table, int32_t table_width,
                           const int32_t *kv_lens, int32_t max_kv, void *out, float *lse, void *ws, size_t ws_bytes,
                           void *stream);

/* Test hook: how later coli_mla_decode_shared calls in this process read the
 * prefix: 0 whichever is faster (default), 1 once for blocks of rows of all
 * sequences, 2 each sequence for itself (where prefix_len + max_kv is a length
 * that coli_mla_decode takes).  Results differ by rounding alone. */
int coli_mla_debug_shared_path(int32_t path);

/*
 * Keys and values of every head out of the paged latents, for a ragged
 * batch: rows cu_k[b] .. cu_k[b + 1] - 1 are tokens 0, 1, .. of sequence b.
 *   cu_k device int32 [batch + 1], from 0, ascending, last <= n_rows; rows behind it are not written
 *   w    device [n_heads, nope + v_dim, rank] of dtype
 *   kv   device [n_rows, n_heads, nope + v_dim] of dtype: w c; k_pe device [n_rows, 64]: the cached rotated keys
 */
int coli_mla_expand(const coli_mla_dims *dims, int32_t batch, int32_t n_rows, const void *pages,
                    const float *kv_scale, int32_t n_pages, const int32_t *table, int32_t table_width,
                    const int32_t *cu_k, const void *w, void *kv, void *k_pe, void *ws, size_t ws_bytes,
                    void *stream);

/*
 * Attention of prompts over expanded keys and values, for a ragged batch of
 * queries (cu_q) and keys (cu_k), offsets as for coli_mla_expand.  The last
 * query of a sequence sees its last key: with causal = 1, query i of n sees
 * keys 0 .. i + m - n of m; a query that sees none gets zeros and lse = -inf.
 *   q      device [n_q_rows, n_heads, nope + 64] of dtype, rotated part last
 *   k_nope device [n_k_rows, n_heads, nope], k_pe device [n_k_rows, 64] (shared by the heads),
 *   v      device [n_k_rows, n_heads, v_dim]; strides of q, k_nope and v in elements, multiples of 8
 *   max_q  host bound of the sequences' query counts; batch * n_heads * ceil(max_q / 128) < 2^28
 *   out    device [n_q_rows, n_heads, v_dim]; lse device f32 [n_q_rows, n_heads], or NULL
 */
int coli_mla_prefill(const coli_mla_dims *dims, int32_t batch, int32_t n_q_rows, int32_t n_k_rows, const void *q,
                     int64_t q_token_stride, int64_t q_head_stride, const void *k_nope, int64_t k_token_stride,
                     int64_t k_head_stride, const void *k_pe, const void *v, int64_t v_token_stride,
                     int64_t v_head_stride, const int32_t *cu_q, const int32_t *cu_k, int32_t max_q, int32_t causal,
                     void *out, float *lse, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* COLI_MLA_H */
