/*
 * coli_w8.h — C ABI of dense 8-bit products on MI355X (gfx950): the
 * projections around the routed-expert MoE layer (coli_moe.h), with weights
 * of one scale an output channel and activations of one scale a token.
 *
 *   s_t = max_k |x_tk| / 127                q_tk = x_tk / s_t, to the nearest integer
 *   out_to = s_t s_o sum_k q_tk w_ok (+ bias_o)
 *
 * Conventions are coli_moe.h's: device pointers, calls that enqueue and
 * return, 0 or a negative COLI_E* code with coli_moe_last_error().  No
 * workspace and no status word: what is not finite shows in the results.
 *
 * Arithmetic: the scale is one division, rounded to binary32; a code is the
 * integer nearest to the exact quotient by that scale, ties to even, in
 * -127 .. 127.  Sums of products are exact (32-bit integers).  A result is
 * (sum * s_t) * s_o, then + bias: in binary64, rounded once, for binary32
 * outputs; for the 16-bit types each step rounded to binary32, then once to the
 * output's type.  A token with a value that is not finite gets the scale
 * NaN and codes 0, so that its results are NaN and no other token's.
 */
#ifndef COLI_W8_H
#define COLI_W8_H

#include "coli_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest sum: 2^16 products of codes (w may hold -128) stay below 2^31. */
#define COLI_W8_MAX_K 65536
/* Most tokens, and most output channels, of one call. */
#define COLI_W8_MAX_ROWS (1 << 24)

/*
 * Tokens as codes and scales.
 *   dtype  of x: COLI_BF16, COLI_FP16 or COLI_F32
 *   x      device [n_tokens, k], at token_stride (elements), rows 16-byte aligned
 *   codes  device int8 [n_tokens, k]; scale device f32 [n_tokens]
 * k a multiple of 16 up to COLI_W8_MAX_K.  A token of zeros gets scale 0 and
 * codes 0.
 */
int coli_w8_quantize(int32_t dtype, int32_t n_tokens, int32_t k, const void *x, int64_t token_stride, int8_t *codes,
                     float *scale, void *stream);

/*
 * out[t, o] = scale[t] w_scale[o] sum_k codes[t, k] w[o, k] (+ bias[o]).
 *   codes    device int8 [n_tokens, k], at code_stride (a multiple of 16)
 *   scale    device f32 [n_tokens]
 *   w        device int8 [n_out, k]; w_scale device f32 [n_out]
 *   bias     device f32 [n_out], or NULL
 *   out      device [n_tokens, n_out] of dtype, at out_stride (elements)
 * k a multiple of 16 up to COLI_W8_MAX_K, any n_out and out_stride >= n_out;
 * elements of out between its rows are not written.
 */
int coli_w8_linear(int32_t dtype, int32_t n_tokens, int32_t k, int32_t n_out, const int8_t *codes, int64_t code_stride,
                   const float *scale, const int8_t *w, const float *w_scale, const float *bias, void *out,
                   int64_t out_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* COLI_W8_H */
