/*
 * headloss_sample.h -- drawing tokens from the head's logits (C ABI).
 *
 * A policy step (GRPO, GSPO) starts from tokens drawn from the head's softmax
 * and their log-probs: the labels and old_logprobs of headloss_forward_backward.
 * This call makes both, a row a request, from the head's logits and one given
 * uniform number a row, with temperature, top-k, top-p and min-p of each
 * request's own.
 *
 * Definition, for a row x[0 .. V) (a NaN counts as -inf, a token at -inf is
 * never drawn and has no mass):
 *   z_j  = c tanh(x_j / c) (softcap c; c = 0: z_j = x_j), zm = z of the largest x
 *   d_j  = (z_j - zm) * (K / T), K = logits_scale * log2(e), in fp32; d_j = 0 where z_j = zm
 *   w_j  = rint(2^30 * 2^d_j), an integer: the row's masses are sums of integers,
 *          exact and the same in any order, so a row's token depends on neither the
 *          launch nor the rows beside it
 *   order: x descending, equal x by ascending index
 *   top-k keeps the first k; top-p keeps, of those, every token before which the mass
 *   is less than top_p times theirs, and the first; min-p keeps those with 2^d_j >= min_p
 *   t    = min(floor(u * W), W - 1), W the kept mass (the product in fp64)
 *   token: the first kept j, by index, with sum of kept w_0 .. w_j > t.
 * T = 0 (or so small that K / T overflows) is greedy: top-k 1 at T = 1.
 *
 * Rows' settings differ freely: greedy, unfiltered and filtered rows share a call.
 * Status codes are those of headloss.h.
 */
#ifndef HEADLOSS_SAMPLE_H
#define HEADLOSS_SAMPLE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * headloss_sample -- one token a row.
 *
 * logits:       N rows of V values of `dtype` (enum headloss_dtype), device; row i starts
 *               at element i * ld (ld >= V: columns past V, a padded vocabulary, are not
 *               read).  The base is aligned to the element; rows need no further alignment.
 * uniforms:     N fp64 in [0, 1), device, 8-byte aligned.
 * temperature:  N fp32, >= 0 and finite, or NULL (1 everywhere).  0 (or -0): greedy.
 * top_k:        N int32 or NULL.  <= 0 or >= V: off.
 * top_p:        N fp32, >= 0, or NULL.  >= 1: off.
 * min_p:        N fp32 in [0, 1] or NULL.  0: off.
 * softcap, logits_scale: as in headloss_create (c >= 0, 0 = off; s > 0), with 1 / c and
 *               s log2(e) inside fp32's range (c = 0 or c > 2.94e-39, s < 2.35e38).
 * tokens:       N int64 (written): the drawn token; -1 for a row without one (every
 *               logit -inf or NaN, or settings outside the ranges above).  The loss calls
 *               take -1 as a masked row.
 * logprobs:     N fp32 or NULL (written): log p(token) of the whole softmax at T = 1 without
 *               filters, the old_logprobs of a GRPO step; 0 for a row without a token.  Summed in
 *               fixed point: the same bits however the row is split over CTAs.
 * draw_logprobs: N fp32 or NULL (written): log(mass of the token / kept mass) at the
 *               row's temperature, the log-prob under the distribution drawn from; 0 likewise.
 * n_kept:       N int32 or NULL (written): the number of tokens that could be drawn.
 * err:          one int, device, 4-byte aligned, zeroed by the caller: bit 0 is set if a
 *               row's settings were out of range (its token is -1), bit 1 if a copy wait gave
 *               up (~2 s; that row's token is -1).
 * stream:       cudaStream_t (NULL = legacy default stream).  Asynchronous, no allocation.
 *
 * N == 0 is valid.  Errors (nothing enqueued): ERR_ARG (N < 0, N >= 2^31, V < 1, V >= 2^31 - 4096, ld < V, a
 * softcap or logits_scale out of range, a NULL logits / uniforms / tokens / err with N > 0),
 * ERR_DTYPE, ERR_ALIGN (logits not aligned to its element; uniforms or tokens not 8-byte, an
 * fp32 or int32 array not 4-byte aligned), ERR_CUDA (launch failure).
 */
int headloss_sample(const void* logits, int64_t N, int64_t V, int64_t ld, int dtype,
                    const double* uniforms, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, float softcap, float logits_scale,
                    int64_t* tokens, float* logprobs, float* draw_logprobs, int32_t* n_kept,
                    int* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HEADLOSS_SAMPLE_H */
