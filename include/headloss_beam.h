/*
 * headloss_beam.h -- a beam search's step behind the head (C ABI): the selection over beams and
 * vocabulary, and the reordering of the beams' states.
 *
 * Status codes are those of headloss.h.
 */
#ifndef HEADLOSS_BEAM_H
#define HEADLOSS_BEAM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * headloss_beam_workspace -- bytes of workspace that headloss_beam_select takes; -1 for sizes that
 * it refuses.  Needs no device.
 */
int64_t headloss_beam_workspace(int64_t requests, int beams, int64_t V, int dtype, int keep);

/*
 * headloss_beam_select -- the `keep` best continuations of each request's beams.
 *
 * A beam b with the running score s_b continues with token j at the score
 *   s_b + log p_b(j),  p_b the softmax of logits_scale * z,  z = c tanh(x / c) (softcap c; c = 0: z = x)
 * of its row x of logits.  A NaN counts as -inf; a token at -inf is no candidate, nor is any of a beam whose
 * score is -inf (or NaN): a first step has the scores 0, -inf, -inf, ...  Without a softcap a row with an
 * infinity has its mass on its infinities.  A beam that has ended has one candidate: itself, with token eos at
 * the score s_b; its row is not read.  Candidates are ordered by score, as fp64 evaluates it from the row's sum
 * of exponentials (which is held in fp32); equal scores by beam, then by falling logit, then by token.
 * Under a softcap the sum is off by a share of 2^-21 softcap * logits_scale at most where that product is up to
 * 1024, and of 2^-19 log V above, beside the roundings of its additions.
 *
 * logits:       requests * beams rows of V values of `dtype` (enum headloss_dtype), device; row i starts at
 *               element i * ld (ld >= V).  The base is aligned to the element; rows need no more.
 * beams, keep:  1 .. 64 and 1 .. 128.
 * scores:       requests x beams fp32, device.
 * ended:        requests x beams bytes (0 or not), device, or NULL (none has ended).
 * eos:          the token that ends a hypothesis, in [0, V), or -1 (none; ended is NULL then).
 * stay:         0: the kept stand in falling order.  1 (keep == beams alone): the first of each parent's
 *               takes the parent's place and the others, in falling order, the free places: states that are
 *               reordered in place then move least.
 * softcap, logits_scale: as in headloss_create, with 1 / c and s log2(e) inside fp32's range.
 * out_scores, parents, tokens: requests x keep fp32, int32, int64 (written): the new score, the beam
 *               within the request that it continues, the token.  Where fewer than `keep` candidates
 *               exist: -inf, -1, -1.
 * out_ended:    requests x keep bytes or NULL (written): 1 where the token is eos, else 0.
 * workspace:    at least headloss_beam_workspace() bytes, device, 16-byte aligned.  Its content is not
 *               kept; calls that may run at once need workspaces of their own.
 * out_scores and scores may be the same memory (as may out_ended and ended) where keep == beams.
 * Asynchronous on `stream`, no allocation; the same candidates in every run.  requests == 0 is valid.
 * Errors (nothing enqueued): ERR_ARG (a size out of range: requests < 0, requests * beams >= 2^31, V < 1 or
 * >= 2^31 - 4096, ld < V; beams, keep, eos, stay, softcap or logits_scale out of range; a NULL pointer;
 * workspace too small), ERR_DTYPE, ERR_ALIGN, ERR_CUDA (launch failure).
 */
int headloss_beam_select(const void* logits, int64_t requests, int beams, int64_t V, int64_t ld, int dtype,
                         const float* scores, const uint8_t* ended, int64_t eos, int keep, int stay,
                         float softcap, float logits_scale, float* out_scores, int32_t* parents,
                         int64_t* tokens, uint8_t* out_ended, void* workspace, int64_t workspace_bytes,
                         void* stream);

/*
 * One tensor of beams' states: rows * outer * positions runs of run_bytes contiguous bytes, that of row i,
 * outer o and position p at i * row_stride + o * outer_stride + p * position_stride bytes (negative strides
 * are refused; runs do not overlap).  A key-value cache (rows, heads, positions, width) has outer = heads; a
 * state of fixed size positions = 1.
 */
typedef struct {
    void* state;
    void* out;              /* state itself: in place; or a buffer of the same layout */
    int64_t outer, positions, run_bytes;
    int64_t row_stride, outer_stride, position_stride;
} headloss_state;

typedef struct headloss_reorder_s* headloss_reorder_t;

/*
 * headloss_reorder_create -- takes n states (1 .. 2^20) of beams, and copies the list to the current
 * device (synchronously).  `states` is in HOST memory.
 * A state that is listed more than once, with the same out and layout, is moved once.
 * Errors: ERR_ARG (n out of range, beams not in 1 .. 64, a NULL pointer, outer, positions or run_bytes < 0, a
 * negative stride, 2^31 outer indices or more), ERR_CUDA.
 */
int headloss_reorder_create(const headloss_state* states, int n, int beams, headloss_reorder_t* out);

/*
 * headloss_reorder -- out[r, b] = state[r, parents[r, b]] for every state of the handle, request r and beam b
 * (row r * beams + b).
 *
 * parents:  requests x beams int32, device.  A parent outside [0, beams) stands for the row itself.
 *           Any map is right in place: all rows are read as they were before the call.
 * begin, end: requests int32 each, device, or both NULL (every position): request r's positions
 *           begin[r] .. end[r] - 1, cut to the state's, are taken; the others of `out` stay as they were.
 * Asynchronous on `stream`, no allocation.  requests == 0 is valid; rows from requests * beams on stay as
 * they were.  In place, a row that is its own parent is neither read nor written.
 * Errors (nothing enqueued): ERR_ARG (NULL handle, parents NULL, one of begin and end NULL, requests < 0 or
 * requests * beams or requests times the handle's outer indices >= 2^31; memory that these rows of one state's out
 * take and another state or out, or the state itself where out is not the same, holds too, whatever begin and end:
 * checked on the first call with so many requests; layouts that interleave beyond what a short search resolves
 * count as such), ERR_ALIGN (an array not 4-byte aligned), ERR_CUDA.
 */
int headloss_reorder(headloss_reorder_t h, const int32_t* parents, int64_t requests, const int32_t* begin,
                     const int32_t* end, void* stream);

void headloss_reorder_destroy(headloss_reorder_t h);

#ifdef __cplusplus
}
#endif

#endif /* HEADLOSS_BEAM_H */
