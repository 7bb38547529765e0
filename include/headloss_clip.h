/*
 * headloss_clip.h -- the global gradient norm over many tensors, and clipping (C ABI).
 *
 * The last step before an update: the 2-norm over every gradient of the model (the head's
 * and the body's), and one factor on all of them where it is too large:
 *   norm   = inv_scale * sqrt(sum over all tensors and elements of g^2)
 *   factor = inv_scale * (norm > max_norm ? max_norm / norm : 1)
 *   out    = g * factor, formed in fp32 and rounded once to the tensor's type.
 * inv_scale takes off what the loss's grad_scale put on.  A norm that is not finite leaves
 * the factor at inv_scale: the caller reads the norm and skips the step.
 *
 * Squares are summed in fp32 over at most a few hundred elements and from there on in fp64, in
 * an order that the sizes, the addresses modulo 16 bytes and the GPU's number of SMs fix (the same
 * result every time for the same list on the same GPU); a run of squares that leaves
 * fp32's range, or comes near its lower end, is summed again from scaled values, so the sum is right
 * over the whole range of the types, subnormal values among them; the norm is its root, rounded to fp32.
 *
 * Status codes are those of headloss.h.
 */
#ifndef HEADLOSS_CLIP_H
#define HEADLOSS_CLIP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct headloss_clip* headloss_clip_t;

/* One gradient tensor: n dense elements of `dtype` (enum headloss_dtype) at grad, device,
 * aligned to the element; the clipped values go to out (same type and size).  out may equal
 * grad (in place) and must not overlap anything else.  n == 0 is valid (pointers unread). */
typedef struct {
    const void* grad;
    void* out;
    int64_t n;
    int dtype;
} headloss_gradient;

/*
 * headloss_clip_create -- a handle with a workspace for lists of up to max_grads tensors on
 * the current device (the only allocation).  One handle is used by one stream at a time.
 * Errors: ERR_ARG (max_grads < 1 or > 2^24, out NULL), ERR_CUDA.
 */
int headloss_clip_create(int max_grads, headloss_clip_t* out);

/*
 * headloss_clip_grads -- norm and clipping of n_grads tensors.
 *
 * grads:     n_grads entries in HOST memory, read before the call returns (they may change
 *            from call to call).
 * max_norm:  > 0 (infinity: never clipped).  inv_scale: > 0, finite.
 * stats_out: 2 fp32, device, 4-byte aligned (written): norm, factor.
 * In place with factor 1 nothing is written but stats_out.
 * Asynchronous on `stream`, no allocation.  The kernel's CTAs wait for one another, for two
 * seconds at most (a GPU that was taken from the process meanwhile): then nothing is written to
 * any out, and norm and factor are NaN (a factor never is otherwise); the handle stays usable.
 * Errors (nothing enqueued): ERR_ARG (NULL handle, grads (n_grads > 0) or stats_out, n_grads < 0 or
 * above the handle's, max_norm or inv_scale out of range, an entry with n < 0 or a NULL pointer), ERR_DTYPE,
 * ERR_ALIGN, ERR_CUDA (launch failure).
 */
int headloss_clip_grads(headloss_clip_t h, const headloss_gradient* grads, int n_grads,
                        float max_norm, float inv_scale, float* stats_out, void* stream);

void headloss_clip_destroy(headloss_clip_t h);

#ifdef __cplusplus
}
#endif

#endif /* HEADLOSS_CLIP_H */
