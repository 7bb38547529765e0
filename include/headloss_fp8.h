/*
 * headloss_fp8.h -- the LM head's product in 8-bit floating point, with one fp32 scale for
 * each block of 128 (C ABI).
 *
 * An 8-bit matrix is a row-major array of codes (enum headloss_fp8) whose rows start every ld
 * bytes, and an array of scales:
 *   block 1:   a scale for each row and 128 columns, scales[k * rows + i] for row i, columns
 *              128 k .. 128 k + 127 (rows consecutive);
 *   block 128: a scale for each 128 x 128 elements, scales[(i / 128) * KB + k], KB = ceil(cols / 128).
 * An element stands for code * scale.
 *
 * A block x is quantised as: s = max(amax * (1 / top), 2^-126) in fp32, amax its largest
 * magnitude, top the type's largest value (448, 57344) and 1 / top rounded to fp32; each code is
 * x * (1 / s), both in fp32, rounded to nearest even (saturating).  A block that holds an infinity
 * or a NaN has the scale NaN, so that every output it enters is NaN.
 *
 * The head's three products, with x the hidden states (tokens x D), w the weight (V x D) and
 * g the loss's gradient (tokens x V):
 *   logits      = x . w^T:   a = x block 1,   b = w block 128
 *   grad_hidden = g . w:     a = g block 1,   b = w^T block 128
 *   grad_weight = g^T . x:   a = g^T block 1, b = x^T block 128
 * headloss_fp8_quantize gives a matrix and its transpose from one read.
 *
 * Status codes are those of headloss.h.
 */
#ifndef HEADLOSS_FP8_H
#define HEADLOSS_FP8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum headloss_fp8 { HEADLOSS_E4M3 = 0, HEADLOSS_E5M2 = 1 };

/*
 * headloss_fp8_quantize -- x and / or its transpose in 8 bits.
 *
 * x:        rows x cols of `dtype` (enum headloss_dtype), device, row i at element i * ld
 *           (ld >= cols), aligned to the element.  Rows on 16-byte boundaries are read fastest.
 * type:     enum headloss_fp8, of both outputs.
 * q:        rows x cols codes or NULL (written), ldq bytes a row; block: 1 or 128; scales as above.
 * qt:       the transpose, cols x rows codes, or NULL (written), ldqt bytes a row; block_t, scales_t
 *           likewise (of the transpose: block_t 1 is a scale for each column of x and 128 rows).
 *           q and qt: 16-byte aligned, ldq >= cols and ldqt >= rows multiples of 16.  A row's bytes
 *           past its columns may be written (zeros).
 * Asynchronous on `stream`, no allocation.  rows == 0 or cols == 0 is valid.
 * Errors (nothing enqueued): ERR_ARG (a negative size, one of 2^31 - 128 or more, 2^31 blocks of 128 x 128
 * or more, ld < cols, a NULL x or scales, both of q and qt NULL, ldq or ldqt too small, block not 1 or 128, type
 * unknown), ERR_DTYPE, ERR_ALIGN, ERR_CUDA (launch failure).
 */
int headloss_fp8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int dtype, int type,
                          void* q, int64_t ldq, float* scales, int block, void* qt, int64_t ldqt,
                          float* scales_t, int block_t, void* stream);

/*
 * headloss_fp8_workspace -- bytes of workspace that headloss_fp8_matmul takes for M x N x K on
 * the current device (0: none); -1 for sizes that it refuses.  Needs a device.
 */
int64_t headloss_fp8_workspace(int64_t M, int64_t N, int64_t K);

/*
 * headloss_fp8_matmul -- out = a . b^T.
 *
 * a:        M x K codes of `a_type`, lda bytes a row, a_scales of block 1.
 * b:        N x K codes of `b_type`, ldb bytes a row, b_scales of block 128.
 *           a and b: 16-byte aligned, lda and ldb multiples of 16 and >= K.  Bytes past K are not used.
 * out:      M x N of `out_dtype` (enum headloss_dtype), row i at element i * ldo (ldo >= N),
 *           aligned to the element (16-byte aligned rows are written fastest; elements past N of a row
 *           are not written).
 *           out[i, j] = sum over blocks k of a_scale[i, k] b_scale[j / 128, k] (sum over the block of
 *           codes' products): products and sums in fp32, one rounding at the end.
 * workspace: at least headloss_fp8_workspace(M, N, K) bytes, device, 16-byte aligned; NULL where
 *           that is 0.  Its content is not kept; calls that may run at once need workspaces of their own.
 * err:      one int, device, 4-byte aligned, zeroed by the caller: bit 0 is set if a wait inside the
 *           kernel gave up (~2 s); the outputs are unreliable then.
 * Asynchronous on `stream`, no allocation; the result has the same bits in every run.
 * M == 0 or N == 0 is valid.
 * Errors (nothing enqueued): ERR_ARG (a negative size, K < 1, a size of 2^31 - 256 or more, 2^31 tiles of 128 x
 * 256 or more, a pitch too small, a NULL pointer, a type unknown, workspace_bytes too small), ERR_DTYPE,
 * ERR_ALIGN, ERR_CUDA.
 */
int headloss_fp8_matmul(const void* a, int64_t lda, const float* a_scales, int a_type, const void* b,
                        int64_t ldb, const float* b_scales, int b_type, int64_t M, int64_t N, int64_t K,
                        void* out, int64_t ldo, int out_dtype, void* workspace,
                        int64_t workspace_bytes, int* err, void* stream);

/*
 * headloss_fp8_linear_workspace -- bytes of workspace of headloss_fp8_linear; -1 for sizes that it
 * refuses.  Needs a device.
 */
int64_t headloss_fp8_linear_workspace(int64_t M, int64_t N, int64_t K);

/*
 * headloss_fp8_linear -- out = x . b^T, x (M x K of `dtype`, row i at element i * ldx) quantised to e4m3 in
 * block 1 on the way: headloss_fp8_quantize and headloss_fp8_matmul in one call, the product's loads of b
 * beginning while x is quantised.  The same bits as the two calls.  Arguments, checks and errors as
 * theirs; workspace at least headloss_fp8_linear_workspace(M, N, K) bytes (never 0 for M, N > 0).
 */
int headloss_fp8_linear(const void* x, int64_t ldx, int dtype, const void* b, int64_t ldb,
                        const float* b_scales, int b_type, int64_t M, int64_t N, int64_t K, void* out,
                        int64_t ldo, int out_dtype, void* workspace, int64_t workspace_bytes, int* err,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HEADLOSS_FP8_H */
