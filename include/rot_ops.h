/*
 * rot_ops.h - training operators next to the optimizer step: dropout from a
 * counter-based generator, layer norm (with the residual stream and dropout
 * in front of it), the clipped policy loss on logits, and products of 8-bit
 * matrices with power-of-two block scales.  Between them they carry a
 * training step from hidden states to the float32 gradients that rot_step
 * reads.
 *
 * Conventions: those of rot.h (0 or a negative ROT_E* code, caller-owned
 * device memory, work enqueued on `stream` without waiting, nothing
 * allocated, no C++ exception crosses).  In addition:
 * - Matrices are row-major with a leading dimension (ld*) in elements, at
 *   least the number of columns; rows of any alignment are accepted except
 *   where stated.  Element counts and offsets are 64-bit.
 * - Element types are ROT_TYPE_*.  Sums, statistics and losses are float32;
 *   each output element is rounded to its type once.
 * - Results do not depend on timing: there are no floating-point atomics.
 * - Outputs must not overlap inputs except where stated.
 * - Sizes of zero rows (tokens) return ROT_OK without a launch where there
 *   is nothing to write.
 * - Every entry point checks its arguments before any device work
 *   (ROT_EINVAL), then the device (ROT_ENOTSUP unless sm_103), and reports a
 *   failed launch as ROT_ECUDA.
 */
#ifndef ROT_OPS_H_
#define ROT_OPS_H_

#include <stdint.h>

#include "rot.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROT_TYPE_F32 0
#define ROT_TYPE_F16 1
#define ROT_TYPE_BF16 2
#define ROT_TYPE_E4M3 3 /* 8-bit float, 4 exponent and 3 mantissa bits, no infinity */
#define ROT_TYPE_E5M2 4 /* 8-bit float, 5 exponent and 2 mantissa bits */

/* ---- dropout -------------------------------------------------------------
 *
 * The mask is a pure function of (seed, offset, i, p), i the element's index
 * in row-major order (row * cols + col, whatever the leading dimensions):
 * element i is kept if word i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror,
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), at counter
 * (i/4 low, i/4 high, offset low, offset high) under the key (seed low, seed
 * high), is >= round(p 2^32) (ties to even).  Nothing is stored: the
 * backward pass computes the mask again.  Give every call of a training run
 * its own (seed, offset).
 */

/* y = residual + kept ? x * (1 / (1 - p)) : 0, in float32 (product, then
 * sum), rounded once.  residual may be NULL (no sum).  The gradient of x is
 * the same call on the gradient of y without a residual; the residual's
 * gradient is that of y itself.  Dropped elements contribute 0 whatever x
 * holds (NaN and infinities included).  y may be x or residual.  type:
 * ROT_TYPE_F32, F16 or BF16 (x, residual and y).  p in [0, 1]; p = 1 drops
 * everything.
 * Errors: ROT_EINVAL (negative sizes, null pointers with rows * cols > 0, a
 * leading dimension below cols, unknown type, p outside [0, 1] or NaN). */
int rot_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y,
                int64_t ldy, int64_t rows, int64_t cols, int32_t type, double p, uint64_t seed,
                uint64_t offset, void* stream);

/* ---- layer norm ----------------------------------------------------------
 *
 * Forward, per row of the hidden stream h:
 *   h    = residual + dropout(x)            (stored in `type`; the norm reads
 *                                            the stored values)
 *   mean = sum h / cols,  rstd = 1 / sqrt(sum (h - mean)^2 / cols + eps)
 *   y    = (h - mean) rstd weight + bias
 * Backward, with wdy = dy weight and hat = (h - mean) rstd:
 *   g  = rstd (wdy - mean(wdy) - hat mean(wdy hat)) + dh
 *   dx = dropout(g), dweight = sum over rows of dy hat, dbias = sum of dy
 */

/* x, h_out, y, residual: rows x cols of `type` (F32, F16, BF16).  weight,
 * bias: cols elements of wtype (F32, or `type`); bias may be NULL.  residual
 * may be NULL; with residual == NULL and p == 0 h is x itself and h_out is
 * not written (may be NULL), otherwise h_out is required (it may be x or
 * residual).  mean, rstd: `rows` float32 each.  Dropout as rot_dropout.
 * Errors: ROT_EINVAL (rows < 0, cols outside [1, ROT_MAX_DIM], null
 * pointers, a leading dimension below cols, unknown types, p outside [0, 1],
 * eps negative or NaN). */
int rot_layer_norm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           const void* weight, const void* bias, int32_t wtype, void* h_out,
                           int64_t ldh, void* y, int64_t ldy, float* mean, float* rstd,
                           int64_t rows, int64_t cols, int32_t type, float eps, double p,
                           uint64_t seed, uint64_t offset, void* stream);

/* Workspace bytes rot_layer_norm_backward needs (256-byte aligned device
 * memory): the weight gradient's partial sums.  0 for sizes it refuses. */
uint64_t rot_layer_norm_work_bytes(int64_t rows, int64_t cols);

/* dy, h, dh, dres_out, dx: rows x cols of `type`.  h, mean, rstd: as the
 * forward pass left them.  dh: gradient that reaches h other than through the
 * norm, or NULL.  dres_out receives g (the residual's gradient) and dx the
 * dropped g; with p == 0 the two are the same array: pass dres_out = NULL and
 * g goes to dx.  With p > 0 both are required.  dweight, dbias: cols float32,
 * overwritten (dbias may be NULL).  dx or dres_out may be dh.  Errors as the
 * forward pass, plus ROT_EINVAL for a missing or misaligned workspace or
 * work_bytes below rot_layer_norm_work_bytes. */
int rot_layer_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                            const float* mean, const float* rstd, const void* weight,
                            int32_t wtype, const void* dh, int64_t lddh, void* dres_out,
                            int64_t lddres, void* dx, int64_t lddx, float* dweight, float* dbias,
                            int64_t rows, int64_t cols, int32_t type, double p, uint64_t seed,
                            uint64_t offset, void* work, uint64_t work_bytes, void* stream);

/* ---- policy loss ---------------------------------------------------------
 *
 * Per token t with logits z (a row of `vocab` entries), target v, old and
 * reference log-probabilities, advantage A and weight w:
 *   logp  = z_v - log sum exp z
 *   ratio = exp(logp - old)
 *   term  = -min(ratio A, clip(ratio, 1 - clip_low, 1 + clip_high) A)
 *           + kl_coef (exp(ref - logp) - (ref - logp) - 1)
 *   loss  = sum over t of w term
 * and the gradient of loss with respect to z is s (onehot(v) - softmax(z)),
 *   s = w (kl_coef (1 - exp(ref - logp)) - [ratio A <= clip(...) A] ratio A).
 * A weight of zero masks its token: nothing of its row, target, old, ref or
 * advantage is looked at, its logp, term and gradient row are 0.  The caller
 * folds the normalisation into the weights.  A target outside [0, vocab) of
 * an unmasked token gives NaN (logp, term, loss and its gradient row).
 */

/* logp (tokens float32) of `targets` (int64) under softmax(logits); weights
 * may be NULL (every token counts).  type: F32, F16 or BF16.
 * Errors: ROT_EINVAL (tokens < 0, vocab < 1 or above 2^30, null pointers
 * with tokens > 0, ldl < vocab, unknown type). */
int rot_token_logprobs(const void* logits, int64_t ldl, const int64_t* targets,
                       const float* weights, float* logp, int64_t tokens, int64_t vocab,
                       int32_t type, void* stream);

/* Loss and gradient.  loss: one float32 (the terms' sum in a fixed order);
 * logp, terms: `tokens` float32 each (terms[t] = w term).  ref_logp may be
 * NULL (kl_coef must then be 0), and with kl_coef == 0 it is not looked at.
 * dlogits (type and vocab as logits, or NULL:
 * loss only) receives grad_scale times the gradient; it may be the logits
 * themselves (same ld).  tokens == 0 sets loss to 0.
 * Errors: as rot_token_logprobs, plus clip bounds or kl_coef negative or NaN,
 * clip_low > 1 and lddl < vocab. */
int rot_policy_loss(const void* logits, int64_t ldl, const int64_t* targets, const float* old_logp,
                    const float* ref_logp, const float* advantages, const float* weights,
                    float* loss, float* logp, float* terms, void* dlogits, int64_t lddl,
                    int64_t tokens, int64_t vocab, int32_t type, float clip_low, float clip_high,
                    float kl_coef, float grad_scale, void* stream);

/* ---- 8-bit matrices ------------------------------------------------------
 *
 * A matrix R x C in 8 bits: `data` (E4M3 or E5M2; rows ld bytes apart, data
 * and ld multiples of 16 bytes for the product) and one power-of-two scale
 * for each block of block_rows x 128 elements, block_rows 1 or 128.  A scale
 * is one byte e standing for 2^(e - 127) (255: NaN), stored column block
 * first: the scale of block (i, j) is scale[j * lds + i], i the row block and
 * j the column block.  The matrix stands for data * scale.
 */

/* data, scale <- x (rows x cols of `type`), and/or the transposed matrix
 * data_t (cols x rows), scale_t.  Per block, e is the least exponent >= -127
 * for which every finite element of the block is within max 2^e (max: 448
 * for E4M3, 57344 for E5M2); elements become round-to-nearest-even of x
 * 2^-e; NaN and infinities become NaN, in their own place only.  Both outputs
 * of one call come from one read of x.  With block_rows 1 the transposed
 * matrix has scales of its own (its blocks are 128 rows of x by one column);
 * with 128 both hold the same blocks.  Either output may be NULL (not both).
 * ldq >= cols, lds >= ceil(rows / block_rows), ldqt >= rows, ldst >=
 * ceil(cols / block_rows).
 * Errors: ROT_EINVAL (sizes < 0, null or too narrow outputs, unknown types,
 * block_rows other than 1 or 128). */
int rot_fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int32_t type,
                     int32_t format, int32_t block_rows, void* data, int64_t ldq, uint8_t* scale,
                     int64_t lds, void* data_t, int64_t ldqt, uint8_t* scale_t, int64_t ldst,
                     void* stream);

/* Workspace bytes rot_fp8_gemm needs for these sizes (may be 0). */
uint64_t rot_fp8_gemm_work_bytes(int64_t M, int64_t N, int64_t K);

/* C (M x N of ctype F32, F16 or BF16) = A B^T, A: M x K and B: N x K in 8
 * bits (formats may differ), or C += A B^T with accumulate != 0 (ctype F32
 * only).  Products are exact; sums are float32 (on the tensor cores over
 * stretches of K, the stretches joined in float32).  K == 0 gives C = 0 (or
 * leaves it, accumulating).  status: device int that receives ROT_ETIMEOUT if
 * a device-side wait gives up (may be NULL).
 * Errors: ROT_EINVAL (sizes < 0 or above 2^31 - 256, null pointers,
 * data pointers or leading dimensions that are not multiples of 16, lds too
 * small, unknown types, accumulate with another ctype than F32, a missing or
 * misaligned (256 bytes) workspace). */
int rot_fp8_gemm(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, int32_t a_format,
                 const uint8_t* a_scale, int64_t a_lds, int32_t a_block_rows, const void* b,
                 int64_t ldb, int32_t b_format, const uint8_t* b_scale, int64_t b_lds,
                 int32_t b_block_rows, void* c, int64_t ldc, int32_t ctype, int32_t accumulate,
                 void* work, uint64_t work_bytes, int32_t* status, void* stream);

/* ---- linear layers in 8 bits ---------------------------------------------
 *
 * y = x W^T with x (tokens x inner, F32, F16 or BF16) quantised by rows
 * (E4M3, blocks of 1 x 128) and W (outer x inner) kept in 8 bits by the
 * caller; and its gradients.  One call runs quantisation and products; the
 * results are those of rot_fp8_quantize and rot_fp8_gemm.
 */

/* Workspace bytes (256-byte aligned device memory); 0 for sizes that are
 * refused. */
uint64_t rot_fp8_linear_work_bytes(int64_t tokens, int64_t inner, int64_t outer);
uint64_t rot_fp8_linear_backward_work_bytes(int64_t tokens, int64_t inner, int64_t outer);

/* y: tokens x outer of x's type.  w, w_scale: W as rot_fp8_gemm takes it.
 * Errors: as rot_fp8_quantize and rot_fp8_gemm. */
int rot_fp8_linear(int64_t tokens, int64_t inner, int64_t outer, const void* x, int64_t ldx,
                   int32_t type, const void* w, int64_t ldw, int32_t w_format,
                   const uint8_t* w_scale, int64_t w_lds, int32_t w_block_rows, void* y,
                   int64_t ldy, void* work, uint64_t work_bytes, int32_t* status, void* stream);

/* dx (tokens x inner of dy's type) = dy W, from W's transpose wt (inner x
 * outer in 8 bits), dy quantised by rows; dw (outer x inner, float32: the
 * optimizer's gradient) = dy^T x, or += with accumulate != 0, both operands
 * quantised along the tokens.  dy: tokens x outer, x: tokens x inner, of one
 * type.  tokens == 0 gives dw = 0 (or leaves it, accumulating).
 * Errors: as rot_fp8_linear. */
int rot_fp8_linear_backward(int64_t tokens, int64_t inner, int64_t outer, const void* dy,
                            int64_t lddy, const void* x, int64_t ldx, int32_t type,
                            const void* wt, int64_t ldwt, int32_t wt_format,
                            const uint8_t* wt_scale, int64_t wt_lds, int32_t wt_block_rows,
                            void* dx, int64_t lddx, float* dw, int64_t lddw, int32_t accumulate,
                            void* work, uint64_t work_bytes, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROT_OPS_H_ */
