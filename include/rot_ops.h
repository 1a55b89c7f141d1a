/*
 * rot_ops.h - training operators next to the optimizer step: dropout from a
 * counter-based generator, layer norm (with the residual stream and dropout
 * in front of it), the heads' entry to attention (rotary positions, the norm
 * of queries and keys), the clipped policy loss on logits, products of 8-bit
 * matrices with power-of-two block scales, and the step of the parameters
 * that are not rot_step's matrices (AdamW over many tensors, the gradient's
 * norm).  Between them they carry a training step from hidden states to the
 * float32 gradients that rot_step reads, and step the rest.
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

/* ---- heads: rotary positions, norm of queries and keys -------------------
 *
 * Queries and keys lie as [batch][token][head][dim] under any strides (a
 * part of a fused projection, heads before tokens), a head's elements next to
 * one another.
 *
 * Rotation of the first `rotated` elements of a head by its token's position
 * p: pair i turns by the angle 2 pi t, t the fractional part of p turns[i] /
 * 2^64.  The product is exact (modulo 2^64), so that an angle is as good at
 * position 2^31 as at 1: turns[i] is the part of a turn that one position
 * adds, to the nearest 2^-64.  With c = magnitude cos, s = magnitude sin:
 *   a' = a c - b s,  b' = b c + a s
 * on the pairs (i, i + rotated / 2), or interleaved (2 i, 2 i + 1).  The rest
 * of the head passes through.  `inverse` turns the other way, with the same
 * magnitude: the rotation's gradient.
 *
 * Norm, per head x with the weight w (dim elements, one for all heads):
 *   r = 1 / sqrt(sum x^2 / dim + eps),  y = rotation(x r w)
 * Backward, with g the inverse rotation of dy and hat = x r:
 *   dx = r (g w - hat mean(g w hat)),  dw = sum over tokens and heads of g hat
 */
#define ROT_MAX_HEAD_DIM 512

typedef struct rot_heads {
  void* data; /* the first head of the first token */
  int64_t heads;
  int64_t batch_stride, token_stride, head_stride; /* in elements */
} rot_heads;

typedef struct rot_rotary {
  const uint64_t* turns; /* rotated / 2 device words */
  int64_t rotated;       /* even, 0 to dim */
  float magnitude;
  int32_t interleaved;
  const void* positions;  /* device, of position_bytes (4 or 8, signed); NULL: token t is at start + t */
  int32_t position_bytes;
  int64_t position_batch_stride, position_token_stride; /* in positions; 0 shares them */
  int64_t start;
} rot_rotary;

/* q_out (and k_out) = the rotation of q (and k) of `type` (F32, F16, BF16).
 * k and k_out may both be NULL.  An output may be its input (same strides).
 * batch * tokens <= 2^30, heads <= 2^16.  Strides are not negative; the
 * outputs' rows must not overlap, the inputs' may (stride 0).
 * Errors: ROT_EINVAL (sizes out of range, dim outside [1, ROT_MAX_HEAD_DIM],
 * null pointers, unknown type, outputs with another number of heads or with
 * rows that overlap, rotated odd, negative or above dim, position_bytes,
 * magnitude NaN). */
int rot_rotate(const rot_heads* q, const rot_heads* q_out, const rot_heads* k,
               const rot_heads* k_out, int64_t batch, int64_t tokens, int64_t dim, int32_t type,
               const rot_rotary* rotary, int32_t inverse, void* stream);

/* The norm with the rotation behind it; rotary may be NULL (no rotation).
 * Weights: dim elements of wtype (F32 or `type`).  k, k_weight and k_out may
 * all be NULL.  An output may be its input.  Squares are float32.
 * Errors: as rot_rotate, plus eps negative or NaN, wtype. */
int rot_head_norm_forward(const rot_heads* q, const void* q_weight, const rot_heads* q_out,
                          const rot_heads* k, const void* k_weight, const rot_heads* k_out,
                          int32_t wtype, int64_t batch, int64_t tokens, int64_t dim, int32_t type,
                          float eps, const rot_rotary* rotary, void* stream);

/* Workspace bytes of rot_head_norm_backward (256-byte aligned device memory);
 * 0 for a dim that it refuses. */
uint64_t rot_head_norm_work_bytes(int64_t dim);

/* dq_out, dq_weight (dim float32, overwritten) from dq and the forward pass's
 * q; the same of k where it is given.  dq_out may be dq or q.
 * Errors: as the forward pass, plus a missing, misaligned or too small
 * workspace. */
int rot_head_norm_backward(const rot_heads* dq, const rot_heads* q, const void* q_weight,
                           const rot_heads* dq_out, float* dq_weight, const rot_heads* dk,
                           const rot_heads* k, const void* k_weight, const rot_heads* dk_out,
                           float* dk_weight, int32_t wtype, int64_t batch, int64_t tokens,
                           int64_t dim, int32_t type, float eps, const rot_rotary* rotary,
                           void* work, uint64_t work_bytes, void* stream);

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

/* ---- AdamW over many tensors ---------------------------------------------
 *
 * Per element (decoupled weight decay; Loshchilov and Hutter, "Decoupled
 * weight decay regularization", ICLR 2019), t the step from 1:
 *   g = scale grad min(1, max_norm / (|scale| norm))
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in float32, p read from and written to `master` where that is given (p then
 * receives its value, rounded to nearest).  A product |scale| norm that is not
 * finite in float32 and a device step below 1 leave every tensor as it was.
 *
 * States in 8 bits: m and sqrt(v) as E4M3 numbers, under one power-of-two
 * scale for every 128 consecutive elements (a byte e for 2^(e - 127), 255 for
 * NaN; e the least for which all finite elements are within 448 of it).
 * Rounding is random: an average that moves by 1 - beta2 = 0.001 of the way
 * each step would stay where it is for good if it were rounded to nearest at
 * three fraction bits.  With w the generator's word of an element, a number
 * between two neighbours goes to the upper one where its place between them,
 * from 0 to 1, plus ((w mod 2^16) + 1/2) / 2^16 is at least 1.  A root above 0
 * is at least the least number above 0.  NaN and infinities become NaN, in
 * their own place only.
 * A bfloat16 p without a master is rounded likewise, by floor(w / 2^16) /
 * 2^16 (a step of it is often below half of p's last place).
 * The word of element i of a tensor: word i mod 4 of Philox4x32-10 at the
 * counter (j low, j high, t low, t high) under the key seed, with j = b / 4 +
 * floor(i / 4) and b the elements of the tensors before it in the list, each
 * rounded up to a multiple of 128.  Calls of the same step need seeds of
 * their own.
 */
typedef struct rot_adamw_tensor {
  void* p;
  const void* g;
  void* m; /* float32; or E4M3 where m_scale is given */
  void* v; /* float32; or E4M3 of the root where v_scale is given */
  uint8_t *m_scale, *v_scale; /* ceil(n / 128) bytes each, or both NULL */
  float* master;              /* NULL: p itself (F32 or BF16) */
  int64_t n;
  int32_t p_type, g_type; /* ROT_TYPE_F32, F16 or BF16 */
} rot_adamw_tensor;

typedef struct rot_adamw_hyper {
  double lr, beta1, beta2, eps, weight_decay, scale, max_norm;
  int64_t step; /* from 1 */
  uint64_t seed;
  const float* lr_device;     /* device word read instead of lr, or NULL */
  const int64_t* step_device; /* device word read instead of step, or NULL */
  const float* norm;          /* device word: the norm of all gradients; NULL: no clipping */
} rot_adamw_hyper;

/* One step of `count` tensors, in place.  Tensors hold n consecutive
 * elements; pointers are aligned to their elements (16 bytes is best).  The
 * written arrays must not overlap.  Tensors of no elements are left out.
 * Errors: ROT_EINVAL (count < 0, n < 0, more than 2^40 elements in all, null
 * or misaligned pointers, unknown types, one scale without the other, F16
 * without a master, F32 with one, an array given twice, hyper-parameters that
 * are negative or NaN, betas not below 1, scale not finite, step < 1, max_norm
 * not above 0). */
int rot_adamw_step(const rot_adamw_tensor* tensors, int32_t count, const rot_adamw_hyper* hyper,
                   void* stream);

/* The same with t counted on the device: `taken` (one int64) holds the steps
 * taken so far, t is one more, and the word moves on to t unless the norm keeps
 * the step from being taken; hyper's step and step_device are not looked at.
 * The corrections 1 - beta^t are float64, rounded as rot_adamw_step's of a step
 * given by the host.  A call of no tensors counts, too.
 * work: ROT_ADAMW_COUNT_BYTES of device memory.
 * Errors: as rot_adamw_step, plus null or misaligned (8 bytes; work 16) taken
 * and work. */
#define ROT_ADAMW_COUNT_BYTES 32
int rot_adamw_step_counted(const rot_adamw_tensor* tensors, int32_t count,
                           const rot_adamw_hyper* hyper, int64_t* taken, void* work, void* stream);

/* Workspace bytes of rot_gradient_norm (256-byte aligned device memory). */
uint64_t rot_gradient_norm_work_bytes(int32_t count);

/* norm (one float32) = sqrt of the sum of the squares of all elements of the
 * tensors (n consecutive elements of `type` each).  Squares and a
 * thread's sums of 32 are float32, sums of those float64: elements near 2^64
 * give infinity, and those below 2^-75 count as 0.
 * Errors: ROT_EINVAL (count < 0, null pointers, n < 0, more than 2^40 elements
 * in all, misaligned elements, unknown types, workspace). */
typedef struct rot_gradient {
  const void* g;
  int64_t n;
  int32_t type;
} rot_gradient;
int rot_gradient_norm(const rot_gradient* gradients, int32_t count, float* norm, void* work,
                      uint64_t work_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROT_OPS_H_ */
