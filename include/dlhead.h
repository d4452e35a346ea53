/*
 * dlhead.h -- C ABI of a merged model's output head on MI355X (gfx950).
 *
 * A merge round leaves several candidates for the next published model: the
 * global, its EMA, the uniform average, averages of snapshots (dlmerge.h).
 * They are told apart by what the output head says of them: the cross-entropy
 * of a probe's tokens (DiffuRefill-1B technical report, section "The final
 * stretch", Table 5; model card, "Training progress"), the confidence of
 * drafted tokens (model card, "Decoding configuration").  The calls below are
 * that head, from the residual stream to log probabilities, with what training
 * needs of it:
 *
 *   dl_rmsnorm            residual addition + root-mean-square norm, output in
 *                         fp32, bf16 or 8 bits with scales
 *   dl_rmsnorm_backward   its gradients
 *   dl_w4_quantize        a merged matrix laid out in 4 bits with group scales
 *   dl_w4_matvec          its product with 1..DL_MAX_VECTORS vectors
 *   dl_logprobs           log probabilities of given tokens, entropy, the most
 *                         likely alternatives
 *   dl_logprobs_backward  the gradient of both in the logits
 *   dl_head_logprobs      log probabilities and entropy straight from the norm's
 *                         output and the embedding, without the logits
 *   dl_head_logprobs_backward  the gradients of both in these inputs
 *   dl_e4m3_quantize      a matrix laid out in 8 bits with a scale for each 128
 *                         x 128 elements, or each 128 of a row
 *   dl_e4m3_matmul        the product of the two kinds, for one token or many
 *
 * Library, status codes and element types are those of dlmerge.h.
 *
 * Memory.  Array arguments are DEVICE pointers to memory the caller owns.
 * Matrices are row-major; ld* is the distance of two rows in elements, at
 * least the number of columns.  The library allocates nothing, keeps nothing
 * from one call for the next, never synchronises and launches every kernel on
 * `stream` (hipStream_t; NULL: the null stream), so calls may be captured into
 * a HIP graph.  Where a call takes a workspace (256-byte aligned), work in
 * flight on several streams, and captured graphs that may run at once, need
 * one each; calls in one stream's order may share one, and its contents do not
 * matter.  Each span from an argument's first element to its last must lie
 * inside one device allocation on the calling thread's current device, which
 * must be the stream's.  An output must not overlap an input or another
 * output unless the call says so (a span counts from first to last element,
 * the gaps between rows included); gaps between rows are left as they were.
 * Pointers must be aligned to their element type (`packed`: 16 bytes); every
 * such alignment and ld gives the same results.
 *
 * Numerics.  Sums, softmax statistics, norms and scales are binary32 or wider
 * in a fixed order: a call gives the same bits every time.
 *
 * Errors.  As in dlmerge.h: every check is made on the host before any
 * launch; DL_E_INVAL, DL_E_ALIGN, or DL_E_HIP (an error already pending, or a
 * launch that failed).
 */
#ifndef DLHEAD_H
#define DLHEAD_H

#include <stdint.h>

#include "dlmerge.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit floating point (one sign, four exponent, three mantissa bits, largest
 * value 448, no infinity): an output of dl_rmsnorm and dl_e4m3_quantize, and an
 * input of dl_w4_matvec and dl_e4m3_matmul. */
enum { DL_E4M3 = 2 };

/* Scales that go with a matrix held in DL_E4M3. */
enum dl_scale {
    DL_SCALE_NONE = 0,     /* none (the other types)                            */
    DL_SCALE_ROW = 1,      /* one fp32 for each row                             */
    DL_SCALE_BLOCK32 = 2,  /* one byte e, standing for 2^(e-127), for each 32
                              columns of a row: rows x ceil(cols/32) bytes,
                              row after row; 255 stands for NaN                 */
    DL_SCALE_TILE128 = 3,  /* such a byte for each 128 rows of 128 columns:
                              ceil(rows/128) x ceil(cols/128) bytes             */
    DL_SCALE_BLOCK128 = 4  /* such a byte for each 128 columns of a row: rows x
                              ceil(cols/128) bytes                              */
};

#define DL_MAX_NORM_COLS 32768
#define DL_MAX_VECTORS 32
#define DL_MAX_TOP 32

/*
 * Residual addition and root-mean-square norm of `rows` rows of `cols`
 * columns:
 *     s = x + residual           (rounded to dtype; s = x without a residual)
 *     inv = 1 / sqrt(mean(s^2) + eps)      (in binary64, rounded to binary32)
 *     y = (s * inv) * weight               (two binary32 roundings)
 *
 *   x, residual  rows x cols of dtype (DL_F32 or DL_BF16); residual may be
 *                NULL.
 *   weight       cols fp32.
 *   eps          >= 0, finite.
 *   sum          rows x cols of dtype, receives s; NULL if not wanted, and
 *                NULL without a residual.  May be x or residual itself (same
 *                pointer and ld).
 *   y            rows x cols of y_dtype: DL_F32, DL_BF16, or DL_E4M3 with
 *                scales:
 *                DL_SCALE_ROW      scale = amax/448 of the row's |y|, elements
 *                                  y * (448/amax); a row whose amax is below
 *                                  2^-100 is held as zeros with scale 0.
 *                DL_SCALE_BLOCK32, DL_SCALE_BLOCK128  for each 32 or 128 columns
 *                                  the smallest power of two b >= 2^-127 with
 *                                  amax <= 448 b, elements y / b.
 *                Elements are rounded to nearest, ties to even; none is
 *                clipped.  A row (block) that holds a NaN or infinity has a
 *                NaN scale and zeros: all of it stands for NaN.
 *   scales       as scale_kind says; NULL for DL_SCALE_NONE.
 *   inv_rms      rows fp32, receives inv (dl_rmsnorm_backward reads it), or
 *                NULL.
 *
 * 1 <= cols <= DL_MAX_NORM_COLS; rows = 0 is a no-op.
 */
int dl_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldres, int dtype,
               const float *weight, float eps, int64_t rows, int64_t cols, void *sum,
               int64_t ldsum, void *y, int64_t ldy, int y_dtype, void *scales, int scale_kind,
               float *inv_rms, void *stream);

/*
 * Gradients of dl_rmsnorm for a gradient dy of y (of the values before any
 * rounding to y_dtype) and, if not NULL, dsum of s:
 *     g = dy * weight ;  h = s * inv ;  c = mean(g * h)
 *     dx = inv * (g - h*c) + dsum        (the gradient of x and of residual)
 *     dweight = sum over rows of dy * h
 * dy, dsum, sum (the norm's s), dx: rows x cols of dtype; dx may be dy or dsum
 * itself.  weight, dweight: cols fp32; dweight may be NULL, otherwise it is
 * written (not added to) and the call needs dl_rmsnorm_workspace_bytes of
 * workspace; a column's sum is off by at most (rows/512 + 64) 2^-24 of its
 * terms' magnitudes.  rows = 0 writes zeros to dweight.
 */
int dl_rmsnorm_workspace_bytes(int64_t rows, int64_t cols, int64_t *bytes);
int dl_rmsnorm_backward(const void *dy, int64_t lddy, const void *dsum, int64_t lddsum,
                        const void *sum, int64_t ldsum, int dtype, const float *weight,
                        const float *inv_rms, int64_t rows, int64_t cols, void *dx, int64_t lddx,
                        float *dweight, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * A matrix in 4 bits.  Each 32 columns of a row share a power of two b, held
 * as a byte e (b = 2^(e-127); 255: the block stands for NaN); an element is
 * one sign bit and a magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6} (codes 0..7)
 * times b.  With kb = ceil(cols/32): `packed` holds rows x kb x 16 bytes, a
 * byte two columns, the lower one in its low half, bit 3 of each half the
 * sign; `scales` holds rows x kb bytes.  `packed` is 16-byte aligned.  Columns
 * past cols in the last block have code 0.
 *
 * dl_w4_quantize lays out w (rows x cols, DL_F32 or DL_BF16, e.g. a weight
 * matrix of a merged global): b is the smallest power of two >= 2^-127 with
 * amax <= 6 b, elements are rounded to the nearest magnitude, ties to the even
 * code, none is clipped; a block that holds a NaN or infinity has e = 255 and
 * code 0.  values, if not NULL, receives what the codes stand for (rows x cols
 * of dtype: exact, infinite where they round up past its range), e.g. to score
 * the published matrix; it may be w itself.
 * 1 <= cols, rows <= 2^31 - 1; rows = 0 is a no-op.
 */
int dl_w4_bytes(int64_t rows, int64_t cols, int64_t *packed_bytes, int64_t *scale_bytes);
int dl_w4_quantize(const void *w, int64_t ldw, int dtype, int64_t rows, int64_t cols,
                   uint8_t *packed, uint8_t *scales, void *values, int64_t ldvalues,
                   void *stream);

/*
 * y[v][r] = sum over k < cols of x[v][k] * W[r][k] for r < rows and
 * v < count, 1 <= count <= DL_MAX_VECTORS: a matrix held in 4 bits times the
 * vectors of the tokens being decoded.
 *
 *   x         count x cols of x_dtype: DL_BF16, or DL_E4M3 with x_scales of
 *             x_scale_kind (DL_SCALE_ROW or DL_SCALE_BLOCK32), as dl_rmsnorm
 *             writes them.
 *   y         count x rows of y_dtype (DL_F32 or DL_BF16).
 *
 * Products are exact and summed in binary32 on the matrix cores (block scales
 * of x are applied in bf16, exact for values of at least 2^-133; a row scale
 * multiplies the sum of its codes' products, which is what has to fit binary32;
 * products and partial sums below 2^-126 may count as 0).  Any code
 * and scale byte is accepted; an element of W that stands for 2^128 or more is
 * infinite.  rows = 0 is a no-op; cols >= 1.
 */
int dl_w4_matvec(const uint8_t *packed, const uint8_t *scales, int64_t rows, int64_t cols,
                 const void *x, int64_t ldx, int x_dtype, const void *x_scales, int x_scale_kind,
                 int count, void *y, int64_t ldy, int y_dtype, void *stream);

/*
 * Of each row of logits (rows x vocab, DL_F32 or DL_BF16), with m its largest
 * element and S = sum exp(l - m):
 *
 *   logprobs      rows fp32: log softmax at targets[row], (l_t - m) - log S.
 *                 A target < 0 means none: 0.  A target >= vocab: NaN.  May be
 *                 NULL (and is without targets).
 *   entropy       rows fp32, or NULL: log S - sum exp(l - m) (l - m) / S.
 *   stats         rows x 2 fp32, or NULL: m and log S (for the backward pass).
 *   top_ids       rows x top_k int64, 0 <= top_k <= min(DL_MAX_TOP, vocab):
 *                 indices of the top_k largest logits, largest first, equal
 *                 ones by the lowest index (NaN before all others).
 *   top_logprobs  rows x top_k fp32: their log probabilities.  Both are NULL
 *                 if top_k is 0, neither otherwise.
 *
 * log S is formed as log1p of the other elements' sum, so the log probability
 * and entropy of a nearly certain token keep their relative accuracy
 * (exponentials below 2^-126 may count as 0).  S is off by at most 1e-5 of itself
 * for up to 2^18 tokens and 4e-5 for more (equal terms; some 1e-7 otherwise).
 * Logits
 * of -infinity (masked tokens) have probability 0 and log probability
 * -infinity.  A row of nothing else has log probability -infinity everywhere,
 * entropy 0 and stats (-infinity, 0).  A row with a NaN or +infinity gives NaN
 * (its top_ids are still as above).
 *
 * workspace: dl_logprobs_workspace_bytes bytes (a few long rows are split over
 * the GPU; 0 for many rows or short ones: then NULL is allowed).  1 <= vocab <=
 * 2^31 - 1; rows = 0 is a no-op.
 */
int dl_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top_k, int64_t *bytes);
int dl_logprobs(const void *logits, int64_t ldl, int dtype, int64_t rows, int64_t vocab,
                const int64_t *targets, float *logprobs, float *entropy, float *stats, int top_k,
                int64_t *top_ids, float *top_logprobs, void *workspace, int64_t workspace_bytes,
                void *stream);

/*
 * The gradient in the logits of dl_logprobs' logprobs and entropy: with
 * p = exp((l - m) - log S), t the row's target, a = dlogprobs[row] (0 without
 * a target) and b = dentropy[row] (0 if dentropy is NULL),
 *     dlogits = a * (delta_t - p) - b * p * (log p + entropy)
 * stats and entropy are the forward call's (entropy is needed with dentropy,
 * else NULL).  dlogits: rows x vocab of dtype; may be logits itself.  1 - p of
 * the target is formed as -expm1(log p).  Masked tokens (-infinity) other than
 * the target have gradient 0; a row with target >= vocab, a NaN or +infinity
 * gives NaN.
 */
int dl_logprobs_backward(const void *logits, int64_t ldl, int dtype, int64_t rows, int64_t vocab,
                         const int64_t *targets, const float *stats, const float *entropy,
                         const float *dlogprobs, const float *dentropy, void *dlogits,
                         int64_t lddl, void *stream);

/*
 * dl_logprobs for the logits l[i][v] = sum over k < width of x[i][k] *
 * embed[v][k], i < rows, v < vocab, which are formed piece by piece and not
 * kept: a probe's log probabilities under a candidate, a training step's loss.
 *
 *   x             rows x width of dtype (DL_F32 or DL_BF16), e.g. dl_rmsnorm's y.
 *   embed         vocab x width of dtype.
 *   targets, logprobs, entropy, stats   as for dl_logprobs.
 *
 * Products are exact and summed in binary32 (DL_F32: a product is off by at
 * most 2^-25 of itself; parts of an element below 2^-126 may count as 0, and
 * 2^128 - 2^119 or more as infinite).  A row of x that holds an infinity or NaN
 * may have results of NaN, and so may all rows if embed holds one.
 *
 * workspace: dl_head_workspace_bytes bytes; `backward` nonzero asks for what the
 * gradients need too (never less than without).  rows = 0 is a no-op.
 * 1 <= vocab, 1 <= width <= DL_MAX_NORM_COLS; rows and vocab at most 2^30, their
 * product at most 2^43.
 */
int dl_head_workspace_bytes(int64_t rows, int64_t vocab, int64_t width, int dtype, int backward,
                            int64_t *bytes);
int dl_head_logprobs(const void *x, int64_t ldx, const void *embed, int64_t lde, int dtype,
                     int64_t rows, int64_t vocab, int64_t width, const int64_t *targets,
                     float *logprobs, float *entropy, float *stats, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * The gradients of dl_head_logprobs' logprobs and entropy: with dlogits as
 * dl_logprobs_backward gives it,
 *     dx = dlogits x embed ;  dembed = dlogits^T x x
 * stats and entropy are the forward call's (entropy is needed with dentropy,
 * else NULL).  dx: rows x width, dembed: vocab x width of dtype, each written (not
 * added to); either may be NULL.  The logits are formed again piece by piece;
 * dlogits, in units of the largest magnitude among the dlogprobs and dentropy that
 * take part, is rounded to dtype, and its products summed in binary32.
 *
 * Without dentropy, a row without a target has no part: its dx is 0 and it adds
 * nothing to dembed, whatever its x, stats and dlogprobs hold.  A row with target
 * >= vocab has NaN for its dx and makes dembed NaN.  rows = 0 writes zeros to
 * dembed.
 */
int dl_head_logprobs_backward(const void *x, int64_t ldx, const void *embed, int64_t lde,
                              int dtype, int64_t rows, int64_t vocab, int64_t width,
                              const int64_t *targets, const float *stats, const float *entropy,
                              const float *dlogprobs, const float *dentropy, void *dx,
                              int64_t lddx, void *dembed, int64_t ldde, void *workspace,
                              int64_t workspace_bytes, void *stream);

/*
 * x (rows x cols, DL_F32 or DL_BF16) in 8 bits: codes, rows x cols in DL_E4M3
 * with rows ldc bytes apart, and scales of scale_kind: DL_SCALE_TILE128 (weights,
 * e.g. a matrix of a merged global) or DL_SCALE_BLOCK128 (activations).  A block's
 * scale b is the smallest power of two >= 2^-127 with amax <= 448 b; elements
 * x / b are rounded to nearest, ties to even, and none is clipped.  A block that
 * holds a NaN or infinity has scale 255 and code 0: all of it stands for NaN.
 * values, if not NULL, receives what the codes stand for (rows x cols of
 * dtype: exact, infinite where they round up past its range), e.g. to score the
 * published matrix; it may be x itself.
 * 1 <= cols, rows <= 2^31 - 1; rows = 0 is a no-op.
 */
int dl_e4m3_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                     uint8_t *codes, int64_t ldc, uint8_t *scales, int scale_kind, void *values,
                     int64_t ldvalues, void *stream);

/*
 * y[i][r] = sum over k < cols of x[i][k] * W[r][k] for r < rows and i < count:
 * a matrix in 8 bits with DL_SCALE_TILE128 times tokens' vectors in 8 bits with
 * DL_SCALE_BLOCK128.
 *
 *   w         rows x cols codes, rows ldw bytes apart;  w_scales its scales.
 *   x         count x cols codes, rows ldx bytes apart;  x_scales its scales.
 *   y         count x rows of y_dtype.  DL_F32: products are exact and summed in
 *             binary32 (products and partial sums below 2^-126 may count as 0).
 *             DL_BF16: the matrix cores' own 8-bit products, which drop low bits
 *             of small addends beside large ones (at most 2^-13 of the sum of
 *             magnitudes of 128 products, some 2e-5 of a typical result), or for
 *             up to 32 vectors exact ones; then bf16's rounding.
 *
 * Block scales may be applied in bf16, exact for values of at least 2^-133; an
 * element that stands for 2^128 or more may count as infinite.
 * Any code and scale byte is accepted.  rows = 0 and count = 0 are no-ops;
 * 1 <= cols, all at most 2^30, rows x count at most 2^43.
 */
int dl_e4m3_matmul(const uint8_t *w, int64_t ldw, const uint8_t *w_scales, int64_t rows,
                   int64_t cols, const uint8_t *x, int64_t ldx, const uint8_t *x_scales,
                   int64_t count, void *y, int64_t ldy, int y_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DLHEAD_H */
