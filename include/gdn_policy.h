/*
 * gdn_policy.h - C ABI of libgdn_policy.so: the policy head that stands after a stack of
 * gated delta rule layers, on AMD Instinct MI355X (gfx950): layer norm and its gradient, an
 * 8-bit integer linear region, the log-probability of the chosen token with its gradient,
 * and a clipped policy loss with its gradient.
 *
 * These operators are not regions of the bitwise contract of gdn_cpr.h and take no identity.
 * What they keep of it: a row's norm, quantised values, products, log-probability and
 * logits gradient are computed from that row alone by a schedule that depends on the row's
 * width and on the types, so the same row gives the same bits in a batch of any size and at
 * any place in it (an engine's decode step and a trainer's packed batch agree bit for bit),
 * and every call gives the same bits on every launch: no floating-point atomics.
 *
 * OWNERSHIP, STREAMS, ERRORS are those of gdn_cpr.h: the caller allocates every buffer, the
 * library allocates no device memory and keeps no state between calls; work is enqueued on
 * the hipStream_t passed as `stream` (NULL = the null stream) of the current HIP device; all
 * argument checks run on the host before anything is enqueued, so a status other than GDN_OK
 * means that nothing was launched, except GDN_E_DEVICE. Every call can be captured into a
 * HIP graph. Values that the host cannot see (token ids, cu_seqlens) never lead to an access
 * out of bounds: an id outside the vocabulary marks a row that is not scored, and token
 * ranges are clamped. Outputs must not alias inputs unless a call says so. Pointers must be
 * aligned to their element; the int8 operands to 16 bytes. gdn_policy_last_error() returns
 * the text of the calling thread's last error. All functions are thread-safe.
 *
 * Row strides are in elements; rows are contiguous inside. An input's stride may be any
 * value in [0, 2^31] (0 repeats one row); outputs are dense.
 */
#ifndef GDN_POLICY_H
#define GDN_POLICY_H

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_POLICY_ABI_VERSION 1
#define GDN_I8_K_ALIGN 128 /* int8 operands hold rows padded with zeros to this many values */

typedef enum gdn_norm_kind { GDN_NORM_LAYER = 0, GDN_NORM_RMS = 1 } gdn_norm_kind_t;
typedef enum gdn_reduction { GDN_REDUCE_TOKEN = 0, GDN_REDUCE_SEQUENCE = 1 } gdn_reduction_t;

/* ABI version of the loaded library, GDN_POLICY_ABI_VERSION. Host only; cannot fail. */
int32_t gdn_policy_abi_version(void);

/* Text of the calling thread's last non-GDN_OK status of this library ("" if none). Valid
 * until the thread's next call into it. Host only; cannot fail. */
const char *gdn_policy_last_error(void);

/* Host struct of the norm calls. Admitted: 0 <= rows < 2^31; 1 <= width <= 16384; x_dtype
 * and w_dtype GDN_DTYPE_F32 or GDN_DTYPE_BF16, w_dtype that of weight and bias. */
typedef struct gdn_norm_shape {
  int64_t rows;
  int32_t width;
  int32_t kind; /* gdn_norm_kind_t */
  int32_t x_dtype, w_dtype;
} gdn_norm_shape_t;

/* Norm of each row x of `width` values, statistics in binary32:
 *   GDN_NORM_LAYER: mean = sum(x) / width, var = sum((x - mean)^2) / width
 *   GDN_NORM_RMS:   mean = 0,              var = sum(x^2) / width
 *   rstd = 1 / sqrt(var + eps),  y = (x - mean) * rstd * weight + bias
 *   x [rows, width] with row stride x_stride; weight [width]; bias [width] or NULL for 0
 *   eps               : finite, >= 0
 *   y [rows, width]   : x's dtype, each value rounded once; may be x itself when x_stride is
 *                       width
 *   mean float [rows] : GDN_NORM_LAYER only (NULL for GDN_NORM_RMS)
 *   rstd float [rows]
 * Errors: GDN_E_NULL, GDN_E_SHAPE (sizes, stride, eps, alignment), GDN_E_UNSUPPORTED (width,
 * kind or dtype not admitted), GDN_E_DEVICE. rows == 0 does nothing. */
gdn_status_t gdn_layer_norm_fwd(const gdn_norm_shape_t *shape, const void *x, int64_t x_stride,
                                const void *weight, const void *bias, double eps, void *y,
                                float *mean, float *rstd, void *stream);

/* Bytes of device workspace that gdn_layer_norm_bwd needs, into *bytes (host). Host only. */
gdn_status_t gdn_layer_norm_bwd_workspace(const gdn_norm_shape_t *shape, size_t *bytes);

/* Gradients through gdn_layer_norm_fwd given dy. With xh = (x - mean) * rstd and
 * g = dy * weight, per row:
 *   dx = rstd * (g - [layer: sum(g) / width] - xh * sum(g * xh) / width)
 * and over rows d_weight = sum(dy * xh), d_bias = sum(dy), binary32 in a fixed order.
 *   dy, x [rows, width], strides dy_stride, x_stride, x's dtype; mean (GDN_NORM_LAYER only)
 *   and rstd as the forward wrote them
 *   dx [rows, width]        : x's dtype; may be dy itself when dy_stride is width
 *   d_weight float [width]  : required; d_bias float [width] or NULL. With rows == 0 both
 *                             are set to 0.
 *   workspace               : device, 256-byte aligned, gdn_layer_norm_bwd_workspace() bytes;
 *                             its contents on entry do not matter
 * Errors as for gdn_layer_norm_fwd; GDN_E_SHAPE also for a short or misaligned workspace. */
gdn_status_t gdn_layer_norm_bwd(const gdn_norm_shape_t *shape, const void *dy,
                                int64_t dy_stride, const void *x, int64_t x_stride,
                                const void *weight, const float *mean, const float *rstd,
                                void *dx, float *d_weight, float *d_bias, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Quantises each row of x [rows, k] (row stride x_stride, x_dtype F32 or BF16) to 8 bits:
 *   a = max |x|,  scale = a / 127,  q = 127 x / a rounded to the nearest integer, ties to even
 * (the exact quotient is rounded). A row of zeros has scale 0 and q 0. A row with a NaN has
 * scale NaN and q 0; one with an infinity has scale infinity, q = +-127 at the infinities and
 * 0 elsewhere: what is multiplied out of either is not finite.
 *   q [rows, k_pad]   : int8, 16-byte aligned, k_pad = k rounded up to GDN_I8_K_ALIGN; the
 *                       padding is set to 0
 *   scale float [rows]
 * Serves a linear layer's inputs (one scale for each token) and its weights [n, k] (one scale
 * for each output channel) alike. Admitted: 0 <= rows < 2^31, 1 <= k <= 65536. */
gdn_status_t gdn_quantize_rows(const void *x, int64_t rows, int64_t k, int64_t x_stride,
                               int32_t x_dtype, int8_t *q, float *scale, void *stream);

/* Bytes of device workspace that gdn_linear_i8_fwd needs, into *bytes (host): 0 but for few
 * tiles of Y and a long k_pad, which is then split over several workgroups. Host only. */
gdn_status_t gdn_linear_i8_fwd_workspace(int64_t m, int64_t n, int64_t k_pad, size_t *bytes);

/* Y [m, n] = (xq wq^T) * x_scale[m] * w_scale[n]: the products of 8-bit integers are summed
 * exactly in 32-bit integers, converted to binary32, multiplied by x_scale, then by w_scale,
 * and rounded to y_dtype.
 *   xq int8 [m, k_pad], wq int8 [n, k_pad], 16-byte aligned, as gdn_quantize_rows writes them
 *   x_scale float [m], w_scale float [n]
 *   y [m, n]  : F32 or BF16
 *   workspace : device, 16-byte aligned, gdn_linear_i8_fwd_workspace() bytes (NULL where that
 *               is 0); its contents on entry do not matter
 * Admitted: 0 <= m, n < 2^31; k_pad a multiple of GDN_I8_K_ALIGN in [128, 65536] (the sum of
 * 65536 products of 8 bits fits 32 bits). m == 0 or n == 0 does nothing. GDN_E_SHAPE also where
 * the tiles of Y take more threads than one launch holds (2^32 - 1), which they never do for m * n
 * under 2^35, m and n rounded up to multiples of 64. */
gdn_status_t gdn_linear_i8_fwd(int64_t m, int64_t n, int64_t k_pad, const int8_t *xq,
                               const float *x_scale, const int8_t *wq, const float *w_scale,
                               int32_t y_dtype, void *y, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Host struct of the token log-probability calls. Admitted: 0 <= rows < 2^31;
 * 1 <= vocab < 2^31; logits_dtype F32 or BF16; id_bytes 4 or 8 (int32 or int64 ids);
 * 2^-40 <= scale <= 2^40. */
typedef struct gdn_logprob_shape {
  int64_t rows, vocab;
  int64_t logits_stride;
  int32_t logits_dtype;
  int32_t id_bytes;
  double scale; /* logits are multiplied by it: the inverse of the sampling temperature */
} gdn_logprob_shape_t;

/* Bytes of device workspace that gdn_token_logprob_fwd needs, into *bytes (host): 0 but for a
 * few rows of a long vocabulary, which are split over several workgroups. Host only. */
gdn_status_t gdn_token_logprob_fwd_workspace(const gdn_logprob_shape_t *shape, size_t *bytes);

/* For each row, with z = scale * logits, lse = log(sum(exp(z))), p = exp(z - lse):
 *   logp = z[id] - lse,  entropy = -sum(p * (z - lse)) = lse - sum(p * z)
 * in one pass over the logits (running maximum and sums in binary32).
 *   ids [rows]     : a row whose id is outside [0, vocab) is not scored: its logits are not
 *                    read and its outputs are 0
 *   logp, lse float [rows]; entropy float [rows] or NULL
 *   workspace      : device, 4-byte aligned, gdn_token_logprob_fwd_workspace() bytes (NULL
 *                    where that is 0); its contents on entry do not matter
 * A logit of -infinity has p = 0 and adds nothing to the entropy; a scored row of nothing but
 * -infinity has lse and logp -infinity and entropy 0; a row with NaN or +infinity gives NaN. An
 * lse past binary32's range is an infinity; logp and entropy come from differences and are not.
 * Errors: GDN_E_NULL, GDN_E_SHAPE (sizes, stride, scale, alignment), GDN_E_UNSUPPORTED
 * (dtype, id_bytes), GDN_E_DEVICE. rows == 0 does nothing. */
gdn_status_t gdn_token_logprob_fwd(const gdn_logprob_shape_t *shape, const void *logits,
                                   const void *ids, float *logp, float *lse, float *entropy,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of gdn_token_logprob_fwd's outputs with respect to the logits:
 *   d_logits[c] = scale * (d_logp * ([c == id] - p[c])
 *                          - d_entropy * p[c] * (log p[c] + entropy))
 * with log p = z - lse. Rows that are not scored get 0. Where p[c] is 0 the entropy's term
 * is 0; a row of nothing but -infinity gets 0.
 *   lse, d_logp float [rows]; entropy, d_entropy float [rows]: both or neither (NULL). lse and
 *                    entropy as the forward wrote them. From |lse| = 64 on, where its rounding
 *                    would be seen in p (and where it overflows), a row's log-sum-exp is formed
 *                    again from its logits, at the price of a second reading of them.
 *   d_logits [rows, vocab]: the logits' dtype; may be the logits themselves when their
 *                    stride is vocab.
 * Errors as for gdn_token_logprob_fwd; GDN_E_SHAPE also where rows * ceil(vocab / 2048) (4096 for
 * BF16) passes 2^31 - 1, which no gradient under 2^41 values does. */
gdn_status_t gdn_token_logprob_bwd(const gdn_logprob_shape_t *shape, const void *logits,
                                   const void *ids, const float *lse, const float *d_logp,
                                   const float *entropy, const float *d_entropy,
                                   void *d_logits, void *stream);

/* Host struct of the policy loss. Admitted: 0 <= tokens < 2^31; 0 <= seqs < 2^31;
 * 0 <= clip_low <= 1; clip_high >= 0; dual_clip 0 (off) or >= 1; coefficients finite. */
typedef struct gdn_policy_shape {
  int64_t tokens, seqs;
  int32_t reduction; /* gdn_reduction_t */
  int32_t reserved;  /* 0 */
  double clip_low, clip_high, dual_clip;
  double kl_coef, entropy_coef;
} gdn_policy_shape_t;

/* Bytes of device workspace that gdn_policy_loss_fwd needs, into *bytes (host). Host only. */
gdn_status_t gdn_policy_loss_workspace(const gdn_policy_shape_t *shape, size_t *bytes);

/* Clipped policy loss of a packed batch, per scored token, in binary64:
 *   r = exp(logp - old_logp),  gain = min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *   where A < 0 and dual_clip > 0: gain = max(gain, dual_clip A);  pg = -gain
 *   u = ref_logp - logp,  kl = exp(u) - u - 1 (next to u = 0 by its series)
 *   cut = 1 where gain is not r A (the token has no policy gradient), else 0
 * GDN_REDUCE_TOKEN: each scored token weighs 1 / (scored tokens); GDN_REDUCE_SEQUENCE: each
 * sequence with scored tokens weighs the same, and its scored tokens share its weight.
 *   stats float [5]     : loss = pg + kl_coef kl - entropy_coef entropy, and the weighted
 *                         means of pg, kl, entropy and cut (0 where there is nothing scored)
 *   seq_weight float [seqs]: the weight of one scored token of each sequence
 *   logp, old_logp, advantages float [tokens]; ref_logp, entropy float [tokens] or NULL (no
 *   KL term, no entropy term); mask: one byte for each token, 0 = not scored, or NULL for all
 *   scored: the other inputs of a token that is not scored may hold anything
 *   cu_seqlens int32 [seqs + 1] as in gdn_cpr.h, or NULL for one sequence (seqs 1)
 *   workspace           : device, 256-byte aligned, gdn_policy_loss_workspace() bytes */
gdn_status_t gdn_policy_loss_fwd(const gdn_policy_shape_t *shape, const float *logp,
                                 const float *old_logp, const float *advantages,
                                 const float *ref_logp, const float *entropy,
                                 const uint8_t *mask, const int32_t *cu_seqlens, float *stats,
                                 float *seq_weight, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* Gradient of d_loss * loss with respect to logp and entropy, given seq_weight w of the
 * forward call: per scored token
 *   d_logp = d_loss w (-[not cut] r A + kl_coef (1 - exp(u))),  d_entropy = -d_loss w entropy_coef
 * and 0 for the others. d_entropy may be NULL. Other arguments as for the forward. */
gdn_status_t gdn_policy_loss_bwd(const gdn_policy_shape_t *shape, const float *logp,
                                 const float *old_logp, const float *advantages,
                                 const float *ref_logp, const uint8_t *mask,
                                 const int32_t *cu_seqlens, const float *seq_weight,
                                 double d_loss, float *d_logp, float *d_entropy, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_POLICY_H */
