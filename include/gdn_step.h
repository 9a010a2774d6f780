/*
 * gdn_step.h - C ABI of libgdn_step.so: what closes an on-policy step around the policy head of
 * gdn_policy.h, on AMD Instinct MI355X (gfx950): tokens drawn from logits (the rollout's end),
 * a linear region in 8-bit floating point with a scale for each block of 128 values, forward
 * and backward, and AdamW over many tensors behind a clipped gradient norm (the trainer's end).
 *
 * As in gdn_policy.h, these operators are not regions of the bitwise contract of gdn_cpr.h and
 * take no identity, and a row's drawn token, quantised values and products are computed from
 * that row alone, with sums whose order depends on the row's width (the product's) or whose
 * terms are integers (the draw's): the same row gives the same bits in a batch of any size and
 * at any place in it. Every call gives the same bits on every launch: no floating-point
 * atomics.
 *
 * OWNERSHIP, STREAMS, ERRORS are those of gdn_policy.h: the caller allocates every buffer, the
 * library allocates no device memory and keeps no state between calls; work is enqueued on
 * the hipStream_t passed as `stream` (NULL = the null stream) of the current HIP device; all
 * argument checks run on the host before anything is enqueued, so a status other than GDN_OK
 * means that nothing was launched, except GDN_E_DEVICE. Every call can be captured into a HIP
 * graph; a workspace belongs to one call at a time, a captured one included. Values that the
 * host cannot see (parameters of a row, random numbers) never lead to an access out of bounds.
 * Outputs must not alias inputs unless a call says so. Pointers must be aligned to their
 * element, the product's operands and scales to 16 bytes. gdn_step_last_error() returns the text
 * of the calling thread's last error. All functions are thread-safe.
 *
 * Row strides are in elements; rows are contiguous inside. An input's stride may be any
 * value in [0, 2^31] (0 repeats one row); outputs are dense.
 */
#ifndef GDN_STEP_H
#define GDN_STEP_H

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_STEP_ABI_VERSION 1
#define GDN_F8_BLOCK 128     /* consecutive values that share a scale */
#define GDN_ADAMW_BLOCK 256  /* values of a tensor whose 8-bit states share a scale */

typedef enum gdn_f8_format { GDN_F8_E4M3 = 0, GDN_F8_E5M2 = 1 } gdn_f8_format_t;
typedef enum gdn_state_format { GDN_STATE_F32 = 0, GDN_STATE_8BIT = 1 } gdn_state_format_t;
typedef enum gdn_moment { GDN_MOMENT_M = 0, GDN_MOMENT_V = 1 } gdn_moment_t;

/* ABI version of the loaded library, GDN_STEP_ABI_VERSION. Host only; cannot fail. */
int32_t gdn_step_abi_version(void);

/* Text of the calling thread's last non-GDN_OK status of this library ("" if none). Valid
 * until the thread's next call into it. Host only; cannot fail. */
const char *gdn_step_last_error(void);

/* ---------------------------------------------------------------- 8-bit floating point
 *
 * A matrix [r, c] in 8 bits is q [r, c_pad], c_pad = c rounded up to GDN_F8_BLOCK, the padding
 * 0, and one scale for each block of 128 consecutive values of a row, a power of two held as
 * its exponent + 127 in a byte (torch's float8_e8m0fnu). The scales lie as the product reads
 * them, four blocks of a row side by side:
 *   scale [ceil(c_pad / 512)][r rounded up to 4][4]: that of row i, block b at [b / 4][i][b % 4]
 * Bytes of rows past the last and blocks past the last hold 127 (a scale of 1). 255, which no
 * block gets, stands for no scale: products with one are unspecified.
 *
 * With a = max |x| of a block, its scale is 2^e for the least whole e >= -127 with
 * a <= 1.75 * 2^emax * 2^e, the format's largest value (448 for E4M3, 57344 for E5M2); a block
 * of zeros has e = 0. q = x / 2^e, which is exact, rounded to the format, ties to even. NaN
 * becomes the format's NaN; an infinity NaN in E4M3, which has none, and infinity in E5M2; the
 * scale of their block comes from its finite values. */

/* Quantises x [rows, k] (row stride x_stride, x_dtype F32 or BF16) by rows, into q [rows,
 * k_pad] with its scale, and by columns, its transpose into qt [k, rows_pad] with its scale_t;
 * either pair may be NULL, and both are made from one reading of x.
 * Admitted: 0 <= rows <= 2^31 - 1 and 1 <= k <= 2^20; with qt also rows <= 2^20 and fewer than
 * 2^24 tiles of 128 x 128 values, which is what one launch holds.
 * Errors: GDN_E_NULL, GDN_E_SHAPE (sizes, stride, alignment), GDN_E_UNSUPPORTED (k, format,
 * dtype), GDN_E_DEVICE. rows == 0 does nothing. */
gdn_status_t gdn_quantize_f8(const void *x, int64_t rows, int64_t k, int64_t x_stride,
                             int32_t x_dtype, int32_t format, uint8_t *q, uint8_t *scale,
                             uint8_t *qt, uint8_t *scale_t, void *stream);

/* Y [m, n] = the sum over k of x[m, k] w[n, k], of the values that xq and wq stand for:
 * added up in binary32 by one chain of matrix instructions over ascending k, the same for every
 * m and n, and rounded to y_dtype once. To F32 the values are taken in bf16, which holds them all
 * but those below 2^-126 (rounded to multiples of 2^-133), products are exact and 16 k are added at
 * a time. To BF16 64 k are, and of eight neighbouring k each product is cut off 13 bits below the
 * power of two of the largest: 1.5e-5 in the 2-norm for random operands, where rounding Y is 1.7e-3.
 * At most that is 2^-10 of the largest product of each eight k, added up over them: where the
 * products of a row cancel it may exceed the rounding of Y, and Y to F32 is the remedy.
 *   xq [m, k_pad] in x_format with x_scale; wq [n, k_pad] in E4M3 with w_scale
 *   y [m, n]  : F32 or BF16
 * Admitted: 0 <= m, n < 2^31; k_pad a multiple of GDN_F8_BLOCK in [0, 2^20]. m == 0 or n == 0
 * does nothing; k_pad == 0 gives zeros (xq, wq and scales may be NULL). GDN_E_SHAPE also where
 * the tiles of Y take more threads than one launch holds (2^32 - 1), which they never do for
 * m * n under 2^35, m and n rounded up to multiples of 64. */
gdn_status_t gdn_linear_f8_fwd(int64_t m, int64_t n, int64_t k_pad, int32_t x_format,
                               const uint8_t *xq, const uint8_t *x_scale, const uint8_t *wq,
                               const uint8_t *w_scale, int32_t y_dtype, void *y, void *stream);

/* Host struct of the product's backward. Admitted: 0 <= m <= 2^20; 1 <= n, k <= 2^20. */
typedef struct gdn_linear_f8_shape {
  int64_t m, n, k;
  int64_t dy_stride;
  int32_t dy_dtype;  /* F32 or BF16 */
  int32_t dy_format; /* gdn_f8_format_t that dy is held in */
  int32_t dx_dtype, dw_dtype; /* F32 or BF16 */
} gdn_linear_f8_shape_t;

/* Bytes of device workspace that gdn_linear_f8_bwd needs, into *bytes (host). Host only. */
gdn_status_t gdn_linear_f8_bwd_workspace(const gdn_linear_f8_shape_t *shape, size_t *bytes);

/* Gradients of Y = X W^T given dy [m, n]: dy is quantised by rows and by columns, and
 *   dx [m, k] = dy w      over n, from wtq [k, n_pad]: W [n, k] quantised by columns
 *   dw [n, k] = dy^T x    over m, from xtq [k, m_pad]: X [m, k] quantised by columns
 * (both in E4M3, with their scales). The gradient passes straight through the rounding of X
 * and W. dx with wtq and wt_scale, or dw with xtq and xt_scale, may be NULL, not both.
 *   workspace : device, 256-byte aligned, gdn_linear_f8_bwd_workspace() bytes (dy quantised both
 *               ways, also where one gradient is wanted); its contents on entry do not matter
 * m == 0 gives dw = 0. Errors as for the forward; GDN_E_SHAPE also where dw is wanted of a dy of
 * 2^24 tiles of 128 x 128 values and more. */
gdn_status_t gdn_linear_f8_bwd(const gdn_linear_f8_shape_t *shape, const void *dy,
                               const uint8_t *wtq, const uint8_t *wt_scale, const uint8_t *xtq,
                               const uint8_t *xt_scale, void *dx, void *dw, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------------ sampling */

/* Host struct of the draw. Admitted: 0 <= rows < 2^31; 1 <= vocab < 2^31; logits_dtype F32 or
 * BF16; u_bytes and id_bytes 4 or 8; temperature 0 or in [2^-40, 2^40]; top_k >= 0; top_p and
 * min_p finite and >= 0. The four parameters hold for every row that has no value of its own. */
typedef struct gdn_sample_shape {
  int64_t rows, vocab;
  int64_t logits_stride;
  int32_t logits_dtype;
  int32_t u_bytes;  /* random numbers in binary32 or binary64 */
  int32_t id_bytes; /* int32 or int64 ids */
  int32_t top_k;    /* 0: off */
  double temperature, top_p, min_p;
} gdn_sample_shape_t;

/* Bytes of device workspace that gdn_sample_tokens needs, into *bytes (host): 0 for a vocabulary
 * of up to 4096, else a few for each row, and more for few rows of a long vocabulary, which are
 * split over several workgroups. Host only. */
gdn_status_t gdn_sample_tokens_workspace(const gdn_sample_shape_t *shape, size_t *bytes);

/* Draws one token of each row. With M the row's largest logit, token i weighs
 *   w_i = exp((logits_i - M) / temperature), rounded to a multiple of 2^-s,
 *   s = min(45, 62 - ceil(log2(vocab)))
 * so that sums of weights are exact. The tokens in order of falling logits, equal ones by
 * rising id, are cut off behind the first of these:
 *   top_k : the first top_k tokens (0, or vocab and more: no cut)
 *   top_p : the shortest run of them that holds top_p of their weight, at least one token
 *           (1 and more: no cut)
 *   min_p : the tokens of weight min_p and more (the largest weighs 1; above 1 counts as 1)
 * and the draw is the smallest id at which the weights of the tokens left, added up by rising
 * id, exceed u times their sum (rounded down). Temperature 0 gives the largest logit's
 * smallest id whatever the others say.
 *   u [rows]          : in [0, 1); values outside are moved to its ends, NaN is 0
 *   temperature, top_p, min_p float [rows], top_k int32 [rows]: or NULL for the shape's
 *   ids [rows]        : the token; -1 for a row without one: no logit above -infinity, a
 *                       logit of NaN or +infinity, a temperature of its own below 0, NaN or
 *                       infinite. A top_k of its own below 0, or a NaN in top_p or min_p, is off
 *   logp float [rows] : its log-probability among the tokens left, at the temperature;
 *                       0 where ids is -1, or where the temperature is 0
 *   workspace         : device, 256-byte aligned, gdn_sample_tokens_workspace() bytes (NULL
 *                       where that is 0); its contents on entry do not matter
 * Errors: GDN_E_NULL, GDN_E_SHAPE (sizes, stride, parameters, alignment), GDN_E_UNSUPPORTED
 * (dtype, u_bytes, id_bytes), GDN_E_DEVICE. rows == 0 does nothing. */
gdn_status_t gdn_sample_tokens(const gdn_sample_shape_t *shape, const void *logits,
                               const void *u, const float *temperature, const int32_t *top_k,
                               const float *top_p, const float *min_p, void *ids, float *logp,
                               void *workspace, size_t workspace_bytes, void *stream);

/* ----------------------------------------------------------------------------- optimiser */

/* One gradient of a list (host array; the pointers are device pointers). */
typedef struct gdn_grad_tensor {
  int64_t numel; /* >= 0 */
  const void *grad;
} gdn_grad_tensor_t;

/* Bytes of device workspace that gdn_grad_norm needs, into *bytes (host). Host only. */
gdn_status_t gdn_grad_norm_workspace(const gdn_grad_tensor_t *tensors, int64_t count,
                                     size_t *bytes);

/* The 2-norm of all values of `count` gradients together, summed in binary64 in a fixed order,
 * and the factor that clips it:
 *   norm float [1]   : sqrt(sum of squares)
 *   factor float [1] : min(1, max_norm / (norm + 1e-6)) of the unrounded norm; NaN where the
 *                      norm is not finite (gdn_adamw_step then does nothing). NULL: not wanted
 *   grad_dtype F32 or BF16; max_norm >= 0, infinity for a factor of 1
 *   workspace : device, 256-byte aligned, gdn_grad_norm_workspace() bytes; its contents on
 *               entry do not matter
 * Admitted: 0 <= count <= 2^20, each numel < 2^40. An empty list has norm 0. One call takes
 * gradients of one type; a norm over both types has to have them in one first. */
gdn_status_t gdn_grad_norm(const gdn_grad_tensor_t *tensors, int64_t count, int32_t grad_dtype,
                           double max_norm, float *norm, float *factor, void *workspace,
                           size_t workspace_bytes, void *stream);

/* One parameter of a list (host array; the pointers are device pointers). */
typedef struct gdn_adamw_tensor {
  int64_t numel;     /* >= 0 */
  void *param;       /* [numel] */
  const void *grad;  /* [numel] */
  void *m, *v;       /* [numel] binary32, or one byte a value */
  float *m_scale, *v_scale; /* [ceil(numel / 256)] with 8-bit states, else NULL */
  float *master;     /* [numel] binary32 weights behind a BF16 param, or NULL */
} gdn_adamw_tensor_t;

/* Host struct of the update. Admitted: 0 <= beta1, beta2 < 1; eps >= 0, weight_decay and lr
 * finite; step >= 1 (the first step is 1). */
typedef struct gdn_adamw_shape {
  int32_t param_dtype, grad_dtype; /* F32 or BF16 */
  int32_t state;                   /* gdn_state_format_t */
  int32_t reserved;                /* 0 */
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
} gdn_adamw_shape_t;

/* One AdamW update of `count` tensors in place. Per value, every operation rounded to binary32
 * by itself, in this order:
 *   g = grad * factor                                  (factor: see gdn_grad_norm)
 *   m = m * beta1 + g * (1 - beta1),  v = v * beta2 + (g * g) * (1 - beta2),  r = sqrt(v)
 *   p = p * (1 - lr weight_decay)
 *       - m / (r * (1 / sqrt(1 - beta2^step)) + eps) * (lr / (1 - beta1^step))
 * the bracketed constants formed in binary64 and rounded once. p is the master where there is
 * one, which param then follows rounded to BF16; else param itself.
 *
 * GDN_STATE_8BIT: a block of 256 values of a tensor (its last one may be shorter) holds m in E4M3
 * with m_scale = max |m| * (1 / 448), and r, the root of v, in an unsigned float of 4 exponent and
 * 4 fraction bits with v_scale = max r * (1 / 248): code c > 0 stands for the binary32 of the bits
 * (c << 19) + (119 << 23), code 0 for 0, times the scale. Values are multiplied by (1 / max) * 448
 * or (1 / max) * 248 (each operation rounded to binary32) and rounded to the format, ties to even;
 * an r above 0 never gets code 0, so that no step divides by eps alone. A block whose largest
 * value is under 2^-100 holds zeros. The update uses m and r of this step before they are rounded.
 *
 *   factor float [1] (device)     : NULL for 1. One that is NaN or infinite leaves everything as
 *                                   it is: a step with gradients that are not finite is skipped
 *   step_at int64 [1], lr_at float [1] (device): the step and the rate where they have to
 *                                   change between replays of a captured call; NULL for the
 *                                   shape's. A step below 1 counts as 1
 * A NaN or an infinity in a block's gradients without such a factor spreads to the values of its
 * block in 8-bit states. Admitted: 0 <= count <= 2^20, each numel < 2^40; no two buffers of the
 * list may overlap (a param that stands in it twice would be updated by two workgroups at once;
 * equal pointers of one tensor are refused), but grad may be NULL where numel is 0. master needs
 * param_dtype BF16.
 * Errors: GDN_E_NULL, GDN_E_SHAPE (sizes, values, alignment, one buffer for two), GDN_E_UNSUPPORTED
 * (dtype, state),
 * GDN_E_DEVICE. */
gdn_status_t gdn_adamw_step(const gdn_adamw_shape_t *shape, const gdn_adamw_tensor_t *tensors,
                            int64_t count, const float *factor, const int64_t *step_at,
                            const float *lr_at, void *stream);

/* The values that 8-bit states stand for: out float [numel] = m, or v = r * r, of `codes`
 * [numel] with `scale` [ceil(numel / 256)] (for a checkpoint in binary32, or to look at).
 * Admitted: 0 <= numel < 2^40. */
gdn_status_t gdn_adamw_state_values(const uint8_t *codes, const float *scale, int64_t numel,
                                    int32_t moment, float *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_STEP_H */
