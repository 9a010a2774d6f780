// Declarations shared by the sources of libgdn_policy.so (host side).
#pragma once

#include "gdn_policy.h"
#include "internal.h"

namespace gdn {

// Arguments of the norm kernels; validated on the host.
struct NormArgs {
  int64_t rows;
  int32_t width, layer, x_bf16, w_bf16;
  int64_t x_stride, dy_stride;
  const void *x, *weight, *bias, *dy;
  float eps;
  void *y;  // forward: y; backward: dx
  float *mean, *rstd;
  // backward
  float *d_weight, *d_bias;
  float *partials;  // [blocks][2][width]: sums of dy * xh and of dy over a block's rows
  int32_t blocks;
  int32_t row_threads;  // set by the launcher: threads that share a row
};
int norm_bwd_blocks(int64_t rows, int32_t width);
hipError_t launch_norm_fwd(const NormArgs &args, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs &args, hipStream_t stream);

struct QuantizeArgs {
  int64_t rows, x_stride;
  int32_t k, k_pad, x_bf16;
  int32_t row_threads;  // set by the launcher: threads that share a row
  const void *x;
  int8_t *q;
  float *scale;
};
hipError_t launch_quantize(const QuantizeArgs &args, hipStream_t stream);

struct LinearI8Args {
  int64_t m, n;
  int32_t k, y_bf16;
  const int8_t *xq, *wq;
  const float *x_scale, *w_scale;
  void *y;
  float *parts;  // sums of parts of K, [splits][m][n] as bits; NULL: a workgroup takes all of K
  int32_t splits, k_part;  // set by the launcher; k_part a multiple of 128
};
int64_t linear_i8_parts_bytes(const LinearI8Args &args);  // 0: no parts
int64_t linear_i8_threads(const LinearI8Args &args);  // of the launch; at most 2^32 - 1 fit one
hipError_t launch_linear_i8(const LinearI8Args &args, hipStream_t stream);

struct LogprobArgs {
  int64_t rows, vocab, stride;
  int32_t bf16, id64;
  float scale, scale_log2e;
  const void *logits, *ids;
  // forward outputs, backward inputs
  float *logp, *lse, *entropy;
  const float *d_logp, *d_entropy;
  void *d_logits;
  float *parts;   // forward of few long rows: the threads' sums, [rows][groups][3][threads]
  int64_t groups;  // of a row; set by the launcher
};
int64_t logprob_parts_bytes(const LogprobArgs &args);  // 0: a row is one workgroup's
hipError_t launch_logprob_fwd(const LogprobArgs &args, hipStream_t stream);
int64_t logprob_bwd_grid(const LogprobArgs &args);
hipError_t launch_logprob_bwd(const LogprobArgs &args, hipStream_t stream);

struct PolicyArgs {
  int64_t tokens, seqs;
  int32_t by_sequence;
  double lo, hi, dual, kl_coef, entropy_coef, d_loss;
  const float *logp, *old_logp, *adv, *ref, *entropy;
  const uint8_t *mask;
  const int32_t *cu;
  float *stats, *seq_weight;
  const float *weight;  // backward
  float *d_logp, *d_entropy;
  double *partials;  // [slots][5]
  double *seq_sums;  // [seqs][5]
  int64_t slots, span;
};
// Tokens of one wave of the forward, and slots of per-(span, sequence) sums: spans meet the
// sequences in order, so span + sequence numbers the pairs that meet without a repeat.
int64_t policy_span(int64_t tokens);
int64_t policy_slots(int64_t tokens, int64_t seqs);
hipError_t launch_policy_fwd(const PolicyArgs &args, hipStream_t stream);
hipError_t launch_policy_bwd(const PolicyArgs &args, hipStream_t stream);

}  // namespace gdn
