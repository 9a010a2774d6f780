// Declarations shared by the sources of libgdn_step.so (host side).
#pragma once

#include "gdn_step.h"
#include "internal.h"

namespace gdn {

// Arguments of the block quantisation; validated on the host.
struct QuantizeF8Args {
  int64_t rows, k, x_stride;
  int32_t x_bf16, e5m2;
  const void *x;
  uint8_t *q, *scale, *qt, *scale_t;
};
int64_t quantize_f8_threads(const QuantizeF8Args &args);  // of the launch; at most 2^32 - 1 fit one
hipError_t launch_quantize_f8(const QuantizeF8Args &args, hipStream_t stream);

struct LinearF8Args {
  int64_t m, n;
  int32_t k, y_bf16, e5m2;
  const uint8_t *xq, *x_scale, *wq, *w_scale;
  void *y;
};
int64_t linear_f8_threads(const LinearF8Args &args);  // of the launch; at most 2^32 - 1 fit one
hipError_t launch_linear_f8(const LinearF8Args &args, hipStream_t stream);
// Two products that have nothing to do with each other, in one launch where that pays.
hipError_t launch_linear_f8(const LinearF8Args &a, const LinearF8Args &b, hipStream_t stream);

// Rows of the scales' layout, and bytes of a matrix's scales.
inline int64_t f8_pad(int64_t c) { return (c + GDN_F8_BLOCK - 1) / GDN_F8_BLOCK * GDN_F8_BLOCK; }
inline int64_t f8_scale_rows(int64_t r) { return (r + 3) / 4 * 4; }
inline int64_t f8_scale_bytes(int64_t r, int64_t c) {
  return (c + 4 * GDN_F8_BLOCK - 1) / (4 * GDN_F8_BLOCK) * f8_scale_rows(r) * 4;
}

struct SampleArgs {
  int64_t rows, vocab, stride;
  int64_t first;  // row of the launch, set by the launcher
  int32_t bf16, u64, id64, top_k, shift;  // a weight of 1 is 2^shift
  double temperature, top_p, min_p;
  const void *logits, *u;
  const float *temperatures, *top_ps, *min_ps;
  const int32_t *top_ks;
  void *ids;
  float *logp;
  void *workspace;
};
int64_t sample_workspace_bytes(const SampleArgs &args);
hipError_t launch_sample(const SampleArgs &args, hipStream_t stream);

struct AdamwArgs {
  int32_t param_bf16, grad_bf16, eight;
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const float *factor, *lr_at;
  const int64_t *step_at;
};
hipError_t launch_adamw(const AdamwArgs &args, const gdn_adamw_tensor_t *tensors, int64_t count,
                        hipStream_t stream);
hipError_t launch_adamw_values(const uint8_t *codes, const float *scale, int64_t numel, bool v,
                               float *out, hipStream_t stream);
int64_t grad_norm_workspace_bytes(const gdn_grad_tensor_t *tensors, int64_t count);
hipError_t launch_grad_norm(const gdn_grad_tensor_t *tensors, int64_t count, bool bf16,
                            double max_norm, float *norm, float *factor, void *workspace,
                            hipStream_t stream);

}  // namespace gdn
