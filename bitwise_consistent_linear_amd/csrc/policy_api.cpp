// C ABI entry points of libgdn_policy.so: host-side claims and dispatch to the HIP kernels.
// Every claim is checked before anything is enqueued, so a refused call leaves all buffers
// untouched.

#include <cmath>
#include <cstdio>

#include "policy_internal.h"

namespace gdn {
namespace {

// A buffer of fixed size: an error's text allocates nothing, so no entry point can throw.
thread_local char g_last_error[256];

constexpr int64_t kMaxInt32 = 2147483647;
// Strides are bounded so that rows * stride elements stay within 64-bit byte offsets.
constexpr int64_t kMaxStride = int64_t(1) << 31;

bool aligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool known_dtype(int32_t d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }
size_t bytes_of(int32_t d) { return d == GDN_DTYPE_BF16 ? 2 : 4; }

gdn_status_t no(gdn_status_t st, const char *fn, const char *what) {
  std::snprintf(g_last_error, sizeof g_last_error, "%s: %s", fn, what);
  return st;
}

gdn_status_t launched(const char *fn, hipError_t e) {
  if (e == hipSuccess) return ok();
  std::snprintf(g_last_error, sizeof g_last_error, "%s: launch failed: %s", fn,
                hipGetErrorString(e));
  return GDN_E_DEVICE;
}

bool any_misaligned(std::initializer_list<const void *> list, size_t bytes) {
  for (const void *p : list)
    if (!aligned(p, bytes)) return true;
  return false;
}

constexpr int32_t kMaxNormWidth = 16384;

gdn_status_t norm_shape(const char *fn, const gdn_norm_shape_t *sh) {
  if (!sh) return no(GDN_E_NULL, fn, "shape is NULL");
  if (sh->rows < 0 || sh->rows > kMaxInt32) return no(GDN_E_SHAPE, fn, "rows must be in [0, 2^31)");
  if (sh->width < 1 || sh->width > kMaxNormWidth)
    return no(GDN_E_UNSUPPORTED, fn, "width must be in [1, 16384]");
  if (sh->kind != GDN_NORM_LAYER && sh->kind != GDN_NORM_RMS)
    return no(GDN_E_UNSUPPORTED, fn, "kind must be GDN_NORM_LAYER or GDN_NORM_RMS");
  if (!known_dtype(sh->x_dtype) || !known_dtype(sh->w_dtype))
    return no(GDN_E_UNSUPPORTED, fn, "x_dtype and w_dtype must be F32 or BF16");
  return GDN_OK;
}

bool bad_stride(int64_t s) { return s < 0 || s > kMaxStride; }

NormArgs norm_args(const gdn_norm_shape_t *sh) {
  NormArgs a{};
  a.rows = sh->rows;
  a.width = sh->width;
  a.layer = sh->kind == GDN_NORM_LAYER;
  a.x_bf16 = sh->x_dtype == GDN_DTYPE_BF16;
  a.w_bf16 = sh->w_dtype == GDN_DTYPE_BF16;
  return a;
}

size_t norm_workspace(const gdn_norm_shape_t *sh) {
  const size_t need = (size_t)norm_bwd_blocks(sh->rows, sh->width) * 2 * sh->width * sizeof(float);
  return (need + 255) / 256 * 256;
}

gdn_status_t linear_i8_shape(const char *fn, int64_t m, int64_t n, int64_t k_pad,
                             LinearI8Args &a) {
  if (m < 0 || m > kMaxInt32 || n < 0 || n > kMaxInt32)
    return no(GDN_E_SHAPE, fn, "m and n must be in [0, 2^31)");
  if (k_pad < GDN_I8_K_ALIGN || k_pad > 65536 || k_pad % GDN_I8_K_ALIGN != 0)
    return no(GDN_E_UNSUPPORTED, fn, "k_pad must be a multiple of 128 in [128, 65536]");
  a = LinearI8Args{};
  a.m = m;
  a.n = n;
  a.k = (int32_t)k_pad;
  return GDN_OK;
}

gdn_status_t logprob_shape(const char *fn, const gdn_logprob_shape_t *sh, LogprobArgs &a) {
  if (!sh) return no(GDN_E_NULL, fn, "shape is NULL");
  if (sh->rows < 0 || sh->rows > kMaxInt32) return no(GDN_E_SHAPE, fn, "rows must be in [0, 2^31)");
  if (sh->vocab < 1 || sh->vocab > kMaxInt32)
    return no(GDN_E_SHAPE, fn, "vocab must be in [1, 2^31)");
  if (bad_stride(sh->logits_stride)) return no(GDN_E_SHAPE, fn, "logits_stride must be in [0, 2^31]");
  if (!known_dtype(sh->logits_dtype))
    return no(GDN_E_UNSUPPORTED, fn, "logits_dtype must be F32 or BF16");
  if (sh->id_bytes != 4 && sh->id_bytes != 8)
    return no(GDN_E_UNSUPPORTED, fn, "id_bytes must be 4 or 8");
  if (!(sh->scale >= 0x1p-40 && sh->scale <= 0x1p+40))
    return no(GDN_E_SHAPE, fn, "scale must be in [2^-40, 2^40]");
  a = LogprobArgs{};
  a.rows = sh->rows;
  a.vocab = sh->vocab;
  a.stride = sh->logits_stride;
  a.bf16 = sh->logits_dtype == GDN_DTYPE_BF16;
  a.id64 = sh->id_bytes == 8;
  a.scale = (float)sh->scale;
  a.scale_log2e = (float)((double)a.scale * 1.4426950408889634074);
  return GDN_OK;
}

gdn_status_t policy_shape(const char *fn, const gdn_policy_shape_t *sh, PolicyArgs &a) {
  if (!sh) return no(GDN_E_NULL, fn, "shape is NULL");
  if (sh->tokens < 0 || sh->tokens > kMaxInt32)
    return no(GDN_E_SHAPE, fn, "tokens must be in [0, 2^31)");
  if (sh->seqs < 0 || sh->seqs > kMaxInt32) return no(GDN_E_SHAPE, fn, "seqs must be in [0, 2^31)");
  if (sh->reduction != GDN_REDUCE_TOKEN && sh->reduction != GDN_REDUCE_SEQUENCE)
    return no(GDN_E_UNSUPPORTED, fn, "reduction must be GDN_REDUCE_TOKEN or GDN_REDUCE_SEQUENCE");
  if (!(sh->clip_low >= 0.0 && sh->clip_low <= 1.0))
    return no(GDN_E_SHAPE, fn, "clip_low must be in [0, 1]");
  if (!(sh->clip_high >= 0.0) || !std::isfinite(sh->clip_high))
    return no(GDN_E_SHAPE, fn, "clip_high must be finite and >= 0");
  if (!(sh->dual_clip == 0.0 || sh->dual_clip >= 1.0) || !std::isfinite(sh->dual_clip))
    return no(GDN_E_SHAPE, fn, "dual_clip must be 0 or >= 1");
  if (!std::isfinite(sh->kl_coef) || !std::isfinite(sh->entropy_coef))
    return no(GDN_E_SHAPE, fn, "coefficients must be finite");
  a = PolicyArgs{};
  a.tokens = sh->tokens;
  a.seqs = sh->seqs;
  a.by_sequence = sh->reduction == GDN_REDUCE_SEQUENCE;
  a.lo = 1.0 - sh->clip_low;
  a.hi = 1.0 + sh->clip_high;
  a.dual = sh->dual_clip;
  a.kl_coef = sh->kl_coef;
  a.entropy_coef = sh->entropy_coef;
  a.span = policy_span(sh->tokens);
  a.slots = policy_slots(sh->tokens, sh->seqs);
  return GDN_OK;
}

size_t policy_partial_bytes(const PolicyArgs &a) {
  return (size_t)(5 * a.slots * 8 + 255) / 256 * 256;
}
size_t policy_workspace(const PolicyArgs &a) {
  return policy_partial_bytes(a) + (size_t)(5 * a.seqs * 8 + 255) / 256 * 256 + 256;
}

gdn_status_t policy_inputs(const char *fn, const gdn_policy_shape_t *sh, const float *logp,
                           const float *old_logp, const float *adv, const float *ref,
                           const int32_t *cu, PolicyArgs &a, const uint8_t *mask) {
  if (sh->tokens > 0 && (!logp || !old_logp || !adv))
    return no(GDN_E_NULL, fn, "logp, old_logp and advantages are required");
  if (!cu && sh->seqs != 1)
    return no(GDN_E_NULL, fn, "cu_seqlens is required unless there is one sequence");
  if (any_misaligned({logp, old_logp, adv, ref, cu}, 4))
    return no(GDN_E_SHAPE, fn, "inputs must be 4-byte aligned");
  a.logp = logp;
  a.old_logp = old_logp;
  a.adv = adv;
  a.ref = ref;
  a.mask = mask;
  a.cu = cu;
  return GDN_OK;
}

}  // namespace

gdn_status_t ok() {
  g_last_error[0] = 0;
  return GDN_OK;
}

}  // namespace gdn

extern "C" {

GDN_EXPORT int32_t gdn_policy_abi_version(void) { return GDN_POLICY_ABI_VERSION; }

GDN_EXPORT const char *gdn_policy_last_error(void) { return gdn::g_last_error; }

GDN_EXPORT gdn_status_t gdn_layer_norm_fwd(const gdn_norm_shape_t *shape, const void *x,
                                           int64_t x_stride, const void *weight, const void *bias,
                                           double eps, void *y, float *mean, float *rstd,
                                           void *stream) {
  const char *fn = "gdn_layer_norm_fwd";
  gdn_status_t st = gdn::norm_shape(fn, shape);
  if (st != GDN_OK) return st;
  if (gdn::bad_stride(x_stride)) return gdn::no(GDN_E_SHAPE, fn, "x_stride must be in [0, 2^31]");
  if (!(eps >= 0.0) || !std::isfinite((float)eps))
    return gdn::no(GDN_E_SHAPE, fn, "eps must be finite and >= 0");
  if (shape->rows == 0) return gdn::ok();
  const bool layer = shape->kind == GDN_NORM_LAYER;
  if (!x || !weight || !y || !rstd || (layer && !mean))
    return gdn::no(GDN_E_NULL, fn, "x, weight, y, rstd and (layer norm) mean are required");
  if (gdn::any_misaligned({x, y}, gdn::bytes_of(shape->x_dtype)) ||
      gdn::any_misaligned({weight, bias}, gdn::bytes_of(shape->w_dtype)) ||
      gdn::any_misaligned({mean, rstd}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  if (y == x && x_stride != shape->width)
    return gdn::no(GDN_E_SHAPE, fn, "y can be x only where x_stride is width");
  gdn::NormArgs a = gdn::norm_args(shape);
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.eps = (float)eps;
  a.y = y;
  a.mean = layer ? mean : nullptr;
  a.rstd = rstd;
  return gdn::launched(fn, gdn::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_layer_norm_bwd_workspace(const gdn_norm_shape_t *shape,
                                                     size_t *bytes) {
  const char *fn = "gdn_layer_norm_bwd_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn_status_t st = gdn::norm_shape(fn, shape);
  if (st != GDN_OK) return st;
  *bytes = gdn::norm_workspace(shape);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_layer_norm_bwd(const gdn_norm_shape_t *shape, const void *dy,
                                           int64_t dy_stride, const void *x, int64_t x_stride,
                                           const void *weight, const float *mean,
                                           const float *rstd, void *dx, float *d_weight,
                                           float *d_bias, void *workspace, size_t workspace_bytes,
                                           void *stream) {
  const char *fn = "gdn_layer_norm_bwd";
  gdn_status_t st = gdn::norm_shape(fn, shape);
  if (st != GDN_OK) return st;
  if (gdn::bad_stride(x_stride) || gdn::bad_stride(dy_stride))
    return gdn::no(GDN_E_SHAPE, fn, "x_stride and dy_stride must be in [0, 2^31]");
  const bool layer = shape->kind == GDN_NORM_LAYER;
  if (!weight || !d_weight || !workspace)
    return gdn::no(GDN_E_NULL, fn, "weight, d_weight and workspace are required");
  if (shape->rows > 0 && (!dy || !x || !dx || !rstd || (layer && !mean)))
    return gdn::no(GDN_E_NULL, fn, "dy, x, dx, rstd and (layer norm) mean are required");
  if (gdn::any_misaligned({x, dy, dx}, gdn::bytes_of(shape->x_dtype)) ||
      gdn::any_misaligned({weight}, gdn::bytes_of(shape->w_dtype)) ||
      gdn::any_misaligned({mean, rstd, d_weight, d_bias}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  if (!gdn::aligned(workspace, 256))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < gdn::norm_workspace(shape))
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_layer_norm_bwd_workspace reports");
  if (shape->rows > 0 && ((dx == dy && dy_stride != shape->width) || dx == x))
    return gdn::no(GDN_E_SHAPE, fn, "dx can be dy only where dy_stride is width, and never x");
  gdn::NormArgs a = gdn::norm_args(shape);
  a.x = x;
  a.x_stride = x_stride;
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.weight = weight;
  a.mean = const_cast<float *>(layer ? mean : nullptr);
  a.rstd = const_cast<float *>(rstd);
  a.y = dx;
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.partials = static_cast<float *>(workspace);
  a.blocks = gdn::norm_bwd_blocks(shape->rows, shape->width);
  return gdn::launched(fn, gdn::launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_quantize_rows(const void *x, int64_t rows, int64_t k,
                                          int64_t x_stride, int32_t x_dtype, int8_t *q,
                                          float *scale, void *stream) {
  const char *fn = "gdn_quantize_rows";
  if (rows < 0 || rows > gdn::kMaxInt32)
    return gdn::no(GDN_E_SHAPE, fn, "rows must be in [0, 2^31)");
  if (k < 1 || k > 65536) return gdn::no(GDN_E_UNSUPPORTED, fn, "k must be in [1, 65536]");
  if (gdn::bad_stride(x_stride)) return gdn::no(GDN_E_SHAPE, fn, "x_stride must be in [0, 2^31]");
  if (!gdn::known_dtype(x_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "x_dtype must be F32 or BF16");
  if (rows == 0) return gdn::ok();
  if (!x || !q || !scale) return gdn::no(GDN_E_NULL, fn, "x, q and scale are required");
  if (!gdn::aligned(x, gdn::bytes_of(x_dtype)) || !gdn::aligned(scale, 4) || !gdn::aligned(q, 16))
    return gdn::no(GDN_E_SHAPE, fn, "x and scale must be element aligned, q 16-byte aligned");
  gdn::QuantizeArgs a{};
  a.rows = rows;
  a.x_stride = x_stride;
  a.k = (int32_t)k;
  a.k_pad = (int32_t)((k + GDN_I8_K_ALIGN - 1) / GDN_I8_K_ALIGN * GDN_I8_K_ALIGN);
  a.x_bf16 = x_dtype == GDN_DTYPE_BF16;
  a.x = x;
  a.q = q;
  a.scale = scale;
  return gdn::launched(fn, gdn::launch_quantize(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_linear_i8_fwd_workspace(int64_t m, int64_t n, int64_t k_pad,
                                                    size_t *bytes) {
  const char *fn = "gdn_linear_i8_fwd_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn::LinearI8Args a;
  gdn_status_t st = gdn::linear_i8_shape(fn, m, n, k_pad, a);
  if (st != GDN_OK) return st;
  *bytes = (size_t)gdn::linear_i8_parts_bytes(a);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_linear_i8_fwd(int64_t m, int64_t n, int64_t k_pad, const int8_t *xq,
                                          const float *x_scale, const int8_t *wq,
                                          const float *w_scale, int32_t y_dtype, void *y,
                                          void *workspace, size_t workspace_bytes,
                                          void *stream) {
  const char *fn = "gdn_linear_i8_fwd";
  gdn::LinearI8Args a;
  gdn_status_t st = gdn::linear_i8_shape(fn, m, n, k_pad, a);
  if (st != GDN_OK) return st;
  if (!gdn::known_dtype(y_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "y_dtype must be F32 or BF16");
  if (m == 0 || n == 0) return gdn::ok();
  if (!xq || !x_scale || !wq || !w_scale || !y)
    return gdn::no(GDN_E_NULL, fn, "xq, x_scale, wq, w_scale and y are required");
  if (gdn::any_misaligned({xq, wq}, 16) || gdn::any_misaligned({x_scale, w_scale}, 4) ||
      !gdn::aligned(y, gdn::bytes_of(y_dtype)))
    return gdn::no(GDN_E_SHAPE, fn, "xq and wq must be 16-byte aligned, the others element aligned");
  const int64_t need = gdn::linear_i8_parts_bytes(a);
  if (need > 0 && !workspace) return gdn::no(GDN_E_NULL, fn, "workspace is required");
  if (need > 0 && !gdn::aligned(workspace, 16))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 16-byte aligned");
  if (workspace_bytes < (size_t)need)
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_linear_i8_fwd_workspace reports");
  a.parts = static_cast<float *>(workspace);
  a.y_bf16 = y_dtype == GDN_DTYPE_BF16;
  a.xq = xq;
  a.wq = wq;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.y = y;
  if (gdn::linear_i8_threads(a) > int64_t(0xFFFFFFFF))
    return gdn::no(GDN_E_SHAPE, fn, "the tiles of m * n values are too many for one launch");
  return gdn::launched(fn, gdn::launch_linear_i8(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_token_logprob_fwd_workspace(const gdn_logprob_shape_t *shape,
                                                        size_t *bytes) {
  const char *fn = "gdn_token_logprob_fwd_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn::LogprobArgs a;
  gdn_status_t st = gdn::logprob_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  *bytes = (size_t)gdn::logprob_parts_bytes(a);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_token_logprob_fwd(const gdn_logprob_shape_t *shape, const void *logits,
                                              const void *ids, float *logp, float *lse,
                                              float *entropy, void *workspace,
                                              size_t workspace_bytes, void *stream) {
  const char *fn = "gdn_token_logprob_fwd";
  gdn::LogprobArgs a;
  gdn_status_t st = gdn::logprob_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  if (shape->rows == 0) return gdn::ok();
  if (!logits || !ids || !logp || !lse)
    return gdn::no(GDN_E_NULL, fn, "logits, ids, logp and lse are required");
  if (!gdn::aligned(logits, gdn::bytes_of(shape->logits_dtype)) ||
      !gdn::aligned(ids, shape->id_bytes) || gdn::any_misaligned({logp, lse, entropy}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  const int64_t need = gdn::logprob_parts_bytes(a);
  if (need > 0 && !workspace) return gdn::no(GDN_E_NULL, fn, "workspace is required");
  if (need > 0 && !gdn::aligned(workspace, 4))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 4-byte aligned");
  if (workspace_bytes < (size_t)need)
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_token_logprob_fwd_workspace reports");
  a.parts = static_cast<float *>(workspace);
  a.logits = logits;
  a.ids = ids;
  a.logp = logp;
  a.lse = lse;
  a.entropy = entropy;
  return gdn::launched(fn, gdn::launch_logprob_fwd(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_token_logprob_bwd(const gdn_logprob_shape_t *shape, const void *logits,
                                              const void *ids, const float *lse,
                                              const float *d_logp, const float *entropy,
                                              const float *d_entropy, void *d_logits,
                                              void *stream) {
  const char *fn = "gdn_token_logprob_bwd";
  gdn::LogprobArgs a;
  gdn_status_t st = gdn::logprob_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  if (!entropy != !d_entropy)
    return gdn::no(GDN_E_NULL, fn, "entropy and d_entropy are given together or not at all");
  if (shape->rows == 0) return gdn::ok();
  if (!logits || !ids || !lse || !d_logp || !d_logits)
    return gdn::no(GDN_E_NULL, fn, "logits, ids, lse, d_logp and d_logits are required");
  if (gdn::any_misaligned({logits, d_logits}, gdn::bytes_of(shape->logits_dtype)) ||
      !gdn::aligned(ids, shape->id_bytes) ||
      gdn::any_misaligned({lse, d_logp, entropy, d_entropy}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  if (d_logits == logits && shape->logits_stride != shape->vocab)
    return gdn::no(GDN_E_SHAPE, fn, "d_logits can be the logits only where their stride is vocab");
  a.logits = logits;
  a.ids = ids;
  a.lse = const_cast<float *>(lse);
  a.d_logp = d_logp;
  a.entropy = const_cast<float *>(entropy);
  a.d_entropy = d_entropy;
  a.d_logits = d_logits;
  if (gdn::logprob_bwd_grid(a) > gdn::kMaxInt32)
    return gdn::no(GDN_E_SHAPE, fn, "rows * ceil(vocab / 2048, BF16 4096) must be under 2^31");
  return gdn::launched(fn, gdn::launch_logprob_bwd(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_policy_loss_workspace(const gdn_policy_shape_t *shape, size_t *bytes) {
  const char *fn = "gdn_policy_loss_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn::PolicyArgs a;
  gdn_status_t st = gdn::policy_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  *bytes = gdn::policy_workspace(a);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_policy_loss_fwd(const gdn_policy_shape_t *shape, const float *logp,
                                            const float *old_logp, const float *advantages,
                                            const float *ref_logp, const float *entropy,
                                            const uint8_t *mask, const int32_t *cu_seqlens,
                                            float *stats, float *seq_weight, void *workspace,
                                            size_t workspace_bytes, void *stream) {
  const char *fn = "gdn_policy_loss_fwd";
  gdn::PolicyArgs a;
  gdn_status_t st = gdn::policy_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  st = gdn::policy_inputs(fn, shape, logp, old_logp, advantages, ref_logp, cu_seqlens, a, mask);
  if (st != GDN_OK) return st;
  if (!stats || (!seq_weight && shape->seqs > 0) || !workspace)
    return gdn::no(GDN_E_NULL, fn, "stats, seq_weight and workspace are required");
  if (gdn::any_misaligned({entropy, stats, seq_weight}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  if (!gdn::aligned(workspace, 256))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < gdn::policy_workspace(a))
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_policy_loss_workspace reports");
  a.entropy = entropy;
  a.stats = stats;
  a.seq_weight = seq_weight;
  a.partials = static_cast<double *>(workspace);
  a.seq_sums = reinterpret_cast<double *>(static_cast<char *>(workspace) +
                                          gdn::policy_partial_bytes(a));
  return gdn::launched(fn, gdn::launch_policy_fwd(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_policy_loss_bwd(const gdn_policy_shape_t *shape, const float *logp,
                                            const float *old_logp, const float *advantages,
                                            const float *ref_logp, const uint8_t *mask,
                                            const int32_t *cu_seqlens, const float *seq_weight,
                                            double d_loss, float *d_logp, float *d_entropy,
                                            void *stream) {
  const char *fn = "gdn_policy_loss_bwd";
  gdn::PolicyArgs a;
  gdn_status_t st = gdn::policy_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  st = gdn::policy_inputs(fn, shape, logp, old_logp, advantages, ref_logp, cu_seqlens, a, mask);
  if (st != GDN_OK) return st;
  if (!std::isfinite(d_loss)) return gdn::no(GDN_E_SHAPE, fn, "d_loss must be finite");
  if (!seq_weight && shape->seqs > 0)
    return gdn::no(GDN_E_NULL, fn, "seq_weight is required");
  if (shape->tokens > 0 && !d_logp) return gdn::no(GDN_E_NULL, fn, "d_logp is required");
  if (gdn::any_misaligned({seq_weight, d_logp, d_entropy}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  a.weight = seq_weight;
  a.d_loss = d_loss;
  a.d_logp = d_logp;
  a.d_entropy = d_entropy;
  return gdn::launched(fn, gdn::launch_policy_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
