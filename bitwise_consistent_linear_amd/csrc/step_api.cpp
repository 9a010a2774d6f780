// C ABI entry points of libgdn_step.so: host-side claims and dispatch to the HIP kernels.
// Every claim is checked before anything is enqueued, so a refused call leaves all buffers
// untouched.

#include <cmath>
#include <cstdio>

#include "step_internal.h"

namespace gdn {
namespace {

// A buffer of fixed size: an error's text allocates nothing, so no entry point can throw.
thread_local char g_last_error[256];

constexpr int64_t kMaxInt32 = 2147483647;
constexpr int64_t kMaxStride = int64_t(1) << 31;
constexpr int64_t kMaxF8Width = int64_t(1) << 20;
constexpr int64_t kMaxTensors = int64_t(1) << 20;
constexpr int64_t kMaxValues = int64_t(1) << 40;
constexpr int64_t kMaxThreads = 0xFFFFFFFF;  // of a launch

bool aligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool known_dtype(int32_t d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }
bool known_format(int32_t f) { return f == GDN_F8_E4M3 || f == GDN_F8_E5M2; }
size_t bytes_of(int32_t d) { return d == GDN_DTYPE_BF16 ? 2 : 4; }
bool bad_stride(int64_t s) { return s < 0 || s > kMaxStride; }

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

gdn_status_t linear_f8_shape(const char *fn, const gdn_linear_f8_shape_t *sh) {
  if (!sh) return no(GDN_E_NULL, fn, "shape is NULL");
  if (sh->m < 0 || sh->m > kMaxF8Width || sh->n < 1 || sh->n > kMaxF8Width || sh->k < 1 ||
      sh->k > kMaxF8Width)
    return no(GDN_E_SHAPE, fn, "m must be in [0, 2^20], n and k in [1, 2^20]");
  if (bad_stride(sh->dy_stride)) return no(GDN_E_SHAPE, fn, "dy_stride must be in [0, 2^31]");
  if (!known_dtype(sh->dy_dtype) || !known_dtype(sh->dx_dtype) || !known_dtype(sh->dw_dtype))
    return no(GDN_E_UNSUPPORTED, fn, "dtypes must be F32 or BF16");
  if (!known_format(sh->dy_format))
    return no(GDN_E_UNSUPPORTED, fn, "dy_format must be GDN_F8_E4M3 or GDN_F8_E5M2");
  return GDN_OK;
}

// The backward's workspace: dy by rows and by columns, each with its scales.
struct F8Room {
  size_t q, scale, qt, scale_t, bytes;
};
F8Room f8_room(const gdn_linear_f8_shape_t *sh) {
  auto up = [](int64_t b) { return (size_t)((b + 255) / 256 * 256); };
  F8Room r;
  r.q = 0;
  r.scale = r.q + up(sh->m * f8_pad(sh->n));
  r.qt = r.scale + up(f8_scale_bytes(sh->m, sh->n));
  r.scale_t = r.qt + up(sh->n * f8_pad(sh->m));
  r.bytes = r.scale_t + up(f8_scale_bytes(sh->n, sh->m));
  return r;
}

gdn_status_t sample_shape(const char *fn, const gdn_sample_shape_t *sh, SampleArgs &a) {
  if (!sh) return no(GDN_E_NULL, fn, "shape is NULL");
  if (sh->rows < 0 || sh->rows > kMaxInt32) return no(GDN_E_SHAPE, fn, "rows must be in [0, 2^31)");
  if (sh->vocab < 1 || sh->vocab > kMaxInt32)
    return no(GDN_E_SHAPE, fn, "vocab must be in [1, 2^31)");
  if (bad_stride(sh->logits_stride)) return no(GDN_E_SHAPE, fn, "logits_stride must be in [0, 2^31]");
  if (!known_dtype(sh->logits_dtype))
    return no(GDN_E_UNSUPPORTED, fn, "logits_dtype must be F32 or BF16");
  if ((sh->u_bytes != 4 && sh->u_bytes != 8) || (sh->id_bytes != 4 && sh->id_bytes != 8))
    return no(GDN_E_UNSUPPORTED, fn, "u_bytes and id_bytes must be 4 or 8");
  if (!(sh->temperature == 0.0 || (sh->temperature >= 0x1p-40 && sh->temperature <= 0x1p+40)))
    return no(GDN_E_SHAPE, fn, "temperature must be 0 or in [2^-40, 2^40]");
  if (sh->top_k < 0) return no(GDN_E_SHAPE, fn, "top_k must be >= 0");
  if (!(sh->top_p >= 0.0) || !std::isfinite(sh->top_p) || !(sh->min_p >= 0.0) ||
      !std::isfinite(sh->min_p))
    return no(GDN_E_SHAPE, fn, "top_p and min_p must be finite and >= 0");
  a = SampleArgs{};
  a.rows = sh->rows;
  a.vocab = sh->vocab;
  a.stride = sh->logits_stride;
  a.bf16 = sh->logits_dtype == GDN_DTYPE_BF16;
  a.u64 = sh->u_bytes == 8;
  a.id64 = sh->id_bytes == 8;
  a.top_k = sh->top_k;
  a.temperature = sh->temperature;
  a.top_p = sh->top_p;
  a.min_p = sh->min_p;
  int bits = 0;  // vocab <= 2^bits
  while ((int64_t(1) << bits) < sh->vocab) ++bits;
  a.shift = 62 - bits < 45 ? 62 - bits : 45;
  return GDN_OK;
}

template <class T>
gdn_status_t tensor_list(const char *fn, const T *tensors, int64_t count) {
  if (count < 0 || count > kMaxTensors) return no(GDN_E_SHAPE, fn, "count must be in [0, 2^20]");
  if (count > 0 && !tensors) return no(GDN_E_NULL, fn, "tensors is NULL");
  for (int64_t i = 0; i < count; ++i)
    if (tensors[i].numel < 0 || tensors[i].numel >= kMaxValues)
      return no(GDN_E_SHAPE, fn, "numel must be in [0, 2^40)");
  return GDN_OK;
}

}  // namespace

gdn_status_t ok() {
  g_last_error[0] = 0;
  return GDN_OK;
}

}  // namespace gdn

extern "C" {

GDN_EXPORT int32_t gdn_step_abi_version(void) { return GDN_STEP_ABI_VERSION; }

GDN_EXPORT const char *gdn_step_last_error(void) { return gdn::g_last_error; }

GDN_EXPORT gdn_status_t gdn_quantize_f8(const void *x, int64_t rows, int64_t k, int64_t x_stride,
                                        int32_t x_dtype, int32_t format, uint8_t *q,
                                        uint8_t *scale, uint8_t *qt, uint8_t *scale_t,
                                        void *stream) {
  const char *fn = "gdn_quantize_f8";
  if (rows < 0 || rows > gdn::kMaxInt32)
    return gdn::no(GDN_E_SHAPE, fn, "rows must be in [0, 2^31)");
  if (k < 1 || k > gdn::kMaxF8Width)
    return gdn::no(GDN_E_UNSUPPORTED, fn, "k must be in [1, 2^20]");
  if (gdn::bad_stride(x_stride)) return gdn::no(GDN_E_SHAPE, fn, "x_stride must be in [0, 2^31]");
  if (!gdn::known_dtype(x_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "x_dtype must be F32 or BF16");
  if (!gdn::known_format(format))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "format must be GDN_F8_E4M3 or GDN_F8_E5M2");
  if (!q != !scale || !qt != !scale_t)
    return gdn::no(GDN_E_NULL, fn, "values and their scales are given together or not at all");
  if (qt && rows > gdn::kMaxF8Width)
    return gdn::no(GDN_E_SHAPE, fn, "rows must be at most 2^20 for the transpose");
  if (rows == 0) return gdn::ok();
  if (!x || (!q && !qt)) return gdn::no(GDN_E_NULL, fn, "x and one pair of outputs are required");
  if (!gdn::aligned(x, gdn::bytes_of(x_dtype)) || gdn::any_misaligned({q, scale, qt, scale_t}, 16))
    return gdn::no(GDN_E_SHAPE, fn, "x must be element aligned, the outputs 16-byte aligned");
  gdn::QuantizeF8Args a{};
  a.rows = rows;
  a.k = k;
  a.x_stride = x_stride;
  a.x_bf16 = x_dtype == GDN_DTYPE_BF16;
  a.e5m2 = format == GDN_F8_E5M2;
  a.x = x;
  a.q = q;
  a.scale = scale;
  a.qt = qt;
  a.scale_t = scale_t;
  if (gdn::quantize_f8_threads(a) > gdn::kMaxThreads)
    return gdn::no(GDN_E_SHAPE, fn, "2^24 tiles of 128 x 128 values are too many for one launch");
  return gdn::launched(fn, gdn::launch_quantize_f8(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_linear_f8_fwd(int64_t m, int64_t n, int64_t k_pad, int32_t x_format,
                                          const uint8_t *xq, const uint8_t *x_scale,
                                          const uint8_t *wq, const uint8_t *w_scale,
                                          int32_t y_dtype, void *y, void *stream) {
  const char *fn = "gdn_linear_f8_fwd";
  if (m < 0 || m > gdn::kMaxInt32 || n < 0 || n > gdn::kMaxInt32)
    return gdn::no(GDN_E_SHAPE, fn, "m and n must be in [0, 2^31)");
  if (k_pad < 0 || k_pad > gdn::kMaxF8Width || k_pad % GDN_F8_BLOCK != 0)
    return gdn::no(GDN_E_UNSUPPORTED, fn, "k_pad must be a multiple of 128 in [0, 2^20]");
  if (!gdn::known_format(x_format))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "x_format must be GDN_F8_E4M3 or GDN_F8_E5M2");
  if (!gdn::known_dtype(y_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "y_dtype must be F32 or BF16");
  if (m == 0 || n == 0) return gdn::ok();
  if (!y || (k_pad > 0 && (!xq || !x_scale || !wq || !w_scale)))
    return gdn::no(GDN_E_NULL, fn, "xq, x_scale, wq, w_scale and y are required");
  if (gdn::any_misaligned({xq, x_scale, wq, w_scale}, 16) ||
      !gdn::aligned(y, gdn::bytes_of(y_dtype)))
    return gdn::no(GDN_E_SHAPE, fn, "operands and scales must be 16-byte aligned, y element aligned");
  gdn::LinearF8Args a{};
  a.m = m;
  a.n = n;
  a.k = (int32_t)k_pad;
  a.y_bf16 = y_dtype == GDN_DTYPE_BF16;
  a.e5m2 = x_format == GDN_F8_E5M2;
  a.xq = xq;
  a.x_scale = x_scale;
  a.wq = wq;
  a.w_scale = w_scale;
  a.y = y;
  if (gdn::linear_f8_threads(a) > gdn::kMaxThreads)
    return gdn::no(GDN_E_SHAPE, fn, "the tiles of m * n values are too many for one launch");
  return gdn::launched(fn, gdn::launch_linear_f8(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_linear_f8_bwd_workspace(const gdn_linear_f8_shape_t *shape,
                                                    size_t *bytes) {
  const char *fn = "gdn_linear_f8_bwd_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn_status_t st = gdn::linear_f8_shape(fn, shape);
  if (st != GDN_OK) return st;
  *bytes = gdn::f8_room(shape).bytes;
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_linear_f8_bwd(const gdn_linear_f8_shape_t *shape, const void *dy,
                                          const uint8_t *wtq, const uint8_t *wt_scale,
                                          const uint8_t *xtq, const uint8_t *xt_scale, void *dx,
                                          void *dw, void *workspace, size_t workspace_bytes,
                                          void *stream) {
  const char *fn = "gdn_linear_f8_bwd";
  gdn_status_t st = gdn::linear_f8_shape(fn, shape);
  if (st != GDN_OK) return st;
  const int64_t m = shape->m, n = shape->n, k = shape->k;
  if (!dx && !dw) return gdn::no(GDN_E_NULL, fn, "dx or dw is required");
  if ((dx && (!wtq || !wt_scale)) || (dw && m > 0 && (!xtq || !xt_scale)))
    return gdn::no(GDN_E_NULL, fn, "dx needs wtq and wt_scale, dw xtq and xt_scale");
  if (m > 0 && (!dy || !workspace)) return gdn::no(GDN_E_NULL, fn, "dy and workspace are required");
  if (!gdn::aligned(dy, gdn::bytes_of(shape->dy_dtype)) ||
      !gdn::aligned(dx, gdn::bytes_of(shape->dx_dtype)) ||
      !gdn::aligned(dw, gdn::bytes_of(shape->dw_dtype)) ||
      gdn::any_misaligned({wtq, wt_scale, xtq, xt_scale}, 16))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned");
  if (!gdn::aligned(workspace, 256))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 256-byte aligned");
  const gdn::F8Room room = gdn::f8_room(shape);
  if (workspace_bytes < room.bytes)
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_linear_f8_bwd_workspace reports");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *const at = static_cast<uint8_t *>(workspace);
  gdn::LinearF8Args a{};
  a.e5m2 = shape->dy_format == GDN_F8_E5M2;
  gdn::LinearF8Args ax = a, aw = a;
  ax.m = m;
  ax.n = k;
  ax.k = (int32_t)gdn::f8_pad(n);
  ax.y_bf16 = shape->dx_dtype == GDN_DTYPE_BF16;
  ax.xq = at + room.q;
  ax.x_scale = at + room.scale;
  ax.wq = wtq;
  ax.w_scale = wt_scale;
  ax.y = dx;
  aw.m = n;
  aw.n = k;
  aw.k = (int32_t)gdn::f8_pad(m);
  aw.y_bf16 = shape->dw_dtype == GDN_DTYPE_BF16;
  aw.xq = at + room.qt;
  aw.x_scale = at + room.scale_t;
  aw.wq = xtq;
  aw.w_scale = xt_scale;
  aw.y = dw;
  gdn::QuantizeF8Args q{};
  q.rows = m;
  q.k = n;
  q.x_stride = shape->dy_stride;
  q.x_bf16 = shape->dy_dtype == GDN_DTYPE_BF16;
  q.e5m2 = a.e5m2;
  q.x = dy;
  if (dx) {
    q.q = at + room.q;
    q.scale = at + room.scale;
  }
  if (dw) {
    q.qt = at + room.qt;
    q.scale_t = at + room.scale_t;
  }
  if (gdn::quantize_f8_threads(q) > gdn::kMaxThreads)
    return gdn::no(GDN_E_SHAPE, fn, "dy's 2^24 tiles of 128 x 128 values are too many for one launch");
  if ((dx && gdn::linear_f8_threads(ax) > gdn::kMaxThreads) ||
      (dw && gdn::linear_f8_threads(aw) > gdn::kMaxThreads))
    return gdn::no(GDN_E_SHAPE, fn, "the tiles of a gradient are too many for one launch");
  hipError_t e = hipSuccess;
  if (m > 0) {
    e = gdn::launch_quantize_f8(q, s);
    if (e == hipSuccess)
      e = !dw ? gdn::launch_linear_f8(ax, s)
              : !dx ? gdn::launch_linear_f8(aw, s) : gdn::launch_linear_f8(ax, aw, s);
  } else if (dw) {
    e = gdn::launch_linear_f8(aw, s);
  }
  return gdn::launched(fn, e);
}

GDN_EXPORT gdn_status_t gdn_sample_tokens_workspace(const gdn_sample_shape_t *shape,
                                                    size_t *bytes) {
  const char *fn = "gdn_sample_tokens_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn::SampleArgs a;
  gdn_status_t st = gdn::sample_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  *bytes = (size_t)gdn::sample_workspace_bytes(a);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_sample_tokens(const gdn_sample_shape_t *shape, const void *logits,
                                          const void *u, const float *temperature,
                                          const int32_t *top_k, const float *top_p,
                                          const float *min_p, void *ids, float *logp,
                                          void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "gdn_sample_tokens";
  gdn::SampleArgs a;
  gdn_status_t st = gdn::sample_shape(fn, shape, a);
  if (st != GDN_OK) return st;
  if (shape->rows == 0) return gdn::ok();
  if (!logits || !u || !ids || !logp)
    return gdn::no(GDN_E_NULL, fn, "logits, u, ids and logp are required");
  if (!gdn::aligned(logits, gdn::bytes_of(shape->logits_dtype)) ||
      !gdn::aligned(u, shape->u_bytes) || !gdn::aligned(ids, shape->id_bytes) ||
      gdn::any_misaligned({temperature, top_k, top_p, min_p, logp}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
  const int64_t need = gdn::sample_workspace_bytes(a);
  if (need > 0 && !workspace) return gdn::no(GDN_E_NULL, fn, "workspace is required");
  if (need > 0 && !gdn::aligned(workspace, 256))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < (size_t)need)
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_sample_tokens_workspace reports");
  a.logits = logits;
  a.u = u;
  a.temperatures = temperature;
  a.top_ks = top_k;
  a.top_ps = top_p;
  a.min_ps = min_p;
  a.ids = ids;
  a.logp = logp;
  a.workspace = workspace;
  return gdn::launched(fn, gdn::launch_sample(a, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_grad_norm_workspace(const gdn_grad_tensor_t *tensors, int64_t count,
                                                size_t *bytes) {
  const char *fn = "gdn_grad_norm_workspace";
  if (!bytes) return gdn::no(GDN_E_NULL, fn, "bytes is NULL");
  gdn_status_t st = gdn::tensor_list(fn, tensors, count);
  if (st != GDN_OK) return st;
  *bytes = (size_t)gdn::grad_norm_workspace_bytes(tensors, count);
  return gdn::ok();
}

GDN_EXPORT gdn_status_t gdn_grad_norm(const gdn_grad_tensor_t *tensors, int64_t count,
                                      int32_t grad_dtype, double max_norm, float *norm,
                                      float *factor, void *workspace, size_t workspace_bytes,
                                      void *stream) {
  const char *fn = "gdn_grad_norm";
  gdn_status_t st = gdn::tensor_list(fn, tensors, count);
  if (st != GDN_OK) return st;
  if (!gdn::known_dtype(grad_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "grad_dtype must be F32 or BF16");
  if (!(max_norm >= 0.0)) return gdn::no(GDN_E_SHAPE, fn, "max_norm must be >= 0");
  if (!norm || !workspace) return gdn::no(GDN_E_NULL, fn, "norm and workspace are required");
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].numel > 0 && !tensors[i].grad) return gdn::no(GDN_E_NULL, fn, "a gradient is NULL");
    if (!gdn::aligned(tensors[i].grad, gdn::bytes_of(grad_dtype)))
      return gdn::no(GDN_E_SHAPE, fn, "a gradient is not aligned to its element");
  }
  if (gdn::any_misaligned({norm, factor}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "norm and factor must be 4-byte aligned");
  if (!gdn::aligned(workspace, 256))
    return gdn::no(GDN_E_SHAPE, fn, "workspace must be 256-byte aligned");
  if (workspace_bytes < (size_t)gdn::grad_norm_workspace_bytes(tensors, count))
    return gdn::no(GDN_E_SHAPE, fn, "workspace smaller than gdn_grad_norm_workspace reports");
  return gdn::launched(fn, gdn::launch_grad_norm(tensors, count, grad_dtype == GDN_DTYPE_BF16,
                                                 max_norm, norm, factor, workspace,
                                                 static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_adamw_step(const gdn_adamw_shape_t *shape,
                                       const gdn_adamw_tensor_t *tensors, int64_t count,
                                       const float *factor, const int64_t *step_at,
                                       const float *lr_at, void *stream) {
  const char *fn = "gdn_adamw_step";
  if (!shape) return gdn::no(GDN_E_NULL, fn, "shape is NULL");
  gdn_status_t st = gdn::tensor_list(fn, tensors, count);
  if (st != GDN_OK) return st;
  if (!gdn::known_dtype(shape->param_dtype) || !gdn::known_dtype(shape->grad_dtype))
    return gdn::no(GDN_E_UNSUPPORTED, fn, "param_dtype and grad_dtype must be F32 or BF16");
  if (shape->state != GDN_STATE_F32 && shape->state != GDN_STATE_8BIT)
    return gdn::no(GDN_E_UNSUPPORTED, fn, "state must be GDN_STATE_F32 or GDN_STATE_8BIT");
  if (!(shape->beta1 >= 0.0 && shape->beta1 < 1.0 && shape->beta2 >= 0.0 && shape->beta2 < 1.0))
    return gdn::no(GDN_E_SHAPE, fn, "beta1 and beta2 must be in [0, 1)");
  if (!(shape->eps >= 0.0) || !std::isfinite(shape->eps) || !std::isfinite(shape->lr) ||
      !std::isfinite(shape->weight_decay))
    return gdn::no(GDN_E_SHAPE, fn, "eps must be finite and >= 0, lr and weight_decay finite");
  if (shape->step < 1) return gdn::no(GDN_E_SHAPE, fn, "step must be >= 1");
  const bool eight = shape->state == GDN_STATE_8BIT;
  for (int64_t i = 0; i < count; ++i) {
    const gdn_adamw_tensor_t &t = tensors[i];
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale)))
      return gdn::no(GDN_E_NULL, fn, "param, grad, m, v and (8-bit states) their scales are required");
    if (t.master && shape->param_dtype != GDN_DTYPE_BF16)
      return gdn::no(GDN_E_UNSUPPORTED, fn, "master needs a BF16 param");
    if (!gdn::aligned(t.param, gdn::bytes_of(shape->param_dtype)) ||
        !gdn::aligned(t.grad, gdn::bytes_of(shape->grad_dtype)) ||
        gdn::any_misaligned({t.m, t.v}, eight ? 1 : 4) ||
        gdn::any_misaligned({t.m_scale, t.v_scale, t.master}, 4))
      return gdn::no(GDN_E_SHAPE, fn, "a buffer is not aligned to its element");
    const void *const one[7] = {t.param, t.grad, t.m, t.v, t.master, eight ? t.m_scale : nullptr,
                                eight ? t.v_scale : nullptr};
    for (int j = 1; j < 7; ++j)
      for (int l = 0; l < j; ++l)
        if (one[j] && one[j] == one[l])
          return gdn::no(GDN_E_SHAPE, fn, "two buffers of a tensor are the same");
  }
  if (!gdn::aligned(factor, 4) || !gdn::aligned(step_at, 8) || !gdn::aligned(lr_at, 4))
    return gdn::no(GDN_E_SHAPE, fn, "factor, step_at and lr_at must be aligned to their element");
  gdn::AdamwArgs a{};
  a.param_bf16 = shape->param_dtype == GDN_DTYPE_BF16;
  a.grad_bf16 = shape->grad_dtype == GDN_DTYPE_BF16;
  a.eight = eight;
  a.lr = shape->lr;
  a.beta1 = shape->beta1;
  a.beta2 = shape->beta2;
  a.eps = shape->eps;
  a.weight_decay = shape->weight_decay;
  a.step = shape->step;
  a.factor = factor;
  a.step_at = step_at;
  a.lr_at = lr_at;
  return gdn::launched(fn, gdn::launch_adamw(a, tensors, count, static_cast<hipStream_t>(stream)));
}

GDN_EXPORT gdn_status_t gdn_adamw_state_values(const uint8_t *codes, const float *scale,
                                               int64_t numel, int32_t moment, float *out,
                                               void *stream) {
  const char *fn = "gdn_adamw_state_values";
  if (numel < 0 || numel >= gdn::kMaxValues)
    return gdn::no(GDN_E_SHAPE, fn, "numel must be in [0, 2^40)");
  if (moment != GDN_MOMENT_M && moment != GDN_MOMENT_V)
    return gdn::no(GDN_E_UNSUPPORTED, fn, "moment must be GDN_MOMENT_M or GDN_MOMENT_V");
  if (numel == 0) return gdn::ok();
  if (!codes || !scale || !out) return gdn::no(GDN_E_NULL, fn, "codes, scale and out are required");
  if (gdn::any_misaligned({scale, out}, 4))
    return gdn::no(GDN_E_SHAPE, fn, "scale and out must be 4-byte aligned");
  return gdn::launched(fn, gdn::launch_adamw_values(codes, scale, numel, moment == GDN_MOMENT_V,
                                                    out, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
