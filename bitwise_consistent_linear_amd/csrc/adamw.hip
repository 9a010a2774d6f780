// AdamW over many tensors in one launch, with states in binary32 or in 8 bits, and the global
// gradient norm whose clip factor it takes, for gfx950.

#include <algorithm>
#include <cmath>

#include "policy_rows.hpp"
#include "step_internal.h"

namespace gdn {
namespace {

using u32x2_a2 = uint32_t __attribute__((ext_vector_type(2), aligned(2)));
using u32_a1 = uint32_t __attribute__((aligned(1)));
using f32x2 = float __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------- values of a tensor

// Four consecutive values at i of n; those past n are 0 and not read. Once: past the caches, for
// what is not looked at again before the next step (60 million values with binary32 states take
// 280 us so, 6.0 TB/s, and 326 through them).
template <bool Once, class T>
__device__ __forceinline__ T fetched(const void *from) {
  return Once ? __builtin_nontemporal_load(static_cast<const T *>(from)) : *static_cast<const T *>(from);
}
template <bool Once, class T>
__device__ __forceinline__ void put(void *to, T v) {
  if (Once)
    __builtin_nontemporal_store(v, static_cast<T *>(to));
  else
    *static_cast<T *>(to) = v;
}

template <bool Once = true>
__device__ __forceinline__ void load4(const float *b, int64_t i, int64_t n, float (&v)[4]) {
  if (i + 4 <= n) {
    const f32x4_a4 r = fetched<Once, f32x4_a4>(b + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? b[i + e] : 0.0f;
  }
}
template <bool Once = true>
__device__ __forceinline__ void load4(const uint16_t *b, int64_t i, int64_t n, float (&v)[4]) {
  if (i + 4 <= n) {
    const u32x2_a2 r = fetched<Once, u32x2_a2>(b + i);
    v[0] = bf16_lo(r[0]);
    v[1] = bf16_hi(r[0]);
    v[2] = bf16_lo(r[1]);
    v[3] = bf16_hi(r[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? bf16_lo(b[i + e]) : 0.0f;
  }
}
__device__ __forceinline__ uint32_t load4(const uint8_t *b, int64_t i, int64_t n) {
  if (i + 4 <= n) return fetched<true, u32_a1>(b + i);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) w |= i + e < n ? (uint32_t)b[i + e] << (8 * e) : 0u;
  return w;
}

template <bool Once>
__device__ __forceinline__ void store4(float *b, int64_t i, int64_t n, const float (&v)[4]) {
  if (i + 4 <= n) {
    put<Once>(b + i, f32x4_a4{v[0], v[1], v[2], v[3]});
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) b[i + e] = v[e];
  }
}
template <bool Once>
__device__ __forceinline__ void store4(uint16_t *b, int64_t i, int64_t n, const float (&v)[4]) {
  if (i + 4 <= n) {
    put<Once>(b + i, u32x2_a2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) b[i + e] = to_bf16(v[e]);
  }
}
__device__ __forceinline__ void store4(uint8_t *b, int64_t i, int64_t n, uint32_t w) {
  if (i + 4 <= n) {
    put<true, u32_a1>(b + i, w);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) b[i + e] = (uint8_t)(w >> (8 * e));
  }
}

// --------------------------------------------------------------------------- 8-bit states

constexpr float kTopM = 448.0f, kTopR = 248.0f, kTiny = 0x1p-100f;
constexpr uint32_t kRootBase = 119u << 23;

template <int N>
__device__ __forceinline__ uint32_t max_rotated(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 | N, 0xF, 0xF, true));
}

// Largest |value| of the wave's block of 256, as binary32: their bits order like integers, a
// NaN above all.
__device__ __forceinline__ float block_peak(const float (&v)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  m = max_rotated<8>(m);
  m = max_rotated<4>(m);
  m = max_rotated<2>(m);
  m = max_rotated<1>(m);
  auto of = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)m, lane); };
  return __uint_as_float(max(max(of(0), of(16)), max(of(32), of(48))));
}

// The factor that takes a block to its format's top, and its scale: 0 and 0 for a block of
// (almost) nothing, so that the factor stays finite.
__device__ __forceinline__ void block_scale(float peak, float top, float &up, float &scale) {
  const bool none = peak < kTiny;
  up = none ? 0.0f : 1.0f / peak * top;
  scale = none ? 0.0f : peak * (1.0f / top);
}

__device__ __forceinline__ uint32_t encode_m(const float (&m)[4], float up) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(m[0] * up, m[1] * up, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m[2] * up, m[3] * up, w, true);
}
__device__ __forceinline__ void decode_m(uint32_t w, float scale, float (&m)[4]) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  m[0] = a[0] * scale;
  m[1] = a[1] * scale;
  m[2] = b[0] * scale;
  m[3] = b[1] * scale;
}

// Codes of the roots: binary32 rounded to 4 fraction bits, ties to even, exponents from -8 on.
__device__ __forceinline__ uint32_t encode_r(const float (&r)[4], float up) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = r[e] * up;
    const uint32_t bits = __float_as_uint(y);
    const int c = (int)(bits - kRootBase + 0x3FFFFu + (bits >> 19 & 1)) >> 19;
    const uint32_t code = (uint32_t)min(max(c, 1), 255);
    w |= (y > 0.0f ? code : 0u) << (8 * e);
  }
  return w;
}
__device__ __forceinline__ void decode_r(uint32_t w, float scale, float (&r)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t c = w >> (8 * e) & 255;
    r[e] = (c ? __uint_as_float((c << 19) + kRootBase) : 0.0f) * scale;
  }
}

// --------------------------------------------------------------------------------- update

// b^n, n >= 0, by squaring: the same steps on the host and on the GPU.
__host__ __device__ inline double power(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, b *= b)
    if (n & 1) r *= b;
  return r;
}

struct Rates {
  float b1, c1, b2, c2, eps, root, decay, rate;
};

__host__ __device__ inline Rates rates_of(const AdamwArgs &a, int64_t step, double lr) {
  Rates r;
  r.b1 = (float)a.beta1;
  r.c1 = (float)(1.0 - a.beta1);
  r.b2 = (float)a.beta2;
  r.c2 = (float)(1.0 - a.beta2);
  r.eps = (float)a.eps;
  r.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, step)));
  r.decay = (float)(1.0 - lr * a.weight_decay);
  r.rate = (float)(lr / (1.0 - power(a.beta1, step)));
  return r;
}

// Tensors of one launch, in its arguments (4 KiB of them are safe): nothing is copied to the GPU
// ahead of the kernel, so the host may change its list as soon as the call is back.
constexpr int kTensors = 52;
// Values a workgroup takes at a time: 4 or 8 a thread. Blocks of 8-bit states are bound by their
// arithmetic and want two on their way (280 million values 667 us, with one 692), binary32 by
// memory and by the latency of short tensors (600000 values 5.2 us, with two 6.4).
constexpr int chunk_of(bool eight) { return eight ? 2048 : 1024; }
constexpr int kGrid = 1 << 20;

struct AdamwLaunch {
  AdamwArgs args;
  Rates rates;
  int32_t count;
  int64_t start[kTensors + 1];  // chunks before each tensor, and in all
  gdn_adamw_tensor_t tensor[kTensors];
};
static_assert(sizeof(AdamwLaunch) <= 4096, "kernel arguments");

// One block of 256 values by a wave, four a lane.
template <bool PB, bool GB, bool Eight>
__device__ __forceinline__ void update(const gdn_adamw_tensor_t &t, int64_t i, const Rates &k,
                                       float factor) {
  using P = std::conditional_t<PB, uint16_t, float>;
  using G = std::conditional_t<GB, uint16_t, float>;
  const int64_t n = t.numel;
  float p[4], g[4], m[4], v[4], r[4];
  uint32_t mc = 0, rc = 0;
  float ms = 0.0f, rs = 0.0f;
  const int64_t block = i / GDN_ADAMW_BLOCK;
  load4(static_cast<const G *>(t.grad), i, n, g);
  if (PB && t.master)
    load4(t.master, i, n, p);
  else
    load4(static_cast<const P *>(t.param), i, n, p);
  if (Eight) {
    mc = load4(static_cast<const uint8_t *>(t.m), i, n);
    rc = load4(static_cast<const uint8_t *>(t.v), i, n);
    ms = t.m_scale[block];
    rs = t.v_scale[block];
  } else {
    load4(static_cast<const float *>(t.m), i, n, m);
    load4(static_cast<const float *>(t.v), i, n, v);
  }
  if (!(fabsf(factor) < __builtin_inff())) return;  // looked at with the values on their way
  if (Eight) {
    decode_m(mc, ms, m);
    decode_r(rc, rs, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r[e] * r[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    g[e] *= factor;
    m[e] = m[e] * k.b1 + g[e] * k.c1;
    v[e] = v[e] * k.b2 + g[e] * g[e] * k.c2;
    r[e] = sqrtf(v[e]);
    p[e] = p[e] * k.decay - m[e] / (r[e] * k.root + k.eps) * k.rate;
  }
  store4<false>(static_cast<P *>(t.param), i, n, p);  // the next forward pass reads it
  if (PB && t.master) store4<true>(t.master, i, n, p);
  if (Eight) {
    if (i + 4 > n)  // values past the tensor's end: no part of the block's peaks
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e >= n) m[e] = r[e] = 0.0f;
    float up, scale;
    block_scale(block_peak(m), kTopM, up, scale);
    store4(static_cast<uint8_t *>(t.m), i, n, encode_m(m, up));
    if (threadIdx.x % 64 == 0) t.m_scale[block] = scale;
    block_scale(block_peak(r), kTopR, up, scale);
    store4(static_cast<uint8_t *>(t.v), i, n, encode_r(r, up));
    if (threadIdx.x % 64 == 0) t.v_scale[block] = scale;
  } else {
    store4<true>(static_cast<float *>(t.m), i, n, m);
    store4<true>(static_cast<float *>(t.v), i, n, v);
  }
}

// One workgroup a chunk, a wave a block of 256 values. 60 million bf16 values with binary32 states
// and masters: 280 us in four launches, 6.0 TB/s; 280 million with 8-bit states 650, 4.3 TB/s, bound
// by 88 vector instructions a value (a correctly rounded root and quotient, and both formats).
template <bool PB, bool GB, bool Eight>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamwLaunch p) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const float factor = p.args.factor ? *p.args.factor : 1.0f;
  Rates k = p.rates;
  if (p.args.step_at || p.args.lr_at) {
    const int64_t step = p.args.step_at ? *p.args.step_at : p.args.step;
    k = rates_of(p.args, step < 1 ? 1 : step, p.args.lr_at ? (double)*p.args.lr_at : p.args.lr);
  }
  constexpr int kChunk = chunk_of(Eight);
  const int64_t first = lane < p.count ? p.start[lane] : INT64_MAX;
  for (int64_t chunk = blockIdx.x; chunk < p.start[p.count]; chunk += gridDim.x) {
    // the tensor: the last one that starts at or before the chunk (empty ones start where the
    // next does)
    const int at = __popcll(__ballot(first <= chunk)) - 1;
    const gdn_adamw_tensor_t &t = p.tensor[at];
    const int64_t base = (chunk - p.start[at]) * kChunk;
#pragma unroll
    for (int b = 0; b < kChunk / 1024; ++b) {
      const int64_t block = base + (b * 4 + wave) * GDN_ADAMW_BLOCK;
      if (block < t.numel) update<PB, GB, Eight>(t, block + 4 * lane, k, factor);
    }
  }
}

// 280 million values: 250 us, 5.6 TB/s.
__global__ __launch_bounds__(256) void adamw_values_kernel(const uint8_t *codes,
                                                           const float *scale, int64_t n,
                                                           bool roots, float *out) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n;
       i += (int64_t)gridDim.x * 1024) {
    float v[4];
    const float s = scale[i / GDN_ADAMW_BLOCK];
    const uint32_t w = load4(codes, i, n);
    if (roots) {
      decode_r(w, s, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= v[e];
    } else {
      decode_m(w, s, v);
    }
    store4<true>(out, i, n, v);
  }
}

// ------------------------------------------------------------------------- gradient norm

constexpr int kNormTensors = 160;
constexpr int kNormChunk = 8192;
constexpr int kNormGrid = 4096;  // workgroups of a launch, a sum each

struct NormLaunch {
  int32_t count;
  int64_t start[kNormTensors + 1];
  gdn_grad_tensor_t tensor[kNormTensors];
  double *sums;  // of this launch's workgroups
};
static_assert(sizeof(NormLaunch) <= 4096, "kernel arguments");

// Sum over the workgroup's threads in a fixed order, in thread 0.
template <int Threads>
__device__ __forceinline__ double workgroup_sum(double v) {
  __shared__ double part[Threads / 64];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_down(v, d);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < Threads / 64; ++i) v += part[i];
  return v;
}

// A sum for each workgroup, in binary64: 280 million bf16 gradients 109 us, 5.1 TB/s.
template <bool GB>
__global__ __launch_bounds__(256) void grad_norm_kernel(const NormLaunch p) {
  using G = std::conditional_t<GB, uint16_t, float>;
  double sum = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < p.start[p.count]; chunk += gridDim.x) {
    int lo = 0, hi = p.count - 1;  // the last tensor that starts at or before the chunk
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.start[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const gdn_grad_tensor_t &t = p.tensor[lo];
    const int64_t base = (chunk - p.start[lo]) * kNormChunk + 4 * threadIdx.x;
#pragma unroll
    for (int j = 0; j < kNormChunk / 1024; ++j) {
      float g[4];
      load4<false>(static_cast<const G *>(t.grad), base + 1024 * j, t.numel, g);  // for the step
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = fma((double)g[e], (double)g[e], sum);
    }
  }
  sum = workgroup_sum<256>(sum);
  if (threadIdx.x == 0) p.sums[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void grad_norm_finish_kernel(const double *sums, int64_t n,
                                                                double max_norm, float *norm,
                                                                float *factor) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += sums[i];
  sum = workgroup_sum<1024>(sum);
  if (threadIdx.x == 0) {
    const double r = sqrt(sum);
    *norm = (float)r;
    if (factor)
      *factor = r < __builtin_inf() ? (float)fmin(1.0, max_norm / (r + 1e-6)) : __builtin_nanf("");
  }
}

int64_t chunks_of(int64_t numel, int64_t chunk) { return (numel + chunk - 1) / chunk; }

// Calls f(first, last, chunks) for the runs of tensors that share a launch.
template <class T, class F>
void each_launch(const T *tensors, int64_t count, int most, int64_t chunk, F f) {
  for (int64_t i = 0; i < count;) {
    int64_t j = i, chunks = 0;
    for (; j < count && j - i < most; ++j) chunks += chunks_of(tensors[j].numel, chunk);
    if (chunks > 0) f(i, j, chunks);
    i = j;
  }
}

template <bool PB, bool GB>
const void *adamw_fn(bool eight) {
  return eight ? (const void *)adamw_kernel<PB, GB, true> : (const void *)adamw_kernel<PB, GB, false>;
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs &a, const gdn_adamw_tensor_t *tensors, int64_t count,
                        hipStream_t stream) {
  const void *fn = a.param_bf16 ? (a.grad_bf16 ? adamw_fn<true, true>(a.eight)
                                               : adamw_fn<true, false>(a.eight))
                                : (a.grad_bf16 ? adamw_fn<false, true>(a.eight)
                                               : adamw_fn<false, false>(a.eight));
  AdamwLaunch p;
  p.args = a;
  p.rates = rates_of(a, a.step, a.lr);
  hipError_t e = hipSuccess;
  const int64_t chunk = chunk_of(a.eight);
  each_launch(tensors, count, kTensors, chunk, [&](int64_t i, int64_t j, int64_t chunks) {
    p.count = (int32_t)(j - i);
    p.start[0] = 0;
    for (int64_t t = i; t < j; ++t) {
      p.tensor[t - i] = tensors[t];
      p.start[t - i + 1] = p.start[t - i] + chunks_of(tensors[t].numel, chunk);
    }
    void *kargs[] = {&p};
    if (e == hipSuccess)
      e = hipLaunchKernel(fn, dim3((unsigned)std::min<int64_t>(chunks, kGrid)), dim3(256), kargs,
                          0, stream);
  });
  return e;
}

hipError_t launch_adamw_values(const uint8_t *codes, const float *scale, int64_t numel, bool v,
                               float *out, hipStream_t stream) {
  void *kargs[] = {&codes, &scale, &numel, &v, &out};
  return hipLaunchKernel((const void *)adamw_values_kernel,
                         dim3((unsigned)std::min<int64_t>(chunks_of(numel, 1024), kGrid)),
                         dim3(256), kargs, 0, stream);
}

int64_t grad_norm_workspace_bytes(const gdn_grad_tensor_t *tensors, int64_t count) {
  int64_t sums = 0;
  each_launch(tensors, count, kNormTensors, kNormChunk, [&](int64_t, int64_t, int64_t chunks) {
    sums += std::min<int64_t>(chunks, kNormGrid);
  });
  return (sums * 8 + 255) / 256 * 256 + 256;
}

hipError_t launch_grad_norm(const gdn_grad_tensor_t *tensors, int64_t count, bool bf16,
                            double max_norm, float *norm, float *factor, void *workspace,
                            hipStream_t stream) {
  double *sums = static_cast<double *>(workspace);
  int64_t n = 0;
  hipError_t e = hipSuccess;
  NormLaunch p;
  each_launch(tensors, count, kNormTensors, kNormChunk, [&](int64_t i, int64_t j, int64_t chunks) {
    p.count = (int32_t)(j - i);
    p.start[0] = 0;
    for (int64_t t = i; t < j; ++t) {
      p.tensor[t - i] = tensors[t];
      p.start[t - i + 1] = p.start[t - i] + chunks_of(tensors[t].numel, kNormChunk);
    }
    p.sums = sums + n;
    const int64_t grid = std::min<int64_t>(chunks, kNormGrid);
    n += grid;
    void *kargs[] = {&p};
    if (e == hipSuccess)
      e = hipLaunchKernel(bf16 ? (const void *)grad_norm_kernel<true>
                               : (const void *)grad_norm_kernel<false>,
                          dim3((unsigned)grid), dim3(256), kargs, 0, stream);
  });
  if (e != hipSuccess) return e;
  const double *from = sums;
  void *kargs[] = {&from, &n, &max_norm, &norm, &factor};
  return hipLaunchKernel((const void *)grad_norm_finish_kernel, dim3(1), dim3(1024), kargs, 0,
                         stream);
}

}  // namespace gdn
