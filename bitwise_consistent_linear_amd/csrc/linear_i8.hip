// The 8-bit integer linear region on gfx950: rows quantised with one scale each, and
// Y = (xq wq^T) x_scale w_scale on the int8 matrix instructions.
//
// The sums of products are exact 32-bit integers, so neither tile nor schedule nor the number
// of rows changes a bit of Y; only the epilogue rounds (integer to binary32, two products,
// and the rounding to Y's type).

#include "policy_internal.h"
#include "policy_rows.hpp"

namespace gdn {
namespace {

using i32x4 = int __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------- quantisation

// max |x| that keeps a NaN.
__device__ __forceinline__ float abs_max(float a, float b) {
  b = fabsf(b);
  return (b > a || b != b) ? b : a;
}

// 127 x / a rounded to the nearest integer, ties to even, for |x| <= a, inv = 1 / a rounded.
// The product with inv is within a unit or two of the quotient's last place, which matters
// only where the exact quotient is a half: one step with the exact remainder then gives the
// half itself, and rint decides the tie. bf16: 127 x is exact in binary32. A quotient q in
// [2^k, 2^(k+1)) of 8-bit numerator and denominator significands that is no half lies at least
// 2^(k-17) from one; the corrected quotient is off by less than 2^(k-23).
__device__ __forceinline__ float quotient(float x, float a, float inv) {
  const float n = 127.0f * x;
  float q = n * inv;
  q = fmaf(fmaf(-q, a, n), inv, q);
  return rintf(q);
}

// binary32 inputs: 127 x takes 31 bits, so the same in binary64.
__device__ __forceinline__ float quotient(double x, double a, double inv) {
  const double n = 127.0 * x;
  double q = n * inv;
  q = fma(fma(-q, a, n), inv, q);
  return (float)rint(q);
}

template <bool B16, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void quantize_kernel(const QuantizeArgs p) {
  constexpr int kThreads = T < 256 ? 256 : T, RPW = kThreads / T;
  __shared__ float slot[kThreads / 64];
  const int t = threadIdx.x % T;
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / T;
  const bool live = row < p.rows;
  if (!live) row = p.rows - 1;
  Vec8<B16> x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_row(x[j], p.x, row * p.x_stride, 8 * (j * T + t), p.k);
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) a = abs_max(a, x[j].get(e));
#pragma unroll
  for (int s = 1; s < (T < 64 ? T : 64); s *= 2) a = abs_max(a, __shfl_xor(a, s, 64));
  if constexpr (T > 64) {
    if (threadIdx.x % 64 == 0) slot[threadIdx.x / 64] = a;
    __syncthreads();
    a = slot[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) a = abs_max(a, slot[i]);
  }
  if (live) {
    if (t == 0) p.scale[row] = a / 127.0f;
    const bool finite = a < __builtin_inff(), some = a > 0.0f;
    // the inverse of a subnormal a is not finite and 127 times a large one neither: scale the
    // row and its maximum by a power of two first
    const float up = a < 0x1p-100f ? 0x1p+120f : a > 0x1p+100f ? 0x1p-100f : 1.0f, as = a * up;
    const float inv = 1.0f / as;
    const double inv64 = B16 ? 0.0 : 1.0 / (double)as;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = 8 * (j * T + t);
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = x[j].get(e);
        float q;
        if (finite)
          q = B16 ? quotient(v * up, as, inv) : quotient((double)(v * up), (double)as, inv64);
        else
          q = a == a && fabsf(v) == a ? copysignf(127.0f, v) : 0.0f;
        o[e / 4] |= ((uint32_t)(some ? (int)q : 0) & 0xFFu) << (8 * (e % 4));
      }
      if (col < p.k_pad)
        *reinterpret_cast<uint2 *>(p.q + row * p.k_pad + col) = make_uint2(o[0], o[1]);
    }
  }
}

template <int T, int NV>
hipError_t quantize_as(const QuantizeArgs &a, hipStream_t stream) {
  constexpr int kThreads = T < 256 ? 256 : T, RPW = kThreads / T;
  QuantizeArgs args = a;
  void *kargs[] = {&args};
  const void *fn = a.x_bf16 ? (const void *)quantize_kernel<true, T, NV>
                            : (const void *)quantize_kernel<false, T, NV>;
  return hipLaunchKernel(fn, dim3((unsigned)((a.rows + RPW - 1) / RPW)), dim3(kThreads), kargs, 0,
                         stream);
}

// ------------------------------------------------------------------------------ product

// Values of one output row at columns n .. n + 3.
template <bool YB>
__device__ __forceinline__ void store4(const LinearI8Args &p, int64_t m, int64_t n, i32x4 acc,
                                       float xs, const float (&ws)[4]) {
  float v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = (float)acc[r] * xs * ws[r];
  const int64_t at = m * p.n + n;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n + r < p.n) {
      if (YB)
        static_cast<uint16_t *>(p.y)[at + r] = (uint16_t)to_bf16(v[r]);
      else
        static_cast<float *>(p.y)[at + r] = v[r];
    }
}

// One wave per 16 x 16 tile of Y, operands straight from memory. v_mfma_i32_16x16x64_i8: lane
// l gives row l % 16 of either operand at k = 16 (l / 16) .. + 15, and holds the results of
// rows 4 (l / 16) .. + 3 of the first operand and row l % 16 of the second. The first operand
// is W, so a lane's four results are neighbours in a row of Y.
template <bool YB>
__global__ __launch_bounds__(64) void linear_i8_kernel(const LinearI8Args p) {
  const int l = threadIdx.x;
  const int64_t tiles_n = (p.n + 15) / 16;
  const int64_t n0 = blockIdx.x % tiles_n * 16, m0 = blockIdx.x / tiles_n * 16;
  const int64_t wrow = n0 + l % 16 < p.n ? n0 + l % 16 : p.n - 1;
  const int64_t xrow = m0 + l % 16 < p.m ? m0 + l % 16 : p.m - 1;
  const int8_t *w = p.wq + wrow * p.k + 16 * (l / 16), *x = p.xq + xrow * p.k + 16 * (l / 16);
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 0; k < p.k; k += 64)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4 *>(w + k),
                                                *reinterpret_cast<const i32x4 *>(x + k), acc, 0, 0, 0);
  const int64_t m = m0 + l % 16, n = n0 + 4 * (l / 16);
  if (m < p.m) {
    float ws[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) ws[r] = n + r < p.n ? p.w_scale[n + r] : 0.0f;
    store4<YB>(p, m, n, acc, p.x_scale[m], ws);
  }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.k_pad <= 512) return quantize_as<64, 1>(a, stream);
  if (a.k_pad <= 2048) return quantize_as<64, 4>(a, stream);
  if (a.k_pad <= 8192) return quantize_as<256, 4>(a, stream);
  if (a.k_pad <= 32768) return quantize_as<1024, 4>(a, stream);
  return quantize_as<1024, 8>(a, stream);
}

int64_t linear_i8_grid(const LinearI8Args &a) { return (a.m + 15) / 16 * ((a.n + 15) / 16); }

hipError_t launch_linear_i8(const LinearI8Args &a, hipStream_t stream) {
  const int64_t grid = linear_i8_grid(a);
  if (grid <= 0) return hipSuccess;
  LinearI8Args args = a;
  void *kargs[] = {&args};
  const void *fn = a.y_bf16 ? (const void *)linear_i8_kernel<true>
                            : (const void *)linear_i8_kernel<false>;
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(64), kargs, 0, stream);
}

}  // namespace gdn
