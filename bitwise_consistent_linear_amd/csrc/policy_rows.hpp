// Device helpers of the policy head's row kernels: eight consecutive values of a row per
// lane, whatever the row's alignment, and sums over the lanes that share a row.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn {

// gfx950 takes 16-byte global accesses at any element alignment, so rows of odd width or
// stride use the same wide loads as aligned ones.
using u32x4_a2 = uint32_t __attribute__((ext_vector_type(4), aligned(2)));
using f32x4_a4 = float __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Eight consecutive values as loaded (bf16 bits or binary32).
template <bool BF16>
struct Vec8;

template <>
struct Vec8<true> {
  u32x4_a2 r;
  __device__ __forceinline__ void zero() { r = u32x4_a2{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const void *base, int64_t idx) {
    r = *reinterpret_cast<const u32x4_a2 *>(static_cast<const uint16_t *>(base) + idx);
  }
  // the first n (0 .. 7) values, `fill` (exact in bf16) after them
  __device__ __forceinline__ void load_part(const void *base, int64_t idx, int n,
                                            float fill = 0.0f) {
    const uint16_t *b = static_cast<const uint16_t *>(base) + idx;
    const uint32_t f = __float_as_uint(fill) >> 16;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 2] |= (e < n ? (uint32_t)b[e] : f) << (16 * (e % 2));
    r = u32x4_a2{w[0], w[1], w[2], w[3]};
  }
  __device__ __forceinline__ float get(int e) const {
    return e % 2 == 0 ? bf16_lo(r[e / 2]) : bf16_hi(r[e / 2]);
  }
  __device__ __forceinline__ static void store(void *base, int64_t idx, const float (&v)[8]) {
    u32x4_a2 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = to_bf16(v[2 * i]) | (to_bf16(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4_a2 *>(static_cast<uint16_t *>(base) + idx) = o;
  }
  __device__ __forceinline__ static void store_part(void *base, int64_t idx, const float (&v)[8],
                                                    int n) {
    uint16_t *b = static_cast<uint16_t *>(base) + idx;
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) b[e] = (uint16_t)to_bf16(v[e]);
  }
};

template <>
struct Vec8<false> {
  f32x4_a4 r[2];
  __device__ __forceinline__ void zero() { r[0] = r[1] = f32x4_a4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const void *base, int64_t idx) {
    const f32x4_a4 *b = reinterpret_cast<const f32x4_a4 *>(static_cast<const float *>(base) + idx);
    r[0] = b[0];
    r[1] = b[1];
  }
  __device__ __forceinline__ void load_part(const void *base, int64_t idx, int n,
                                            float fill = 0.0f) {
    const float *b = static_cast<const float *>(base) + idx;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e / 4][e % 4] = e < n ? b[e] : fill;
  }
  __device__ __forceinline__ float get(int e) const { return r[e / 4][e % 4]; }
  __device__ __forceinline__ static void store(void *base, int64_t idx, const float (&v)[8]) {
    f32x4_a4 *b = reinterpret_cast<f32x4_a4 *>(static_cast<float *>(base) + idx);
    b[0] = f32x4_a4{v[0], v[1], v[2], v[3]};
    b[1] = f32x4_a4{v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ static void store_part(void *base, int64_t idx, const float (&v)[8],
                                                    int n) {
    float *b = static_cast<float *>(base) + idx;
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) b[e] = v[e];
  }
};

// Values of a row of `width` at [col, col + 8); zeros past its end. n: how many are the row's.
template <bool BF16>
__device__ __forceinline__ void load_row(Vec8<BF16> &v, const void *base, int64_t row_off,
                                         int64_t col, int64_t width) {
  if (col + 8 <= width)
    v.load(base, row_off + col);
  else if (col < width)
    v.load_part(base, row_off + col, (int)(width - col));
  else
    v.zero();
}

template <bool BF16>
__device__ __forceinline__ void store_row(void *base, int64_t row_off, int64_t col, int64_t width,
                                          const float (&v)[8]) {
  if (col + 8 <= width)
    Vec8<BF16>::store(base, row_off + col, v);
  else if (col < width)
    Vec8<BF16>::store_part(base, row_off + col, v, (int)(width - col));
}

// Sum over groups of G neighbouring lanes (a power of two up to 64), in every lane.
template <int G>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int s = G / 2; s > 0; s /= 2) v += __shfl_xor(v, s, 64);
  return v;
}

// Sum over the T threads that share a row, in every one of them: the lanes of a wave by
// lane_sum, waves in ascending order through `slot` (one float per wave of the workgroup,
// which must not be written again before the workgroup's next barrier after this one).
template <int T>
__device__ __forceinline__ float row_sum(float v, float *slot) {
  if constexpr (T <= 64) {
    return lane_sum<T>(v);
  } else {
    v = lane_sum<64>(v);
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) slot[wave] = v;
    __syncthreads();
    const int first = wave / (T / 64) * (T / 64);
    float s = slot[first];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) s += slot[first + i];
    return s;
  }
}

// Two such sums at once, through one barrier.
template <int T, int N>
__device__ __forceinline__ void row_sum2(float a, float b, float (&slot)[2][N], float &sa,
                                         float &sb) {
  sa = lane_sum<(T < 64 ? T : 64)>(a);
  sb = lane_sum<(T < 64 ? T : 64)>(b);
  if constexpr (T > 64) {
    const int wave = threadIdx.x / 64, first = wave / (T / 64) * (T / 64);
    if (threadIdx.x % 64 == 0) {
      slot[0][wave] = sa;
      slot[1][wave] = sb;
    }
    __syncthreads();
    sa = slot[0][first];
    sb = slot[1][first];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) {
      sa += slot[0][first + i];
      sb += slot[1][first + i];
    }
  }
}

}  // namespace gdn
