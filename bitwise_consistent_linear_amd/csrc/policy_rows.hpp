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

// Two values rounded to bf16 (to nearest even; one instruction on gfx950), `a` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
  using f32x2 = float __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float f) { return (uint16_t)pack_bf16(f, 0.0f); }

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
  __device__ __forceinline__ void load_part(const void *base, int64_t idx, int n, float fill) {
    const uint16_t *b = static_cast<const uint16_t *>(base) + idx;
    const uint32_t f = __float_as_uint(fill) >> 16;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 2] |= (e < n ? (uint32_t)b[e] : f) << (16 * (e % 2));
    r = u32x4_a2{w[0], w[1], w[2], w[3]};
  }
  // the values from the n-th on are `fill` (its upper half; n may be below 0)
  __device__ __forceinline__ void fill_from(int n, float fill) {
    const uint32_t h = __float_as_uint(fill);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i >= n) r[i] = (r[i] & 0xFFFF0000u) | h >> 16;
      if (2 * i + 1 >= n) r[i] = (r[i] & 0xFFFFu) | (h & 0xFFFF0000u);
    }
  }
  // the last 8 - s values first, `fill` (its upper half) after them; s in 0 .. 8
  __device__ __forceinline__ void drop(int s, float fill) {
    const uint32_t h = __float_as_uint(fill), f = (h & 0xFFFF0000u) | h >> 16;
    if (s & 12) r = u32x4_a2{r[2], r[3], f, f};
    if (s & 8) r = u32x4_a2{f, f, f, f};
    if (s & 2) r = u32x4_a2{r[1], r[2], r[3], f};
    if (s & 1) {
      auto half = [](uint32_t lo, uint32_t hi) { return lo >> 16 | hi << 16; };
      r = u32x4_a2{half(r[0], r[1]), half(r[1], r[2]), half(r[2], r[3]), half(r[3], f)};
    }
  }
  __device__ __forceinline__ float get(int e) const {
    return e % 2 == 0 ? bf16_lo(r[e / 2]) : bf16_hi(r[e / 2]);
  }
  __device__ __forceinline__ static void store(void *base, int64_t idx, const float (&v)[8]) {
    u32x4_a2 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4_a2 *>(static_cast<uint16_t *>(base) + idx) = o;
  }
  __device__ __forceinline__ static void store_part(void *base, int64_t idx, const float (&v)[8],
                                                    int n) {
    uint16_t *b = static_cast<uint16_t *>(base) + idx;
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) b[e] = to_bf16(v[e]);
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
  __device__ __forceinline__ void load_part(const void *base, int64_t idx, int n, float fill) {
    const float *b = static_cast<const float *>(base) + idx;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e / 4][e % 4] = e < n ? b[e] : fill;
  }
  __device__ __forceinline__ void fill_from(int n, float fill) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= n) r[e / 4][e % 4] = fill;
  }
  __device__ __forceinline__ void drop(int s, float fill) {
    const f32x4_a4 f = {fill, fill, fill, fill};
    if (s & 12) {
      r[0] = r[1];
      r[1] = f;
    }
    if (s & 8) r[0] = f;
    if (s & 2) {
      r[0] = f32x4_a4{r[0][2], r[0][3], r[1][0], r[1][1]};
      r[1] = f32x4_a4{r[1][2], r[1][3], fill, fill};
    }
    if (s & 1) {
      r[0] = f32x4_a4{r[0][1], r[0][2], r[0][3], r[1][0]};
      r[1] = f32x4_a4{r[1][1], r[1][2], r[1][3], fill};
    }
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

// Values of a row of `width` at [col, col + 8), to be settled before their use: a row's end
// inside them makes the load one of its last eight values, whole, and settle_row moves them into
// place. (Value by value, each load waits for the one before it: the layer norm's backward of
// 16384 x 4095 bf16 took 150 us that way and takes 85.) Rows of fewer than eight are loaded so.
template <bool BF16>
__device__ __forceinline__ void load_row(Vec8<BF16> &v, const void *base, int64_t row_off,
                                         int64_t col, int64_t width, float fill = 0.0f) {
  if (width >= 8)
    v.load(base, row_off + (col + 8 <= width ? col : width - 8));
  else
    v.load_part(base, row_off + col, col < width ? (int)(width - col) : 0, fill);
}

// `fill` past the row's end.
template <bool BF16>
__device__ __forceinline__ void settle_row(Vec8<BF16> &v, int64_t col, int64_t width,
                                           float fill = 0.0f) {
  if (width >= 8 && col + 8 > width)
    v.drop(col < width ? (int)(col + 8 - width) : 8, fill);
}

template <bool BF16>
__device__ __forceinline__ void store_row(void *base, int64_t row_off, int64_t col, int64_t width,
                                          const float (&v)[8]) {
  if (col + 8 <= width)
    Vec8<BF16>::store(base, row_off + col, v);
  else if (col < width)
    Vec8<BF16>::store_part(base, row_off + col, v, (int)(width - col));
}

// A lane's neighbour n places on in its row of 16 lanes, around the row's end.
template <int N>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 | N, 0xF, 0xF, true));
}

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum over each row of 16 lanes or over the wave's 64, in every lane (pairs are added in an
// order that all lanes share up to commutation, so all have the same bits).
template <int G>
__device__ __forceinline__ float lane_sum(float v) {
  static_assert(G == 16 || G == 64, "a row of lanes or the wave");
  v += rotated<8>(v);
  v += rotated<4>(v);
  v += rotated<2>(v);
  v += rotated<1>(v);
  if constexpr (G == 64) v = (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
  return v;
}

// Maximum over the wave's lanes, in every lane (a NaN is passed over).
__device__ __forceinline__ float lane_max(float v) {
  v = fmaxf(v, rotated<8>(v));
  v = fmaxf(v, rotated<4>(v));
  v = fmaxf(v, rotated<2>(v));
  v = fmaxf(v, rotated<1>(v));
  return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}

// K sums at once over the `waves` waves that share a row (the wave's alone, or a row of 16
// lanes, for G lanes a row): lanes first, then the waves, whose sums a row of 16 lanes adds.
// `slot` must not be written again before the workgroup's next barrier after this one.
template <int G, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int waves, float (&slot)[K][16]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<G>(v[k]);
  if (G < 64 || waves == 1) return;
  const int wave = threadIdx.x / 64, first = wave / waves * waves, at = threadIdx.x % 16;
  if (threadIdx.x % 64 == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) slot[k][wave] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<16>(at < waves ? slot[k][first + at] : 0.0f);
}

}  // namespace gdn
