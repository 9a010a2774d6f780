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

// v_mfma_i32_16x16x64_i8: lane l gives row l % 16 of either operand at k = 16 (l / 16) .. + 15,
// and holds the results of rows 4 (l / 16) .. + 3 of the first operand and row l % 16 of the
// second. The first operand is W, so a lane's four results are neighbours in a row of Y; two
// products whose W rows are 8 (i / 4) + 4 j + i % 4 (j = 0, 1) give a lane eight neighbours.
__device__ __forceinline__ i32x4 mfma(i32x4 w, i32x4 x, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}
__device__ __forceinline__ int pair_row(int i, int j) { return 8 * (i / 4) + 4 * j + i % 4; }

// Eight neighbouring results of row m from column n on.
template <bool YB>
__device__ __forceinline__ void store8(const LinearI8Args &p, int64_t m, int64_t n, i32x4 lo,
                                       i32x4 hi, float xs, const float (&ws)[8]) {
  float v[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] = (float)lo[r] * xs * ws[r];
    v[4 + r] = (float)hi[r] * xs * ws[4 + r];
  }
  store_row<YB>(p.y, m * p.n, n, p.n, v);
}

__device__ __forceinline__ void load_scales(const LinearI8Args &p, int64_t n, float (&ws)[8]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) ws[r] = n + r < p.n ? p.w_scale[n + r] : 0.0f;
}

// Few rows: W's bytes are what counts, each read once, straight into the operand registers. A
// workgroup takes 32 columns and MT groups of 16 rows; its eight waves take the 128-byte lines
// of K in turn and their integer sums are added in LDS.
template <int MT, bool YB>
__global__ __launch_bounds__(512) void linear_i8_rows_kernel(const LinearI8Args p) {
  constexpr int U = MT == 4 ? 1 : MT == 2 ? 2 : 4;  // lines of K in flight
  __shared__ i32x4 part[8][2 * MT][64];
  const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n0 = (int64_t)blockIdx.x * 32;
  const int8_t *w[2], *x[MT];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t row = n0 + pair_row(l % 16, j);
    w[j] = p.wq + (row < p.n ? row : p.n - 1) * p.k + 16 * (l / 16);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = 16 * i + l % 16;
    x[i] = p.xq + (row < p.m ? row : p.m - 1) * p.k + 16 * (l / 16);
  }
  i32x4 acc[2][MT];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  auto at = [](const int8_t *b, int k) { return *reinterpret_cast<const i32x4 *>(b + k); };
  const int lines = p.k / 128;
  int line = wave;
  for (; line + 8 * (U - 1) < lines; line += 8 * U) {
    i32x4 wf[U][2][2], xf[U][2][MT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (line + 8 * u) * 128 + 64 * h;
#pragma unroll
        for (int j = 0; j < 2; ++j) wf[u][h][j] = at(w[j], k);
#pragma unroll
        for (int i = 0; i < MT; ++i) xf[u][h][i] = at(x[i], k);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[j][i] = mfma(wf[u][h][j], xf[u][h][i], acc[j][i]);
  }
  for (; line < lines; line += 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = line * 128 + 64 * h;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const i32x4 wf = at(w[j], k);
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = mfma(wf, at(x[i], k), acc[j][i]);
      }
    }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][2 * i + j][l] = acc[j][i];
  __syncthreads();
  if (wave < MT) {  // wave i finishes rows 16 i .. + 15
    i32x4 lo = part[0][2 * wave][l], hi = part[0][2 * wave + 1][l];
#pragma unroll
    for (int v = 1; v < 8; ++v) {
      lo += part[v][2 * wave][l];
      hi += part[v][2 * wave + 1][l];
    }
    const int64_t m = 16 * wave + l % 16, n = n0 + 8 * (l / 16);
    if (m < p.m) {
      float ws[8];
      load_scales(p, n, ws);
      store8<YB>(p, m, n, lo, hi, p.x_scale[m], ws);
    }
  }
}

// A BN x BM tile of Y by (BN / TN) x (BM / TM) waves, each TN columns by TM rows. K goes
// through LDS 128 bytes at a time, two stages: the loads of the next one, straight from memory
// into LDS, are in flight while the matrix units work on the current one. A line of 128 bytes
// is held as eight 16-byte chunks, chunk c of row r at place c ^ key(r), so that the lanes of
// an operand read, which want the same chunk of 16 rows, spread over the banks. The loads
// write LDS in the order of the lanes, so the permutation is in which chunk a lane fetches.
__device__ __forceinline__ int x_key(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int w_key(int r) { return ((r >> 3) & 3) << 1 | ((r >> 1) & 1); }

template <int BM, int BN, int TM, int TN, bool YB>
__global__ __launch_bounds__(BM / TM *(BN / TN) * 64) void linear_i8_tile_kernel(const LinearI8Args p) {
  constexpr int kWaves = BM / TM * (BN / TN), MI = TM / 16, NP = TN / 32;
  constexpr int kLoads = (BM + BN) / 8 / kWaves;  // 1 KiB (8 rows) each, per wave and stage
  static_assert((BM + BN) / 8 % kWaves == 0 && BN / 8 % 1 == 0, "whole loads");
  __shared__ __align__(128) int8_t stage0[(BM + BN) * 128];
  __shared__ __align__(128) int8_t stage1[(BM + BN) * 128];
  const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // tiles: each XCD (workgroup % 8) a run of neighbours, in bands of 8 tiles of rows
  const int64_t tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
  const int64_t total = tiles_m * tiles_n, per = (total + 7) / 8;
  const int64_t tile = blockIdx.x % 8 * per + blockIdx.x / 8;
  if (blockIdx.x / 8 >= per || tile >= total) return;
  const int64_t band = tile / (8 * tiles_n), in_band = tile % (8 * tiles_n);
  const int64_t height = tiles_m - 8 * band < 8 ? tiles_m - 8 * band : 8;
  const int64_t m0 = (8 * band + in_band % height) * BM, n0 = in_band / height * BN;

  // the wave's loads of a stage: a base in scalar registers and an offset per lane; rows past
  // the end repeat the last one
  const int8_t *wbase = p.wq + n0 * p.k, *xbase = p.xq + m0 * p.k;
  const int last_w = (int)(p.n - n0 < BN ? p.n - n0 : BN) - 1;
  const int last_x = (int)(p.m - m0 < BM ? p.m - m0 : BM) - 1;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (wave * kLoads + i) * 8 + l / 8;  // W's rows, then X's
    if ((wave * kLoads + i) * 8 < BN)
      off[i] = (uint32_t)(r < last_w ? r : last_w) * p.k + 16 * (l % 8 ^ w_key(r));
    else
      off[i] = (uint32_t)(r - BN < last_x ? r - BN : last_x) * p.k + 16 * (l % 8 ^ x_key(r - BN));
  }
  auto fetch = [&](int8_t *to, int k) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int8_t *base = ((wave * kLoads + i) * 8 < BN ? wbase : xbase) + k;
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)(base + off[i]),
          (__attribute__((address_space(3))) void *)(to + (wave * kLoads + i) * 1024), 16, 0, 0);
    }
  };

  i32x4 acc[2 * NP][MI];
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j)
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  const int wn = wave % (BN / TN) * TN, wm = wave / (BN / TN) * TM;
  auto compute = [&](const int8_t *from) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 xf[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = wm + 16 * i + l % 16;
        xf[i] = *reinterpret_cast<const i32x4 *>(from + (BN + r) * 128 + 16 * ((4 * h + l / 16) ^ x_key(r)));
      }
#pragma unroll
      for (int j = 0; j < 2 * NP; ++j) {
        const int r = wn + j / 2 * 32 + pair_row(l % 16, j % 2);
        const i32x4 wf = *reinterpret_cast<const i32x4 *>(from + r * 128 + 16 * ((4 * h + l / 16) ^ w_key(r)));
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = mfma(wf, xf[i], acc[j][i]);
      }
    }
  };

  fetch(stage0, 0);
  for (int k = 0; k + 256 <= p.k; k += 256) {
    __syncthreads();  // stage0 has arrived; stage1's last reader is done
    fetch(stage1, k + 128);
    compute(stage0);
    __syncthreads();
    fetch(stage0, k + 256 < p.k ? k + 256 : k);  // after the last stage: one not needed
    compute(stage1);
  }
  if (p.k % 256 != 0) {
    __syncthreads();
    compute(stage0);
  }

#pragma unroll
  for (int q = 0; q < NP; ++q) {
    const int64_t n = n0 + wn + 32 * q + 8 * (l / 16);
    float ws[8];
    load_scales(p, n, ws);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t m = m0 + wm + 16 * i + l % 16;
      if (m < p.m) store8<YB>(p, m, n, acc[2 * q][i], acc[2 * q + 1][i], p.x_scale[m], ws);
    }
  }
}

struct Launch {
  const void *fn;
  int threads;
  int64_t grid;
};

template <int MT>
Launch rows_launch(const LinearI8Args &a) {
  return {a.y_bf16 ? (const void *)linear_i8_rows_kernel<MT, true>
                   : (const void *)linear_i8_rows_kernel<MT, false>,
          512, (a.n + 31) / 32};
}

template <int BM, int BN, int TM, int TN>
Launch tile_launch(const LinearI8Args &a) {
  const int64_t total = (a.m + BM - 1) / BM * ((a.n + BN - 1) / BN);
  return {a.y_bf16 ? (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, true>
                   : (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, false>,
          BM / TM * (BN / TN) * 64, (total + 7) / 8 * 8};
}

Launch pick(const LinearI8Args &a) {
  if (a.m <= 16) return rows_launch<1>(a);
  if (a.m <= 32) return rows_launch<2>(a);
  if (a.m <= 64) return rows_launch<4>(a);
  const int64_t big = (a.m + 255) / 256 * ((a.n + 255) / 256);
  if (big >= 200) return tile_launch<256, 256, 64, 128>(a);
  return tile_launch<128, 128, 64, 64>(a);
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

int64_t linear_i8_grid(const LinearI8Args &a) { return pick(a).grid; }

hipError_t launch_linear_i8(const LinearI8Args &a, hipStream_t stream) {
  if (a.m == 0 || a.n == 0) return hipSuccess;
  const Launch go = pick(a);
  LinearI8Args args = a;
  void *kargs[] = {&args};
  return hipLaunchKernel(go.fn, dim3((unsigned)go.grid), dim3(go.threads), kargs, 0, stream);
}

}  // namespace gdn
