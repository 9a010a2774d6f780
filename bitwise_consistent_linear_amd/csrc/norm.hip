// Layer norm and root-mean-square norm, forward and backward, on gfx950.
//
// Both are bound by memory: the forward reads x and writes y, the backward reads x and dy and
// writes dx. T threads hold a row in registers, 8 consecutive values at a time, so the
// statistics take two passes over registers and one over memory: the mean first, then the
// sum of squared distances from it, which keeps the variance exact to a few roundings where
// a sum of squares less the squared mean would cancel. A workgroup walks over several rows
// with weight and bias in registers.
//
// The reduction order depends on the width alone, so a row has the same bits in every batch.

#include "policy_internal.h"
#include "policy_rows.hpp"

namespace gdn {
namespace {

constexpr int kFwdGrid = 2048;  // workgroups of a forward launch; more rows are walked over

template <bool XB, bool WB, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_fwd_kernel(const NormArgs p) {
  constexpr int kThreads = T < 256 ? 256 : T, RPW = kThreads / T;
  __shared__ float slot[2][kThreads / 64];
  const int t = threadIdx.x % T, D = p.width;
  const bool layer = p.layer;
  const float inv = 1.0f / (float)D;
  Vec8<WB> w[NV], b[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_row(w[j], p.weight, 0, 8 * (j * T + t), D);
    if (p.bias)
      load_row(b[j], p.bias, 0, 8 * (j * T + t), D);
    else
      b[j].zero();
  }
  // one group of T threads per row; the rows past the end repeat the last one, unwritten
  for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < p.rows; r0 += (int64_t)gridDim.x * RPW) {
    int64_t row = r0 + threadIdx.x / T;
    const bool live = row < p.rows;
    if (!live) row = p.rows - 1;
    Vec8<XB> x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_row(x[j], p.x, row * p.x_stride, 8 * (j * T + t), D);
    float mean = 0.0f;
    if (layer) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[j].get(e);
      mean = row_sum<T>(s, slot[0]) * inv;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int left = D - 8 * (j * T + t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < left ? x[j].get(e) - mean : 0.0f;
        q = fmaf(d, d, q);
      }
    }
    const float var = row_sum<T>(q, slot[1]) * inv;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (live) {
      if (t == 0) {
        if (layer) p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = fmaf((x[j].get(e) - mean) * rstd, w[j].get(e), b[j].get(e));
        store_row<XB>(p.y, row * D, 8 * (j * T + t), D, y);
      }
    }
    // rms writes slot[1] again without a barrier of the mean's in between
    if (!layer && T > 64) __syncthreads();
  }
}

// Backward of one block of rows: dx, and the block's sums of dy * xh and of dy for every
// column. G groups of T threads take rows in turn; a thread keeps its columns' sums.
template <bool XB, bool WB, int T, int NV, int G>
__global__ __launch_bounds__(T *G) void norm_bwd_kernel(const NormArgs p) {
  __shared__ float slot[2][2][T * G / 64];
  __shared__ float share[G > 1 ? T * NV * 8 : 1];
  const int t = threadIdx.x % T, g = threadIdx.x / T, D = p.width;
  const bool layer = p.layer;
  const float inv = 1.0f / (float)D;
  Vec8<WB> w[NV];
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_row(w[j], p.weight, 0, 8 * (j * T + t), D);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.0f;
  }
  const int64_t per = (p.rows + p.blocks - 1) / p.blocks;
  const int64_t lo = per * blockIdx.x, hi = lo + per < p.rows ? lo + per : p.rows;
  int par = 0;
  auto load = [&](Vec8<XB> (&x)[NV], Vec8<XB> (&dy)[NV], float &mean, float &rstd, int64_t row) {
    if (row >= hi) row = hi - 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_row(x[j], p.x, row * p.x_stride, 8 * (j * T + t), D);
      load_row(dy[j], p.dy, row * p.dy_stride, 8 * (j * T + t), D);
    }
    mean = layer ? p.mean[row] : 0.0f;
    rstd = p.rstd[row];
  };
  Vec8<XB> x[NV], dy[NV];
  float mean, rstd;
  if (lo < hi) load(x, dy, mean, rstd, lo + g);
  for (int64_t r0 = lo; r0 < hi; r0 += G, par ^= 1) {
    const bool live = r0 + g < hi;
    const int64_t row = r0 + g;
    // the next row's loads are in flight under this one's sums
    Vec8<XB> nx[NV], ndy[NV];
    float nmean, nrstd;
    load(nx, ndy, nmean, nrstd, row + G);
    float s1 = 0.0f, s2 = 0.0f;  // zeros past the row's end: dy is 0 there
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (x[j].get(e) - mean) * rstd, d = dy[j].get(e);
        const float gw = d * w[j].get(e);
        s1 = fmaf(gw, xh, s1);
        s2 += gw;
        if (live) {
          dw[j][e] = fmaf(d, xh, dw[j][e]);
          db[j][e] += d;
        }
      }
    float c1, c2;
    row_sum2<T>(s1, s2, slot[par], c1, c2);
    c1 *= inv;
    c2 = layer ? c2 * inv : 0.0f;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = (x[j].get(e) - mean) * rstd;
          const float gw = dy[j].get(e) * w[j].get(e);
          o[e] = (fmaf(-xh, c1, gw) - c2) * rstd;
        }
        store_row<XB>(p.y, row * D, 8 * (j * T + t), D, o);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = nx[j];
      dy[j] = ndy[j];
    }
    mean = nmean;
    rstd = nrstd;
  }
  // groups in ascending order
  auto gather = [&](float (&acc)[NV][8]) {
    if constexpr (G > 1) {
      for (int k = 1; k < G; ++k) {
        if (g == k)
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) share[(j * T + t) * 8 + e] = acc[j][e];
        __syncthreads();
        if (g == 0)
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[j][e] += share[(j * T + t) * 8 + e];
        __syncthreads();
      }
    }
  };
  gather(dw);
  gather(db);
  if (g == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      store_row<false>(p.partials, (int64_t)blockIdx.x * 2 * D, 8 * (j * T + t), D, dw[j]);
      if (p.d_bias)
        store_row<false>(p.partials, (int64_t)(blockIdx.x * 2 + 1) * D, 8 * (j * T + t), D, db[j]);
    }
  }
}

// The blocks' column sums, added: 64 columns per workgroup, wave i takes the blocks
// i, i + 16, ... in order, then the waves in order. blockIdx.y: d_weight or d_bias.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const NormArgs p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int col = blockIdx.x * 64 + lane, D = p.width;
  float *out = blockIdx.y == 0 ? p.d_weight : p.d_bias;
  float s = 0.0f;
  if (col < D)
#pragma unroll 8
    for (int b = wave; b < p.blocks; b += 16)
      s += p.partials[((int64_t)b * 2 + blockIdx.y) * D + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    out[col] = s;
  }
}

template <int T, int NV>
const void *fwd_fn(const NormArgs &a) {
  return a.x_bf16 ? (a.w_bf16 ? (const void *)norm_fwd_kernel<true, true, T, NV>
                              : (const void *)norm_fwd_kernel<true, false, T, NV>)
                  : (a.w_bf16 ? (const void *)norm_fwd_kernel<false, true, T, NV>
                              : (const void *)norm_fwd_kernel<false, false, T, NV>);
}

template <int T, int NV, int G>
const void *bwd_fn(const NormArgs &a) {
  return a.x_bf16 ? (a.w_bf16 ? (const void *)norm_bwd_kernel<true, true, T, NV, G>
                              : (const void *)norm_bwd_kernel<true, false, T, NV, G>)
                  : (a.w_bf16 ? (const void *)norm_bwd_kernel<false, true, T, NV, G>
                              : (const void *)norm_bwd_kernel<false, false, T, NV, G>);
}

hipError_t run(const void *fn, const NormArgs &a, dim3 grid, int threads, hipStream_t stream) {
  NormArgs args = a;
  void *kargs[] = {&args};
  return hipLaunchKernel(fn, grid, dim3(threads), kargs, 0, stream);
}

}  // namespace

// Blocks of rows of a backward launch, by rows and width alone (the same bits on any device).
int norm_bwd_blocks(int64_t rows, int32_t width) {
  const int64_t most = 512;
  return (int)(rows < most ? (rows < 1 ? 1 : rows) : most);
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  int T, threads = 256;
  const void *fn;
  if (a.width <= 128) { T = 16; fn = fwd_fn<16, 1>(a); }
  else if (a.width <= 512) { T = 64; fn = fwd_fn<64, 1>(a); }
  else if (a.width <= 2048) { T = 64; fn = fwd_fn<64, 4>(a); }
  else if (a.width <= 8192) { T = 256; fn = fwd_fn<256, 4>(a); }
  else { T = threads = 1024; fn = fwd_fn<1024, 2>(a); }
  const int64_t need = (a.rows + threads / T - 1) / (threads / T);
  return run(fn, a, dim3((unsigned)(need < kFwdGrid ? need : kFwdGrid)), threads, stream);
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream) {
  int threads;
  const void *fn;
  if (a.width <= 128) { threads = 256; fn = bwd_fn<16, 1, 16>(a); }
  else if (a.width <= 512) { threads = 256; fn = bwd_fn<64, 1, 4>(a); }
  else if (a.width <= 2048) { threads = 256; fn = bwd_fn<256, 1, 1>(a); }
  else if (a.width <= 4096) { threads = 512; fn = bwd_fn<512, 1, 1>(a); }
  else if (a.width <= 8192) { threads = 1024; fn = bwd_fn<1024, 1, 1>(a); }
  else { threads = 1024; fn = bwd_fn<1024, 2, 1>(a); }
  // rows == 0: one block that writes zeros
  hipError_t e = run(fn, a, dim3((unsigned)a.blocks), threads, stream);
  if (e != hipSuccess) return e;
  return run((const void *)norm_columns_kernel, a,
             dim3((unsigned)((a.width + 63) / 64), a.d_bias ? 2 : 1), 1024, stream);
}

}  // namespace gdn
