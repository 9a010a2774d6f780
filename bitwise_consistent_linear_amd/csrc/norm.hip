// Layer norm and root-mean-square norm, forward and backward, on gfx950.
//
// Both are bound by memory: the forward reads x and writes y, the backward reads x and dy and
// writes dx. A row is held in registers, eight consecutive values (times NV) per thread, by as
// many waves as it fills (or by a row of 16 lanes up to 128 values), so the statistics take
// two passes over registers and one over memory: the mean first, then the sum of squared
// distances from it, which keeps the variance exact to a few roundings where a sum of squares
// less the squared mean would cancel. A workgroup walks over rows with the weight (and bias)
// in registers, the next row's loads in flight under the current one.
//
// Measured (bf16): forward of 16384 x 4096 45 us (6.0 TB/s), backward 78 us with its column
// sums (5.2 TB/s of the x, dy and dx that it cannot do without; a large copy reaches 4.7 to 4.9).
// Rows of odd width use the same 16-byte accesses at their element's alignment: backward of
// 4099 x 2049 binary32 24 us (4.2 TB/s: 257 of a row's 320 threads have values, and 4 us are
// the second launch).
//
// The reduction order depends on the width alone, so a row has the same bits in every batch.

#include "policy_internal.h"
#include "policy_rows.hpp"

namespace gdn {
namespace {

// Workgroups of a forward launch; more rows are walked over. Of the widest rows a workgroup of
// 1024 threads for each compute unit: 2000 x 16384 bf16 takes 25 us so and 37 with 2048 of them
// (16384 x 4096 the other way round, 45 with 2048 and 49 with 512).
constexpr int kFwdGrid = 2048, kFwdGridWide = 256, kWide = 8192;
constexpr int kBwdGrid = 256;   // blocks of rows of a backward launch

// How a row is split: threads of one row, rows at a time, threads of a workgroup.
struct Split {
  int row_threads, groups, nv;
  int threads() const { return row_threads * groups; }
};

// G: lanes that share a row, 16 or 64 (then p.row_threads / 64 waves do).
template <bool XB, bool WB, int G, int NV>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(const NormArgs p) {
  __shared__ float slot[2][1][16];
  const int T = G == 64 ? p.row_threads : G, groups = (int)blockDim.x / T;
  const int t = threadIdx.x % T, g = threadIdx.x / T, D = p.width;
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
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    settle_row(w[j], 8 * (j * T + t), D);
    if (p.bias) settle_row(b[j], 8 * (j * T + t), D);
  }
  // rows past the end repeat the last one, unwritten
  auto load = [&](Vec8<XB> (&x)[NV], int64_t row) {
    if (row >= p.rows) row = p.rows - 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) load_row(x[j], p.x, row * p.x_stride, 8 * (j * T + t), D);
  };
  const int64_t step = (int64_t)gridDim.x * groups;
  Vec8<XB> x[NV], next[NV];
  load(x, (int64_t)blockIdx.x * groups + g);
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + g;
    if (r0 + step < p.rows) load(next, row + step);
#pragma unroll
    for (int j = 0; j < NV; ++j) settle_row(x[j], 8 * (j * T + t), D);
    float mean[1] = {0.0f};
    if (layer) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) mean[0] += x[j].get(e);
      row_sums<G>(mean, T / 64, slot[0]);
      mean[0] *= inv;
    }
    float var[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int left = D - 8 * (j * T + t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < left ? x[j].get(e) - mean[0] : 0.0f;
        var[0] = fmaf(d, d, var[0]);
      }
    }
    row_sums<G>(var, T / 64, slot[1]);
    const float rstd = 1.0f / sqrtf(fmaf(var[0], inv, p.eps));
    if (row < p.rows) {
      if (t == 0) {
        if (layer) p.mean[row] = mean[0];
        p.rstd[row] = rstd;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = fmaf((x[j].get(e) - mean[0]) * rstd, w[j].get(e), b[j].get(e));
        store_row<XB>(p.y, row * D, 8 * (j * T + t), D, y);
      }
    }
    // rms writes slot[1] again without the mean's barrier in between
    if (!layer && T > 64) __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = next[j];
  }
}

// Backward of one block of rows: dx, and the block's sums of dy * xh and of dy for every
// column. Groups of T threads take rows in turn; a thread keeps its columns' sums. Blocks that
// took a run of rows each were all at the same offset of equal distances and got 4.6 TB/s
// where rows taken in turn get 5.2; holding two rows ahead or storing past the caches changed
// nothing beyond the noise.
template <bool XB, bool WB, int G, int NV>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(const NormArgs p) {
  __shared__ float slot[2][2][16];
  __shared__ float share[8 * (1024 + 8)];  // all threads' columns, where there are several groups
  const int T = G == 64 ? p.row_threads : G, groups = (int)blockDim.x / T;
  const int t = threadIdx.x % T, g = threadIdx.x / T, D = p.width;
  const bool layer = p.layer;
  const float inv = 1.0f / (float)D;
  Vec8<WB> w[NV];
  float dw[NV][8], db[NV][8];
  constexpr bool kAhead = NV == 1;  // with NV = 2 the next row would not fit the registers
  auto load_weight = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_row(w[j], p.weight, 0, 8 * (j * T + t), D);
  };
  auto settle_weight = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j) settle_row(w[j], 8 * (j * T + t), D);
  };
  if (kAhead) load_weight();
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.0f;
  // blocks take groups of rows in turn, so that together they walk through memory in order
  const int64_t step = (int64_t)gridDim.x * groups;
  struct Row {
    Vec8<XB> x[NV], dy[NV];
    float mean, rstd;
  };
  auto load = [&](Row &r, int64_t row) {  // past the end the last one again, unused
    if (row >= p.rows) row = p.rows - 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_row(r.x[j], p.x, row * p.x_stride, 8 * (j * T + t), D);
      load_row(r.dy[j], p.dy, row * p.dy_stride, 8 * (j * T + t), D);
    }
    r.mean = layer ? p.mean[row] : 0.0f;
    r.rstd = p.rstd[row];
  };
  Row cur, next;
  if (kAhead && p.rows > 0) load(cur, (int64_t)blockIdx.x * groups + g);
  if (kAhead) settle_weight();
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += step, par ^= 1) {
    const int64_t row = r0 + g;
    if (kAhead) {
      if (r0 + step < p.rows) load(next, row + step);
    } else {
      load(cur, row);
      load_weight();
      settle_weight();
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      settle_row(cur.x[j], 8 * (j * T + t), D, cur.mean);
      if constexpr (G == 16)
        if (D < 8) cur.x[j].fill_from(D - 8 * t, cur.mean);
      settle_row(cur.dy[j], 8 * (j * T + t), D);
    }
    // Sums of g xh and of g. Past the row's end dy is 0 and x the mean: with x 0 there, xh would be
    // -mean rstd, an infinity in a row of equal large values, and 0 times it would reach the sums.
    // A bf16 x is the mean cut to its upper half: where mean rstd passes the range the row's values
    // are equal, so the mean is one of them and the cut takes nothing. (A choice of xh = 0 for every
    // value took 87.9 us for 16384 x 4095 bf16, this 84.6.)
    float c[2] = {0.0f, 0.0f};
    float xh[NV][8], gw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = cur.dy[j].get(e);
        xh[j][e] = (cur.x[j].get(e) - cur.mean) * cur.rstd;
        gw[j][e] = d * w[j].get(e);
        c[0] = fmaf(gw[j][e], xh[j][e], c[0]);
        c[1] += gw[j][e];
        if (row < p.rows) {
          dw[j][e] = fmaf(d, xh[j][e], dw[j][e]);
          db[j][e] += d;
        }
      }
    row_sums<G>(c, T / 64, slot[par]);
    const float rs = cur.rstd, c1 = c[0] * inv * rs, c2 = layer ? c[1] * inv * rs : 0.0f;
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(-xh[j][e], c1, fmaf(gw[j][e], rs, -c2));
        store_row<XB>(p.y, row * D, 8 * (j * T + t), D, o);
      }
    }
    if (kAhead) cur = next;
  }
  // the columns of all groups, groups in ascending order, into the block's row of sums
  auto put = [&](float (&acc)[NV][8], int64_t at) {
    if (groups == 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) store_row<false>(p.partials, at, 8 * (j * T + t), D, acc[j]);
      return;
    }
    // several groups hold one run of eight columns a thread (NV = 1): value e of a thread at
    // e * (threads + 8), so that neither its neighbours' nor a column's neighbours share banks
    const int stride = (int)blockDim.x + 8;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) share[e * stride + threadIdx.x] = acc[0][e];
    __syncthreads();
    for (int col = threadIdx.x; col < D; col += blockDim.x) {
      const float *own = share + col % 8 * stride + col / 8;
      float s = own[0];
#pragma unroll 8
      for (int k = 1; k < groups; ++k) s += own[k * T];
      p.partials[at + col] = s;
    }
  };
  put(dw, (int64_t)blockIdx.x * 2 * D);
  if (p.d_bias) put(db, (int64_t)(blockIdx.x * 2 + 1) * D);
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

template <int G, int NV>
const void *fwd_fn(const NormArgs &a) {
  return a.x_bf16 ? (a.w_bf16 ? (const void *)norm_fwd_kernel<true, true, G, NV>
                              : (const void *)norm_fwd_kernel<true, false, G, NV>)
                  : (a.w_bf16 ? (const void *)norm_fwd_kernel<false, true, G, NV>
                              : (const void *)norm_fwd_kernel<false, false, G, NV>);
}

template <int G, int NV>
const void *bwd_fn(const NormArgs &a) {
  return a.x_bf16 ? (a.w_bf16 ? (const void *)norm_bwd_kernel<true, true, G, NV>
                              : (const void *)norm_bwd_kernel<true, false, G, NV>)
                  : (a.w_bf16 ? (const void *)norm_bwd_kernel<false, true, G, NV>
                              : (const void *)norm_bwd_kernel<false, false, G, NV>);
}

// Eight values a thread up to `single` values of a row, sixteen above; a row of 16 lanes for 128
// values and less. `most` threads of a workgroup where a row needs fewer. The forward takes two
// runs of eight from 4096 on: 8192 x 8192 bf16 43 us so, 61 with 1024 threads a row; the backward,
// which has the columns' sums in registers too, from 8192 on.
constexpr int kFwdSingle = 4096, kBwdSingle = 8192;
Split split_of(int width, int most, int single) {
  Split s;
  s.nv = width <= single ? 1 : 2;
  const int vecs = (width + 8 * s.nv - 1) / (8 * s.nv);
  s.row_threads = vecs <= 16 ? 16 : (vecs + 63) / 64 * 64;
  s.groups = s.row_threads >= most ? 1 : most / s.row_threads;
  return s;
}

hipError_t run(const void *fn, const NormArgs &a, dim3 grid, int threads, hipStream_t stream) {
  NormArgs args = a;
  void *kargs[] = {&args};
  return hipLaunchKernel(fn, grid, dim3(threads), kargs, 0, stream);
}

}  // namespace

// Blocks of a backward launch, by rows and width alone (the same bits on any device). More
// blocks than compute units only add partial sums to write and read: 16384 x 4096 bf16 took
// 88.6 us with 256 blocks of two rows at a time, 93.0 with 512 and 99.9 with 1024.
int norm_bwd_blocks(int64_t rows, int32_t width) {
  const int groups = split_of(width, 1024, kBwdSingle).groups;
  const int64_t need = (rows + groups - 1) / groups;
  return (int)(need < 1 ? 1 : need < kBwdGrid ? need : kBwdGrid);  // no rows: one writes zeros
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const Split s = split_of(a.width, 256, kFwdSingle);
  NormArgs args = a;
  args.row_threads = s.row_threads;
  const void *fn = s.row_threads == 16 ? fwd_fn<16, 1>(a) : s.nv == 1 ? fwd_fn<64, 1>(a)
                                                                      : fwd_fn<64, 2>(a);
  const int64_t need = (a.rows + s.groups - 1) / s.groups;
  const int64_t most = a.width > kWide ? kFwdGridWide : kFwdGrid;
  return run(fn, args, dim3((unsigned)(need < most ? need : most)), s.threads(), stream);
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream) {
  const Split s = split_of(a.width, 1024, kBwdSingle);
  NormArgs args = a;
  args.row_threads = s.row_threads;
  const void *fn = s.row_threads == 16 ? bwd_fn<16, 1>(a) : s.nv == 1 ? bwd_fn<64, 1>(a)
                                                                      : bwd_fn<64, 2>(a);
  hipError_t e = run(fn, args, dim3((unsigned)a.blocks), s.threads(), stream);
  if (e != hipSuccess) return e;
  return run((const void *)norm_columns_kernel, args,
             dim3((unsigned)((a.width + 63) / 64), a.d_bias ? 2 : 1), 1024, stream);
}

}  // namespace gdn
