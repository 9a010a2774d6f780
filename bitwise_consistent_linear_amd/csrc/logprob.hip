// Log-probability of the chosen token of each row of logits, and its gradient, on gfx950.
//
// Forward: bound by the one read of the logits. A workgroup takes a row; each thread keeps a
// running maximum m of its logits and, relative to it, the sums s of the exponentials and t
// of the exponentials times the differences, the next tile's loads in flight under this one's
// arithmetic; the threads' triples are then merged over lanes and waves in a fixed order. lse = scale m + log s, logp = scale (v[id] - m) - log s,
// entropy = log s - scale t / s: differences from the maximum keep what differences of large
// logits would lose. The order depends on the vocabulary alone, so a row has the same bits
// in any batch.
//
// Backward: elementwise in the logits, bound by reading them and writing the gradient: 8192 x
// 65536 bf16 with the entropy's term 348 us (6.0 TB/s), 1021 x 50021 binary32 74 us (5.3 TB/s).

#include "policy_internal.h"
#include "policy_rows.hpp"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ int64_t id_of(const LogprobArgs &p, int64_t row) {
  return p.id64 ? static_cast<const int64_t *>(p.ids)[row]
                : (int64_t)static_cast<const int32_t *>(p.ids)[row];
}

// Over some logits v (not yet scaled): their maximum m (the lowest finite value if there are
// none), s = sum(exp(scale (v - m))) and t = sum(exp(scale (v - m)) (v - m)). Differences
// come before the scale, so neither overflows a sum, and c = scale / ln 2 turns them into
// powers of two. A v of -infinity has exp 0, and its difference is held finite in t.
// kFar: a distance whose exponential is 0 for every admitted scale (>= 2^-40) and whose
// product with a count of values is finite.
constexpr float kFar = -1.0e28f;
struct Softmax {
  float m, s, t;
};

// The sums taken relative to `to` >= a.m. Where a.m is the lowest value and s is 0 they stay 0.
__device__ __forceinline__ void rebase(Softmax &a, float to, float c) {
  const float d = fmaxf(a.m - to, kFar), k = __builtin_amdgcn_exp2f(d * c);
  a.t = k * fmaf(a.s, d, a.t);
  a.s = k * a.s;
  a.m = to;
}

// The wave's lanes together, in every lane.
__device__ __forceinline__ Softmax over_lanes(Softmax a, float c) {
  rebase(a, lane_max(a.m), c);
  a.s = lane_sum<64>(a.s);
  a.t = lane_sum<64>(a.t);
  return a;
}

// Eight logits of a row at [col, col + 8), -infinity past its end.
template <bool B16>
__device__ __forceinline__ void load_logits(Vec8<B16> &v, const void *base, int64_t off,
                                            int64_t col, int64_t vocab) {
  if (col + 8 <= vocab) {
    v.load(base, off + col);
  } else {
    const int n = col < vocab ? (int)(vocab - col) : 0;
    v.load_part(base, off + col, n, kNegInf);
  }
}

constexpr int kFwdVecs = 4;

template <bool B16, bool ENT>
__global__ __launch_bounds__(512) void logprob_fwd_kernel(const LogprobArgs p) {
  __shared__ Softmax part[8];
  const int64_t row = blockIdx.x, V = p.vocab;
  const int threads = blockDim.x, lane = threadIdx.x % 64, waves = threads / 64;
  const int64_t id = id_of(p, row);
  if (id < 0 || id >= V) {
    if (threadIdx.x == 0) {
      p.logp[row] = p.lse[row] = 0.0f;
      if (ENT) p.entropy[row] = 0.0f;
    }
    return;
  }
  const int64_t off = row * p.stride;
  const float c = p.scale_log2e;
  const float chosen = B16 ? bf16_lo(static_cast<const uint16_t *>(p.logits)[off + id])
                           : static_cast<const float *>(p.logits)[off + id];
  const int64_t tile = (int64_t)threads * 8 * kFwdVecs;
  auto load = [&](Vec8<B16> (&x)[kFwdVecs], int64_t c0) {
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j)
      load_logits(x[j], p.logits, off, c0 + 8 * (int64_t)(j * threads + threadIdx.x), V);
  };
  Softmax a{kLowest, 0.0f, 0.0f};
  Vec8<B16> x[kFwdVecs], next[kFwdVecs];
  load(x, 0);
  for (int64_t c0 = 0; c0 < V; c0 += tile) {
    if (c0 + tile < V) load(next, c0 + tile);
    float top = a.m;
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, x[j].get(e));
    rebase(a, top, c);
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = x[j].get(e) - top, k = __builtin_amdgcn_exp2f(d * c);
        a.s += k;
        if (ENT) a.t = fmaf(k, fmaxf(d, kFar), a.t);
      }
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j) x[j] = next[j];
  }
  a = over_lanes(a, c);
  if (waves > 1) {
    if (lane == 0) part[threadIdx.x / 64] = a;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    a = lane < waves ? part[lane] : Softmax{kLowest, 0.0f, 0.0f};
    a = over_lanes(a, c);
  }
  if (threadIdx.x == 0) {
    const float ls = logf(a.s);
    const bool none = a.s == 0.0f;  // every logit is -inf
    p.lse[row] = none ? kNegInf : fmaf(a.m, p.scale, ls);
    p.logp[row] = none ? kNegInf : fmaf(chosen - a.m, p.scale, -ls);
    if (ENT) p.entropy[row] = none ? 0.0f : fmaf(-a.t / a.s, p.scale, ls);
  }
}

// Threads of a row, by the vocabulary alone: one tile of 32 values a thread up to 8192 values
// and 512 threads from there. 8192 rows of 65536 bf16 values take 179 us at 512 threads (6.0
// TB/s), 191 at 256 and 221 at 1024; of 2048 values 11.0 us at 64 threads, 44 at 512. A row
// by itself is bound by what one compute unit can fetch: 131072 binary32 values take 12 us.
int fwd_threads(int64_t vocab) {
  return vocab <= 2048 ? 64 : vocab <= 4096 ? 128 : vocab <= 8192 ? 256 : 512;
}

// Runs of eight values a thread: 32 bytes of either type (4096 x 65536 binary32 takes 344 us
// with one run and 372 with two, 8192 x 65536 bf16 355 with two and 402 with one).
constexpr int kBwdThreads = 256;
constexpr int bwd_vecs(bool bf16) { return bf16 ? 2 : 1; }
constexpr int bwd_span(bool bf16) { return kBwdThreads * 8 * bwd_vecs(bf16); }

template <bool B16, bool ENT>
__global__ __launch_bounds__(kBwdThreads) void logprob_bwd_kernel(const LogprobArgs p) {
  constexpr int J = bwd_vecs(B16), kSpan = bwd_span(B16);
  const int64_t V = p.vocab, spans = (V + kSpan - 1) / kSpan;
  const int64_t row = blockIdx.x / spans, c0 = (blockIdx.x % spans) * kSpan;
  const int64_t id = id_of(p, row);
  const float lse = p.lse[row];
  const bool use = id >= 0 && id < V && lse != kNegInf;
  const float scale = p.scale;
  const float g = use ? p.d_logp[row] * scale : 0.0f;
  const float h = ENT && use ? p.d_entropy[row] * scale : 0.0f;
  const float H = ENT && use ? p.entropy[row] : 0.0f;
  Vec8<B16> x[J];
  if (use) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      load_row(x[j], p.logits, row * p.stride, c0 + 8 * (j * kBwdThreads + threadIdx.x), V);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t c = c0 + 8 * (j * kBwdThreads + threadIdx.x);
    float d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
    if (use) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = fmaf(x[j].get(e), scale, -lse), q = exp_of(z);
        float k = g;
        if (ENT) k = fmaf(h, z + H, g);
        d[e] = q == 0.0f ? 0.0f : -q * k;
        if (c + e == id) d[e] += g;
      }
    }
    store_row<B16>(p.d_logits, row * V, c, V, d);
  }
}

// A launch holds at most 2^32 - 1 threads, so more rows go in several: `fn` over runs of rows
// of at most kMostThreads threads, `per` workgroups of `threads` for each row.
constexpr int64_t kMostThreads = int64_t(1) << 31;

hipError_t run(const void *fn, const LogprobArgs &a, int64_t per, int threads,
               hipStream_t stream) {
  const int64_t most = kMostThreads / (per * threads);  // at least 8: per is at most 2^20
  const int64_t bytes = a.bf16 ? 2 : 4;
  for (int64_t r = 0; r < a.rows; r += most) {
    LogprobArgs args = a;
    args.rows = a.rows - r < most ? a.rows - r : most;
    auto past = [&](const void *p, int64_t by) {
      return p ? static_cast<const char *>(p) + r * by : nullptr;
    };
    auto out = [&](float *p) { return p ? p + r : nullptr; };
    args.logits = past(a.logits, a.stride * bytes);
    args.ids = past(a.ids, a.id64 ? 8 : 4);
    args.logp = out(a.logp);
    args.lse = out(a.lse);
    args.entropy = out(a.entropy);
    args.d_logp = reinterpret_cast<const float *>(past(a.d_logp, 4));
    args.d_entropy = reinterpret_cast<const float *>(past(a.d_entropy, 4));
    args.d_logits = const_cast<char *>(past(a.d_logits, a.vocab * bytes));
    void *kargs[] = {&args};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(args.rows * per)), dim3(threads),
                                         kargs, 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int64_t bwd_spans(const LogprobArgs &a) {
  const int64_t span = bwd_span(a.bf16);
  return (a.vocab + span - 1) / span;
}

}  // namespace

hipError_t launch_logprob_fwd(const LogprobArgs &a, hipStream_t stream) {
  const void *fn = a.bf16 ? (a.entropy ? (const void *)logprob_fwd_kernel<true, true>
                                       : (const void *)logprob_fwd_kernel<true, false>)
                          : (a.entropy ? (const void *)logprob_fwd_kernel<false, true>
                                       : (const void *)logprob_fwd_kernel<false, false>);
  return run(fn, a, 1, fwd_threads(a.vocab), stream);
}

int64_t logprob_bwd_grid(const LogprobArgs &a) { return a.rows * bwd_spans(a); }

hipError_t launch_logprob_bwd(const LogprobArgs &a, hipStream_t stream) {
  const void *fn = a.bf16 ? (a.d_entropy ? (const void *)logprob_bwd_kernel<true, true>
                                         : (const void *)logprob_bwd_kernel<true, false>)
                          : (a.d_entropy ? (const void *)logprob_bwd_kernel<false, true>
                                         : (const void *)logprob_bwd_kernel<false, false>);
  return run(fn, a, bwd_spans(a), kBwdThreads, stream);
}

}  // namespace gdn
