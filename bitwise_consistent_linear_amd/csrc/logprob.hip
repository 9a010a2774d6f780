// Log-probability of the chosen token of each row of logits, and its gradient, on gfx950.
//
// Forward: bound by the one read of the logits (8192 x 65536 bf16 with entropies 168 us, 6.0
// TB/s). A workgroup takes a row; each thread keeps a running maximum m of its logits and,
// relative to it, the sums s of the exponentials and t of the exponentials times the
// differences, the next tile's loads in flight under this one's arithmetic; the threads' triples
// are then merged over lanes and waves in a fixed order. lse = scale m + log s, logp =
// scale (v[id] - m) - log s, entropy = log s - scale t / s: differences from the maximum keep
// what differences of large logits would lose. A few rows of a long vocabulary are split over
// workgroups at fixed places where the sums begin anew in either way, so the order depends on
// the vocabulary alone and a row has the same bits in any batch.
//
// Backward: elementwise in the logits, bound by reading them and writing the gradient: 8192 x
// 65536 bf16 with the entropy's term 338 us (6.2 TB/s), 1021 x 50021 binary32 73 us (5.4 TB/s).
// It takes differences too: from the lse where that is next to zero, else from the row's maximum.

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

// Two sets of logits together.
__device__ __forceinline__ void merge(Softmax &a, Softmax b, float c) {
  const float top = fmaxf(a.m, b.m);
  rebase(a, top, c);
  rebase(b, top, c);
  a.s += b.s;
  a.t += b.t;
}

// Runs of eight logits into a.
template <bool ENT, bool B16, int N>
__device__ __forceinline__ void add_values(Softmax &a, const Vec8<B16> (&x)[N], float c) {
  float top = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, x[j].get(e));
  rebase(a, top, c);
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = x[j].get(e) - top, k = __builtin_amdgcn_exp2f(d * c);
      a.s += k;
      if (ENT) a.t = fmaf(k, fmaxf(d, kFar), a.t);
    }
}

// A thread's 32 logits of a tile: four runs of eight, `threads` runs apart, -infinity past the
// row's end.
constexpr int kFwdVecs = 4;
template <bool B16>
struct Tile {
  Vec8<B16> x[kFwdVecs];
  __device__ __forceinline__ static int64_t col(int64_t c0, int j) {
    return c0 + 8 * (int64_t)(j * (int)blockDim.x + (int)threadIdx.x);
  }
  __device__ __forceinline__ void load(const LogprobArgs &p, int64_t off, int64_t c0) {
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j) x[j].load(p.logits, off + col(c0, j));
  }
  // the row's last tile, not a whole one
  __device__ __forceinline__ void load_last(const LogprobArgs &p, int64_t off, int64_t c0) {
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j)
      load_row(x[j], p.logits, off, col(c0, j), p.vocab, kNegInf);
#pragma unroll
    for (int j = 0; j < kFwdVecs; ++j) settle_row(x[j], col(c0, j), p.vocab, kNegInf);
  }
};

// Tiles that a thread adds up from nothing before it merges the sum into its row's: 65536
// values of a workgroup of 512 threads. Rows of more can be split there with the same bits.
constexpr int kGroupTiles = 4, kMostFwdThreads = 512;
constexpr int64_t kGroupValues = (int64_t)kGroupTiles * kMostFwdThreads * 8 * kFwdVecs;

// A thread's logits of a row from `from` to `end`, groups of tiles in turn.
template <bool B16, bool ENT>
__device__ __forceinline__ Softmax thread_sums(const LogprobArgs &p, int64_t off, int64_t from,
                                               int64_t end) {
  const int64_t tile = (int64_t)blockDim.x * 8 * kFwdVecs;
  const float c = p.scale_log2e;
  Softmax a{kLowest, 0.0f, 0.0f}, g = a;
  Tile<B16> x, next;
  int tiles = 0;
  auto add = [&]() {
    add_values<ENT>(g, x.x, c);
    if (++tiles == kGroupTiles) {
      merge(a, g, c);
      g = Softmax{kLowest, 0.0f, 0.0f};
      tiles = 0;
    }
  };
  int64_t c0 = from;
  if (c0 + tile <= end) x.load(p, off, c0);
  for (; c0 + tile <= end; c0 += tile) {
    if (c0 + 2 * tile <= end) next.load(p, off, c0 + tile);
    add();
    x = next;
  }
  if (c0 < end) {
    x.load_last(p, off, c0);
    add();
  }
  if (tiles > 0) merge(a, g, c);
  return a;
}

__device__ __forceinline__ bool scored(const LogprobArgs &p, int64_t id) {
  return id >= 0 && id < p.vocab;
}

__device__ __forceinline__ float logit_of(const LogprobArgs &p, int64_t at) {
  return p.bf16 ? bf16_lo(static_cast<const uint16_t *>(p.logits)[at])
                : static_cast<const float *>(p.logits)[at];
}

// The outputs of a row from all its logits and the chosen one; none: it is not scored.
template <bool ENT>
__device__ __forceinline__ void put_row(const LogprobArgs &p, int64_t row, bool none, Softmax a,
                                        float chosen) {
  const float ls = logf(a.s);
  const bool empty = a.s == 0.0f;  // every logit is -inf
  p.lse[row] = none ? 0.0f : empty ? kNegInf : fmaf(a.m, p.scale, ls);
  p.logp[row] = none ? 0.0f : empty ? kNegInf : fmaf(chosen - a.m, p.scale, -ls);
  if (ENT) p.entropy[row] = none || empty ? 0.0f : fmaf(-a.t / a.s, p.scale, ls);
}

// The threads' sums of a row together and its outputs: lanes, then waves.
template <bool ENT>
__device__ __forceinline__ void finish_row(const LogprobArgs &p, int64_t row, Softmax a,
                                           float chosen) {
  __shared__ Softmax part[8];
  const int lane = threadIdx.x % 64, waves = (int)blockDim.x / 64;
  const float c = p.scale_log2e;
  a = over_lanes(a, c);
  if (waves > 1) {
    if (lane == 0) part[threadIdx.x / 64] = a;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    a = over_lanes(lane < waves ? part[lane] : Softmax{kLowest, 0.0f, 0.0f}, c);
  }
  if (threadIdx.x == 0) put_row<ENT>(p, row, false, a, chosen);
}

// A row by a workgroup.
template <bool B16, bool ENT>
__global__ __launch_bounds__(kMostFwdThreads) void logprob_fwd_kernel(const LogprobArgs p) {
  const int64_t row = blockIdx.x, id = id_of(p, row);
  if (!scored(p, id)) {
    if (threadIdx.x == 0) put_row<ENT>(p, row, true, Softmax{0.0f, 0.0f, 0.0f}, 0.0f);
    return;
  }
  const int64_t off = row * p.stride;
  const float chosen = logit_of(p, off + id);
  finish_row<ENT>(p, row, thread_sums<B16, ENT>(p, off, 0, p.vocab), chosen);
}

// A group of tiles of a row by a workgroup, its threads' sums put down for the next kernel:
// 6 KiB for the group's 128 or 256.
template <bool B16, bool ENT>
__global__ __launch_bounds__(kMostFwdThreads) void logprob_groups_kernel(const LogprobArgs p) {
  const int64_t row = blockIdx.x / p.groups, from = blockIdx.x % p.groups * kGroupValues;
  if (!scored(p, id_of(p, row))) return;
  const int64_t end = p.vocab - from < kGroupValues ? p.vocab : from + kGroupValues;
  const Softmax a = thread_sums<B16, ENT>(p, row * p.stride, from, end);
  float *part = p.parts + (int64_t)blockIdx.x * 3 * kMostFwdThreads + threadIdx.x;
  part[0] = a.m;
  part[kMostFwdThreads] = a.s;
  if (ENT) part[2 * kMostFwdThreads] = a.t;
}

// The groups of a row together, each thread's in turn as the kernel of a whole row adds them:
// the same bits.
template <bool ENT>
__global__ __launch_bounds__(kMostFwdThreads) void logprob_join_kernel(const LogprobArgs p) {
  const int64_t row = blockIdx.x, id = id_of(p, row);
  if (!scored(p, id)) {
    if (threadIdx.x == 0) put_row<ENT>(p, row, true, Softmax{0.0f, 0.0f, 0.0f}, 0.0f);
    return;
  }
  const float c = p.scale_log2e, chosen = logit_of(p, row * p.stride + id);
  const float *part = p.parts + row * p.groups * 3 * kMostFwdThreads + threadIdx.x;
  Softmax a{kLowest, 0.0f, 0.0f};
#pragma unroll 8
  for (int64_t g = 0; g < p.groups; ++g, part += 3 * kMostFwdThreads)
    merge(a, Softmax{part[0], part[kMostFwdThreads], ENT ? part[2 * kMostFwdThreads] : 0.0f}, c);
  finish_row<ENT>(p, row, a, chosen);
}

// Threads of a row, by the vocabulary alone: as many tiles of 32 values a thread as 512 threads
// would need, spread evenly, and 512 threads beyond a group. 8192 rows of 65536 bf16 values take
// 169 us at 512 threads (6.0 TB/s), 191 at 256 and 221 at 1024; 4096 rows of 20000 29 us in two
// tiles of 320 threads, 40 in one of 512 and a rest; of 2048 values 11.0 us at 64, 44 at 512.
int fwd_threads(int64_t vocab) {
  constexpr int64_t kMost = kMostFwdThreads * 8 * kFwdVecs;
  if (vocab > kGroupValues) return kMostFwdThreads;
  const int64_t tiles = (vocab + kMost - 1) / kMost, each = (vocab + tiles - 1) / tiles;
  return (int)((each + 64 * 8 * kFwdVecs - 1) / (64 * 8 * kFwdVecs)) * 64;
}
// Runs of eight values a thread: 32 bytes of either type (4096 x 65536 binary32 takes 342 us
// with one run and 363 with two, 8192 x 65536 bf16 345 with two and 405 with one).
constexpr int kBwdThreads = 256;
constexpr int bwd_vecs(bool bf16) { return bf16 ? 2 : 1; }
constexpr int bwd_span(bool bf16) { return kBwdThreads * 8 * bwd_vecs(bf16); }

// Rows whose |lse| is below this take log p = scale x - lse with the lse of the forward, whose
// rounding (half a step, at most 2^-19) is then no more than the exponential's own of a distance
// of 32. In an lse far from zero the logarithm of the sum is lost, or it is past binary32's range,
// so such a row's maximum and sum are formed again and log p = scale (x - max) - log(sum).
constexpr float kNearLse = 64.0f;

// Maximum and sum of the exponentials of a row by a workgroup, in every thread.
template <bool B16>
__device__ __forceinline__ Softmax row_again(const LogprobArgs &p, int64_t off) {
  constexpr int J = bwd_vecs(B16), kWaves = kBwdThreads / 64;
  __shared__ Softmax part[kWaves];
  const float c = p.scale_log2e;
  Softmax a{kLowest, 0.0f, 0.0f};
  for (int64_t c0 = 0; c0 < p.vocab; c0 += bwd_span(B16)) {
    Vec8<B16> x[J];
    auto col = [&](int j) { return c0 + 8 * (j * kBwdThreads + (int)threadIdx.x); };
#pragma unroll
    for (int j = 0; j < J; ++j) load_row(x[j], p.logits, off, col(j), p.vocab, kNegInf);
#pragma unroll
    for (int j = 0; j < J; ++j) settle_row(x[j], col(j), p.vocab, kNegInf);
    add_values<false>(a, x, c);
  }
  a = over_lanes(a, c);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = a;
  __syncthreads();
  a = part[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) merge(a, part[i], c);
  return a;
}

// What a row's gradient is made of: scale d_logp, scale d_entropy, the entropy.
struct RowGrad {
  float g, h, H;
};

// The gradient of the span of a row that begins at c0, with log p = scale (x - m) - ls; zeros
// where the row is not used.
template <bool B16, bool ENT>
__device__ __forceinline__ void put_gradient(const LogprobArgs &p, int64_t row, int64_t id,
                                             bool use, RowGrad r, float m, float ls, int64_t c0) {
  constexpr int J = bwd_vecs(B16);
  const int64_t V = p.vocab;
  const float scale = p.scale;
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
      settle_row(x[j], c, V);
      const int at = id >= c && id < c + 8 ? (int)(id - c) : -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = fmaf(x[j].get(e) - m, scale, -ls), q = exp_of(z);
        float k = r.g;
        if (ENT) k = fmaf(r.h, z + r.H, r.g);
        d[e] = q == 0.0f ? 0.0f : -q * k;
        if (e == at) d[e] += r.g;
      }
    }
    store_row<B16>(p.d_logits, row * V, c, V, d);
  }
}

// A workgroup takes a span of a row. All of a row far from zero is one workgroup's, and the row's
// others have nothing to do; which one it is changes with the row so that they spread over the
// XCDs, which take workgroups in turn (8192 x 65536 bf16 674 us where near rows take 337, and
// 4600 with the first workgroup of every row; 8 x 131072 binary32 55 and 4). The registers of the
// far rows' loops are the near ones' too: with 66 of them 64 x 131072 bf16 near zero took 8.2 us,
// with 34 7.2. The row's values are read before the branch, where they are scalar loads: after
// it, through the vector memory, the 337 us were 356.
template <bool B16, bool ENT>
__global__ __launch_bounds__(kBwdThreads) void logprob_bwd_kernel(const LogprobArgs p) {
  constexpr int kSpan = bwd_span(B16);
  const int64_t spans = (p.vocab + kSpan - 1) / kSpan;
  const int64_t row = blockIdx.x / spans, span = blockIdx.x % spans;
  const int64_t id = id_of(p, row);
  const float lse = p.lse[row];
  const bool use = scored(p, id);
  RowGrad r{0.0f, 0.0f, 0.0f};
  if (use) {
    r.g = p.d_logp[row] * p.scale;
    if (ENT) r.h = p.d_entropy[row] * p.scale;
    if (ENT) r.H = p.entropy[row];
  }
  if (__builtin_expect(!use || fabsf(lse) < kNearLse, 1)) {
    put_gradient<B16, ENT>(p, row, id, use, r, 0.0f, lse, span * kSpan);
    return;
  }
  const int64_t low = spans % 8 == 0 ? 8 : spans & -spans;  // row * spans mod 8: 8 / low places
  if (span != row * low / 8 % spans) return;
  const Softmax a = row_again<B16>(p, row * p.stride);
  const bool any = a.s != 0.0f;  // else every logit is -infinity; a NaN stays
  const float ls = logf(a.s);
  for (int64_t c0 = 0; c0 < p.vocab; c0 += kSpan)
    put_gradient<B16, ENT>(p, row, id, any, r, a.m, ls, c0);
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
    args.parts = a.parts ? a.parts + r * a.groups * 3 * kMostFwdThreads : nullptr;
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

// Groups that a row is split into, 0 where a workgroup takes it whole. A row by itself is bound
// by the arithmetic of its compute unit (1.2 us for 16384 values of either type), so a few long
// rows leave the others idle; the second kernel costs 3 us. 8 rows in the two ways, whole and
// split: of 131072 binary32 values 10.1 and 9.2 us, of 262144 21.6 and 11.2, of 300001 25.7
// and 11.4; 64 rows of 262144 25.0 and 16.8, 128 rows 26.7 and 26.2, 256 rows 41 and 45.
int64_t split_groups(const LogprobArgs &a) {
  const bool split = a.rows <= 64 && a.vocab > kGroupValues / 2 * 3;
  return split ? (a.vocab + kGroupValues - 1) / kGroupValues : 0;
}

int64_t logprob_parts_bytes(const LogprobArgs &a) {
  return a.rows * split_groups(a) * 3 * kMostFwdThreads * (int64_t)sizeof(float);
}

hipError_t launch_logprob_fwd(const LogprobArgs &a, hipStream_t stream) {
  LogprobArgs args = a;
  args.groups = split_groups(a);
  if (args.groups > 0) {
    const void *fn = a.bf16 ? (a.entropy ? (const void *)logprob_groups_kernel<true, true>
                                         : (const void *)logprob_groups_kernel<true, false>)
                            : (a.entropy ? (const void *)logprob_groups_kernel<false, true>
                                         : (const void *)logprob_groups_kernel<false, false>);
    const hipError_t e = run(fn, args, args.groups, kMostFwdThreads, stream);
    if (e != hipSuccess) return e;
    return run(a.entropy ? (const void *)logprob_join_kernel<true>
                         : (const void *)logprob_join_kernel<false>,
               args, 1, kMostFwdThreads, stream);
  }
  const void *fn = a.bf16 ? (a.entropy ? (const void *)logprob_fwd_kernel<true, true>
                                       : (const void *)logprob_fwd_kernel<true, false>)
                          : (a.entropy ? (const void *)logprob_fwd_kernel<false, true>
                                       : (const void *)logprob_fwd_kernel<false, false>);
  return run(fn, args, 1, fwd_threads(a.vocab), stream);
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
