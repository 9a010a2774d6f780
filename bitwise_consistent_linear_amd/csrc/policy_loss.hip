// Clipped policy loss of a packed ragged batch, and its gradient, on gfx950.
//
// A token costs two exponentials and some thirty bytes, so both directions are bound by
// latency up to millions of tokens. The ratio is compared with the clip borders and the sums
// are long, so the arithmetic is binary64 (its vector rate is far from the bound here).
//
// Forward: a wave takes 256 consecutive tokens, 4 per lane, and adds them up for each
// sequence that meets them; a pair (block of tokens, sequence) has the slot block + sequence,
// which no other pair has, since the pairs that meet form a staircase. One workgroup then adds
// each sequence's slots in order, forms the weights and the loss. No atomics: the same bits
// on every launch. Backward: elementwise, each token's sequence found from its wave's first.

#include "policy_internal.h"

namespace gdn {
namespace {

constexpr int kSpan = 256, kPer = kSpan / 64;  // tokens per wave and per lane
constexpr int kSums = 5;                       // pg, kl, entropy, cut, count

struct Token {
  double ratio_adv, pg, kl, kl_slope;  // r A, -gain, exp(u) - u - 1, 1 - exp(u)
  bool moves;
};

__device__ __forceinline__ Token token_terms(const PolicyArgs &p, int64_t t) {
  Token o;
  const double lp = p.logp[t], adv = p.adv[t];
  const double r = exp(lp - (double)p.old_logp[t]);
  const double clamped = r < p.lo ? p.lo : (r > p.hi ? p.hi : r);
  const double plain = r * adv, clipped = clamped * adv;
  o.ratio_adv = plain;
  o.moves = plain <= clipped;
  double gain = o.moves ? plain : clipped;
  if (p.dual > 0.0 && adv < 0.0 && gain < p.dual * adv) {
    gain = p.dual * adv;
    o.moves = false;
  }
  o.pg = -gain;
  o.kl = 0.0;
  o.kl_slope = 0.0;
  if (p.ref) {
    const double u = (double)p.ref[t] - lp, e = exp(u);
    o.kl = e - u - 1.0;
    o.kl_slope = 1.0 - e;
  }
  return o;
}

// Start of sequence n, clamped to [0, tokens]; n == seqs gives the end of the last one.
__device__ __forceinline__ int64_t start_of(const PolicyArgs &p, int64_t n) {
  if (!p.cu) return n == 0 ? 0 : p.tokens;
  const int64_t v = p.cu[n];
  return v < 0 ? 0 : (v > p.tokens ? p.tokens : v);
}

// The last sequence that starts at or before token t (sequences of no tokens before it are
// passed over): the one that holds t if any does.
__device__ __forceinline__ int64_t find_seq(const PolicyArgs &p, int64_t t) {
  int64_t lo = 0, hi = p.seqs - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (start_of(p, mid) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s > 0; s /= 2) v += __shfl_xor(v, s, 64);
  return v;
}

__global__ __launch_bounds__(256) void policy_tokens_kernel(const PolicyArgs p) {
  const int64_t block = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  const int64_t t0 = block * kSpan;
  if (t0 >= p.tokens) return;
  const int64_t t1 = t0 + kSpan < p.tokens ? t0 + kSpan : p.tokens;
  double v[kPer][4];
  bool use[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t t = t0 + 64 * j + lane;
    use[j] = t < t1 && (!p.mask || p.mask[t]);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j][k] = 0.0;
    if (use[j]) {
      const Token o = token_terms(p, t);
      v[j][0] = o.pg;
      v[j][1] = o.kl;
      v[j][2] = p.entropy ? (double)p.entropy[t] : 0.0;
      v[j][3] = o.moves ? 0.0 : 1.0;
    }
  }
  // cu_seqlens that fall are clamped: a slot is written for every sequence from the first
  // that meets the block on, within the slots there are
  for (int64_t n = find_seq(p, t0); n < p.seqs; ++n) {
    const int64_t s = start_of(p, n);
    if (s >= t1) break;
    const int64_t e = start_of(p, n + 1);
    if (e <= s || e <= t0) continue;
    double sum[kSums] = {0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t t = t0 + 64 * j + lane;
      if (use[j] && t >= s && t < e) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] += v[j][k];
        sum[4] += 1.0;
      }
    }
#pragma unroll
    for (int k = 0; k < kSums; ++k) sum[k] = wave_sum(sum[k]);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) p.partials[k * p.slots + block + n] = sum[k];
    }
  }
}

// Sum over a workgroup of 1024 threads, in every thread, waves in order.
__device__ __forceinline__ double group_sum(double v, double *slot) {
  v = wave_sum(v);
  __syncthreads();
  if (threadIdx.x % 64 == 0) slot[threadIdx.x / 64] = v;
  __syncthreads();
  double s = slot[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) s += slot[i];
  return s;
}

__global__ __launch_bounds__(1024) void policy_finish_kernel(const PolicyArgs p) {
  __shared__ double slot[16];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  constexpr int kFew = 8;  // a sequence of at most so many slots is one thread's, else a wave's
  double count = 0.0, live = 0.0;
  for (int64_t n = tid; n < p.seqs; n += 1024) {
    const int64_t s = start_of(p, n), e = start_of(p, n + 1);
    const int64_t lo = s / kSpan + n, hi = e > s ? (e - 1) / kSpan + n : lo - 1;
    if (hi - lo >= kFew) continue;
    for (int k = 0; k < kSums; ++k) {
      double v = 0.0;
      for (int64_t i = lo; i <= hi; ++i) v += p.partials[k * p.slots + i];
      p.seq_sums[k * p.seqs + n] = v;
    }
  }
  for (int64_t n = wave; n < p.seqs; n += 16) {
    const int64_t s = start_of(p, n), e = start_of(p, n + 1);
    const int64_t lo = s / kSpan + n, hi = e > s ? (e - 1) / kSpan + n : lo - 1;
    if (hi - lo < kFew) continue;
    for (int k = 0; k < kSums; ++k) {
      double v = 0.0;
      for (int64_t i = lo + lane; i <= hi; i += 64) v += p.partials[k * p.slots + i];
      v = wave_sum(v);
      if (lane == 0) p.seq_sums[k * p.seqs + n] = v;
    }
  }
  __syncthreads();
  for (int64_t n = tid; n < p.seqs; n += 1024) {
    const double c = p.seq_sums[4 * p.seqs + n];
    count += c;
    live += c > 0.0 ? 1.0 : 0.0;
  }
  count = group_sum(count, slot);
  live = group_sum(live, slot);
  double out[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t n = tid; n < p.seqs; n += 1024) {
    const double c = p.seq_sums[4 * p.seqs + n];
    const double w = c > 0.0 ? (p.by_sequence ? 1.0 / (c * live) : 1.0 / count) : 0.0;
    p.seq_weight[n] = (float)w;
    if (c > 0.0)
      for (int k = 0; k < 4; ++k) out[k] += w * p.seq_sums[k * p.seqs + n];
  }
  for (int k = 0; k < 4; ++k) out[k] = group_sum(out[k], slot);
  if (tid == 0) {
    p.stats[0] = (float)(out[0] + p.kl_coef * out[1] - p.entropy_coef * out[2]);
    for (int k = 0; k < 4; ++k) p.stats[k + 1] = (float)out[k];
  }
}

__global__ __launch_bounds__(256) void policy_grad_kernel(const PolicyArgs p) {
  const int64_t block = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  const int64_t t0 = block * kSpan;
  if (t0 >= p.tokens) return;
  int64_t n = find_seq(p, t0);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t t = t0 + 64 * j + lane;
    if (t >= p.tokens) break;
    while (n + 1 < p.seqs && start_of(p, n + 1) <= t) ++n;
    const bool in = t >= start_of(p, n) && t < start_of(p, n + 1);
    float dl = 0.0f, de = 0.0f;
    if (in && (!p.mask || p.mask[t])) {
      const Token o = token_terms(p, t);
      const double w = (double)p.weight[n] * p.d_loss;
      dl = (float)(w * (p.kl_coef * o.kl_slope - (o.moves ? o.ratio_adv : 0.0)));
      de = (float)(-w * p.entropy_coef);
    }
    p.d_logp[t] = dl;
    if (p.d_entropy) p.d_entropy[t] = de;
  }
}

hipError_t run(const void *fn, const PolicyArgs &a, int64_t grid, int threads,
               hipStream_t stream) {
  PolicyArgs args = a;
  void *kargs[] = {&args};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(threads), kargs, 0, stream);
}

}  // namespace

int64_t policy_slots(int64_t tokens, int64_t seqs) { return (tokens + kSpan - 1) / kSpan + seqs; }

hipError_t launch_policy_fwd(const PolicyArgs &a, hipStream_t stream) {
  const int64_t blocks = (a.tokens + kSpan - 1) / kSpan;
  if (blocks > 0) {
    const hipError_t e = run((const void *)policy_tokens_kernel, a, (blocks + 3) / 4, 256, stream);
    if (e != hipSuccess) return e;
  }
  return run((const void *)policy_finish_kernel, a, 1, 1024, stream);
}

hipError_t launch_policy_bwd(const PolicyArgs &a, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t blocks = (a.tokens + kSpan - 1) / kSpan;
  return run((const void *)policy_grad_kernel, a, (blocks + 3) / 4, 256, stream);
}

}  // namespace gdn
