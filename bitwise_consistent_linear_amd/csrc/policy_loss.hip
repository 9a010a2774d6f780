// Clipped policy loss of a packed ragged batch, and its gradient, on gfx950.
//
// A token costs two exponentials and some thirty bytes, so both directions are bound by
// latency up to millions of tokens. The ratio is compared with the clip borders and the sums
// are long, so the arithmetic is binary64 (its vector rate is far from the bound here).
//
// Forward: a wave takes a span of consecutive tokens, 256 at a time and 4 per lane, and adds
// them up for each sequence that meets the span; a pair (span, sequence) has the slot span +
// sequence, which no other pair has, since the pairs that meet form a staircase. One workgroup
// then adds each sequence's slots (a grid before it, of more than 512 sequences), forms the
// weights and the loss. No atomics: the same bits on every launch. Backward: elementwise, each token's sequence found from its
// wave's first.
//
// What a wave waits for is memory: it issues all loads of its tokens first and finds its first
// sequence by a search of 64 lanes (one round of loads for 64 sequences, two for 4096), the
// last round's starts held in its lanes. 262144 tokens in 64 sequences: tokens 6.0 us,
// finish 6.2, gradient 6.3; 16384 in 4: 5.5, 4.5 and 5.8, of which a kernel that does nothing
// would take 2 to 3 each.

#include "policy_internal.h"

namespace gdn {
namespace {

constexpr int kChunk = 256, kPer = kChunk / 64;  // tokens of a wave at a time, and per lane
constexpr int kSums = 5;                         // pg, kl, entropy, cut, count
constexpr int64_t kMostSpans = 4096;             // longer batches have longer spans

int64_t span_of(int64_t tokens) {  // tokens of a wave, by their number alone
  const int64_t chunks = (tokens + kChunk - 1) / kChunk;
  return kChunk * (chunks > kMostSpans ? (chunks + kMostSpans - 1) / kMostSpans : 1);
}

struct Inputs {  // of one token
  float logp, old, adv, ref, entropy;
  bool use;
};

struct Token {
  double ratio_adv, pg, kl, kl_slope;  // r A, -gain, exp(u) - 1 - u, 1 - exp(u)
  bool moves;
};

// Tokens past `end` are not used; nothing of them is read.
__device__ __forceinline__ Inputs load_token(const PolicyArgs &p, int64_t t, int64_t end,
                                             bool want_entropy) {
  Inputs v{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, false};
  if (t < end) {
    v.logp = p.logp[t];
    v.old = p.old_logp[t];
    v.adv = p.adv[t];
    if (p.ref) v.ref = p.ref[t];
    if (want_entropy && p.entropy) v.entropy = p.entropy[t];
    v.use = !p.mask || p.mask[t];
  }
  return v;
}

__device__ __forceinline__ Token token_terms(const PolicyArgs &p, const Inputs &v) {
  Token o;
  const double lp = v.logp, adv = v.adv;
  const double r = exp(lp - (double)v.old);
  const double clamped = r < p.lo ? p.lo : (r > p.hi ? p.hi : r);
  const double plain = r * adv, clipped = clamped * adv;
  o.ratio_adv = plain;
  o.moves = !(plain > clipped);  // a NaN stays one, in the loss and in the gradient
  double gain = o.moves ? plain : clipped;
  if (p.dual > 0.0 && adv < 0.0 && gain < p.dual * adv) {
    gain = p.dual * adv;
    o.moves = false;
  }
  o.pg = -gain;
  o.kl = 0.0;
  o.kl_slope = 0.0;
  if (p.ref) {
    // Policies near their reference have u next to 0, where exp(u) - 1 - u loses u^2 / 2 among
    // the roundings of 1: below 2^-6 six terms of the series, the next under 2^-49 of the sum.
    const double u = (double)v.ref - lp, e = exp(u);
    const double series =
        u * u * fma(u, fma(u, fma(u, fma(u, fma(u, 1.0 / 5040, 1.0 / 720), 1.0 / 120), 1.0 / 24),
                           1.0 / 6), 0.5);
    const bool near = fabs(u) < 0x1p-6;
    o.kl = near ? series : e - u - 1.0;
    o.kl_slope = near ? -(u + series) : 1.0 - e;
  }
  return o;
}

// Start of sequence n, clamped to [0, tokens]; n >= seqs gives the end of the last one.
__device__ __forceinline__ int64_t start_of(const PolicyArgs &p, int64_t n) {
  if (n > p.seqs) n = p.seqs;
  if (!p.cu) return n == 0 ? 0 : p.tokens;
  const int64_t v = p.cu[n];
  return v < 0 ? 0 : (v > p.tokens ? p.tokens : v);
}

// A cursor over the sequences that meet a wave's tokens: lane i holds the start of sequence
// first + i.
struct Starts {
  int64_t first;
  int held;
  __device__ __forceinline__ void load(const PolicyArgs &p, int64_t n) {
    first = n;
    held = (int)start_of(p, n + threadIdx.x % 64);
  }
  // The last sequence that starts at or before token t (sequences of no tokens before it are
  // passed over): the one that holds t if any does. Uniform over the wave; 64 starts a round,
  // those of the last round held.
  __device__ __forceinline__ int64_t seek(const PolicyArgs &p, int64_t t) {
    int64_t lo = 0, len = p.seqs;  // the answer is in [lo, lo + len)
    while (len > 64) {
      const int64_t step = (len + 63) / 64, at = lo + step * (int64_t)(threadIdx.x % 64);
      const int below = __popcll(__ballot(at < lo + len && start_of(p, at) <= t));
      const int64_t end = lo + len;
      lo += step * (below > 0 ? below - 1 : 0);
      len = end - lo < step ? end - lo : step;
    }
    load(p, lo);
    const int below = __popcll(__ballot((int64_t)(threadIdx.x % 64) < len && held <= t));
    return lo + (below > 0 ? below - 1 : 0);
  }
  // start of sequence n in [first, first + 64)
  __device__ __forceinline__ int64_t at(int64_t n) const {
    return __builtin_amdgcn_readlane(held, __builtin_amdgcn_readfirstlane((int)(n - first)));
  }
  // starts of n and of the next one, with the 64 from n on held if they are not yet
  __device__ __forceinline__ void span(const PolicyArgs &p, int64_t n, int64_t &s, int64_t &e) {
    if (n - first >= 63) load(p, n);
    s = at(n);
    e = at(n + 1);
  }
};

// v plus its neighbour's by a DPP move, 0 where there is none.
template <int Ctrl, int Rows>
__device__ __forceinline__ double plus_moved(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, Ctrl, Rows, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), Ctrl, Rows, 0xF, true);
  return v + __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// Sum over each row of 16 lanes, in its last lane: runs of 2, 4, 8, 16 lanes.
__device__ __forceinline__ double row_total(double v) {
  v = plus_moved<0x111, 0xF>(v);  // from one lane below in the row, two, four, eight
  v = plus_moved<0x112, 0xF>(v);
  v = plus_moved<0x114, 0xF>(v);
  return plus_moved<0x118, 0xF>(v);
}

// Sum over the wave's lanes, in lane 63: the rows of 16, then their sums.
__device__ __forceinline__ double wave_total(double v) {
  v = row_total(v);
  v = plus_moved<0x142, 0xA>(v);  // the row before, into rows 1 and 3
  return plus_moved<0x143, 0xC>(v);  // the first two rows, into the others
}

__global__ __launch_bounds__(256) void policy_tokens_kernel(const PolicyArgs p) {
  const int64_t block = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64;
  const int64_t t0 = block * p.span;
  if (t0 >= p.tokens) return;
  const int64_t end = t0 + p.span < p.tokens ? t0 + p.span : p.tokens;
  Inputs in[kPer];
  auto load = [&](int64_t c0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) in[j] = load_token(p, c0 + 64 * j + lane, end, true);
  };
  load(t0);
  Starts starts;
  int64_t n = starts.seek(p, t0), s, e;
  starts.span(p, n, s, e);
  double sum[3] = {0.0, 0.0, 0.0};  // of the lane's tokens of sequence n so far
  int cut = 0, count = 0;           // of the wave's
  auto flush = [&]() {
    double *out = p.partials + (block + n) * kSums;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const double v = wave_total(sum[k]);
      if (lane == 63) out[k] = v;
      sum[k] = 0.0;
    }
    if (lane == 63) {
      out[3] = (double)cut;
      out[4] = (double)count;
    }
    cut = count = 0;
  };
  for (int64_t c0 = t0; c0 < end; c0 += kChunk) {
    const int64_t c1 = c0 + kChunk < end ? c0 + kChunk : end;
    if (c0 > t0) load(c0);
    Token o[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = token_terms(p, in[j]);
    // the sequences that meet [c0, c1), those that end in it put down
    while (s < c1) {
      if (e > s && e > c0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int64_t t = c0 + 64 * j + lane;
          const bool mine = in[j].use && t >= s && t < e;
          if (mine) {
            sum[0] += o[j].pg;
            sum[1] += o[j].kl;
            sum[2] += (double)in[j].entropy;
          }
          count += __popcll(__ballot(mine));
          cut += __popcll(__ballot(mine && !o[j].moves));
        }
      }
      if (e > c1) break;
      if (e > s && e > t0) flush();
      if (++n >= p.seqs) {
        s = e = p.tokens;
        break;
      }
      starts.span(p, n, s, e);
    }
  }
  if (s < end && e > end) flush();
}

// Sums over a workgroup of 1024 threads, in every thread, waves in order.
template <int K>
__device__ __forceinline__ void group_total(double (&v)[K], double (&slot)[16][K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const double t = wave_total(v[k]);
    if (threadIdx.x % 64 == 63) slot[threadIdx.x / 64][k] = t;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = slot[0][k];
#pragma unroll
    for (int i = 1; i < 16; ++i) v[k] += slot[i][k];
  }
}

constexpr int kInLds = 512;  // sequences whose sums the finish forms itself, in LDS
constexpr int kGroup = 64;   // sequences of a workgroup of the sums kernel otherwise

// Sums of the slots of sequences [n0, n1) by a workgroup of 1024 threads: 16 lanes for a
// sequence of up to kFew slots, a wave for a longer one. `start` gives a sequence's start.
template <class Start>
__device__ __forceinline__ void add_slots(const PolicyArgs &p, int64_t n0, int64_t n1,
                                          Start start, double *sums) {
  constexpr int kFew = 256;
  const int tid = threadIdx.x, lane = tid % 64;
  const uint32_t span = (uint32_t)p.span;  // starts are below 2^31
  auto slots = [&](int64_t n, int64_t &lo, int64_t &hi) {
    const uint32_t s = (uint32_t)start(n), e = (uint32_t)start(n + 1);
    lo = s / span + n;
    hi = e > s ? (e - 1) / span + n + 1 : lo;
  };
  for (int64_t n = n0 + tid / 16; n < n1; n += 64) {
    int64_t lo, hi;
    slots(n, lo, hi);
    if (hi - lo > kFew) continue;
    double v[kSums] = {};
#pragma unroll 2
    for (int64_t i = lo + tid % 16; i < hi; i += 16)
#pragma unroll
      for (int k = 0; k < kSums; ++k) v[k] += p.partials[i * kSums + k];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      v[k] = row_total(v[k]);
      if (tid % 16 == 15) sums[n * kSums + k] = v[k];
    }
  }
  for (int64_t n = n0 + tid / 64; n < n1; n += 16) {
    int64_t lo, hi;
    slots(n, lo, hi);
    if (hi - lo <= kFew) continue;
    double v[kSums] = {};
#pragma unroll 4
    for (int64_t i = lo + lane; i < hi; i += 64)
#pragma unroll
      for (int k = 0; k < kSums; ++k) v[k] += p.partials[i * kSums + k];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      v[k] = wave_total(v[k]);
      if (lane == 63) sums[n * kSums + k] = v[k];
    }
  }
}

// Many sequences: their sums by a grid, before the finish.
constexpr int64_t kSumsGrid = 1 << 16;  // workgroups; more sequences are walked over

__global__ __launch_bounds__(1024) void policy_sums_kernel(const PolicyArgs p) {
  const int64_t step = (int64_t)gridDim.x * kGroup;
  for (int64_t n0 = (int64_t)blockIdx.x * kGroup; n0 < p.seqs; n0 += step)
    add_slots(p, n0, n0 + kGroup < p.seqs ? n0 + kGroup : p.seqs,
              [&](int64_t n) { return start_of(p, n); }, p.seq_sums);
}

__global__ __launch_bounds__(1024) void policy_finish_kernel(const PolicyArgs p) {
  __shared__ double held[kInLds * kSums], slot2[16][2], slot4[16][4];
  __shared__ int starts[kInLds + 1];
  const int tid = threadIdx.x;
  const double *sums = p.seq_sums;  // [seqs][kSums]
  if (p.seqs <= kInLds) {
    for (int n = tid; n <= (int)p.seqs; n += 1024) starts[n] = (int)start_of(p, n);
    __syncthreads();
    add_slots(p, 0, p.seqs, [&](int64_t n) { return (int64_t)starts[n]; }, held);
    __syncthreads();
    sums = held;
  }
  double all[2] = {0.0, 0.0};  // scored tokens, sequences with any
  for (int64_t n = tid; n < p.seqs; n += 1024) {
    const double c = sums[n * kSums + 4];
    all[0] += c;
    all[1] += c > 0.0 ? 1.0 : 0.0;
  }
  group_total(all, slot2);
  double out[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t n = tid; n < p.seqs; n += 1024) {
    const double c = sums[n * kSums + 4];
    const double w = c > 0.0 ? (p.by_sequence ? 1.0 / (c * all[1]) : 1.0 / all[0]) : 0.0;
    p.seq_weight[n] = (float)w;
    if (c > 0.0)
#pragma unroll
      for (int k = 0; k < 4; ++k) out[k] += w * sums[n * kSums + k];
  }
  group_total(out, slot4);
  if (tid == 0) {
    p.stats[0] = (float)(out[0] + p.kl_coef * out[1] - p.entropy_coef * out[2]);
#pragma unroll
    for (int k = 0; k < 4; ++k) p.stats[k + 1] = (float)out[k];
  }
}

__global__ __launch_bounds__(256) void policy_grad_kernel(const PolicyArgs p) {
  const int64_t block = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64;
  const int64_t t0 = block * kChunk;
  if (t0 >= p.tokens) return;
  const int64_t end = t0 + kChunk < p.tokens ? t0 + kChunk : p.tokens;
  Inputs in[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) in[j] = load_token(p, t0 + 64 * j + lane, end, false);
  Starts starts;
  int64_t n = starts.seek(p, t0), held = -1;
  float weight = 0.0f, w[kPer] = {};  // weight: of sequence first + lane
  for (; n < p.seqs; ++n) {
    int64_t s, e;
    starts.span(p, n, s, e);
    if (s >= end) break;
    if (starts.first != held) {
      held = starts.first;
      weight = held + lane < p.seqs ? p.weight[held + lane] : 0.0f;
    }
    const float wn = __int_as_float(__builtin_amdgcn_readlane(
        __float_as_int(weight), __builtin_amdgcn_readfirstlane((int)(n - starts.first))));
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t t = t0 + 64 * j + lane;
      if (t >= s && t < e) w[j] = wn;
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t t = t0 + 64 * j + lane;
    if (t >= end) break;
    float dl = 0.0f, de = 0.0f;
    if (in[j].use && w[j] != 0.0f) {  // a scored token of a sequence has a weight
      const Token o = token_terms(p, in[j]);
      const double v = (double)w[j] * p.d_loss;
      dl = (float)(v * (p.kl_coef * o.kl_slope - (o.moves ? o.ratio_adv : 0.0)));
      de = (float)(-v * p.entropy_coef);
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

int64_t policy_span(int64_t tokens) { return span_of(tokens); }

int64_t policy_slots(int64_t tokens, int64_t seqs) {
  const int64_t span = span_of(tokens);
  return (tokens + span - 1) / span + seqs;
}

hipError_t launch_policy_fwd(const PolicyArgs &a, hipStream_t stream) {
  const int64_t spans = (a.tokens + a.span - 1) / a.span;
  if (spans > 0) {
    const hipError_t e = run((const void *)policy_tokens_kernel, a, (spans + 3) / 4, 256, stream);
    if (e != hipSuccess) return e;
  }
  if (a.seqs > kInLds) {
    const int64_t need = (a.seqs + kGroup - 1) / kGroup;
    const hipError_t e = run((const void *)policy_sums_kernel, a,
                             need < kSumsGrid ? need : kSumsGrid, 1024, stream);
    if (e != hipSuccess) return e;
  }
  return run((const void *)policy_finish_kernel, a, 1, 1024, stream);
}

hipError_t launch_policy_bwd(const PolicyArgs &a, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t blocks = (a.tokens + kChunk - 1) / kChunk;
  return run((const void *)policy_grad_kernel, a, (blocks + 3) / 4, 256, stream);
}

}  // namespace gdn
