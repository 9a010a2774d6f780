// Clipped policy loss of a packed ragged batch, and its gradient, on gfx950.
//
// A token costs two exponentials and some thirty bytes, so both directions are bound by
// latency up to millions of tokens. The ratio is compared with the clip borders and the sums
// are long, so the arithmetic is binary64 (its vector rate is far from the bound here).
//
// Forward: a wave takes a span of consecutive tokens, 256 at a time and 4 per lane, and adds
// them up for each sequence that meets the span; a pair (span, sequence) has the slot span +
// sequence, which no other pair has, since the pairs that meet form a staircase. Sequences inside
// a run of 256 tokens are taken together, so many short ones cost what a few long ones do
// (5372 tokens in 216 sequences 24 us with the gradient, 34 one after the other; 116 in 124 18.5
// and 94). One workgroup then adds each sequence's slots (a grid before it, of more than 512
// sequences), forms the weights and the loss; a small batch takes one launch in all. No atomics:
// the same bits on every launch. Backward: elementwise, each token's sequence found from its
// wave's first.
//
// What a wave waits for is memory: it issues all loads of its tokens first and finds its first
// sequence by a search of 64 lanes (one round of loads for 64 sequences, two for 4096), the
// last round's starts held in its lanes. 262144 tokens in 64 sequences: tokens 6.4 us, finish
// 6.1, gradient 6.9; 16384 in 4: 5.9, 4.1 and 5.8, of which a kernel that does nothing would
// take 2 to 3 each.

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

// Which of the sequences whose starts are held (lanes from `from` to `to` of the window) each of
// a chunk's tokens belongs to, found for all of them at once: every sequence with tokens marks the
// place of its start, and a token's sequence is the one marked last at or before it. One wave's
// LDS, no barrier: its accesses to LDS are in order.
struct Marks {
  uint8_t at[kChunk];
};
__device__ __forceinline__ void lds_in_order() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}
// own: this lane's sequence has a start at token c0 + place inside the chunk, and tokens. Gives in
// seq[j] the lane of the sequence of token c0 + 64 j + lane, -1 for a token before all of them.
__device__ __forceinline__ void find_sequences(Marks &m, bool own, int place, int (&seq)[kPer]) {
  const int lane = threadIdx.x % 64;
  lds_in_order();  // earlier reads are done
  reinterpret_cast<uint32_t *>(m.at)[lane] = 0;
  lds_in_order();
  if (own) m.at[place] = (uint8_t)(lane + 1);
  lds_in_order();
  uint8_t mark[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) mark[j] = m.at[64 * j + lane];
  int before = -1;  // the place marked last in the runs of 64 so far
  const uint64_t below = (~0ull) >> (63 - lane);
  int place_of[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint64_t all = __ballot(mark[j] != 0), mine = all & below;
    place_of[j] = mine ? 64 * j + 63 - __builtin_clzll(mine) : before;
    if (all) before = 64 * j + 63 - __builtin_clzll(all);
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    seq[j] = place_of[j] < 0 ? -1 : (int)m.at[place_of[j]] - 1;
}

// The value that lane `from` holds (any lane where from < 0).
__device__ __forceinline__ double of_lane(double v, int from) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (from & 63), (int)(uint32_t)b);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (from & 63), (int)(uint32_t)(b >> 32));
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ int of_lane(int v, int from) {
  return __builtin_amdgcn_ds_bpermute(4 * (from & 63), v);
}

// Bits [a, b) of a chunk's 256 flags set.
__device__ __forceinline__ int count_bits(const uint64_t (&f)[kPer], int a, int b) {
  int n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int lo = max(a - 64 * j, 0), hi = min(b - 64 * j, 64);
    if (lo < hi) n += __popcll((f[j] >> lo) << (64 - (hi - lo)));
  }
  return n;
}

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

// The sums of the span `block` by a wave.
__device__ __forceinline__ void add_span(const PolicyArgs &p, int64_t block, Marks &mark) {
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
  // Sequences that lie inside a chunk are taken together, each token with its weight but for a
  // factor of the whole batch: 1, or 1 / (its sequence's scored tokens). Their counts are exact
  // from the tokens' flags. The sum stands in the slot of the last of them, over that weight.
  double inner[3] = {0.0, 0.0, 0.0}, last_over = 0.0;
  int64_t last = -1;
  int last_lane = 0;
  for (int64_t c0 = t0; c0 < end; c0 += kChunk) {
    const int64_t c1 = c0 + kChunk < end ? c0 + kChunk : end;
    if (c0 > t0) load(c0);
    Token o[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = token_terms(p, in[j]);
    // the sequences that meet [c0, c1), those that end in it put down
    while (s < c1) {
      if (s >= c0 && e <= c1) {
        const int base = (int)(n - starts.first), from = starts.held - (int)c0;
        const int to = of_lane(starts.held, lane + 1) - (int)c0, size = (int)(c1 - c0);
        const bool inside = lane >= base && lane < 63 && starts.first + lane < p.seqs &&
                            from >= 0 && to <= size;
        const uint64_t rest = ~__ballot(inside) >> base;  // bit 63 is never inside: not 0
        const int more = __builtin_ctzll(rest), run = more > 0 ? more : 1;
        const bool own = inside && lane < base + run && to > from;
        uint64_t used[kPer], cuts[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          used[j] = __ballot(in[j].use);
          cuts[j] = __ballot(in[j].use && !o[j].moves);
        }
        const int c = own ? count_bits(used, from, to) : 0;
        const double w = c > 0 ? (p.by_sequence ? 1.0 / (double)c : 1.0) : 0.0;
        int seq[kPer];
        find_sequences(mark, own, from, seq);
        const int run_end = __builtin_amdgcn_readlane(starts.held, base + run) - (int)c0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const double wt = of_lane(w, seq[j]);
          if (in[j].use && seq[j] >= 0 && 64 * j + lane < run_end) {
            inner[0] += wt * o[j].pg;
            inner[1] += wt * o[j].kl;
            inner[2] += wt * (double)in[j].entropy;
          }
        }
        if (own) {
          double *out = p.partials + (block + starts.first + lane) * kSums;
          out[0] = out[1] = out[2] = 0.0;
          out[3] = (double)count_bits(cuts, from, to);
          out[4] = (double)c;
        }
        if (const uint64_t any = __ballot(c > 0)) {
          last_lane = 63 - __builtin_clzll(any);
          last = starts.first + last_lane;
          last_over = p.by_sequence ? (double)__builtin_amdgcn_readlane(c, last_lane) : 1.0;
        }
        n += run;
        if (n >= p.seqs) {
          s = e = p.tokens;
          break;
        }
        starts.span(p, n, s, e);
        continue;
      }
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
  if (last >= 0) {
    double *out = p.partials + (block + last) * kSums;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const double v = of_lane(wave_total(inner[k]), 63) * last_over;
      if (lane == last_lane) out[k] = v;  // the lane that wrote 0 there
    }
  }
}

__global__ __launch_bounds__(256) void policy_tokens_kernel(const PolicyArgs p) {
  __shared__ __align__(4) Marks marks[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  add_span(p, (int64_t)blockIdx.x * 4 + wave, marks[wave]);
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

// Sequences' sums, weights and the loss, by a workgroup of 1024 threads.
__device__ __forceinline__ void finish(const PolicyArgs &p) {
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

__global__ __launch_bounds__(1024) void policy_finish_kernel(const PolicyArgs p) { finish(p); }

// A small batch in one launch, a span for each of its first waves: loss and gradient of 64 tokens
// 12.9 us against 17.1, of 1024 15.9 against 17.1 (4096, with every wave at work on the one
// compute unit, 18.2 against 15.3).
constexpr int64_t kSmall = 4 * kChunk;
__global__ __launch_bounds__(1024) void policy_small_kernel(const PolicyArgs p) {
  __shared__ __align__(4) Marks marks[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (wave < 4) add_span(p, wave, marks[wave]);
  __threadfence_block();
  __syncthreads();
  finish(p);
}

__global__ __launch_bounds__(256) void policy_grad_kernel(const PolicyArgs p) {
  __shared__ __align__(4) Marks marks[4];
  const int64_t block = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64;
  const int64_t t0 = block * kChunk;
  if (t0 >= p.tokens) return;
  const int64_t end = t0 + kChunk < p.tokens ? t0 + kChunk : p.tokens;
  Inputs in[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) in[j] = load_token(p, t0 + 64 * j + lane, end, false);
  Starts starts;
  int64_t n = starts.seek(p, t0);
  float w[kPer] = {};
  const int size = (int)(end - t0);
  int64_t s, e;
  starts.span(p, n, s, e);
  if (n < p.seqs && s <= t0 && e >= end) {  // all of one sequence
    const float weight = p.weight[n];
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = weight;
    n = p.seqs;
  }
  while (n < p.seqs) {  // 63 sequences at a time
    if (n - starts.first >= 63) starts.load(p, n);
    const int64_t mine = starts.first + lane;
    const bool held = lane >= (int)(n - starts.first) && lane < 63 && mine < p.seqs;
    const float weight = held ? p.weight[mine] : 0.0f;
    const int from = max(starts.held - (int)t0, 0), to = of_lane(starts.held, lane + 1) - (int)t0;
    int seq[kPer];
    find_sequences(marks[threadIdx.x / 64], held && from < size && to > from, from, seq);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int stop = of_lane(to, seq[j]);
      const float wt = __int_as_float(of_lane(__float_as_int(weight), seq[j]));
      if (seq[j] >= 0 && 64 * j + lane < stop) w[j] = wt;
    }
    n = starts.first + 63;
    if (starts.at(n) >= end) break;
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
  if (a.tokens <= kSmall && a.seqs <= kInLds)
    return run((const void *)policy_small_kernel, a, 1, 1024, stream);
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
