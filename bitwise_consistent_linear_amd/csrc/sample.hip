// Tokens drawn from logits with temperature, top-k, top-p and min-p, for gfx950.
//
// A token's weight is a whole number, exp((x - max) / T) in units of 2^-shift, so sums of weights
// are exact and the order of the additions, in LDS atomics too, changes nothing: a row's token is
// the same whichever kernel draws it. Every filter keeps the head of one order, falling logits
// and rising ids among equal ones; a token's place in it is a 64-bit number (the logit's bits made
// to order like integers above, the inverted id below) and a filter is the least such number that
// it keeps. The draw goes by rising id.

#include <algorithm>

#include "policy_rows.hpp"
#include "step_internal.h"

namespace gdn {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;       // a weight above 0 lies in the first 46.5 * 32
constexpr int kList = 4096;       // candidates that LDS holds
constexpr int kFew = 64;          // candidates that one wave ranks
constexpr float kBinsPerNat = 64.0f;
constexpr int kTable = 64;        // steps of an octave in the table of powers of two

__device__ __forceinline__ uint32_t key_of(float x) {  // a NaN above all, -0 as 0
  const uint32_t b = __float_as_uint(x + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kInfinity = 0xFF800000u, kMinusInfinity = 0x007FFFFFu;  // keys

__device__ __forceinline__ u64 place_of(float x, int64_t id) {
  return (u64)key_of(x) << 32 | (uint32_t)~(uint32_t)id;
}

// f * m rounded down, for a finite f in [0, 1); up: rounded up. Exact.
__device__ __forceinline__ u64 part_of(double f, u64 m, bool up) {
  if (!(f > 0.0)) return 0;
  const u64 bits = (u64)__double_as_longlong(f);
  const int e = (int)(bits >> 52);
  const u64 mant = (bits & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0);
  const int s = 1075 - (e ? e : 1);  // f = mant 2^-s, s >= 53
  const u64 lo = mant * m, hi = __umul64hi(mant, m);
  u64 q;
  bool rest;
  if (s < 64) {
    q = hi << (64 - s) | lo >> s;
    rest = (lo & ((1ull << s) - 1)) != 0;
  } else if (s < 128) {
    q = s == 64 ? hi : hi >> (s - 64);
    rest = lo != 0 || (s > 64 && (hi & ((1ull << (s - 64)) - 1)) != 0);
  } else {
    q = 0;
    rest = lo != 0 || hi != 0;
  }
  return q + (up && rest);
}

// What a row's draw goes by, as the caller gave it.
struct Request {
  double T, top_p, min_p, u;
  int64_t k;
  __device__ __forceinline__ Request(const SampleArgs &p, int64_t row) {
    T = p.temperatures ? (double)p.temperatures[row] : p.temperature;
    k = p.top_ks ? (int64_t)p.top_ks[row] : p.top_k;
    top_p = p.top_ps ? (double)p.top_ps[row] : p.top_p;
    min_p = p.min_ps ? (double)p.min_ps[row] : p.min_p;
    u = p.u64 ? static_cast<const double *>(p.u)[row]
              : (double)static_cast<const float *>(p.u)[row];
  }
  __device__ __forceinline__ bool drawn(uint32_t top_key) const {
    return top_key > kMinusInfinity && top_key < kInfinity && T >= 0.0 && T < __builtin_inf();
  }
  // the least weight that min_p keeps
  __device__ __forceinline__ u64 floor(int shift) const {
    const u64 unit = 1ull << shift;
    return !(min_p > 0.0) ? 0 : min_p >= 1.0 ? unit : part_of(min_p, unit, true);
  }
  // where in a sum of `all` the draw falls
  __device__ __forceinline__ u64 point(u64 all) const {
    return u >= 1.0 ? all - 1 : part_of(u, all, false);
  }
};

// exp((x - top) / T) in units of 2^-shift, to the nearest: y = (x - top) log2(e) / T in steps of
// the table is split into a whole number and a rest of at most half a step, whose power of two
// five terms of its series give to 2^-44. The table holds 2^(shift + i / kTable); a whole power
// is added to its exponent, and the last product rounds to whole numbers by the sum with 2^52. Its
// 64 values lie two to a bank of LDS, so that lanes hardly wait for each other (1024 values and
// four terms: a random read takes 23 cycles a wave, as long as the terms that it saves).
struct Weigh {
  const double *power;
  double top, rate, least;  // rate: kTable log2(e) / T
  __device__ __forceinline__ Weigh(const double *power, float top, double T)
      : power(power), top(top), rate(1.4426950408889634074 * kTable / T),
        least(-64.0 * kTable / rate) {}  // from there on down the weight is 0
  __device__ __forceinline__ static void fill(double *power, int shift, int thread, int threads) {
    for (int i = thread; i < kTable; i += threads)
      power[i] = exp2((double)i / kTable + (double)shift);
  }
  static constexpr u64 kNone = 0x4330000000000000ull;  // the bits of 2^52
  static constexpr double kMagic = 0x1.8p52;
  // y to the nearest whole number, in the low word
  __device__ __forceinline__ double whole(double d) const { return fma(d, rate, kMagic); }
  __device__ __forceinline__ static int low(double t) { return (int)(uint32_t)(u64)__double_as_longlong(t); }
  __device__ __forceinline__ double below(float x) const { return fmax((double)x - top, least); }
  // Two steps to a bin, from the top down: bin b of y in [-2 b - 1.5, -2 b + 0.5].
  static constexpr int kPerOctave = kTable / 2;
  __device__ __forceinline__ int bin_at(double d) const { return -low(whole(d)) >> 1; }
  __device__ __forceinline__ int bin(float x) const { return bin_at(below(x)); }
  // the weight added to kNone
  __device__ __forceinline__ u64 raw(float x) const { return raw_at(below(x)); }
  __device__ __forceinline__ u64 raw_at(double d) const {
    constexpr double c = 0.69314718055994530942 / kTable;
    const double t = whole(d), r = fma(d, rate, kMagic - t);
    const int n = low(t);
    const double q = fma(r, fma(r, fma(r, fma(r, c * c * c * c / 24, c * c * c / 6), c * c / 2), c), 1.0);
    const u64 bits = (u64)__double_as_longlong(power[n & (kTable - 1)]);
    const uint32_t high = (uint32_t)(bits >> 32) + ((uint32_t)(n & ~(kTable - 1)) << 14);
    const double w = __longlong_as_double((long long)((u64)high << 32 | (uint32_t)bits));
    return (u64)__double_as_longlong(fma(w, q, 0x1p52));
  }
  __device__ __forceinline__ u64 operator()(float x) const { return raw(x) - kNone; }
  __device__ __forceinline__ u64 operator()(u64 place) const {
    return (*this)(logit_of((uint32_t)(place >> 32)));
  }
};

// f(vec, id) for the whole runs of eight ids in [from, to) of a row at `off`, a thread of
// `threads` each, Ahead loads ahead of their use, and g(x, id) for the ids behind the last one.
template <bool B16, int Ahead, class F, class G>
__device__ __forceinline__ void over_runs(const SampleArgs &p, int64_t off, int64_t from, int64_t to,
                                          int thread, int threads, F f, G g) {
  if (from >= to) return;
  const int64_t first = off + from;
  const int runs = (int)((to - from) / 8);
  int i = thread;
  if constexpr (Ahead > 1) {
#pragma unroll 1
    for (; i + (Ahead - 1) * threads < runs; i += Ahead * threads) {
      Vec8<B16> v[Ahead];
#pragma unroll
      for (int u = 0; u < Ahead; ++u) v[u].load(p.logits, first + 8 * (int64_t)(i + u * threads));
#pragma unroll
      for (int u = 0; u < Ahead; ++u) {
        f(v[u], from + 8 * (int64_t)(i + u * threads));
        __builtin_amdgcn_sched_barrier(0);  // one run at a time: all at once would spill
      }
    }
  }
#pragma unroll 1
  for (; i < runs; i += threads) {
    Vec8<B16> v;
    v.load(p.logits, first + 8 * (int64_t)i);
    f(v, from + 8 * (int64_t)i);
  }
  if (thread == runs % threads)  // the next thread in turn
#pragma unroll 1
    for (int64_t id = from + 8 * (int64_t)runs; id < to; ++id) {
      const float x = B16 ? bf16_lo(static_cast<const uint16_t *>(p.logits)[off + id])
                          : static_cast<const float *>(p.logits)[off + id];
      g(x, id);
    }
}
// f(x, id) for ids [from, to): eight neighbours a thread, which are taken one by one.
template <bool B16, int Ahead = 1, class F>
__device__ __forceinline__ void over(const SampleArgs &p, int64_t off, int64_t from, int64_t to,
                                     int thread, int threads, F f) {
  over_runs<B16, Ahead>(
      p, off, from, to, thread, threads,
      [&](const Vec8<B16> &v, int64_t id) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f(v.get(e), id + e);
          if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
      },
      f);
}

// Sum of the weights of ids [from, to) that this thread sees: of those at or above `floor`.
template <bool B16>
__device__ __forceinline__ u64 thread_mass(const SampleArgs &p, int64_t off, int64_t from, int64_t to,
                                           int thread, int threads, const Weigh &weigh, u64 floor) {
  u64 sum = 0, n = 0;
  if (floor == 0) {
    over<B16, 4>(p, off, from, to, thread, threads, [&](float x, int64_t) {
      sum += weigh.raw(x);
      ++n;
    });
    return sum - n * Weigh::kNone;
  }
  over<B16, 1>(p, off, from, to, thread, threads, [&](float x, int64_t) {
    const u64 w = weigh(x);
    sum += w >= floor ? w : 0;
  });
  return sum;
}

// Largest key of ids [from, to) that this thread sees.
template <bool B16>
__device__ __forceinline__ uint32_t thread_top(const SampleArgs &p, int64_t off, int64_t from,
                                               int64_t to, int thread, int threads) {
  float top = -__builtin_inff();
  uint32_t all = 0;  // a NaN is passed over by the maximum, not by that of the magnitudes' bits
  auto one = [&](float x, int64_t) {
    top = fmaxf(top, x);
    all = max(all, __float_as_uint(x) & 0x7FFFFFFFu);
  };
  if constexpr (B16) {
    using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
    u16x2 pair = {0, 0};
    over_runs<B16, 8>(
        p, off, from, to, thread, threads,
        [&](const Vec8<true> &v, int64_t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pair = __builtin_elementwise_max(pair, __builtin_bit_cast(u16x2, v.r[i] & 0x7FFF7FFFu));
            top = fmaxf(fmaxf(top, bf16_lo(v.r[i])), bf16_hi(v.r[i]));
          }
        },
        one);
    all = max(all, (uint32_t)max(pair[0], pair[1]) << 16);
  } else {
    over<B16, 4>(p, off, from, to, thread, threads, one);
  }
  return all > 0x7F800000u ? 0xFFFFFFFFu : key_of(top);
}

// Lanes talk by DPP and readlane: the permutes that shuffles compile to go through LDS, which all
// waves of a unit share (a search of 1024 places took 8 us with them).
template <int Ctrl>
__device__ __forceinline__ u64 dpp(u64 v) {  // 0 from outside the row of 16 lanes
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, Ctrl, 0xF, 0xF, true);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), Ctrl, 0xF, 0xF, true);
  return (u64)(uint32_t)hi << 32 | (uint32_t)lo;
}
__device__ __forceinline__ u64 of_lane(u64 v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (u64)hi << 32 | lo;
}
// f over each row of 16 lanes, in all of them, and over the wave; f's order of arguments is free.
template <class F>
__device__ __forceinline__ u64 row_all(u64 v, F f) {
  v = f(v, dpp<0x128>(v));  // rotated by 8, 4, 2, 1
  v = f(v, dpp<0x124>(v));
  v = f(v, dpp<0x122>(v));
  return f(v, dpp<0x121>(v));
}
template <class F>
__device__ __forceinline__ u64 wave_all(u64 v, F f) {
  v = row_all(v, f);
  return f(f(of_lane(v, 0), of_lane(v, 16)), f(of_lane(v, 32), of_lane(v, 48)));
}
__device__ __forceinline__ u64 add(u64 a, u64 b) { return a + b; }
__device__ __forceinline__ u64 least_of(u64 a, u64 b) { return a < b ? a : b; }
__device__ __forceinline__ u64 most_of(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_top(uint32_t k) { return (uint32_t)wave_all(k, most_of); }
__device__ __forceinline__ u64 wave_sum(u64 v) { return wave_all(v, add); }
// Sums of the lanes up to each.
__device__ __forceinline__ uint32_t wave_run(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);
  auto of = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); };
  const uint32_t a = of(15), b = a + of(31), c = b + of(47);
  const int row = threadIdx.x % 64 / 16;
  return v + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}
__device__ __forceinline__ u64 wave_run(u64 v) {
  v += dpp<0x111>(v);  // from 1, 2, 4, 8 lanes below
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  const u64 a = of_lane(v, 15), b = a + of_lane(v, 31), c = b + of_lane(v, 47);
  const int row = threadIdx.x % 64 / 16;
  return v + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}

// Sum of value(x, id) over ids [from, to) by a wave.
template <bool B16, class F>
__device__ __forceinline__ u64 wave_mass(const SampleArgs &p, int64_t off, int64_t from, int64_t to,
                                         F value) {
  u64 sum = 0;
  over<B16>(p, off, from, to, threadIdx.x % 64, 64, [&](float x, int64_t i) { sum += value(x, i); });
  return wave_sum(sum);
}

// Where the running sum of value(x, id) over ids [from, to) passes `rest` (less than the whole):
// a part of the range for each wave, then of that part, down to eight ids a lane. from is a
// multiple of 512, to too or the row's end. The place, in every thread; `sums` holds a value for
// each wave.
template <bool B16, int Waves, class F>
__device__ __forceinline__ u64 descend(const SampleArgs &p, int64_t off, int64_t from, int64_t to,
                                       u64 rest, u64 *sums, u64 *found, F value) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  while (to - from > Waves * 512) {
    const int64_t each = ((to - from + Waves - 1) / Waves + 511) / 512 * 512;
    const int64_t begin = from + wave * each;
    const u64 sum = wave_mass<B16>(p, off, begin, begin + each < to ? begin + each : to, value);
    __syncthreads();
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    int w = 0;
    while (w < Waves - 1 && rest >= sums[w]) rest -= sums[w++];
    from += w * each;
    to = from + each < to ? from + each : to;
  }
  const int64_t col = from + 512 * wave + 8 * lane;
  u64 w[8] = {}, sum = 0;
  float x[8] = {};
  if (col < to) {
    Vec8<B16> v;
    load_row(v, p.logits, off, col, p.vocab);
    settle_row(v, col, p.vocab, -__builtin_inff());  // of weight 0
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = v.get(e);
      sum += w[e] = value(x[e], col + e);
    }
  }
  const u64 run = wave_run(sum);
  __syncthreads();
  if (lane == 63) sums[wave] = run;
  __syncthreads();
  u64 before = run - sum;
  for (int i = 0; i < wave; ++i) before += sums[i];
  if (before <= rest && rest < before + sum)  // one thread's
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (before <= rest && rest < before + w[e]) *found = place_of(x[e], col + e);
      before += w[e];
    }
  __syncthreads();
  return *found;
}

// The first id of the largest logit.
template <bool B16>
__device__ __forceinline__ u64 first_of(const SampleArgs &p, int64_t off, uint32_t top_key,
                                        int threads, u64 *found) {
  if (threadIdx.x == 0) *found = 0;
  __syncthreads();
  over<B16>(p, off, 0, p.vocab, threadIdx.x, threads, [&](float x, int64_t i) {
    if (key_of(x) == top_key) atomicMax(found, place_of(x, i));
  });
  __syncthreads();
  return *found;
}

__device__ __forceinline__ void answer(const SampleArgs &p, int64_t row, int64_t id, double logp) {
  if (p.id64)
    static_cast<int64_t *>(p.ids)[row] = id;
  else
    static_cast<int32_t *>(p.ids)[row] = (int32_t)id;
  p.logp[row] = (float)logp;
}
// ... of a place drawn among weights that sum to `all`.
__device__ __forceinline__ void answer(const SampleArgs &p, int64_t row, u64 place, float top,
                                       double T, u64 all) {
  const double z = ((double)logit_of((uint32_t)(place >> 32)) - (double)top) / T;
  answer(p, row, (uint32_t)~(uint32_t)place, z - log(ldexp((double)all, -p.shift)));
}

// ------------------------------------------------------------------------- without cuts

// No top-k or top-p: two readings of the row, its maximum and the sum of its weights, and a few
// of ever smaller parts of it. A row a workgroup at a time. 512 x 131072 bf16 take 71 us: the maximum
// 25 (134 MB, memory), the sums the rest (22 instructions a logit, most of them in 64 bits).
template <bool B16>
__global__ __launch_bounds__(kThreads) void sample_plain_kernel(const SampleArgs p) {
  constexpr int kWaves = kThreads / 64;
  __shared__ double power[kTable];
  __shared__ u64 sums[kWaves], found;
  __shared__ uint32_t tops[kWaves];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int64_t V = p.vocab, each = ((V + kWaves - 1) / kWaves + 511) / 512 * 512;
  const int64_t begin = wave * each, end = begin + each < V ? begin + each : V;
  const int64_t row = p.first + blockIdx.x, off = row * p.stride;
  Weigh::fill(power, p.shift, tid, kThreads);
  uint32_t top_key = wave_top(thread_top<B16>(p, off, begin, end, lane, 64));
  if (lane == 0) tops[wave] = top_key;
  __syncthreads();
  for (int i = 0; i < kWaves; ++i) top_key = max(top_key, tops[i]);
  const Request r(p, row);
  if (!r.drawn(top_key)) {
    if (tid == 0) answer(p, row, -1, 0.0);
    return;
  }
  if (r.T == 0.0) {
    const u64 place = first_of<B16>(p, off, top_key, kThreads, &found);
    if (tid == 0) answer(p, row, (uint32_t)~(uint32_t)place, 0.0);
    return;
  }
  const float top = logit_of(top_key);
  const Weigh weigh(power, top, r.T);
  const u64 floor = r.floor(p.shift);
  const u64 sum = wave_sum(thread_mass<B16>(p, off, begin, end, lane, 64, weigh, floor));
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  u64 all = 0;
  for (int i = 0; i < kWaves; ++i) all += sums[i];
  u64 rest = r.point(all);
  int w = 0;
  while (w < kWaves - 1 && rest >= sums[w]) rest -= sums[w++];
  const int64_t from = w * each;
  const u64 place = descend<B16, kWaves>(p, off, from, from + each < V ? from + each : V, rest, sums,
                                         &found, [&](float x, int64_t) {
                                           const u64 w = weigh(x);
                                           return w >= floor ? w : 0;
                                         });
  if (tid == 0) answer(p, row, place, top, r.T, all);
}

// Few rows: a row in slices, a workgroup each, in three launches: the slices' maxima, their sums,
// and the draw within one slice. 8 x 131072 f32: 3.0 + 4.4 + 5.1 us, mostly each launch's own 2 to 3.
constexpr int kSliceThreads = 256, kSliceWaves = kSliceThreads / 64;

struct Slices {
  int64_t count, each;  // of a row; each a multiple of 512 * kSliceWaves ids
  uint32_t *tops;       // [rows][count]
  u64 *sums;            // [rows][count]
};

__device__ __forceinline__ uint32_t row_top(const Slices &s, int64_t row, uint32_t *tops) {
  uint32_t k = 0;
  for (int64_t i = threadIdx.x; i < s.count; i += kSliceThreads) k = max(k, s.tops[row * s.count + i]);
  k = wave_top(k);
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = k;
  __syncthreads();
  for (int i = 0; i < kSliceWaves; ++i) k = max(k, tops[i]);
  return k;
}

template <bool B16>
__global__ __launch_bounds__(kSliceThreads) void sample_tops_kernel(const SampleArgs p, const Slices s) {
  __shared__ uint32_t tops[kSliceWaves];
  const int64_t row = blockIdx.x / s.count, from = blockIdx.x % s.count * s.each;
  const int64_t to = from + s.each < p.vocab ? from + s.each : p.vocab;
  uint32_t k = wave_top(thread_top<B16>(p, row * p.stride, from, to, threadIdx.x, kSliceThreads));
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = k;
  __syncthreads();
  for (int i = 0; i < kSliceWaves; ++i) k = max(k, tops[i]);
  if (threadIdx.x == 0) s.tops[blockIdx.x] = k;
}

template <bool B16>
__global__ __launch_bounds__(kSliceThreads) void sample_sums_kernel(const SampleArgs p, const Slices s) {
  __shared__ double power[kTable];
  __shared__ u64 sums[kSliceWaves];
  __shared__ uint32_t tops[kSliceWaves];
  Weigh::fill(power, p.shift, threadIdx.x, kSliceThreads);
  const int64_t row = blockIdx.x / s.count, from = blockIdx.x % s.count * s.each;
  const int64_t to = from + s.each < p.vocab ? from + s.each : p.vocab;
  const uint32_t top_key = row_top(s, row, tops);
  const Request r(p, row);
  if (!r.drawn(top_key) || r.T == 0.0) return;
  const Weigh weigh(power, logit_of(top_key), r.T);
  const u64 floor = r.floor(p.shift);
  u64 sum = 0;
  over<B16>(p, row * p.stride, from, to, threadIdx.x, kSliceThreads, [&](float x, int64_t) {
    const u64 w = weigh(x);
    sum += w >= floor ? w : 0;
  });
  sum = wave_sum(sum);
  if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSliceWaves; ++i) sum += sums[i];
    s.sums[blockIdx.x] = sum;
  }
}

template <bool B16>
__global__ __launch_bounds__(kSliceThreads) void sample_slice_kernel(const SampleArgs p, const Slices s) {
  __shared__ double power[kTable];
  __shared__ u64 sums[kSliceWaves], found, slice, rest, total;
  __shared__ uint32_t tops[kSliceWaves];
  const int64_t row = blockIdx.x, off = row * p.stride;
  Weigh::fill(power, p.shift, threadIdx.x, kSliceThreads);
  const uint32_t top_key = row_top(s, row, tops);
  const Request r(p, row);
  if (!r.drawn(top_key)) {
    if (threadIdx.x == 0) answer(p, row, -1, 0.0);
    return;
  }
  if (r.T == 0.0) {
    const u64 place = first_of<B16>(p, off, top_key, kSliceThreads, &found);
    if (threadIdx.x == 0) answer(p, row, (uint32_t)~(uint32_t)place, 0.0);
    return;
  }
  if (threadIdx.x < 64) {  // the wave's lanes take the slices in turn
    const int lane = threadIdx.x;
    u64 all = 0;
    for (int64_t i = lane; i < s.count; i += 64) all += s.sums[row * s.count + i];
    all = wave_sum(all);
    u64 left = r.point(all), before = 0;
    for (int64_t i0 = 0; i0 < s.count; i0 += 64) {
      const u64 sum = i0 + lane < s.count ? s.sums[row * s.count + i0 + lane] : 0;
      const u64 run = wave_run(sum);
      if (before + run - sum <= left && left < before + run) {
        slice = (u64)(i0 + lane);
        rest = left - (before + run - sum);
        total = all;
      }
      before += of_lane(run, 63);
    }
  }
  __syncthreads();
  const float top = logit_of(top_key);
  const Weigh weigh(power, top, r.T);
  const u64 floor = r.floor(p.shift);
  const int64_t from = (int64_t)slice * s.each;
  const u64 place = descend<B16, kSliceWaves>(
      p, off, from, from + s.each < p.vocab ? from + s.each : p.vocab, rest, sums, &found,
      [&](float x, int64_t) {
        const u64 w = weigh(x);
        return w >= floor ? w : 0;
      });
  if (threadIdx.x == 0) answer(p, row, place, top, r.T, total);
}

// ---------------------------------------------------------------------------- with cuts

struct Shared {
  double power[kTable];
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 list[kList];
  u64 few[kFew], few_value[kFew], few_sum[kFew];
  u64 wave[4][kThreads / 64], wave2[kThreads / 64], part[kThreads / 64];
  u64 found, before;
  uint32_t n, bin;
};

struct Range {
  u64 sum, count, lo, hi;
};
constexpr Range kNothing = {0, 0, ~0ull, 0};
__device__ __forceinline__ void join(Range &a, u64 sum, u64 count, u64 lo, u64 hi) {
  a.sum += sum;
  a.count += count;
  a.lo = lo < a.lo ? lo : a.lo;
  a.hi = hi > a.hi ? hi : a.hi;
}
// Sums, least and largest over the workgroup.
__device__ __forceinline__ Range block_range(Shared &s, Range v) {
  static_assert(kThreads == 1024, "a row of lanes holds a value of each wave");
  const int wave = threadIdx.x / 64, at = threadIdx.x % 16;
  v = {wave_all(v.sum, add), wave_all(v.count, add), wave_all(v.lo, least_of), wave_all(v.hi, most_of)};
  __syncthreads();
  if (threadIdx.x % 64 == 0) {
    s.wave[0][wave] = v.sum;
    s.wave[1][wave] = v.count;
    s.wave[2][wave] = v.lo;
    s.wave[3][wave] = v.hi;
  }
  __syncthreads();
  return {of_lane(row_all(s.wave[0][at], add), 0), of_lane(row_all(s.wave[1][at], add), 0),
          of_lane(row_all(s.wave[2][at], least_of), 0), of_lane(row_all(s.wave[3][at], most_of), 0)};
}

// The bin, of those that `value(b)` weighs, in which the running sum passes `target` (at least
// 1, at most all of them): its number in s.bin, the sum before it in s.before.
template <class F>
__device__ __forceinline__ void find_bin(Shared &s, u64 target, F value) {
  constexpr int each = kBins / kThreads;
  const int t = threadIdx.x;
  u64 v[each], sum = 0;
#pragma unroll
  for (int i = 0; i < each; ++i) sum += v[i] = value(each * t + i);
  const u64 run = wave_run(sum);
  if (t % 64 == 63) s.wave2[t / 64] = run;  // s.wave may still be read
  __syncthreads();
  u64 before = run - sum;
  for (int i = 0; i < t / 64; ++i) before += s.wave2[i];
  if (before < target && target <= before + sum) {
#pragma unroll
    for (int i = 0; i < each; ++i) {
      if (before < target && target <= before + v[i]) {
        s.bin = each * t + i;
        s.before = before;
      }
      before += v[i];
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void clear_bins(Shared &s) {
  for (int b = threadIdx.x; b < kBins; b += kThreads) {
    s.mass[b] = 0;
    s.count[b] = 0;
  }
  __syncthreads();
}

// The candidate at which the running sum of value(c), by falling order(c), passes `target`.
// walk(f) calls f(c) for every candidate; those whose order is in [lo, hi] count, `count` of
// them, with a sum of target and more.
template <class Walk, class Order, class Value>
__device__ __forceinline__ u64 resolve(Shared &s, u64 lo, u64 hi, u64 count, u64 target, Walk walk,
                                       Order order, Value value) {
  while (count > kFew) {
    const int bits = 64 - __clzll((long long)(hi - lo) | 1);
    const int shift = bits > 11 ? bits - 11 : 0;
    clear_bins(s);
    walk([&](u64 c) {
      const u64 o = order(c);
      if (o >= lo && o <= hi) {
        const int b = (int)((hi - o) >> shift);
        atomicAdd(&s.mass[b], value(c));
        atomicAdd(&s.count[b], 1u);
      }
    });
    __syncthreads();
    find_bin(s, target, [&](int b) { return s.mass[b]; });
    const u64 bin = s.bin;
    count = s.count[bin];
    target -= s.before;
    const u64 end = hi - (bin << shift), span = (1ull << shift) - 1;
    hi = end;
    if (hi - lo > span) lo = hi - span;
    __syncthreads();
  }
  if (threadIdx.x == 0) s.n = 0;
  __syncthreads();
  walk([&](u64 c) {
    const u64 o = order(c);
    if (o >= lo && o <= hi) s.few[atomicAdd(&s.n, 1u)] = c;
  });
  __syncthreads();
  // every one of them against four others by each wave
  const int n = (int)s.n, i = threadIdx.x % 64, part = threadIdx.x / 64 * (kFew / 16);
  if (threadIdx.x < kFew) {
    s.few_sum[i] = 0;
    s.few_value[i] = i < n ? value(s.few[i]) : 0;
  }
  __syncthreads();
  if (i < n && part < n) {
    const u64 o = order(s.few[i]);
    u64 before = 0;
#pragma unroll
    for (int j = 0; j < kFew / 16; ++j)
      if (part + j < n && order(s.few[part + j]) > o) before += s.few_value[part + j];
    if (before) atomicAdd(&s.few_sum[i], before);
  }
  __syncthreads();
  if (threadIdx.x < n) {
    const u64 before = s.few_sum[i];
    if (before < target && target <= before + s.few_value[i]) s.found = s.few[i];
  }
  __syncthreads();
  const u64 c = s.found;
  __syncthreads();
  return c;
}

__device__ __forceinline__ u64 share(double top_p, u64 all) {  // where top_p cuts a sum off
  const u64 t = part_of(top_p, all, true);
  return t > 0 ? t : 1;
}

// The weight of a logit that a cut (a place, 0 for none) and min_p keep, else 0.
struct Kept {
  const Weigh &weigh;
  float last;
  int64_t last_id;
  u64 floor;
  __device__ __forceinline__ Kept(const Weigh &weigh, u64 cut, u64 floor, int64_t vocab)
      : weigh(weigh), last(cut ? logit_of((uint32_t)(cut >> 32)) : -__builtin_inff()),
        last_id(cut ? (int64_t)(uint32_t)~(uint32_t)cut : vocab), floor(floor) {}
  __device__ __forceinline__ u64 operator()(float x, int64_t id) const {
    const u64 w = x > last || (x == last && id <= last_id) ? weigh(x) : 0;
    return w >= floor ? w : 0;
  }
};

// Rows whose cuts keep more than LDS holds, or whose candidates did not fit there: bins of the
// logits and then of places narrow every cut down in the row itself. A kernel of its own, as its
// registers would make the common path's spill. The workspace holds a word for each row: whether
// it is one.
template <bool B16>
__global__ __launch_bounds__(kThreads) void sample_left_kernel(const SampleArgs p) {
  constexpr int kWaves = kThreads / 64;
  __shared__ Shared s;
  const int tid = threadIdx.x;
  const int64_t row = p.first + blockIdx.x, off = row * p.stride, V = p.vocab;
  if (!static_cast<const uint32_t *>(p.workspace)[row]) return;
  Weigh::fill(s.power, p.shift, tid, kThreads);
  const uint32_t mine = thread_top<B16>(p, off, 0, V, tid, kThreads);
  const uint32_t top_key = (uint32_t)block_range(s, {0, 0, mine, mine}).hi;
  const Request r(p, row);
  const float top = logit_of(top_key);
  const Weigh weigh(s.power, top, r.T);
  const float bins = (float)fmin((double)kBinsPerNat / r.T, 0x1p100);
  auto bin_of = [&](float x) { return (int)fminf((top - x) * bins, (float)(kBins - 1)); };
  const u64 floor = r.floor(p.shift);
  u64 cut = 0;  // the least place that is kept
  for (int by_mass = 0; by_mass < 2; ++by_mass) {
    if (by_mass ? !(r.top_p < 1.0) : !(r.k > 0 && r.k < V)) continue;
    auto value = [&](u64 c) { return by_mass ? weigh(c) : 1ull; };
    clear_bins(s);
    over<B16>(p, off, 0, V, tid, kThreads, [&](float x, int64_t i) {
      const u64 c = place_of(x, i);
      if (c >= cut) {
        const int b = bin_of(x);
        atomicAdd(&s.mass[b], value(c));
        atomicAdd(&s.count[b], 1u);
      }
    });
    __syncthreads();
    Range w = kNothing;
    for (int b = tid; b < kBins; b += kThreads) w.sum += s.mass[b];
    const u64 all = block_range(s, w).sum;
    const u64 target = by_mass ? share(r.top_p, all) : (u64)r.k;
    find_bin(s, target, [&](int b) { return s.mass[b]; });
    const int bin = (int)s.bin;
    const uint32_t count = s.count[bin];
    const u64 rest = target - s.before;
    __syncthreads();
    // the bin's places into the list if they fit, and how far they go
    const bool fits = count <= kList;
    if (tid == 0) s.n = 0;
    __syncthreads();
    w = kNothing;
    over<B16>(p, off, 0, V, tid, kThreads, [&](float x, int64_t i) {
      const u64 c = place_of(x, i);
      if (c >= cut && bin_of(x) == bin) {
        join(w, 0, 0, c, c);
        if (fits) s.list[atomicAdd(&s.n, 1u)] = c;
      }
    });
    w = block_range(s, w);
    cut = resolve(s, w.lo, w.hi, count, rest,
                  [&](auto f) {
                    if (fits)
                      for (uint32_t i = tid; i < count; i += kThreads) f(s.list[i]);
                    else
                      over<B16>(p, off, 0, V, tid, kThreads,
                                [&](float x, int64_t i) { f(place_of(x, i)); });
                  },
                  [](u64 c) { return c; }, value);
  }
  const Kept value(weigh, cut, floor, V);
  const int wave = tid / 64;
  const int64_t each = ((V + kWaves - 1) / kWaves + 511) / 512 * 512, begin = wave * each;
  u64 sum = 0;
  over<B16, 4>(p, off, begin, begin + each < V ? begin + each : V, tid % 64, 64,
               [&](float x, int64_t i) { sum += value(x, i); });
  sum = wave_sum(sum);
  __syncthreads();
  if (tid % 64 == 0) s.wave2[wave] = sum;
  __syncthreads();
  u64 all = 0;
  for (int i = 0; i < kWaves; ++i) all += s.wave2[i];
  u64 rest = r.point(all);
  int w = 0;
  while (w < kWaves - 1 && rest >= s.wave2[w]) rest -= s.wave2[w++];
  const int64_t from = w * each;
  const u64 place = descend<B16, kWaves>(p, off, from, from + each < V ? from + each : V, rest,
                                         s.wave2, &s.found, value);
  if (tid == 0) answer(p, row, place, top, r.T, all);
}

// A row by a workgroup. What the cuts can keep is gathered into LDS first:
//   top-k : the k-th largest of the threads' maxima has k logits at or above it;
//   top-p alone : the weights are added up in bins of a 32nd of an octave, so that the run's
//           end is known to a bin, and the logits down to there are gathered;
// then each cut and the draw itself is a search among these, by the same steps. Of a run too long
// for LDS the last bin's logits alone are gathered, and on the way the weights of the bins before
// it added up for sixteen parts of the row: the cut is found in the bin, and the token in one part.
// 256 x 65536 bf16, top-p 0.95: 58 us, of them the maximum 6, the bins 16 to 20, gathering the bin
// and the sums 18, a search 4 to 6 (with the sums in a launch of their own behind the cut 51 + 23);
// 100 x 50021 f32 with every filter 27. Both are bound by the instructions of one workgroup. Slices
// of a row over several, in five launches, made a top-k slower (1 x 131072 32 us against 24) and a
// top-p of few rows faster (62 against 86), measured while both forms drew behind a long top-p in a
// launch of their own: not taken. 1 x 131072 top-p takes 61 here now, 8 rows 79.
template <bool B16>
__global__ __launch_bounds__(kThreads) void sample_cut_kernel(const SampleArgs p) {
  __shared__ Shared s;
  const int tid = threadIdx.x;
  const int64_t row = p.first + blockIdx.x, off = row * p.stride, V = p.vocab;
  constexpr int kWaves = kThreads / 64;
  uint32_t *const left = static_cast<uint32_t *>(p.workspace);  // of a row: sample_left_kernel's
  const bool small = V <= kList;  // the list takes the row
  Weigh::fill(s.power, p.shift, tid, kThreads);
  if (tid == 0 && !small) left[row] = 0;
  const Request r(p, row);
  const uint32_t mine = thread_top<B16>(p, off, 0, V, tid, kThreads);
  const Range tops = block_range(s, {0, 0, mine, mine});
  const uint32_t top_key = (uint32_t)tops.hi;
  if (!r.drawn(top_key)) {
    if (tid == 0) answer(p, row, -1, 0.0);
    return;
  }
  if (r.T == 0.0) {
    const u64 place = first_of<B16>(p, off, top_key, kThreads, &s.found);
    if (tid == 0) answer(p, row, (uint32_t)~(uint32_t)place, 0.0);
    return;
  }
  const float top = logit_of(top_key);
  const Weigh weigh(s.power, top, r.T);
  const u64 floor = r.floor(p.shift);
  const bool by_count = r.k > 0 && r.k < V, by_mass = r.top_p < 1.0;
  if (!small && (by_count ? r.k > kThreads : !by_mass)) {
    if (tid == 0) left[row] = 1;
    return;
  }
  u64 cut = 0;     // the least place that is kept
  u64 goal = 0;    // where top_p cuts the sum off, if that is known
  uint32_t n = 0;  // places in the list
  bool whole = true;  // the list holds all that is kept
  const uint32_t each = ((uint32_t)V + kWaves * 512 - 1) / (kWaves * 512) * 512;  // of a wave
  // Logits from `lowest` on into the list; a wave takes room for its eight times 64 at once.
  auto gather = [&](float lowest) {
    if (tid == 0) s.n = 0;
    __syncthreads();
    auto append = [&](uint32_t mine, auto get, int64_t id) {  // bit e: get(e) may go in
      if (__ballot(mine != 0) == 0) return;
      const uint32_t run = wave_run((uint32_t)__popc(mine));
      uint32_t room = 0;
      if (tid % 64 == 63 && run > 0) room = atomicAdd(&s.n, run);
      uint32_t to = (uint32_t)__builtin_amdgcn_readlane((int)room, 63) + run - __popc(mine);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (mine >> e & 1) {
          if (to < kList) s.list[to] = place_of(get(e), id + e);
          ++to;
        }
    };
    constexpr int kAhead = 4;
    const int64_t whole_runs = V / 8 * 8;
    const int runs = (int)(V / 8);
#pragma unroll 1
    for (int i0 = 0; i0 < runs; i0 += kAhead * kThreads) {  // all lanes stay: append speaks to them
      Vec8<B16> v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads + tid;
        v[u].load(p.logits, off + 8 * (int64_t)(i < runs ? i : runs - 1));
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads + tid;
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          mine |= v[u].get(e) >= lowest ? 1u << e : 0u;
        append(i < runs ? mine : 0, [&](int e) { return v[u].get(e); }, 8 * (int64_t)i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (tid < V - whole_runs) {  // the last few, one each
      const int64_t id = whole_runs + tid;
      const float x = B16 ? bf16_lo(static_cast<const uint16_t *>(p.logits)[off + id])
                          : static_cast<const float *>(p.logits)[off + id];
      if (x >= lowest) {
        const uint32_t to = atomicAdd(&s.n, 1u);
        if (to < kList) s.list[to] = place_of(x, id);
      }
    }
    __syncthreads();
    n = s.n;
    __syncthreads();
  };
  // Those of bin `only` into the list, and the weights of the bins before it added up for a part
  // of the row each.
  auto gather_bin = [&](int only) {
    if (tid == 0) s.n = 0;
    __syncthreads();
    const int lane = tid % 64, wave = tid / 64;
    const int64_t begin = (int64_t)wave * each;
    u64 sum = 0;
    over<B16, 2>(p, off, begin, begin + each < V ? begin + each : V, lane, 64,
                 [&](float x, int64_t id) {
                   const double d = weigh.below(x);
                   const int bin = weigh.bin_at(d);
                   const u64 w = weigh.raw_at(d) - Weigh::kNone;
                   sum += bin < only && w >= floor ? w : 0;
                   if (bin == only) {
                     const uint32_t to = atomicAdd(&s.n, 1u);
                     if (to < kList) s.list[to] = place_of(x, id);
                   }
                 });
    sum = wave_sum(sum);
    if (lane == 0) s.part[wave] = sum;
    __syncthreads();
    n = s.n;
    __syncthreads();
  };
  enum { kTops, kCount, kMass, kDraw };
  int stage = kCount;
  // what the next search goes over, where that is known without a look at the list
  Range known = kNothing;
  auto between = [&](uint32_t lo, uint32_t hi) {
    known = {0, n, (u64)lo << 32, (u64)hi << 32 | 0xFFFFFFFFu};
  };
  if (small) {
    gather(-__builtin_inff());
  } else if (by_count) {
    stage = kTops;
    s.list[tid] = (u64)mine << 32 | (uint32_t)~tid;
    n = kThreads;
    between((uint32_t)tops.lo, top_key);
    __syncthreads();
  } else {
    // The run ends above a weight of (1 - top_p) / vocab: from such a one on all weigh less than
    // 1 - top_p together, and the sum is at least 1. Smaller ones need no bin.
    const double part = r.top_p > 0.0 ? 1.0 - r.top_p : 1.0;
    const u64 tail = part_of(part / (double)V * (1.0 - 0x1p-50), 1ull << p.shift, false);
    clear_bins(s);
    Range w = kNothing;
    over<B16, 4>(p, off, 0, V, tid, kThreads, [&](float x, int64_t) {
      const double d = weigh.below(x);
      const u64 wx = weigh.raw_at(d) - Weigh::kNone;
      w.sum += wx;
      if (wx > tail) atomicAdd(&s.mass[weigh.bin_at(d)], wx);
    });
    goal = share(r.top_p, block_range(s, w).sum);
    find_bin(s, goal, [&](int b) { return s.mass[b]; });
    const int bin = (int)s.bin;
    const u64 before = s.before;
    __syncthreads();
    // how many logits that is, at most: none of a bin weighs as little as the next one's first
    w = kNothing;
    for (int b = tid; b <= bin; b += kThreads) {
      // 2^(shift - (b + 1) / kPerOctave)
      const double next = ldexp(s.power[-2 * (b + 1) & (kTable - 1)],
                                -(b + Weigh::kPerOctave) / Weigh::kPerOctave);
      w.sum += (u64)fmin((double)s.mass[b] / fmax(next - 1.0, 1.0) + 1.0, 0x1p40);
    }
    whole = block_range(s, w).sum <= kList;
    if (!whole) goal -= before;
    // from a little below the bin, which is behind the cut anyway; else a little more than the bin
    auto edge = [&](double steps, double slack) {
      const double x = (double)top - steps / weigh.rate;
      return (float)(x + slack * fabs(x));
    };
    const float lowest = edge(2 * bin + 1.75, -0x1p-20), highest = edge(2 * bin - 0.75, 0x1p-20);
    if (whole)
      gather(lowest);
    else
      gather_bin(bin);
    between(key_of(lowest), whole ? top_key : key_of(highest));
    if (n > kList) {
      if (tid == 0) left[row] = 1;
      return;
    }
  }
  for (; stage <= kDraw; ++stage) {
    if ((stage == kCount && !by_count) || (stage == kMass && !by_mass)) continue;
    if (stage == kDraw && !whole) break;
    const u64 least = stage == kDraw ? floor : 0;
    auto value = [&](u64 c) {
      if (stage < kMass) return 1ull;
      const u64 w = c >= cut ? weigh(c) : 0;
      return w >= least ? w : 0;
    };
    auto order = [&](u64 c) { return stage == kDraw ? (u64)(uint32_t)c : c; };
    auto walk = [&](auto f) {
      for (uint32_t i = tid; i < n; i += kThreads) {
        const u64 c = s.list[i];
        if (c >= cut && (stage != kDraw || value(c) > 0)) f(c);
      }
    };
    Range w = known;
    known = kNothing;
    if (w.count == 0) {
      walk([&](u64 c) { join(w, value(c), 1, order(c), order(c)); });
      w = block_range(s, w);
    }
    u64 target = (u64)r.k;
    if (stage == kMass) target = goal ? goal : share(r.top_p, w.sum);
    if (stage == kDraw) target = r.point(w.sum) + 1;
    const u64 found = resolve(s, w.lo, w.hi, w.count, target, walk, order, value);
    if (stage == kDraw) {
      if (tid == 0) answer(p, row, found, top, r.T, w.sum);
    } else if (stage == kTops) {
      gather(logit_of((uint32_t)(found >> 32)));
      between((uint32_t)(found >> 32), top_key);
      if (n > kList) {
        if (tid == 0) left[row] = 1;
        return;
      }
    } else {
      cut = found;
    }
  }
  if (whole) return;
  // the bin's part of the cut among the parts of the row, then the draw from one of them
  for (uint32_t i = tid; i < n; i += kThreads) {
    const u64 c = s.list[i], w = weigh(c);
    if (c >= cut && w >= floor)
      atomicAdd(&s.part[~(uint32_t)c / each], w);
  }
  __syncthreads();
  u64 all = 0;
  for (int i = 0; i < kWaves; ++i) all += s.part[i];
  u64 rest = r.point(all);
  int w = 0;
  while (w < kWaves - 1 && rest >= s.part[w]) rest -= s.part[w++];
  const int64_t from = (int64_t)w * each;
  const u64 place = descend<B16, kWaves>(p, off, from, from + each < V ? from + each : V, rest,
                                         s.wave2, &s.found, Kept(weigh, cut, floor, V));
  if (tid == 0) answer(p, row, place, top, r.T, all);
}

bool cuts(const SampleArgs &a) { return a.top_ks || a.top_k > 0 || a.top_ps || a.top_p < 1.0; }

// Slices where rows alone leave half of the 256 compute units idle and a row is long enough to
// pay for three launches.
constexpr int64_t kSliceUnit = 512 * kSliceWaves;
Slices slices_of(const SampleArgs &a) {
  Slices s{1, 0, nullptr, nullptr};
  if (a.rows == 0 || cuts(a) || a.rows > 128 || a.vocab < 16384) return s;
  const int64_t want = std::min<int64_t>(512 / a.rows, (a.vocab + kSliceUnit - 1) / kSliceUnit);
  s.each = ((a.vocab + want - 1) / want + kSliceUnit - 1) / kSliceUnit * kSliceUnit;
  s.count = (a.vocab + s.each - 1) / s.each;
  return s;
}

}  // namespace

int64_t sample_workspace_bytes(const SampleArgs &a) {
  const Slices s = slices_of(a);
  const int64_t slices = s.count > 1 ? a.rows * s.count * 12 : 0;
  // what is left of each row; a row's own parameters, which the sizes do not show, may cut too
  const int64_t left = a.vocab > kList ? a.rows * 4 : 0;
  return (std::max(slices, left) + 255) / 256 * 256;
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  SampleArgs args = a;
  Slices s = slices_of(a);
  if (s.count > 1) {
    s.sums = static_cast<u64 *>(a.workspace);
    s.tops = reinterpret_cast<uint32_t *>(s.sums + a.rows * s.count);
    void *kargs[] = {&args, &s};
    const void *fns[3] = {
        a.bf16 ? (const void *)sample_tops_kernel<true> : (const void *)sample_tops_kernel<false>,
        a.bf16 ? (const void *)sample_sums_kernel<true> : (const void *)sample_sums_kernel<false>,
        a.bf16 ? (const void *)sample_slice_kernel<true> : (const void *)sample_slice_kernel<false>};
    for (int i = 0; i < 3; ++i) {
      const hipError_t e = hipLaunchKernel(
          fns[i], dim3((unsigned)(i < 2 ? a.rows * s.count : a.rows)), dim3(kSliceThreads), kargs, 0, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const void *fn = cuts(a) ? (a.bf16 ? (const void *)sample_cut_kernel<true>
                                     : (const void *)sample_cut_kernel<false>)
                           : (a.bf16 ? (const void *)sample_plain_kernel<true>
                                     : (const void *)sample_plain_kernel<false>);
  const void *left = a.bf16 ? (const void *)sample_left_kernel<true>
                            : (const void *)sample_left_kernel<false>;
  constexpr int64_t kMost = 1 << 21;  // rows of a launch: 2^31 threads
  for (args.first = 0; args.first < a.rows; args.first += kMost) {
    void *kargs[] = {&args};
    const dim3 grid((unsigned)std::min<int64_t>(a.rows - args.first, kMost));
    hipError_t e = hipLaunchKernel(fn, grid, dim3(kThreads), kargs, 0, stream);
    if (e == hipSuccess && cuts(a) && a.vocab > kList)
      e = hipLaunchKernel(left, grid, dim3(kThreads), kargs, 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gdn
