// Tokens drawn from logits with temperature, top-k, top-p and min-p, for gfx950.
//
// A token's weight is a whole number, exp((x - max) / T) in units of 2^-shift, so sums of weights
// are exact and the order of the additions, in LDS atomics too, changes nothing. Every filter
// keeps the head of one order, falling logits and rising ids among equal ones; a token's place in
// it is a 64-bit number (the logit's bits made to order like integers above, the inverted id
// below) and a filter is the least such number that it keeps. The draw goes by rising id.

#include <algorithm>

#include "policy_rows.hpp"
#include "step_internal.h"

namespace gdn {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kList = 4096;       // candidates that LDS holds
constexpr int kFew = 64;          // candidates that one wave ranks
constexpr float kBinsPerNat = 64.0f;
constexpr int kTable = 1024;      // steps of an octave in the table of powers of two

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

struct Shared {
  double power[kTable];  // 2^(i / kTable)
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 list[kList];
  u64 few[kFew];
  u64 wave[kWaves], wave2[kWaves];
  u64 found, before;
  uint32_t n, bin, held;
};

template <class F>
__device__ __forceinline__ u64 block_reduce(Shared &s, u64 v, F f) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v = f(v, (u64)__shfl_xor(v, d));
  __syncthreads();
  if (threadIdx.x % 64 == 0) s.wave[threadIdx.x / 64] = v;
  __syncthreads();
  v = s.wave[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v = f(v, s.wave[i]);
  return v;
}

// exp((x - top) / T) in units of 2^-shift, to the nearest: y = (x - top) log2(e) / T in steps of
// the table is split into a whole number and a rest of at most half a step, whose power of two
// four terms of its series give to 2^-51.
struct Weigh {
  const double *power;
  double top, rate;  // rate: kTable log2(e) / T
  int shift;
  __device__ __forceinline__ u64 operator()(float x) const {
    double y = ((double)x - top) * rate;
    y = fmax(y, -64.0 * kTable);  // a weight of 0
    const double magic = 0x1.8p52, t = y + magic;
    const int n = (int)(uint32_t)(u64)__double_as_longlong(t);
    const double r = y - (t - magic);
    constexpr double c = 0.69314718055994530942 / kTable;
    const double q = r * (c + r * (c * c / 2 + r * (c * c * c / 6)));
    const double w = power[n & (kTable - 1)];
    const double e = ldexp(fma(w, q, w), (n >> 10) + shift);
    return (u64)__double_as_longlong(e + 0x1p52) - (u64)__double_as_longlong(0x1p52);
  }
  __device__ __forceinline__ u64 operator()(u64 place) const {
    return (*this)(logit_of((uint32_t)(place >> 32)));
  }
};

// The bin, of those that `value(b)` weighs, in which the running sum passes `target` (at least
// 1, at most all of them): its number in s.bin, the sum before it in s.before.
template <class F>
__device__ __forceinline__ void find_bin(Shared &s, u64 target, F value) {
  constexpr int each = kBins / kThreads;
  const int t = threadIdx.x;
  u64 v[each], sum = 0;
#pragma unroll
  for (int i = 0; i < each; ++i) sum += v[i] = value(each * t + i);
  u64 run = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const u64 o = __shfl_up(run, d);
    if (t % 64 >= d) run += o;
  }
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

// The candidate at which the running sum of weigh(c), by falling order(c), passes `target`.
// walk(f) calls f(c) for every candidate; those whose order is in [lo, hi] count, `count` of
// them, with a sum of target and more.
template <class Walk, class Order, class Value>
__device__ __forceinline__ u64 resolve(Shared &s, u64 lo, u64 hi, uint32_t count, u64 target,
                                       Walk walk, Order order, Value weigh) {
  while (count > kFew) {
    const int bits = 64 - __clzll((long long)(hi - lo) | 1);
    const int shift = bits > 11 ? bits - 11 : 0;
    clear_bins(s);
    walk([&](u64 c) {
      const u64 o = order(c);
      if (o >= lo && o <= hi) {
        const int b = (int)((hi - o) >> shift);
        atomicAdd(&s.mass[b], weigh(c));
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
  if (threadIdx.x < 64) {
    const int n = (int)s.n;
    const u64 c = threadIdx.x < n ? s.few[threadIdx.x] : 0;
    const u64 w = threadIdx.x < n ? weigh(c) : 0, o = order(c);
    u64 before = 0;
    for (int j = 0; j < n; ++j) {
      const u64 oj = __shfl(o, j), wj = __shfl(w, j);
      if (oj > o) before += wj;
    }
    if (before < target && target <= before + w) s.found = c;
  }
  __syncthreads();
  const u64 c = s.found;
  __syncthreads();
  return c;
}

// One row a workgroup at a time.
template <bool B16>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs p) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int64_t V = p.vocab;
  s.power[tid] = exp2((double)tid / kTable);
  auto add = [](u64 a, u64 b) { return a + b; };
  auto most = [](u64 a, u64 b) { return a > b ? a : b; };
  auto least = [](u64 a, u64 b) { return a < b ? a : b; };

  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t off = row * p.stride;
    // f(x, id) for ids [from, to) of the row: `threads` threads from `first` on, eight ids each
    auto over = [&](int64_t from, int64_t to, int first, int threads, auto f) {
      for (int64_t col = from + 8 * first; col < to; col += 8 * threads) {
        Vec8<B16> v;
        load_row(v, p.logits, off, col, V);
        settle_row(v, col, V);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < to) f(v.get(e), col + e);
      }
    };
    uint32_t best = 0;
    uint32_t at = 0;
    over(0, V, tid, kThreads, [&](float x, int64_t id) {
      const uint32_t k = key_of(x);
      if (k > best) {
        best = k;
        at = (uint32_t)id;
      }
    });
    const u64 head = block_reduce(s, (u64)best << 32 | (uint32_t)~at, most);
    const uint32_t top_key = (uint32_t)(head >> 32);
    const double T = p.temperatures ? (double)p.temperatures[row] : p.temperature;
    int64_t id = -1;
    double logp = 0.0;
    const bool drawn = top_key > kMinusInfinity && top_key < kInfinity && T >= 0.0 &&
                       T < __builtin_inf();
    if (drawn && T == 0.0) {
      id = (uint32_t)~(uint32_t)head;
    } else if (drawn) {
      const float top = logit_of(top_key);
      const Weigh weigh{s.power, (double)top, 1.4426950408889634074 * kTable / T, p.shift};
      const float bins = (float)fmin((double)kBinsPerNat / T, 0x1p100);
      auto bin_of = [&](float x) { return (int)fminf((top - x) * bins, (float)(kBins - 1)); };
      const int64_t k = p.top_ks ? (int64_t)p.top_ks[row] : p.top_k;
      const double top_p = p.top_ps ? (double)p.top_ps[row] : p.top_p;
      const double min_p = p.min_ps ? (double)p.min_ps[row] : p.min_p;
      const double u = p.u64 ? static_cast<const double *>(p.u)[row]
                             : (double)static_cast<const float *>(p.u)[row];
      const u64 unit = 1ull << p.shift;
      const u64 floor = !(min_p > 0.0) ? 0 : min_p >= 1.0 ? unit : part_of(min_p, unit, true);
      u64 cut = 0;  // the least place that is kept
      bool listed = false;  // s.list holds the places that are kept, n of them
      uint32_t n = 0;
      auto in_row = [&](auto f) {
        over(0, V, tid, kThreads, [&](float x, int64_t i) { f(place_of(x, i)); });
      };
      auto in_list = [&](auto f) {
        for (uint32_t i = tid; i < n; i += kThreads) f(s.list[i]);
      };
      auto itself = [](u64 c) { return c; };
      // The places from `from` on, of bin `only` where it is one, into the list, or none if
      // there are more than it holds.
      auto gather = [&](u64 from, int only) {
        if (tid == 0) s.n = 0;
        __syncthreads();
        over(0, V, tid, kThreads, [&](float x, int64_t i) {
          const u64 c = place_of(x, i);
          if (c >= from && (only < 0 || bin_of(x) == only)) {
            const uint32_t to = atomicAdd(&s.n, 1u);
            if (to < kList) s.list[to] = c;
          }
        });
        __syncthreads();
        n = s.n;
        __syncthreads();
        return n <= kList;
      };
      // The place in the row, of those from `cut` on, at which the sum of value(place) passes
      // target(sum of all).
      auto select = [&](auto target_of, auto value) {
        clear_bins(s);
        over(0, V, tid, kThreads, [&](float x, int64_t i) {
          const u64 c = place_of(x, i);
          if (c >= cut) {
            const int b = bin_of(x);
            atomicAdd(&s.mass[b], value(c));
            atomicAdd(&s.count[b], 1u);
          }
        });
        __syncthreads();
        u64 all = 0;
        for (int b = tid; b < kBins; b += kThreads) all += s.mass[b];
        const u64 target = target_of(block_reduce(s, all, add));
        find_bin(s, target, [&](int b) { return s.mass[b]; });
        const int bin = (int)s.bin;
        const uint32_t count = s.count[bin];
        const u64 rest = target - s.before;
        __syncthreads();
        u64 lo = ~0ull, hi = 0;
        auto widen = [&](u64 c) {
          lo = least(lo, c);
          hi = most(hi, c);
        };
        const bool fits = count <= kList && gather(cut, bin);
        if (fits)
          in_list(widen);
        else
          over(0, V, tid, kThreads, [&](float x, int64_t i) {
            const u64 c = place_of(x, i);
            if (c >= cut && bin_of(x) == bin) widen(c);
          });
        lo = block_reduce(s, lo, least);
        hi = block_reduce(s, hi, most);
        return fits ? resolve(s, lo, hi, count, rest, in_list, itself, value)
                    : resolve(s, lo, hi, count, rest, in_row, itself, value);
      };
      if (k > 0 && k < V) {
        cut = select([&](u64) { return (u64)k; }, [](u64) { return 1ull; });
        listed = k <= kList && gather(cut, -1);
      }
      if (top_p < 1.0) {
        auto target = [&](u64 all) { return most(part_of(top_p, all, true), 1ull); };
        if (listed) {
          u64 all = 0, lo = ~0ull, hi = 0;
          in_list([&](u64 c) {
            all += weigh(c);
            lo = least(lo, c);
            hi = most(hi, c);
          });
          all = block_reduce(s, all, add);
          lo = block_reduce(s, lo, least);
          hi = block_reduce(s, hi, most);
          cut = resolve(s, lo, hi, n, target(all), in_list, itself, weigh);
        } else {
          cut = select(target, weigh);
          listed = gather(cut, -1);
        }
      }
      auto kept = [&](u64 c) {
        const u64 w = c >= cut ? weigh(c) : 0;
        return w >= floor ? w : 0;
      };
      u64 all = 0, pick = 0;
      auto point = [&]() { return u >= 1.0 ? all - 1 : part_of(u, all, false); };
      if (listed) {
        u64 lo = ~0ull, hi = 0;
        in_list([&](u64 c) {
          all += kept(c);
          lo = least(lo, (uint32_t)c);
          hi = most(hi, (uint32_t)c);
        });
        all = block_reduce(s, all, add);
        lo = block_reduce(s, lo, least);
        hi = block_reduce(s, hi, most);
        pick = resolve(s, lo, hi, n, point() + 1, in_list,
                       [](u64 c) { return (u64)(uint32_t)c; }, kept);
      } else {
        // a part of the row for each wave, then of that part, down to 512 ids
        int64_t from = 0, to = V;
        u64 rest = 0;
        for (bool first = true; first || to - from > 512; first = false) {
          const int64_t each = ((to - from + kWaves - 1) / kWaves + 511) / 512 * 512;
          const int64_t begin = from + wave * each, end = begin + each < to ? begin + each : to;
          u64 sum = 0;
          over(begin, end, lane, 64, [&](float x, int64_t i) { sum += kept(place_of(x, i)); });
#pragma unroll
          for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
          __syncthreads();
          if (lane == 0) s.wave2[wave] = sum;
          __syncthreads();
          if (first) {
            for (int i = 0; i < kWaves; ++i) all += s.wave2[i];
            rest = point();
          }
          int w = 0;
          while (w < kWaves - 1 && rest >= s.wave2[w]) rest -= s.wave2[w++];
          from += w * each;
          to = from + each < to ? from + each : to;
        }
        if (wave == 0) {
          u64 sum = 0;
          over(from, to, lane, 64, [&](float x, int64_t i) { sum += kept(place_of(x, i)); });
          u64 run = sum;
#pragma unroll
          for (int d = 1; d < 64; d *= 2) {
            const u64 o = __shfl_up(run, d);
            if (lane >= d) run += o;
          }
          u64 before = run - sum;
          if (before <= rest && rest < run)
            over(from, to, lane, 64, [&](float x, int64_t i) {
              const u64 c = place_of(x, i), w = kept(c);
              if (before <= rest && rest < before + w) s.found = c;
              before += w;
            });
        }
        __syncthreads();
        pick = s.found;
      }
      id = (uint32_t)~(uint32_t)pick;
      logp = ((double)logit_of((uint32_t)(pick >> 32)) - (double)top) / T -
             log(ldexp((double)all, -p.shift));
    }
    if (tid == 0) {
      if (p.id64)
        static_cast<int64_t *>(p.ids)[row] = id;
      else
        static_cast<int32_t *>(p.ids)[row] = (int32_t)id;
      p.logp[row] = (float)logp;
    }
    __syncthreads();
  }
}

}  // namespace

int64_t sample_workspace_bytes(const SampleArgs &) { return 0; }

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  SampleArgs args = a;
  void *kargs[] = {&args};
  const void *fn = a.bf16 ? (const void *)sample_kernel<true> : (const void *)sample_kernel<false>;
  return hipLaunchKernel(fn, dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(kThreads),
                         kargs, 0, stream);
}

}  // namespace gdn
