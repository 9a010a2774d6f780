// The 8-bit integer linear region on gfx950: rows quantised with one scale each, and
// Y = (xq wq^T) x_scale w_scale on the int8 matrix instructions.
//
// The sums of products are exact 32-bit integers, so neither tile nor schedule nor the number
// of rows changes a bit of Y; only the epilogue rounds (integer to binary32, two products,
// and the rounding to Y's type).

#include <algorithm>

#include "policy_internal.h"
#include "policy_rows.hpp"

namespace gdn {
namespace {

using i32x4 = int __attribute__((ext_vector_type(4)));
using f32x4 = float __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------- quantisation

// The rounding of 127 x / a goes through the sum with 1.5 * 2^23, whose last place is 1: the
// sum rounds to an integer, ties to even, and its low byte is that integer's.
constexpr float kToInteger = 12582912.0f;

// 127 x / a rounded to the nearest integer, ties to even, in the low byte, for |x| <= a;
// n = 127 x (exact in binary32 for bf16 x), inv = 1 / a rounded. The product with inv is
// within a unit or two of the quotient's last place, which matters only where the exact
// quotient is a half: one step with the exact remainder then gives the half itself, and the
// sum decides the tie. A quotient q in [2^k, 2^(k+1)) of 8-bit numerator and denominator
// significands that is no half lies at least 2^(k-17) from one; the corrected quotient is off
// by less than 2^(k-23).
__device__ __forceinline__ uint32_t quotient(float n, float a, float inv) {
  float q = n * inv;
  q = fmaf(fmaf(-q, a, n), inv, q);
  return __float_as_uint(q + kToInteger);
}

// binary32 x: 127 x takes 31 bits, so the same in binary64.
__device__ __forceinline__ uint32_t quotient(double n, double a, double inv) {
  double q = n * inv;
  q = fma(fma(-q, a, n), inv, q);
  return __float_as_uint((float)rint(q) + kToInteger);
}

// Bytes 0 of four words, the first lowest.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
  return ab | cd;
}

// Largest |x| of eight values as binary32 bits: those order like integers, a NaN above all.
__device__ __forceinline__ uint32_t abs_top(const Vec8<true> &v) {
  using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v.r[i] & 0x7FFF7FFFu));
  return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}
__device__ __forceinline__ uint32_t abs_top(const Vec8<false> &v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v.get(e)) & 0x7FFFFFFFu);
  return m;
}

template <int N>
__device__ __forceinline__ uint32_t max_rotated(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 | N, 0xF, 0xF, true));
}

// Workgroups; more rows are walked over. Rows of more than kLongRow values: 262144 threads in all
// (2000 x 30000 bf16 34.5 us, with 2048 workgroups 41).
constexpr int kQuantizeGrid = 2048, kLongRow = 16384, kLongThreads = 262144;

// G lanes share a row: 16, or 64 (then row_threads / 64 waves do). NV runs of eight values a
// thread. A workgroup walks over rows, the next row's loads in flight under this one. Bound by
// memory: 16384 x 4096 bf16 39 us (5.1 TB/s).
template <bool B16, int G, int NV>
__global__ __launch_bounds__(1024) void quantize_kernel(const QuantizeArgs p) {
  __shared__ uint32_t slot[2][16];
  const int T = G == 64 ? p.row_threads : G, groups = (int)blockDim.x / T;
  const int t = threadIdx.x % T, g = threadIdx.x / T, waves = T / 64;
  auto load = [&](Vec8<B16> (&x)[NV], int64_t row) {  // past the end the last row, unwritten
    if (row >= p.rows) row = p.rows - 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) load_row(x[j], p.x, row * p.x_stride, 8 * (j * T + t), p.k);
  };
  const int64_t step = (int64_t)gridDim.x * groups;
  constexpr bool kAhead = NV <= 4;
  Vec8<B16> x[NV], next[kAhead ? NV : 1];
  if (kAhead) load(x, (int64_t)blockIdx.x * groups + g);
  int par = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += step, par ^= 1) {
    const int64_t row = r0 + g;
    if constexpr (kAhead) {
      if (r0 + step < p.rows) load(next, row + step);
    } else {
      load(x, row);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) settle_row(x[j], 8 * (j * T + t), p.k);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) top = max(top, abs_top(x[j]));
    top = max_rotated<8>(top);
    top = max_rotated<4>(top);
    top = max_rotated<2>(top);
    top = max_rotated<1>(top);
    if constexpr (G == 64) {
      auto of = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)top, lane); };
      top = max(max(of(0), of(16)), max(of(32), of(48)));
      if (waves > 1) {
        const int wave = threadIdx.x / 64, first = wave / waves * waves;
        if (threadIdx.x % 64 == 0) slot[par][wave] = top;
        __syncthreads();
        for (int i = 0; i < waves; ++i) top = max(top, slot[par][first + i]);
      }
    }
    if (row < p.rows) {
      const float a = __uint_as_float(top);
      if (t == 0) p.scale[row] = a / 127.0f;
      // the inverse of a subnormal a is not finite and 127 times a large one neither: scale the
      // row and its maximum by a power of two first
      const float up = a < 0x1p-100f ? 0x1p+120f : a > 0x1p+100f ? 0x1p-100f : 1.0f, as = a * up;
      const bool plain = a > 0.0f && a < __builtin_inff();
      const float inv = 1.0f / as;
      const double inv64 = B16 ? 0.0 : 1.0 / (double)as;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = 8 * (j * T + t);
        if (col >= p.k_pad) break;
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[j].get(e);
          if (plain)
            q[e] = B16 ? quotient(127.0f * up * v, as, inv)
                       : quotient(127.0 * (double)(v * up), (double)as, inv64);
          else  // +-127 at the infinities of a row without NaN, else 0
            q[e] = a > 0.0f && fabsf(v) == a ? (v > 0.0f ? 127 : -127) : 0;
        }
        *reinterpret_cast<uint2 *>(p.q + row * p.k_pad + col) =
            make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
      }
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < NV; ++j) x[j] = next[j];
    }
  }
}

template <int G, int NV>
const void *quantize_fn(const QuantizeArgs &a) {
  return a.x_bf16 ? (const void *)quantize_kernel<true, G, NV>
                  : (const void *)quantize_kernel<false, G, NV>;
}

// ------------------------------------------------------------------------------ product

// v_mfma_i32_16x16x64_i8: lane l gives row l % 16 of either operand at k = 16 (l / 16) .. + 15,
// and holds the results of rows 4 (l / 16) .. + 3 of the first operand and row l % 16 of the
// second. The first operand is W, so a lane's four results are neighbours in a row of Y.
__device__ __forceinline__ i32x4 mfma(i32x4 w, i32x4 x, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}

__device__ __forceinline__ f32x4 scaled(i32x4 acc, float xs, f32x4 ws) {
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = (float)acc[r] * xs * ws[r];
  return v;
}

// Results of a lane as they are stored: sums of a part of K as their bits.
__device__ __forceinline__ f32x4 results(const LinearI8Args &p, i32x4 acc, float xs, f32x4 ws) {
  return p.parts ? __builtin_bit_cast(f32x4, acc) : scaled(acc, xs, ws);
}

__device__ __forceinline__ f32x4 column_scales(const LinearI8Args &p, int64_t n) {
  f32x4 ws;
#pragma unroll
  for (int r = 0; r < 4; ++r) ws[r] = p.w_scale[n + r < p.n ? n + r : p.n - 1];
  return ws;
}

// Few rows (16 x 4096 x 4096: 7.2 us of which 2 to 3 are a launch; its 16.8 MB of W at 4.9
// TB/s are 3.4): W's bytes are what counts, each read once by a group of 16 MT rows, straight into
// the operand registers. A workgroup takes 16 NT columns; its eight waves take the 128-byte
// lines of K in turn and their integer sums are added in LDS.
template <int MT, int NT, bool YB>
__global__ __launch_bounds__(512) void linear_i8_rows_kernel(const LinearI8Args p) {
  constexpr int U = MT * NT == 4 ? 1 : 2;  // lines of K a turn, the next in flight
  __shared__ i32x4 part[8][NT * MT][64];
  const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t tiles_n = (p.n + 16 * NT - 1) / (16 * NT);
  const int64_t n0 = blockIdx.x % tiles_n * (16 * NT), m0 = blockIdx.x / tiles_n * (16 * MT);
  const int k0 = (int)blockIdx.y * p.k_part, kn = min(p.k_part, p.k - k0);
  const int8_t *w[NT], *x[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t row = n0 + 16 * j + l % 16;
    w[j] = p.wq + (row < p.n ? row : p.n - 1) * p.k + k0 + 16 * (l / 16);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = m0 + 16 * i + l % 16;
    x[i] = p.xq + (row < p.m ? row : p.m - 1) * p.k + k0 + 16 * (l / 16);
  }
  i32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  auto at = [](const int8_t *b, int k) { return *reinterpret_cast<const i32x4 *>(b + k); };
  const int lines = kn / 128;
  struct Turn {
    i32x4 w[U][2][NT], x[U][2][MT];
  };
  auto load = [&](Turn &t, int line) {  // a line past the end is zeros
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = line + 8 * u < lines;
        const int k = in ? (line + 8 * u) * 128 + 64 * h : 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) t.w[u][h][j] = in ? at(w[j], k) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MT; ++i) t.x[u][h][i] = in ? at(x[i], k) : i32x4{0, 0, 0, 0};
      }
  };
  auto multiply = [&](const Turn &t) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[j][i] = mfma(t.w[u][h][j], t.x[u][h][i], acc[j][i]);
  };
  Turn t0, t1;
  load(t0, wave);
  for (int line = wave; line < lines; line += 16 * U) {
    load(t1, line + 8 * U);
    multiply(t0);
    load(t0, line + 16 * U);
    multiply(t1);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][j * MT + i][l] = acc[j][i];
  __syncthreads();
  if (wave < NT * MT) {  // wave j MT + i finishes columns 16 j .. + 15 of rows 16 i .. + 15
    i32x4 sum = part[0][wave][l];
#pragma unroll
    for (int v = 1; v < 8; ++v) sum += part[v][wave][l];
    const int64_t m = m0 + wave % MT * 16 + l % 16, n = n0 + wave / MT * 16 + 4 * (l / 16);
    if (m < p.m) {
      const f32x4 v = results(p, sum, p.x_scale[m], column_scales(p, n));
      float *part = p.parts ? p.parts + blockIdx.y * p.m * p.n : static_cast<float *>(p.y);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < p.n) {
          if (YB)
            static_cast<uint16_t *>(p.y)[m * p.n + n + r] = to_bf16(v[r]);
          else
            part[m * p.n + n + r] = v[r];
        }
    }
  }
}

// Sixteen bytes of row m of Y from column n on: 4 binary32 or 8 bf16 values.
template <bool YB, bool Through>
__device__ __forceinline__ void store_chunk(const LinearI8Args &p, void *to, int64_t m, int64_t n,
                                            i32x4 v) {
  using unaligned = int __attribute__((ext_vector_type(4), aligned(YB ? 2 : 4)));
  constexpr int kChunk = YB ? 8 : 4;
  if (n + kChunk <= p.n) {
    char *y = static_cast<char *>(to) + (m * p.n + n) * (YB ? 2 : 4);
    if (Through)
      __builtin_nontemporal_store(v, reinterpret_cast<unaligned *>(y));
    else
      *reinterpret_cast<unaligned *>(y) = v;
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (n + e < p.n) {
        if (YB)
          static_cast<uint16_t *>(to)[m * p.n + n + e] =
              (uint16_t)((uint32_t)v[e / 2] >> (16 * (e % 2)));
        else
          static_cast<int *>(to)[m * p.n + n + e] = v[e];
      }
  }
}

// A BN x BM tile of Y by (BN / TN) x (BM / TM) waves, each TN columns by TM rows.
//
// K goes through LDS in stages of 64 bytes of every row of the tile, four buffers of one
// stage each: loads straight from memory into LDS run three stages ahead, and the operands
// of the next stage are read from LDS under the products of the current one, interleaved
// with them. A stage has one barrier: past it, the next stage has arrived for every wave and
// the buffer of the current one, in registers by now, is free for the stage four ahead.
//
// The loads are the instruction itself: it has no destination register, and as the compiler's
// builtin every later read of LDS waits for all of them. So the waits for them are written
// out (arrive), and nothing else in the loop goes through the vector memory counter.
//
// A row's 64 bytes are four 16-byte chunks, chunk c of row r at place c ^ key(r), so that the
// lanes of an operand read spread over the LDS banks. 16 lanes are served together, measured
// by which keys conflict: 0 - 3, 12 - 15 and 20 - 27, that is chunk c of rows 0 - 3 and 12 - 15
// with chunk c ^ 1 of rows 4 - 11, and the same for the other half of the wave; the keys 0, 0,
// 3, 3 of four rows each give these 16 places of the 256 bytes that the banks hold. The loads
// fill LDS in the order of their lanes, so the permutation is in which chunk a lane fetches.
//
// Bound by the matrix units and the power they draw: 8192 x 8192 x 8192 to bf16 takes 456 us
// (2410 TOP/s), 16384 x 4096 x 4096 228 us to bf16 (2410) and 237 to binary32 (2320); products
// of random bytes in registers alone reach 3200 TOP/s (4700 of zeros, at a higher clock).
// Tried and slower: waves of 128 x 128 (300 us), two workgroups a unit with tiles of 256 x 128
// and three stages (282), tiles taken in turn by 256 workgroups (its state did not fit beside
// 128 sums a lane).
//
// Results go through LDS as well, 16 rows of a wave at a time, so that neighbouring lanes
// store neighbouring values. With Through the stores bypass the caches, which hold the operands
// (16384 x 4096 x 4096 to binary32 237 us against 263, 256 x 65536 x 4096 to bf16 75 against
// 82). Where rows start inside a 16-byte chunk the caches put the parts of a line together:
// 597 x 38941 x 293 to binary32 took 47 us past them and 33 through them.
__device__ __forceinline__ int chunk_key(int r) { return (r >> 3 & 1) * 3; }

// 16 bytes per lane from base + offset to LDS, lane after lane from `to` (uniform) on.
__device__ __forceinline__ void load_to_lds(const int8_t *base, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"  // a wait state between writing m0 and its use
      "global_load_lds_dwordx4 %1, %2"
      :: "s"(to), "v"(offset), "s"(base) : "memory", "m0");
}

// At most `Loads` of the wave's loads are still on their way, every read of LDS is done, and
// all waves are here.
template <int Loads>
__device__ __forceinline__ void arrive() {
  static_assert(Loads < 64, "six bits of the counter");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Loads) : "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt = 0, which the compiler then knows
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int BM, int BN, int TM, int TN, bool YB, bool Through>
__global__ __launch_bounds__(BM / TM *(BN / TN) * 64) __attribute__((amdgpu_waves_per_eu(TM * TN > 8192 ? 1 : 2)))
void linear_i8_tile_kernel(const LinearI8Args p) {
  constexpr int kWaves = BM / TM * (BN / TN), MI = TM / 16, NJ = TN / 16;
  constexpr int kLoads = (BM + BN) / 16 / kWaves;  // 1 KiB (16 rows) each, per wave and stage
  constexpr int kStage = (BM + BN) * 64;
  static_assert((BM + BN) / 16 % kWaves == 0, "whole loads");
  static_assert(kStage * 4 / kWaves >= 16 * TN * 4, "a wave's share of LDS holds 16 rows");
  __shared__ __align__(128) int8_t lds[4 * kStage];
  const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // tiles: each XCD (workgroup % 8) a run of neighbours, in bands of 8 tiles of rows
  const int64_t tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
  const int64_t total = tiles_m * tiles_n, per = (total + 7) / 8;
  const int64_t tile = blockIdx.x % 8 * per + blockIdx.x / 8;
  if (tile >= total) return;
  const int64_t band = tile / (8 * tiles_n), in_band = tile % (8 * tiles_n);
  const int64_t height = tiles_m - 8 * band < 8 ? tiles_m - 8 * band : 8;
  const int64_t m0 = (8 * band + in_band % height) * BM, n0 = in_band / height * BN;

  // the wave's loads of a stage: a base in scalar registers and an offset per lane (below
  // 256 rows of 2^16 bytes); rows past the end repeat the last one
  const int k0 = (int)blockIdx.y * p.k_part, kn = min(p.k_part, p.k - k0);
  const int8_t *wbase = p.wq + n0 * p.k + k0, *xbase = p.xq + m0 * p.k + k0;
  const int last_w = (int)(p.n - n0 < BN ? p.n - n0 : BN) - 1;
  const int last_x = (int)(p.m - m0 < BM ? p.m - m0 : BM) - 1;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = (wave * kLoads + i) * 16, r = at + l / 4;  // W's rows, then X's
    const int row = at < BN ? (r < last_w ? r : last_w) : (r - BN < last_x ? r - BN : last_x);
    off[i] = (uint32_t)row * p.k + 16 * (l % 4 ^ chunk_key(r));
  }
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)lds + wave * kLoads * 1024);
  // Each XCD takes the stages around K from a place of its own: were all workgroups at the same
  // k of rows 2^n bytes apart, they would ask the same few memory channels (16 x 65536 x 4096
  // takes 61 us that way against 51, 256 rows 83 against 75). Those of an XCD keep in step,
  // for the operands they share in its L2. The sums are integers: the order changes nothing.
  int fk = (int)(blockIdx.x % 8) * (kn / 64) / 8 * 64;
  auto fetch = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds(((wave * kLoads + i) * 16 < BN ? wbase : xbase) + fk, off[i],
                  lds_at + buf * kStage + i * 1024);
    fk = fk + 64 < kn ? fk + 64 : 0;
  };

  i32x4 acc[NJ][MI], xf[2][MI], wf[2][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  const int wn = wave % (BN / TN) * TN, wm = wave / (BN / TN) * TM;
  const int lane_at = l % 16 * 64 + 16 * ((l / 16) ^ chunk_key(l % 16));
  auto read = [&](int buf, int b) {
    const int8_t *from = lds + buf * kStage;
#pragma unroll
    for (int i = 0; i < MI; ++i)
      xf[b][i] = *reinterpret_cast<const i32x4 *>(from + (BN + wm + 16 * i) * 64 + lane_at);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      wf[b][j] = *reinterpret_cast<const i32x4 *>(from + (wn + 16 * j) * 64 + lane_at);
  };
  // One stage: the two stages after the next one may still be on their way.
  auto step = [&](int cur, int b) {
    arrive<2 * kLoads>();
    fetch(cur);
    read((cur + 1) % 4, 1 - b);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[j][i] = mfma(wf[b][j], xf[b][i], acc[j][i]);
    // an operand read, two products, ...
#pragma unroll
    for (int q = 0; q < MI + NJ; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, MI * NJ / (MI + NJ), 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) fetch(i);
  arrive<3 * kLoads>();
  read(0, 0);
  int k = 0;
  for (; k + 256 <= kn; k += 256) {
    step(0, 0);
    step(1, 1);
    step(2, 0);
    step(3, 1);
  }
  if (k < kn) {  // 128 bytes left
    step(0, 0);
    step(1, 1);
  }

  arrive<0>();  // every load has landed and every operand been read: LDS is free
  int8_t *own = lds + wave * (kStage * 4 / kWaves);
  void *const to = p.parts ? p.parts + blockIdx.y * p.m * p.n : p.y;
  f32x4 ws[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) ws[j] = column_scales(p, n0 + wn + 16 * j + 4 * (l / 16));
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t mi = m0 + wm + 16 * i;
    const float xs = p.x_scale[mi + l % 16 < p.m ? mi + l % 16 : p.m - 1];
    // row r of 16: TN values as 16-byte chunks (4 binary32 or 8 bf16), chunk c at c ^ r
    constexpr int kChunk = YB ? 8 : 4, kChunks = TN / kChunk;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const f32x4 v = results(p, acc[j][i], xs, ws[j]);
      const int r = l % 16, n = 16 * j + 4 * (l / 16), c = (n / kChunk) ^ (r % kChunks);
      int8_t *at = own + (r * kChunks + c) * 16;
      if (YB)
        *reinterpret_cast<uint2 *>(at + n % kChunk * 2) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      else
        *reinterpret_cast<f32x4 *>(at) = v;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int g = 0; g < kChunks / 4; ++g) {
      const int q = 64 * g + l, r = q / kChunks, c = q % kChunks;
      const i32x4 v = *reinterpret_cast<const i32x4 *>(own + (r * kChunks + (c ^ (r % kChunks))) * 16);
      const int64_t m = mi + r, n = n0 + wn + kChunk * c;
      if (m < p.m) store_chunk<YB, Through>(p, to, m, n, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The parts' sums together, scaled: a row of Y a blockIdx.y, a value a thread.
template <bool YB>
__global__ __launch_bounds__(256) void linear_i8_join_kernel(const LinearI8Args p) {
  const int64_t m = blockIdx.y, n = (int64_t)blockIdx.x * 256 + threadIdx.x, each = p.m * p.n;
  if (n >= p.n) return;
  const int *part = reinterpret_cast<const int *>(p.parts) + m * p.n + n;
  int sum = part[0];
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) sum += part[s * each];
  const float v = (float)sum * p.x_scale[m] * p.w_scale[n];
  if (YB)
    static_cast<uint16_t *>(p.y)[m * p.n + n] = to_bf16(v);
  else
    static_cast<float *>(p.y)[m * p.n + n] = v;
}

struct Launch {
  const void *fn;
  int threads;
  int64_t grid;
  double us;  // of one round over the units, for 1024 k
};

template <int MT, int NT>
Launch rows_launch(const LinearI8Args &a) {
  return {a.y_bf16 ? (const void *)linear_i8_rows_kernel<MT, NT, true>
                   : (const void *)linear_i8_rows_kernel<MT, NT, false>,
          512, (a.m + 16 * MT - 1) / (16 * MT) * ((a.n + 16 * NT - 1) / (16 * NT)), 0.8};
}

template <int BM, int BN, int TM, int TN>
Launch tile_launch(const LinearI8Args &a, double round) {
  const int64_t total = (a.m + BM - 1) / BM * ((a.n + BN - 1) / BN);
  const bool whole = a.n % (a.y_bf16 ? 8 : 4) == 0;  // rows of Y of whole 16-byte chunks
  return {a.y_bf16 ? (whole ? (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, true, true>
                            : (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, true, false>)
                   : (whole ? (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, false, true>
                            : (const void *)linear_i8_tile_kernel<BM, BN, TM, TN, false, false>),
          BM / TM * (BN / TN) * 64, (total + 7) / 8 * 8, round / 4};
}

// The kernel of a size. Up to 256 workgroups (one for each compute unit) the rows kernels'
// split of K over the waves pays: 16 x 4096 x 4096 takes 9.8 us in 256 workgroups of 16 x 16
// against 13.4 in 64 of 64 x 64 tiles, and twice the columns or rows for a workgroup costs 1
// to 3 us. Past that, the tile whose rounds over the units take the least: a round of 4096
// k takes 10.5 us in tiles of 64 x 64, 17 of 64 x 128, 23 of 128 x 128, 37 of 128 x 256 and
// 62 of 256 x 256 (measured from 512 x 4096 x 4096 to 16384 x 4096 x 4096).
Launch pick(const LinearI8Args &a) {
  auto count = [&](int rows, int cols) {
    return (a.m + rows - 1) / rows * ((a.n + cols - 1) / cols);
  };
  if (count(16, 16) <= 256) return rows_launch<1, 1>(a);
  if (count(16, 32) <= 256) return rows_launch<1, 2>(a);
  if (count(32, 16) <= 256) return rows_launch<2, 1>(a);
  if (count(32, 32) <= 256) return rows_launch<2, 2>(a);
  auto time = [&](int rows, int cols, double round) {
    return (double)((count(rows, cols) + 255) / 256) * round;
  };
  const double t[5] = {time(256, 256, 62.0), time(128, 256, 37.0), time(128, 128, 23.0),
                       time(64, 128, 17.0), time(64, 64, 10.5)};
  switch (std::min_element(t, t + 5) - t) {
    case 0: return tile_launch<256, 256, 64, 128>(a, 62.0);
    case 1: return tile_launch<128, 256, 64, 64>(a, 37.0);
    case 2: return tile_launch<128, 128, 64, 64>(a, 23.0);
    case 3: return tile_launch<64, 128, 32, 64>(a, 17.0);
    default: return tile_launch<64, 64, 32, 32>(a, 10.5);
  }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // fewer threads with more values each: 16384 x 2100 bf16 24 us with two runs a thread and 32
  // with one, 8192 x 8192 36 with four and 58 with one
  const int nv = a.k_pad <= 2048 ? 1 : a.k_pad <= 4096 ? 2 : a.k_pad <= kLongRow ? 4 : 8;
  const int vecs = (a.k_pad + 8 * nv - 1) / (8 * nv);
  QuantizeArgs args = a;
  args.row_threads = vecs <= 16 ? 16 : (vecs + 63) / 64 * 64;
  const int groups = args.row_threads >= 256 ? 1 : 256 / args.row_threads;
  const void *fn = vecs <= 16 ? quantize_fn<16, 1>(a)
                   : nv == 1  ? quantize_fn<64, 1>(a)
                   : nv == 2  ? quantize_fn<64, 2>(a)
                   : nv == 4  ? quantize_fn<64, 4>(a)
                              : quantize_fn<64, 8>(a);
  const int threads = args.row_threads * groups;
  const int64_t need = (a.rows + groups - 1) / groups;
  const int64_t most = a.k_pad > kLongRow ? kLongThreads / threads : kQuantizeGrid;
  void *kargs[] = {&args};
  return hipLaunchKernel(fn, dim3((unsigned)(need < most ? need : most)), dim3(threads), kargs, 0,
                         stream);
}

int64_t linear_i8_threads(const LinearI8Args &a) {
  const Launch go = pick(a);
  return go.grid * go.threads;
}

// Parts of K by workgroups of their own, where a launch would leave at least half of the compute
// units idle for long enough: a unit fetches some 45 bytes/ns whatever its waves (16 x 4096 x
// 4096 takes the same with 4, 8 or 16 of them), so only other units help. The second kernel with
// its launch costs about 5.5 us. Whole and split: 85 x 69 x 15744 15.9 and 7.3 us, 21 x 568 x
// 10752 11.7 and 7.9, 700 x 700 x 9344 24.6 and 19.0, 1 x 64 x 65536 36.4 and 8.7; 512 x 1024 x
// 4096, which the rule leaves whole, 8.4 and 10.4.
constexpr double kJoin = 5.5;
int32_t linear_i8_splits(const LinearI8Args &a) {
  const Launch go = pick(a);
  if (go.grid > 128 || a.m > 65535) return 1;
  const int64_t most = std::min<int64_t>(256 / go.grid, a.k / 1024);
  const int64_t lines = a.k / 128, part = most > 1 ? (lines + most - 1) / most : lines;
  const int64_t splits = (lines + part - 1) / part;  // none of them empty
  const double saved = go.us * a.k / 1024 * (1.0 - 1.0 / (double)splits);
  return saved > kJoin ? (int32_t)splits : 1;
}

int64_t linear_i8_parts_bytes(const LinearI8Args &a) {
  if (a.m == 0 || a.n == 0) return 0;
  const int64_t splits = linear_i8_splits(a);
  return splits > 1 ? splits * a.m * a.n * 4 : 0;
}

hipError_t launch_linear_i8(const LinearI8Args &a, hipStream_t stream) {
  if (a.m == 0 || a.n == 0) return hipSuccess;
  LinearI8Args args = a;
  args.splits = linear_i8_splits(a);
  void *kargs[] = {&args};
  if (args.splits == 1) {
    const Launch go = pick(a);
    args.k_part = a.k;
    args.parts = nullptr;
    return hipLaunchKernel(go.fn, dim3((unsigned)go.grid), dim3(go.threads), kargs, 0, stream);
  }
  args.k_part = (a.k / 128 + args.splits - 1) / args.splits * 128;
  LinearI8Args sums = a;  // 4 bytes a sum
  sums.y_bf16 = 0;
  const Launch go = pick(sums);
  hipError_t e = hipLaunchKernel(go.fn, dim3((unsigned)go.grid, (unsigned)args.splits),
                                 dim3(go.threads), kargs, 0, stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel(a.y_bf16 ? (const void *)linear_i8_join_kernel<true>
                                  : (const void *)linear_i8_join_kernel<false>,
                         dim3((unsigned)((a.n + 255) / 256), (unsigned)a.m), dim3(256), kargs, 0,
                         stream);
}

}  // namespace gdn
