// Helpers of the products whose tiles go through LDS: which workgroup takes which tile, loads
// straight from memory into LDS, the wait that goes with them, and stores of a tile's rows.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn {

using i32x4 = int __attribute__((ext_vector_type(4)));

// The tile of Y, counted in tiles, that a workgroup takes; rows below 0: none. Each XCD (workgroup
// % 8) has a run of neighbours, in bands of 8 tiles of rows. The grid may be larger than the
// product's own, as where two products share one.
struct TilePlace {
  int64_t row, col;
};
__host__ __device__ __forceinline__ TilePlace tile_place(int64_t workgroup, int64_t tiles_m,
                                                         int64_t tiles_n) {
  const int64_t total = tiles_m * tiles_n, per = (total + 7) / 8, turn = workgroup / 8;
  const int64_t tile = workgroup % 8 * per + turn;
  if (turn >= per || tile >= total) return {-1, 0};  // past its XCD's run: another one's tiles
  const int64_t band = tile / (8 * tiles_n), in_band = tile % (8 * tiles_n);
  const int64_t height = tiles_m - 8 * band < 8 ? tiles_m - 8 * band : 8;
  return {8 * band + in_band % height, in_band / height};
}

// 16 bytes per lane from base + offset to LDS, lane after lane from `to` (uniform) on.
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t offset, uint32_t to) {
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

// Sixteen bytes of row m of Y [.., width] from column n on: 4 binary32 or 8 bf16 values.
// Through: past the caches.
template <bool YB, bool Through>
__device__ __forceinline__ void store_chunk(int64_t width, void *to, int64_t m, int64_t n,
                                            i32x4 v) {
  using unaligned = int __attribute__((ext_vector_type(4), aligned(YB ? 2 : 4)));
  constexpr int kChunk = YB ? 8 : 4;
  if (n + kChunk <= width) {
    char *y = static_cast<char *>(to) + (m * width + n) * (YB ? 2 : 4);
    if (Through)
      __builtin_nontemporal_store(v, reinterpret_cast<unaligned *>(y));
    else
      *reinterpret_cast<unaligned *>(y) = v;
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (n + e < width) {
        if (YB)
          static_cast<uint16_t *>(to)[m * width + n + e] =
              (uint16_t)((uint32_t)v[e / 2] >> (16 * (e % 2)));
        else
          static_cast<int *>(to)[m * width + n + e] = v[e];
      }
  }
}

}  // namespace gdn
