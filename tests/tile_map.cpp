// Host-side check of lds_tiles.hpp's map from workgroups to tiles: for products of tiles_m x
// tiles_n tiles, by a grid of their own (whole rounds of 8 workgroups) and by larger ones, as where
// two products share a launch. Prints "case m=<m> n=<n> grid=<g> least=<l> most=<h> outside=<o>":
// how many workgroups take a tile, at least and at most, and how many places are no tile.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "lds_tiles.hpp"

static void run(int64_t m, int64_t n, int64_t grid) {
  std::vector<int> taken(m * n, 0);
  int outside = 0;
  for (int64_t b = 0; b < grid; ++b) {
    const gdn::TilePlace at = gdn::tile_place(b, m, n);
    if (at.row < 0) continue;
    if (at.row >= m || at.col < 0 || at.col >= n)
      ++outside;
    else
      ++taken[at.row * n + at.col];
  }
  std::printf("case m=%lld n=%lld grid=%lld least=%d most=%d outside=%d\n", (long long)m,
              (long long)n, (long long)grid, *std::min_element(taken.begin(), taken.end()),
              *std::max_element(taken.begin(), taken.end()), outside);
}

int main() {
  for (int64_t m : {1, 2, 7, 8, 9, 17, 33, 64})
    for (int64_t n : {1, 3, 8, 9, 17, 65}) {
      const int64_t own = (m * n + 7) / 8 * 8;
      for (int64_t grid : {own, own + 8, 2 * own, 5 * own + 24, own + 4096}) run(m, n, grid);
    }
  run(8, 9, 160);  // dx of 1021 x 2049 x 1111 in 128 x 128 tiles, in dw's grid
  return 0;
}
