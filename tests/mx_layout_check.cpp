// Enumerates the rows of B that the MXFP4 tile kernel deals to its LDS rows
// (csrc/mx_layout.h) and checks that
//   - every column of a tile (of gated products every gate and every up row)
//     has one LDS row, and a load's eight rows lie within the tile;
//   - the block that a wave's s-th load fills is its first one's moved by
//     tile_step columns, in the same half;
//   - the four values that the matrix instruction leaves a lane for each of two
//     subtiles are eight consecutive columns, and gate and up of a column are
//     values of the same lane.
#include <cstdio>
#include <set>
#include <utility>

#include "mx_layout.h"

using namespace fgg;

static long long checks = 0, failed = 0;
static bool quiet = false;
static void expect(bool ok, const char* what, int a, int b, int c) {
  ++checks;
  if (!ok && ++failed <= 20 && !quiet) std::printf("FAILED %s: %d %d %d\n", what, a, b, c);
}

// (half, column) of LDS row `row` of a tile; planted: two columns change places
static std::pair<int, int> held(int row, bool gated, bool plant) {
  int c = mx::tile_column(row >> 3, row & 7, gated);
  if (plant) c ^= row & 1;
  return {mx::tile_half(row >> 3, gated), c};
}

static void tile(int bn, int waves, bool gated, bool plant) {
  const int cols = gated ? bn / 2 : bn;
  std::set<std::pair<int, int>> seen;
  for (int row = 0; row < bn; ++row) {
    const auto h = held(row, gated, plant);
    expect(h.second >= 0 && h.second < cols, "a column of the tile", bn, gated, row);
    expect(seen.insert(h).second, "a column held twice", bn, gated, row);
  }
  expect((int)seen.size() == bn, "every column held", bn, gated, 0);
  for (int w = 0; w < waves; ++w)
    for (int s = 0; s < bn / 8 / waves; ++s) {
      const int b = s * waves + w;
      // with four waves the half of a gated load is its number's, with eight its wave's
      expect(mx::tile_half(b, gated) == (waves == 8 ? mx::tile_half(w, gated) : mx::tile_half(s * waves, gated)), "half", bn, w, s);
      for (int r = 0; r < 8; ++r)
        expect(mx::tile_column(b, r, gated) == mx::tile_column(w, r, gated) + mx::tile_step(s, waves, gated), "step", b, r, gated);
    }
  const int step = gated ? 4 : 2;  // subtiles of 16 rows that 32 columns take
  for (int j = 0; j < bn / 16; ++j)
    for (int q = 0; q < 4; ++q)
      for (int t = 0; t < 4; ++t) {
        const auto h = held(j * 16 + 4 * q + t, gated, plant);
        expect(h.first == (gated ? j % 4 / 2 : 0), "gate subtiles before up subtiles", j, q, t);
        expect(h.second == j / step * 32 + 8 * q + 4 * (j % 2) + t, "a lane's columns", j, q, t);
      }
}

int main() {
  for (int gated = 0; gated < 2; ++gated) {
    tile(256, 8, gated, false);
    tile(128, 4, gated, false);
  }
  std::printf("%lld checks, %lld failed\n", checks, failed);
  const long long bad = failed;
  quiet = true;
  tile(256, 8, true, true);
  std::printf("planted mistake %s\n", failed > bad ? "seen" : "missed");
  return bad || failed == bad;
}
