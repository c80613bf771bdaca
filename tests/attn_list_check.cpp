// Checks the arithmetic of paged_decode_attention's list of work
// (csrc/attn_list.h) at the ends of its range:
//   - the tiles of a row cover its tokens and no tile is empty, for every length
//     that a 32-bit count holds, and no token that a wave looks at passes 2^31;
//   - the slices of a list follow each other without a gap, none is empty, and
//     slice_of finds the slice that holds a tile.
#include <cstdio>
#include <initializer_list>

#include "attn_list.h"

using namespace fgg::attn_list;

static long long checks = 0, failed = 0;
static void expect(bool ok, const char* what, long long a, long long b) {
  ++checks;
  if (!ok && ++failed <= 20) std::printf("FAILED %s: %lld %lld\n", what, a, b);
}

static void row(long long len) {
  const long long n = tiles_of((int)len);
  expect(n >= 1 && n * kTile >= len, "tiles cover the row", len, n);
  expect(len == 0 ? n == 1 : (n - 1) * kTile < len, "no tile is empty", len, n);
  if (n < 1 || len == 0) return;
  for (int wave = 0; wave < kWaves; ++wave) {
    const long long tok = (n - 1) * (long long)kTile + wave * kWaveTokens;
    expect(tok + kWaveTokens - 1 <= 0x7FFFFFFFLL, "tokens of the last tile in 32 bits", len, tok);
    expect(first_token((int)n - 1, kTile, wave) == tok, "first token of a wave", len, tok);
  }
}

static void list(int total, int workgroups) {
  const int n = slices_of(total, workgroups);
  long long at = 0;
  for (int i = 0; i < workgroups; ++i) {
    const int a = slice_start(i, total, workgroups), b = slice_start(i + 1, total, workgroups);
    expect(a == at && b <= total && (i < n ? b > a : b == a), "slices follow each other", total, i);
    if (i < n)
      for (int t : {a, a + (b - a) / 2, b - 1}) expect(slice_of(t, total, workgroups) == i, "slice of a tile", total, t);
    at = b;
  }
  expect(at == total, "the slices hold the list", total, at);
}

int main() {
  for (long long len = 0; len < 4000; ++len) row(len);
  for (long long len = 0x7FFFFFFFLL - 4000; len <= 0x7FFFFFFFLL; ++len) row(len);
  for (int p = 12; p < 31; ++p)
    for (int e = -1; e <= 1; ++e) row((1LL << p) + e);
  for (int workgroups : {1, 3, 767, 768})
    for (int total : {1, 2, 5, 766, 767, 768, 769, 1535, 100003, (1 << 30) - 1, 1 << 30}) list(total, workgroups);
  std::printf("%lld checks, %lld failed\n", checks, failed);
  return failed != 0;
}
