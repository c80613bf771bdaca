// Enumerates every staging load and fragment read of prompt_attention's blocks
// (csrc/attn_layout.h) and checks that
//   - a load that is made reads inside its row, and inside the span that the
//     buffer's range check allows for its vector offset;
//   - every byte of a block is written once, and a fragment read finds the row
//     and chunk that it is for;
//   - a cycle's lanes of a fragment read touch different banks.
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "attn_layout.h"

using namespace fgg::attn_layout;

static long long checks = 0, failed = 0;
static bool quiet = false;
static void expect(bool ok, const char* what, int D, int a, int b) {
  ++checks;
  if (!ok && ++failed <= 20 && !quiet) std::printf("FAILED %s: D=%d %d %d\n", what, D, a, b);
}

// (row, logical chunk) that staging puts at each physical 16-byte place
static std::vector<std::pair<int, int>> staged(int D, bool value, bool plant) {
  std::vector<std::pair<int, int>> at(32 * D * 2 / 16, {-1, -1});
  const long long stride = 5 * D + 8;
  for (int j = 0; j < stage_loads(D); ++j)
    for (int t = 0; t < kThreads; ++t) {
      uint32_t off = stage_off(D, t, value, stride);
      if (plant) off ^= (uint32_t)(t & 16);  // a planted mistake: another chunk
      const long long byte = off + (long long)j * stage_rows(D) * stride * 2;
      const int row = (int)(byte / (stride * 2)), in = (int)(byte % (stride * 2));
      expect(in % 16 == 0 && in + 16 <= D * 2, "chunk inside its row", D, j, t);
      auto& place = at[j * kThreads + t];
      expect(place.first < 0, "a place written twice", D, j, t);
      place = {row, in / 16};
    }
  return at;
}

static void reads(int D, bool plant) {
  const auto k_at = staged(D, false, plant), v_at = staged(D, true, plant);
  for (int lane = 0; lane < 64; ++lane)
    for (int k = 0; k < D / 16; ++k) {
      const int a = k_read(D, lane, k);
      expect(a % 16 == 0 && a >= 0 && a + 16 <= 32 * D * 2, "K read in its block", D, lane, k);
      expect(k_at[a / 16] == std::make_pair(lane & 31, 2 * k + (lane >> 5)), "K read finds its chunk", D, lane, k);
    }
  for (int lane = 0; lane < 64; ++lane)
    for (int k = 0; k < 2; ++k)
      for (int i = 0; i < D / 32; ++i)
        for (int e = 0; e < 2; ++e) {
          const int a = v_read(D, lane, k, i, e);
          expect(a % 8 == 0 && a >= 0 && a + 8 <= 32 * D * 2, "V read in its block", D, lane, i);
          const int row = 16 * k + 8 * e + 4 * (lane / 32) + lane % 16 / 4;
          const int dim = 32 * i + 16 * (lane / 16 % 2) + 4 * (lane % 4);
          expect(v_at[a / 16] == std::make_pair(row, dim / 8) && a % 16 == dim % 8 * 2, "V read finds its values", D,
                 lane, i);
        }
}

static void banks(int D) {
  for (int k = 0; k < D / 16; ++k) {
    std::map<int, std::set<int>> cycle;
    for (int lane = 0; lane < 64; ++lane) {
      const int g = (lane >> 5) * 2 + (((lane >> 2) ^ (lane >> 3) ^ (lane >> 4)) & 1);
      for (int w = 0; w < 4; ++w)
        expect(cycle[g].insert((k_read(D, lane, k) / 4 + w) % 64).second, "K bank conflict", D, lane, k);
    }
  }
  for (int k = 0; k < 2; ++k)
    for (int i = 0; i < D / 32; ++i)
      for (int e = 0; e < 2; ++e) {
        std::map<int, std::set<int>> cycle;
        for (int lane = 0; lane < 64; ++lane)
          for (int w = 0; w < 2; ++w)
            expect(cycle[lane / 32].insert((v_read(D, lane, k, i, e) / 4 + w) % 64).second, "V bank conflict", D, lane, i);
      }
}

// Loads of a block of which `left` rows exist.
static void tails(int D, long long stride) {
  for (int left = -3; left <= 32; ++left) {
    const uint32_t bytes = stage_bytes(D, left < 32 ? left : 32, stride);
    for (int value = 0; value < 2; ++value)
      for (int j = 0; j < stage_loads(D); ++j)
        for (int t = 0; t < kThreads; ++t) {
          const int row = t / (D / 8) + j * stage_rows(D);
          if (row >= left) continue;  // not loaded
          const uint32_t voff = stage_off(D, t, value, stride);
          const unsigned long long at = voff + (unsigned long long)j * stage_rows(D) * stride * 2;
          expect((unsigned long long)voff + 16 <= bytes, "vector offset within the range check", D, left, t);
          expect(at + 16 <= ((unsigned long long)(left - 1) * stride + D) * 2, "load within the rows", D, left, t);
        }
  }
}

int main() {
  for (int D : {64, 128}) {
    reads(D, false);
    banks(D);
    for (long long stride : {(long long)D, 6LL * D, 12288LL, 1LL << 22}) tails(D, stride);
  }
  const long long sound = failed;
  quiet = true;
  reads(128, true);  // the checks see a planted mistake
  const bool seen = failed > sound;
  std::printf("%lld checks, %lld failed, planted mistake %s\n", checks, sound, seen ? "seen" : "MISSED");
  return sound || !seen;
}
