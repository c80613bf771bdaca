// The list of work of paged_decode_attention, shared by the kernels (device) and
// a host check (tests/attn_list_check.cpp).  Plain integer arithmetic, no HIP
// types.
//
// Rows of work are cut into tiles of 128 tokens, 32 to a wave; the tiles of all
// rows make one list, and the list is cut into slices for the workgroups.  Lengths
// go up to 2^31 - 1 tokens and the list up to 2^30 tiles.
#pragma once

#include "offsets.h"

namespace fgg {
namespace attn_list {

constexpr int kWaveTokens = 32;
constexpr int kWaves = 4;
constexpr int kTile = kWaves * kWaveTokens;

// An empty row has a tile too: the one that writes its zeros.  (Rounded up from len - 1:
// len + kTile - 1 may pass 2^31.)
FGG_HD int tiles_of(int len) { return len ? (len - 1) / kTile + 1 : 1; }

// First token of a wave in step t of waves that take `step` tokens at once.
FGG_HD int first_token(int t, int step, int wave) { return t * step + wave * kWaveTokens; }

// The list in slices that differ by at most one tile, none of them empty (a
// row's pieces come from consecutive slices): where one begins, and which one
// holds a tile.  Workgroups past the last slice have nothing to do.
FGG_HD int slices_of(int total, int workgroups) { return workgroups < total ? workgroups : total; }
FGG_HD int slice_start(int i, int total, int workgroups) {
  const int n = slices_of(total, workgroups);
  return i < n ? (int)((long long)i * total / n) : total;
}
FGG_HD int slice_of(int tile, int total, int workgroups) {
  return (int)(((long long)(tile + 1) * slices_of(total, workgroups) - 1) / total);
}

}  // namespace attn_list
}  // namespace fgg
