// Which rows of B a tile's LDS rows hold in the MXFP4 tile kernel: shared by the
// kernel and a host check that enumerates them (tests/mx_layout_check.cpp).
//
// The tile's LDS rows come in blocks of eight, b = 0, 1, ..: two blocks are a
// subtile of 16 rows, and two subtiles (of gated products four: gate, gate, up,
// up) hold 32 columns of C.  The matrix instruction leaves lane (r, q) with
// values t < 4 of subtile rows 4 q + t, so row 4 q + t of the first subtile is
// column 8 q + t of the 32 and of the second column 8 q + 4 + t.
#pragma once

#include "offsets.h"

namespace fgg {
namespace mx {

// Column of C, from the tile's first, of row r8 of block b.
FGG_HD int tile_column(int b, int r8, bool gated) {
  return (gated ? b >> 3 : b >> 2) * 32 + 8 * ((b & 1) * 2 + (r8 >> 2)) + 4 * ((b >> 1) & 1) + (r8 & 3);
}
// 1 where block b holds up rows.
FGG_HD int tile_half(int b, bool gated) { return gated ? (b >> 2) & 1 : 0; }
// What block s * waves + w is columns further than block w: waves is a multiple
// of 4, so the blocks' places among the 32 columns are the same.
FGG_HD int tile_step(int s, int waves, bool gated) { return (s * waves >> (gated ? 3 : 2)) * 32; }

}  // namespace mx
}  // namespace fgg
