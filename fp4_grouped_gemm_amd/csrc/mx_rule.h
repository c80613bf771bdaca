// Which kernel computes an MXFP4 product, and how the one for few rows splits K:
// host code, shared by the launchers and a host check of what the tests reach
// (tests/mx_rule_check.cpp).
#pragma once

#include <algorithm>

namespace fgg {
namespace mx {

enum class Kernel { kRows, kTiles, kLargeTiles };

// Which kernel, by rows an expert has on average, and columns (a gated column
// counts as two, its gate and its up row).
//
// Few rows: the stream of weights.  It passes over an expert's weights once for
// every 32 rows of it in each scan of 1024 rows, one pass after the other, where a
// tile costs nearly the same whatever rows it holds.  Measured at 16, 24, 32 and 40
// rows for each of 32 experts of 2048 columns, 7168 K, stream | 128 x 128 tiles, us:
// 52 | 57, 57 | 59, 62 | 60 and 99 | 61; of 64 experts of 2048 columns, 1024 K, 22 | 29,
// 26 | 29 and 27 | 30; 16 rows on average, but the r-th expert's share as 1 / r: 94 |
// 62 and 37 | 33.  Where rows in no order take several scans an expert has some in
// each, and a pass for them: 8, 16 and 24 rows for each of 256 experts of 2048
// columns, 2048 K, in runs 123 | 129, 150 | 130 and 182 | 138, in no order 180 | 743,
// 326 | 968 and 472 | 1607.
//
// The rows of a decode batch often come in no order, and windows then hold all
// experts; so batches of up to 256 rows go to the stream up to 64 rows an expert.  64
// rows for each of 4 experts of 8192 columns, 8192 K, 57 | 53 in runs and 58 | 142 in no
// order; of 4 of 4096 gated columns, 4096 K, 32 | 32 and 33 | 85; 32 rows for each of
// 8 of 8192 columns, 8192 K, 65 | 84 and 68 | 267.  In no order the stream stays ahead
// far beyond that, in runs it does not, and the launch cannot tell them apart: 256 is
// about where runs of unequal length cross (shares as 1 / r; 8 experts of 2048 gated
// columns, 4096 K: 256 rows 29 | 25, of 4096 columns, 8192 K 49 | 48; no order 30 | 127
// and 45 | 264).  Past it the stream costs runs more and more: 512 rows
// over 8 experts of 1024 gated columns, 2048 K, equal shares 17 | 17, 1 / r 31 | 18, no
// order 17 | 82; 512 over 8 of 8192, 8192 K, 145 | 80 and 136 | 278; 1024 over 16 of 512,
// 7168 K, 25 | 30, 55 | 31 and 24 | 346.
//
// Of one expert: 28672 columns, 4096 K, 18 | 23 at 32 rows and 27 | 24 at 64.  With few
// columns K is split over waves, which tiles do not do: 4096 columns and K, 9.5 | 16
// at 64 rows, 16 | 18 at 128 and 23 | 18 at 192.
//
// Of the tiles the large ones read their operands half as often; they need rows
// to fill them and enough of them to fill the card.  128 x 128 | 256 x 256, us: 125,
// 150, 200 and 300 rows for each of 8 experts of 8192 columns, 8192 K, 91 | 87, 164 |
// 93, 121 | 96 and 185 | 169; 125 and 250 rows for each of 64 of 1024 gated columns,
// 2048 K, 54 | 65 and 89 | 78; of one expert, 4096 columns and K, 2048 rows (128 large
// tiles) 31 | 32, 3000 rows 41 | 37; 6144 columns, 4096 K, 777 rows 26 | 29; 28672
// columns, 4096 K, 512 rows 59 | 42.
inline Kernel kernel_for(int M, int N, int G, bool gated, int num_cus) {
  const long long cols = (long long)N * (gated ? 2 : 1);
  const bool few = M <= std::max(32ll, 24ll * G) || (M <= 256 && G > 1 && M <= 64ll * G);
  if (few || (M <= 128 && cols * G <= 8192)) return Kernel::kRows;
  const long long large = std::max((M + 255) / 256, G) * ((cols + 255) / 256);
  return M > 128ll * G && 2 * large > num_cus ? Kernel::kLargeTiles : Kernel::kTiles;
}

// Columns of C that a wave of the kernel for few rows makes.
constexpr int rows_columns(bool gated) { return gated ? 16 : 32; }

// K is split over 4, 2 or 1 of a workgroup's four waves: as much as leaves the card's
// waves, eight a compute unit, something to do.  Measured with 4 | 2 | 1, us, one row
// unless said: 4096 columns of 4096 K 5.6 | 6.4 | 9.0, 8192 of 4096 6.5 | 6.8 |
// 9.0, 16384 of 4096 10.0 | 9.6 | 12.1, 28672 of 4096 16.5 | 14.2 | 14.1; 192
// rows over 64 experts, 2048 columns of 1024 K, 38 | 26 | 19.  MXFP4 results
// need whole blocks of 32 columns in a workgroup, so at most 2 there.  Both limits
// are the card's 256 compute units, once and four times.
inline int rows_ksplit(int M, int N, int G, bool gated, bool mx_result, int num_cus) {
  const long long waves = (long long)((N + rows_columns(gated) - 1) / rows_columns(gated)) * std::min(M, G);
  return waves <= num_cus && !mx_result ? 4 : waves <= 4ll * num_cus ? 2 : 1;
}

}  // namespace mx
}  // namespace fgg
