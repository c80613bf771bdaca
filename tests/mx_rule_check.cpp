// Reads products "M N G gated mx_result" and prints the kernel that each goes to (csrc/mx_rule.h) with 256
// compute units, "rows" with the number of waves that K is split over.
#include <cstdio>

#include "mx_rule.h"

using namespace fgg;

int main() {
  int M, N, G, gated, mx_result;
  while (std::scanf("%d %d %d %d %d", &M, &N, &G, &gated, &mx_result) == 5) {
    const mx::Kernel k = mx::kernel_for(M, N, G, gated, 256);
    if (k == mx::Kernel::kRows)
      std::printf("rows %d\n", mx::rows_ksplit(M, N, G, gated, mx_result));
    else
      std::printf("%s\n", k == mx::Kernel::kTiles ? "tiles" : "large tiles");
  }
}
