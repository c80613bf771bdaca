// Reads products "M N G gated mx_result [on num_cus]" a line and prints the kernel that each goes to
// (csrc/mx_rule.h), "rows" with the number of waves that K is split over; 256 compute units unless said.
#include <cstdio>

#include "mx_rule.h"

using namespace fgg;

int main() {
  int M, N, G, gated, mx_result, cus;
  char line[256];
  while (std::fgets(line, sizeof line, stdin)) {
    const int n = std::sscanf(line, "%d %d %d %d %d on %d", &M, &N, &G, &gated, &mx_result, &cus);
    if (n < 5) return 1;
    if (n == 5) cus = 256;
    const mx::Kernel k = mx::kernel_for(M, N, G, gated, cus);
    if (k == mx::Kernel::kRows)
      std::printf("rows %d\n", mx::rows_ksplit(M, N, G, gated, mx_result, cus));
    else
      std::printf("%s\n", k == mx::Kernel::kTiles ? "tiles" : "large tiles");
  }
}
