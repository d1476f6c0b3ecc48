// The tile rule over the sizes that the microscaled products take: prints the
// number of sizes and how many launches would reach 2^32 threads.
#include <cstdio>

#include "../../bit_nf4_quantized_03_amd/csrc/mx_tiles.h"

int main() {
  long sizes = 0, over = 0;
  for (int e = -1; e <= 10; ++e)
    for (int m = 0; m <= 24; ++m)
      for (int n = 0; n <= 24; ++n)
        for (int k = 0; k < 9; ++k) {
          const int experts = e < 0 ? 0 : 1 << e;
          const int64_t top = int64_t(1) << 24;
          int64_t M = (int64_t(1) << m) + k % 3 - 1, N = (int64_t(1) << n) + k / 3 - 1;
          M = M < top ? M : top, N = N < top ? N : top;
          if (M < 1 || N < 1 || M > (int64_t(1) << 37) / N || N * (experts ? experts : 1) > int64_t(1) << 28) continue;
          for (int fp4 = 0; fp4 < 2; ++fp4) {
            const int t = qnf4::mx_choose_tile(M, N, experts, fp4);
            const int64_t groups = qnf4::mx_tile_groups(qnf4::kMxTile[t].bm, qnf4::kMxTile[t].bn, M, N, experts);
            ++sizes;
            if (groups * qnf4::kMxTile[t].threads >= int64_t(1) << 32) {
              if (over++ == 0) std::printf("%lld x %lld, %d experts: tile %d\n", (long long)M, (long long)N, experts, t);
            }
          }
        }
  std::printf("%ld sizes, %ld over\n", sizes, over);
  return over != 0;
}
