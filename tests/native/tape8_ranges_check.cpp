// Host check of the 8-bit tape's buffer ranges (ranges.h).  Reads lines
// "d_v T W R" and prints, per line, 1 when the code and scale descriptors are
// valid, else 0.
#include <cstdio>

#include "../../sparse_memory_linear_sdm_amd/csrc/ranges.h"

int main() {
  long long d, t, w, r;
  while (std::scanf("%lld %lld %lld %lld", &d, &t, &w, &r) == 4)
    std::printf("%d\n", sdm::ranges::tape8_ok((int)d, t, (int)w, (int)r) ? 1 : 0);
  return 0;
}
