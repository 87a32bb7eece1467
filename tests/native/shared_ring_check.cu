// Prints the stages of the wide kernel's ring: bits of a row, 1 when a call has
// more than 128 query rows, stages (tests/test_shared_ring.py; no GPU).
#include <cstdio>

#include "shared_ring.cuh"

using bpkv::shared::wide::Shape;

int main() {
  for (int dual = 0; dual < 2; ++dual) {
    std::printf("16 %d %d\n", dual, Shape<16>::stages(dual));
    std::printf("8 %d %d\n", dual, Shape<8>::stages(dual));
  }
  return 0;
}
