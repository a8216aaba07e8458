// Prints how the latent attention splits its units over CTA pairs, as the
// kernel computes it, for "units pairs" read from stdin: one line each, the
// first unit of pairs 0 .. pairs. Host code only: no GPU is needed to run it.
#include <cstdio>

#include "mla_attention.cu"

// (The library's own asks the driver; nothing here launches.)
int fp8blk::current_device(const DevInfo**) { return FP8BLK_ERR_CUDA; }

int main() {
  int units, pairs;
  while (std::scanf("%d %d", &units, &pairs) == 2) {
    const fp8blk::Divisor by_pairs = fp8blk::divisor(pairs);
    for (int q = 0; q <= pairs; ++q) std::printf("%d ", fp8blk::unit_of_pair(by_pairs, units, pairs, q));
    std::printf("\n");
  }
  return 0;
}
