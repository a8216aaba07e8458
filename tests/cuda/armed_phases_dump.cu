// Prints what the few-token MoE layer's producer keeps of the copies it has in
// flight, for lines of barrier numbers read from stdin (a copy armed on each, in
// order): "used parity" as bit masks. Host code only: no GPU is needed to run it.
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>

#include "moe_layer.cu"

// (The library's own; nothing here launches.)
int fp8blk::current_device(const DevInfo**) { return FP8BLK_ERR_CUDA; }
int fp8blk::gate_shape_status(const float*, int64_t, int64_t, int64_t, int64_t, int64_t, int, float) { return 0; }

int main() {
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    fp8blk::Armed a{0, 0};
    for (int s; in >> s;) a.arm(s);
    std::printf("%u %u\n", a.used, a.parity);
  }
  return 0;
}
