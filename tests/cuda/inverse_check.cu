// Checks of the norm's arithmetic over every fp32 input (csrc/quotient.cuh): the
// reciprocal and the reciprocal root against their bounds, in fp64, and
// max(amax, 1e-4) / 448 by Markstein's correction against CUDA's IEEE division.
// Prints one line each and exits non-zero where a bound does not hold.
#include <cuda_runtime.h>
#include <cstdint>
#include <cstdio>

#include "quotient.cuh"

enum { kInverse, kRoot, kScale };

__global__ void check(int what, uint32_t first, uint32_t last, unsigned long long* counts) {
  unsigned long long n = 0, bad = 0;
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  for (uint64_t b = first + static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; b <= last; b += step) {
    const float a = __uint_as_float(static_cast<uint32_t>(b));
    ++n;
    if (what == kInverse) {
      const double off = fabs(static_cast<double>(a) * fp8blk::inverse(a) - 1.0);
      bad += !(off <= 0x1p-24 * (1.0 + 0x1p-10));
    } else if (what == kRoot) {
      const double y = fp8blk::inverse_root(a), off = fabs(y * y * static_cast<double>(a) - 1.0);  // twice y's error
      bad += !(off <= 2.0 * 1.5 * 0x1p-24 * (1.0 + 0x1p-8));
    } else {
      bad += fp8blk::div_by_scale(a, 448.0f, 1.0f / 448.0f) != __fdiv_rn(a, 448.0f);
    }
  }
  atomicAdd(counts, n);
  atomicAdd(counts + 1, bad);
}

uint32_t bits(float f) {
  union { float f; uint32_t u; } v = {f};
  return v.u;
}

int main() {
  unsigned long long* d;
  if (cudaMalloc(&d, 16) != cudaSuccess) return 2;
  struct { const char* name; int what; float first, last; } runs[] = {
      {"inverse", kInverse, 0x1p-126f, 0x1.fffffep125f},
      {"inverse_root", kRoot, 0x1p-149f, 0x1.fffffep127f},
      {"scale", kScale, 1e-4f, 0x1.fffffep127f},
  };
  int rc = 0;
  for (const auto& r : runs) {
    unsigned long long h[2] = {0, 0};
    cudaMemset(d, 0, 16);
    check<<<1216, 256>>>(r.what, bits(r.first), bits(r.last), d);
    if (cudaMemcpy(h, d, 16, cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
    std::printf("%s values %llu outside %llu\n", r.name, h[0], h[1]);
    if (h[1] != 0 || h[0] < 1000000000ull) rc = 1;
  }
  return rc;
}
