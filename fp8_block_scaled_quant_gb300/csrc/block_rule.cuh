// The quantisation rule of a block: its scale and the e4m3 codes.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8blk {

// Scale of a 128-element (or 128x128) block: max(amax, 1e-4) / 448 as an IEEE
// fp32 division; with ue8m0, rounded up to a power of two on the bits
// (2^ceil(log2 s) exactly: unchanged when the mantissa is zero, otherwise the
// next power of two above).
__device__ __forceinline__ float block_scale(float amax, bool ue8m0) {
  float s = __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f);
  if (ue8m0) {
    uint32_t b = __float_as_uint(s);
    if (b & 0x007FFFFFu) b = (b & 0x7F800000u) + 0x00800000u;
    s = __uint_as_float(b);
  }
  return s;
}

// Two fp32 values -> two e4m3 codes (round to nearest even, saturating), low
// byte = a.
__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {
  return static_cast<uint16_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

}  // namespace fp8blk
