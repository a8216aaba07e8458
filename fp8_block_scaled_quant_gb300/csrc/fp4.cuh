// Microscaled 4-bit floats: the e2m1 codes, the rules for their scales, where a
// scale byte sits, and the tensor-core instructions that multiply them.
//
// Two formats. FP8BLK_FP4_E4M3: an e4m3 scale s for every 16 columns and an fp32
// scale g for every row; with a = max(row amax, 2^-100),
//   g = a / 2688,  s = e4m3(amax_block * (448 / a)),  q = e2m1(x * (1 / (s g)))
// (2688 = 6 * 448: the row's largest block has s = 448, its largest element
// q = 6). FP8BLK_FP4_UE8M0: a power of two for every 32 columns, the least that
// is not below amax_block / 6, no row scale. Every step is rounded to fp32.
//
// Scale bytes are kept in the order in which tensor memory wants them: the byte
// of (row, block) at [row / 128][block / 4][row % 32][row % 128 / 32][block % 4],
// so 128 rows x 4 blocks are one tile of 512 bytes, 16 bytes to a lane.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "ptx.cuh"

namespace fp8blk {

constexpr int kFp4E4M3 = FP8BLK_FP4_E4M3, kFp4UE8M0 = FP8BLK_FP4_UE8M0;
constexpr int kScaleTile = 512;  // bytes of 128 rows x 4 blocks

// Columns of a scale tile (4 blocks).
__host__ __device__ constexpr int fp4_tile_cols(int fmt) { return fmt == kFp4E4M3 ? 64 : 128; }

__host__ __device__ inline int64_t fp4_scale_bytes(int64_t rows, int64_t K, int fmt) {
  return (rows + 127) / 128 * (K / fp4_tile_cols(fmt)) * kScaleTile;
}

// Where the scale byte of (row, block) sits; ktiles = K / fp4_tile_cols.
__device__ __forceinline__ int64_t fp4_scale_at(int64_t row, int block, int64_t ktiles) {
  return ((row >> 7) * ktiles + (block >> 2)) * kScaleTile + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

// ---- codes and scales ---------------------------------------------------------

// Eight values to e2m1 codes (nearest, ties to the even code, saturating), the
// first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

// Absolute values compared by their bits: a NaN is above infinity.
__device__ __forceinline__ bool finite_bits(uint32_t abs_bits) { return abs_bits < 0x7F800000u; }

struct RowScale {
  float g, c;  // the row's scale, and 448 / amax
  bool finite;
};

__device__ __forceinline__ RowScale fp4_row_scale(uint32_t amax_bits) {
  RowScale r;
  r.finite = finite_bits(amax_bits);
  const float a = fmaxf(__uint_as_float(amax_bits), 7.8886090522101181e-31f);  // 2^-100
  r.g = r.finite ? __fdiv_rn(a, 2688.0f) : __uint_as_float(0x7FFFFFFFu);
  r.c = __fdiv_rn(448.0f, a);
  return r;
}

// The scale byte of a block, and *mul: what its values are multiplied by before
// the rounding to e2m1 (0: all codes are zero).
__device__ __forceinline__ uint8_t fp4_block_scale_e4m3(uint32_t amax_bits, const RowScale& row, float* mul) {
  if (!row.finite) {
    *mul = 0.0f;
    return 0;
  }
  const uint8_t code = __nv_cvt_float_to_fp8(__fmul_rn(__uint_as_float(amax_bits), row.c), __NV_SATFINITE, __NV_E4M3);
  *mul = code ? __frcp_rn(__fmul_rn(e4m3_value(code), row.g)) : 0.0f;
  return code;
}

__device__ __forceinline__ uint8_t fp4_block_scale_ue8m0(uint32_t amax_bits, float* mul) {
  if (!finite_bits(amax_bits)) {
    *mul = 0.0f;
    return 0xFF;
  }
  uint32_t b = __float_as_uint(__fdiv_rn(__uint_as_float(amax_bits), 6.0f));
  uint32_t e = (b >> 23) + ((b & 0x7FFFFFu) ? 1u : 0u);  // biased exponent of the least power of two not below
  e = max(e, 1u);
  *mul = __uint_as_float((254u - e) << 23);  // 2^-(e - 127), exact: e <= 253
  return static_cast<uint8_t>(e);
}

// Quantises a row's columns 16 unit .. 16 unit + 15, of a warp whose lanes have
// consecutive units (lane 0 a multiple of 32) and call it together: a scale word
// is put together from the lanes of its four blocks. Lanes with unit >= units
// store nothing. amax: the bits of the unit's largest |v|.
template <int FMT>
__device__ __forceinline__ void fp4_store16(const float2* v, uint32_t amax, const RowScale& rs, int64_t row, int unit,
                                            int units, uint2* q, uint8_t* s, int64_t ktiles) {
  const uint32_t lane = threadIdx.x & 31;
  float mul;
  uint32_t word;
  if constexpr (FMT == kFp4E4M3) {
    word = static_cast<uint32_t>(fp4_block_scale_e4m3(amax, rs, &mul)) << (8 * (lane & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  } else {
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    word = static_cast<uint32_t>(fp4_block_scale_ue8m0(amax, &mul)) << (8 * ((lane >> 1) & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  }
  if (unit >= units) return;
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(v[i], make_float2(mul, mul));
  // mul == 0: a block of zeros, or one that is not finite
  q[row * units + unit] = mul == 0.0f ? make_uint2(0, 0) : make_uint2(e2m1x8(&y[0].x), e2m1x8(&y[4].x));
  constexpr int kPer = FMT == kFp4E4M3 ? 4 : 8;  // lanes of a scale word
  if ((unit & (kPer - 1)) == 0)
    *reinterpret_cast<uint32_t*>(s + fp4_scale_at(row, unit / (kPer / 4), ktiles)) = word;
}

// ---- tensor cores -------------------------------------------------------------

// Instruction descriptor of the 4-bit block-scaled MMA: e2m1 A and B, both
// K-major, fp32 accumulation, an M x N tile; bit 23: UE8M0 scales (else e4m3);
// `sf_id`: the first byte of each 32-bit scale word that is used.
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, int fmt, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (fmt == kFp4UE8M0 ? 1u << 23 : 0u) | (static_cast<uint32_t>(M >> 4) << 24) | (sf_id << 29);
}

// D[tmem] (+)= A B^T for 64 columns, each product scaled by its blocks' scales.
// A scale word (a row's four blocks) is in lane row % 32 of column sf + row / 32,
// the same in all four lane quarters.
template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (FMT == kFp4E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes, no swizzle,
// groups of eight rows 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scale_tile(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// A scale tile from shared memory into four columns of tensor memory, the 32
// lanes repeated in every lane quarter. Ordered with the issuing thread's MMAs.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// `bytes` (a multiple of 16) from a 16-byte aligned address into shared memory;
// they complete on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

}  // namespace fp8blk
