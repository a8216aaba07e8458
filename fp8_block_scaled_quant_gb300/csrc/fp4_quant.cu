// Quantisation to microscaled 4-bit floats and back (fp4.cuh has the rules).
//
// fp4_quant: one row to a block of threads, 16 columns (one e4m3 block, half a
// ue8m0 block) to a thread and pass. The row stays in registers between its amax
// and its codes (up to 16384 columns; longer rows are read again). fp4_dequant: 16
// columns to a thread. Both are bound by HBM, single rows by launch latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kHeld = 4;  // passes whose values stay in registers

struct QuantParams {
  const void* x;
  uint2* q;
  uint8_t* s;
  float* g;
  int64_t x_stride, ktiles;
  int units;  // K / 16
};

__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* v) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load16(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + i);
    v[4 * i] = a.x;
    v[4 * i + 1] = a.y;
    v[4 * i + 2] = a.z;
    v[4 * i + 3] = a.w;
  }
}

__device__ __forceinline__ uint32_t amax16(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// The codes and the scale bytes of a unit. All lanes of a group of eight (four)
// call it together: a scale word is put together from eight (four) lanes.
template <int FMT>
__device__ __forceinline__ void store_unit(const QuantParams& p, int64_t row, int unit, const float* v, uint32_t amax,
                                           const RowScale& rs) {
  float mul;
  uint32_t word;
  const int lane = threadIdx.x & 31;
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
  if (unit >= p.units) return;
  p.q[row * p.units + unit] = e2m1x16_scaled(v, mul);
  const int per = FMT == kFp4E4M3 ? 4 : 8;
  if ((unit & (per - 1)) == 0) {
    const int block = FMT == kFp4E4M3 ? unit : unit / 2;
    *reinterpret_cast<uint32_t*>(p.s + fp4_scale_at(row, block, p.ktiles)) = word;
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kMaxThreads) fp4_quant_kernel(const QuantParams p) {
  __shared__ uint32_t part[kMaxThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const int n = blockDim.x, tid = threadIdx.x;
  const int passes = (p.units + n - 1) / n;
  float v[kHeld][16];
  uint32_t am[kHeld];
  RowScale rs{};
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    am[u] = 0;
    if (u < passes && tid + u * n < p.units) load16(x + static_cast<int64_t>(tid + u * n) * 16, v[u]);
    else
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) am[u] = amax16(v[u]);
  if constexpr (FMT == kFp4E4M3) {
    uint32_t m = max(max(am[0], am[1]), max(am[2], am[3]));
    for (int i = tid + kHeld * n; i < p.units; i += n) {
      float w[16];
      load16(x + static_cast<int64_t>(i) * 16, w);
      m = max(m, amax16(w));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
    for (int i = 0; i < n / 32; ++i) m = max(m, part[i]);
    rs = fp4_row_scale(m);
    if (tid == 0) p.g[row] = rs.g;
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (u < passes) store_unit<FMT>(p, row, tid + u * n, v[u], am[u], rs);
  for (int u = kHeld; u < passes; ++u) {
    float w[16] = {};
    if (tid + u * n < p.units) load16(x + static_cast<int64_t>(tid + u * n) * 16, w);
    store_unit<FMT>(p, row, tid + u * n, w, amax16(w), rs);
  }
}

struct DequantParams {
  const uint2* q;
  const uint8_t* s;
  const float* g;
  uint4* out;
  int64_t total, ktiles;  // units of 16 columns
  int units;
};

template <int FMT>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const DequantParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.total) return;
  const int64_t row = i / p.units;
  const int unit = static_cast<int>(i - row * p.units);
  const uint2 codes = __ldcs(p.q + i);
  float v[16];
  e2m1x8_values(codes.x, v);
  e2m1x8_values(codes.y, v + 8);
  uint32_t w[8];
  if constexpr (FMT == kFp4E4M3) {
    const float s = e4m3_value(__ldg(p.s + fp4_scale_at(row, unit, p.ktiles))), g = __ldg(p.g + row);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j] * s, g);  // v s is exact
  } else {
    const uint32_t e = __ldg(p.s + fp4_scale_at(row, unit / 2, p.ktiles));
    // 2^(e - 127): a subnormal for e = 0, NaN for e = 255
    const float s = e == 255 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(e ? e << 23 : 1u << 22);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= s;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  __stcs(p.out + 2 * i, make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(p.out + 2 * i + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

int launch(const void* kernel, dim3 grid, int threads, void* params, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {params};
  return cuda_status(cudaLaunchKernelExC(&cfg, kernel, args));
}

}  // namespace

bool fp4_fmt_valid(int fmt) { return fmt == kFp4E4M3 || fmt == kFp4UE8M0; }

// Arguments checked by the caller.
int fp4_quant_launch(const void* x, bool fp32, int64_t x_stride, int64_t M, int64_t K, int fmt, void* q, void* s, float* g,
                     cudaStream_t stream) {
  QuantParams p{};
  p.x = x;
  p.q = static_cast<uint2*>(q);
  p.s = static_cast<uint8_t*>(s);
  p.g = g;
  p.x_stride = x_stride;
  p.ktiles = K / fp4_tile_cols(fmt);
  p.units = static_cast<int>(K / 16);
  int threads = (p.units + 31) / 32 * 32;
  if (threads > kMaxThreads) threads = kMaxThreads;
  const void* kernel =
      fp32 ? (fmt == kFp4E4M3 ? reinterpret_cast<const void*>(fp4_quant_kernel<float, kFp4E4M3>)
                              : reinterpret_cast<const void*>(fp4_quant_kernel<float, kFp4UE8M0>))
           : (fmt == kFp4E4M3 ? reinterpret_cast<const void*>(fp4_quant_kernel<__nv_bfloat16, kFp4E4M3>)
                              : reinterpret_cast<const void*>(fp4_quant_kernel<__nv_bfloat16, kFp4UE8M0>));
  return launch(kernel, dim3(static_cast<unsigned>(M)), threads, &p, stream);
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_fp4_scale_bytes(int64_t rows, int64_t K, int fmt) {
  if (rows < 0 || K < 0 || K % kBlock || !fp4_fmt_valid(fmt)) return 0;
  return static_cast<size_t>(fp4_scale_bytes(rows, K, fmt));
}

extern "C" int fp8blk_fp4_quant(const void* x, int is_fp32, int64_t x_stride, int64_t M, int64_t K, int fmt, void* q,
                                void* s, float* g, fp8blk_stream_t stream) {
  if (M < 0 || K < 0 || K % kBlock || M >= int64_t{1} << 31 || K >= int64_t{1} << 30 || x_stride < K)
    return FP8BLK_ERR_SHAPE;
  if (!fp4_fmt_valid(fmt) || (is_fp32 != 0 && is_fp32 != 1)) return FP8BLK_ERR_ARG;
  if (M == 0 || K == 0) return FP8BLK_OK;
  if (!x || !q || !s || (fmt == kFp4E4M3 && !g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(x, 16) || x_stride % (is_fp32 ? 4 : 8) || !is_aligned(q, 16) || !is_aligned(s, 16) || !is_aligned(g, 4))
    return FP8BLK_ERR_ALIGN;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  return fp4_quant_launch(x, is_fp32 == 1, x_stride, M, K, fmt, q, s, g, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fp8blk_fp4_dequant(const void* q, const void* s, const float* g, int64_t M, int64_t K, int fmt,
                                  void* out_bf16, fp8blk_stream_t stream) {
  if (M < 0 || K < 0 || K % kBlock || M >= int64_t{1} << 31 || K >= int64_t{1} << 30) return FP8BLK_ERR_SHAPE;
  if (!fp4_fmt_valid(fmt)) return FP8BLK_ERR_ARG;
  if (M == 0 || K == 0) return FP8BLK_OK;
  if (!q || !s || !out_bf16 || (fmt == kFp4E4M3 && !g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(q, 16) || !is_aligned(s, 16) || !is_aligned(out_bf16, 16) || !is_aligned(g, 4)) return FP8BLK_ERR_ALIGN;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  DequantParams p{};
  p.q = static_cast<const uint2*>(q);
  p.s = static_cast<const uint8_t*>(s);
  p.g = g;
  p.out = static_cast<uint4*>(out_bf16);
  p.units = static_cast<int>(K / 16);
  p.total = M * p.units;
  p.ktiles = K / fp4_tile_cols(fmt);
  if (p.total > ((int64_t{1} << 31) - 1) * 256) return FP8BLK_ERR_SHAPE;
  const void* kernel = fmt == kFp4E4M3 ? reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4E4M3>)
                                       : reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4UE8M0>);
  return launch(kernel, dim3(static_cast<unsigned>((p.total + 255) / 256)), 256, &p,
                reinterpret_cast<cudaStream_t>(stream));
}
