// Quantisation to microscaled 4-bit floats and back (fp4.cuh has the rules).
//
// fp4_quant: a block of threads to a row, 8 columns to a thread and pass, so that a
// warp reads and writes whole lines. The row stays in registers between its amax and
// its codes (up to 8192 columns; longer rows are read again). fp4_dequant: 8
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
  uint32_t* q;
  uint8_t* s;
  float* g;
  int64_t x_stride, ktiles;
  int vecs;  // K / 8
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kMaxThreads) fp4_quant_kernel(const QuantParams p) {
  __shared__ uint32_t part[kMaxThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const int n = blockDim.x, tid = threadIdx.x;
  float v[kHeld][8];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    if (tid + u * n < p.vecs) load8(x + static_cast<int64_t>(tid + u * n) * 8, v[u]);
  }
  RowScale rs{};
  if constexpr (FMT == kFp4E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) m = max(m, amax8(v[u]));
    for (int i = tid + kHeld * n; i < p.vecs; i += n) {
      float w[8];
      load8(x + static_cast<int64_t>(i) * 8, w);
      m = max(m, amax8(w));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
    const int lane = tid & 31;
    m = __reduce_max_sync(0xFFFFFFFFu, lane < n / 32 ? part[lane] : 0u);
    rs = fp4_row_scale(m);
    if (tid == 0) p.g[row] = rs.g;
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if ((tid & ~31) + u * n < p.vecs) fp4_store8<FMT>(v[u], amax8(v[u]), rs, row, tid + u * n, p.vecs, p.q, p.s, p.ktiles);
  for (int u = kHeld; (tid & ~31) + u * n < p.vecs; ++u) {
    float w[8] = {};
    if (tid + u * n < p.vecs) load8(x + static_cast<int64_t>(tid + u * n) * 8, w);
    fp4_store8<FMT>(w, amax8(w), rs, row, tid + u * n, p.vecs, p.q, p.s, p.ktiles);
  }
}

struct DequantParams {
  const uint32_t* q;
  const uint8_t* s;
  const float* g;
  uint4* out;
  int64_t ktiles;
  int vecs;
};

// A block of threads to 256 vectors (2048 columns) of a row.
template <int FMT>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const DequantParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  float g = 1.0f;
  if constexpr (FMT == kFp4E4M3) g = __ldg(p.g + row);
  for (int vec = blockIdx.y * 256 + threadIdx.x; vec < p.vecs; vec += gridDim.y * 256) {
    float v[8];
    e2m1x8_values(__ldcs(p.q + row * p.vecs + vec), v);
    if constexpr (FMT == kFp4E4M3) {
      const float s = e4m3_value(__ldg(p.s + fp4_scale_at(row, vec / 2, p.ktiles)));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j] * s, g);  // v s is exact
    } else {
      const uint32_t e = __ldg(p.s + fp4_scale_at(row, vec / 4, p.ktiles));
      // 2^(e - 127): a subnormal for e = 0, NaN for e = 255
      const float s = e == 255 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(e ? e << 23 : 1u << 22);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(p.out + row * p.vecs + vec, make_uint4(w[0], w[1], w[2], w[3]));
  }
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
  p.q = static_cast<uint32_t*>(q);
  p.s = static_cast<uint8_t*>(s);
  p.g = g;
  p.x_stride = x_stride;
  p.ktiles = K / fp4_tile_cols(fmt);
  p.vecs = static_cast<int>(K / 8);
  int threads = (p.vecs + 31) / 32 * 32;
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
  p.q = static_cast<const uint32_t*>(q);
  p.s = static_cast<const uint8_t*>(s);
  p.g = g;
  p.out = static_cast<uint4*>(out_bf16);
  p.vecs = static_cast<int>(K / 8);
  p.ktiles = K / fp4_tile_cols(fmt);
  const void* kernel = fmt == kFp4E4M3 ? reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4E4M3>)
                                       : reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4UE8M0>);
  const unsigned across = static_cast<unsigned>((p.vecs + 255) / 256);
  return launch(kernel, dim3(static_cast<unsigned>(M), across < 65535u ? across : 65535u), 256, &p,
                reinterpret_cast<cudaStream_t>(stream));
}
