// The seam between two blocks of a transformer layer: the block's output is
// normed (optionally), gated, added to the scaled residual, and the sum normed
// for the next block, whose product reads it in bf16, e4m3 or e2m1.
//
//   z = post_w ? y * rsqrt(mean(y^2) + eps) * post_w : y
//   r = residual_scale * x + gate * z          -> bf16
//   h = r * rsqrt(mean(r^2) + eps) * norm_w    -> bf16, or act_quant, or fp4_quant
//
// fp32 from the inputs to the one rounding of each output (the norm reads r
// before it is rounded). One block of threads to a token, 16 columns to a thread and
// pass (a quantisation block of e2m1, an eighth of an e4m3 block), the row in
// registers from the first read to the last write.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_rule.cuh"
#include "fp4.cuh"
#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"
#include "quotient.cuh"

namespace fp8blk {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCols = 16384;

// What h is written as.
enum : int { kOutBf16 = 0, kOutE4m3 = 1, kOutFp4E4M3 = 2, kOutFp4UE8M0 = 3 };

struct NormParams {
  const __nv_bfloat16* y;
  const __nv_bfloat16* x;   // null: no residual
  const float* post_w;      // null: no norm of y
  const float* gate_col;    // null, or one factor per column
  const __nv_bfloat16* gate_tok;  // null, or one factor per token and column
  const float* norm_w;
  __nv_bfloat16* r;         // null: not written
  void* h;
  void* h_s;                // e4m3: fp32 scales; e2m1: scale tiles
  float* h_g;               // e2m1 with e4m3 scales: row scales
  int64_t y_stride, x_stride, gate_stride, ktiles;
  float residual_scale, eps, inv_n;
  int cols;
  int ue8m0;
};

__device__ __forceinline__ void unpack8(const uint4& a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Columns c .. c + 15 of a bf16 row; those past `cols` (a multiple of 8) are zeros.
__device__ __forceinline__ void load16(const __nv_bfloat16* row, int c, int cols, float* v) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  unpack8(c < cols ? *reinterpret_cast<const uint4*>(row + c) : zero, v);
  unpack8(c + 8 < cols ? *reinterpret_cast<const uint4*>(row + c + 8) : zero, v + 8);
}

__device__ __forceinline__ void load16(const float* row, int c, int cols, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = c + 4 * i < cols ? __ldg(reinterpret_cast<const float4*>(row + c) + i) : make_float4(0, 0, 0, 0);
    v[4 * i] = a.x;
    v[4 * i + 1] = a.y;
    v[4 * i + 2] = a.z;
    v[4 * i + 3] = a.w;
  }
}

// The sum over the block, the same in every thread: lanes, then warps in order.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 1 / sqrt(mean of v^2 + eps) over the block's row. Squares that overflow fp32 (a
// row near 2^60), or that vanish where eps does not hide it, are summed again
// with v times a power of two; the sum is the same in all threads, so they turn together.
template <int V>
__device__ __forceinline__ float rms_factor(const float (&v)[V][16], float inv_n, float eps, float* part) {
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < V; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[u][i], v[u][i], sum);
  sum = block_sum(sum, part);
  const bool huge = sum == __uint_as_float(0x7F800000u);
  if (huge || (sum < 7.9e-31f && eps < 8.7e-19f)) {  // 2^-100, 2^-60
    const float s = __uint_as_float(huge ? (127u - 80u) << 23 : (127u + 60u) << 23);
    sum = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = fmaf(v[u][i] * s, v[u][i] * s, sum);
    __syncthreads();  // every warp has read the first sums
    return __frsqrt_rn(fmaf(block_sum(sum, part), inv_n, eps * s * s)) * s;
  }
  return __frsqrt_rn(fmaf(sum, inv_n, eps));
}

template <int OUT, int V>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_kernel(const NormParams p) {
  __shared__ float part[3][32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31;
  float v[V][16];
#pragma unroll
  for (int u = 0; u < V; ++u) load16(p.y + row * p.y_stride, (tid + u * n) * 16, p.cols, v[u]);
  if (p.post_w) {
    const float k = rms_factor<V>(v, p.inv_n, p.eps, part[0]);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float w[16];
      load16(p.post_w, (tid + u * n) * 16, p.cols, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] *= k * w[i];
    }
  }
  if (p.gate_col || p.gate_tok) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float w[16];
      if (p.gate_col) load16(p.gate_col, (tid + u * n) * 16, p.cols, w);
      else load16(p.gate_tok + row * p.gate_stride, (tid + u * n) * 16, p.cols, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] *= w[i];
    }
  }
  if (p.x) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float w[16];
      load16(p.x + row * p.x_stride, (tid + u * n) * 16, p.cols, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] = fmaf(w[i], p.residual_scale, v[u][i]);
    }
  }
  if (p.r) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int c = (tid + u * n) * 16;
      if (c < p.cols) *reinterpret_cast<uint4*>(p.r + row * p.cols + c) = pack8(v[u]);
      if (c + 8 < p.cols) *reinterpret_cast<uint4*>(p.r + row * p.cols + c + 8) = pack8(v[u] + 8);
    }
  }
  const float k = rms_factor<V>(v, p.inv_n, p.eps, part[1]);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    float w[16];
    load16(p.norm_w, (tid + u * n) * 16, p.cols, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[u][i] *= k * w[i];
  }

  if constexpr (OUT == kOutBf16) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int c = (tid + u * n) * 16;
      __nv_bfloat16* h = static_cast<__nv_bfloat16*>(p.h) + row * p.cols + c;
      if (c < p.cols) *reinterpret_cast<uint4*>(h) = pack8(v[u]);
      if (c + 8 < p.cols) *reinterpret_cast<uint4*>(h + 8) = pack8(v[u] + 8);
    }
  } else if constexpr (OUT == kOutE4m3) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int c = (tid + u * n) * 16;
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[u][i]));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));  // eight lanes: 128 columns
      if (c >= p.cols) continue;
      const float s = block_scale(m, p.ue8m0 != 0), ri = __frcp_rn(s);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = div_by_scale(v[u][4 * i + j], s, ri);
        w[i] = e4m3x2(q[0], q[1]) | (static_cast<uint32_t>(e4m3x2(q[2], q[3])) << 16);
      }
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.h) + row * p.cols + c) = make_uint4(w[0], w[1], w[2], w[3]);
      if ((lane & 7) == 0) static_cast<float*>(p.h_s)[row * (p.cols / kBlock) + c / kBlock] = s;
    }
  } else {
    uint32_t am[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      am[u] = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) am[u] = max(am[u], __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
    }
    RowScale rs{};
    if constexpr (OUT == kOutFp4E4M3) {
      uint32_t m = am[0];
#pragma unroll
      for (int u = 1; u < V; ++u) m = max(m, am[u]);
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      uint32_t* top = reinterpret_cast<uint32_t*>(part[2]);
      if (lane == 0) top[tid >> 5] = m;
      __syncthreads();
      m = __reduce_max_sync(0xFFFFFFFFu, lane < (n >> 5) ? top[lane] : 0u);
      rs = fp4_row_scale(m);
      if (tid == 0) p.h_g[row] = rs.g;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int unit = tid + u * n;
      float mul;
      uint32_t word;
      if constexpr (OUT == kOutFp4E4M3) {
        word = static_cast<uint32_t>(fp4_block_scale_e4m3(am[u], rs, &mul)) << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
      } else {
        const uint32_t m = max(am[u], __shfl_xor_sync(0xFFFFFFFFu, am[u], 1));
        word = static_cast<uint32_t>(fp4_block_scale_ue8m0(m, &mul)) << (8 * ((lane >> 1) & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
      }
      if (unit * 16 >= p.cols) continue;
      static_cast<uint2*>(p.h)[row * (p.cols / 16) + unit] = e2m1x16_scaled(v[u], mul);
      constexpr int per = OUT == kOutFp4E4M3 ? 4 : 8;
      if ((unit & (per - 1)) == 0)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.h_s) +
                                     fp4_scale_at(row, OUT == kOutFp4E4M3 ? unit : unit / 2, p.ktiles)) = word;
    }
  }
}

template <int OUT>
const void* kernel_for(int v) {
  return v == 1 ? reinterpret_cast<const void*>(residual_norm_kernel<OUT, 1>)
                : reinterpret_cast<const void*>(residual_norm_kernel<OUT, 2>);
}

}  // namespace

bool fp4_fmt_valid(int fmt);

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_residual_norm(const void* y_bf16, int64_t y_stride, const void* x_bf16, int64_t x_stride,
                                    const float* post_w, const float* gate_col, const void* gate_tok_bf16,
                                    int64_t gate_stride, float residual_scale, const float* norm_w, float eps, int64_t T,
                                    int64_t D, int out_kind, int scale_fmt, void* r_bf16, void* h, void* h_s, float* h_g,
                                    fp8blk_stream_t stream) {
  const bool fp8 = out_kind == FP8BLK_NORM_E4M3, fp4 = out_kind == FP8BLK_NORM_E2M1;
  if (out_kind != FP8BLK_NORM_BF16 && !fp8 && !fp4) return FP8BLK_ERR_ARG;
  if (T < 0 || T >= int64_t{1} << 31 || D < 1 || D > kMaxCols || D % (out_kind == FP8BLK_NORM_BF16 ? 8 : kBlock) ||
      y_stride < D || (x_bf16 && x_stride < D) || (gate_tok_bf16 && gate_stride < D))
    return FP8BLK_ERR_SHAPE;
  if ((fp8 && !scale_fmt_valid(scale_fmt)) || (fp4 && !fp4_fmt_valid(scale_fmt)) || !(eps >= 0.0f) ||
      (gate_col && gate_tok_bf16))
    return FP8BLK_ERR_ARG;
  if (T == 0) return FP8BLK_OK;
  if (!y_bf16 || !norm_w || !h || ((fp8 || fp4) && !h_s) || (fp4 && scale_fmt == kFp4E4M3 && !h_g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(y_bf16, 16) || y_stride % 8 || !is_aligned(x_bf16, 16) || (x_bf16 && x_stride % 8) ||
      !is_aligned(post_w, 16) || !is_aligned(gate_col, 16) || !is_aligned(gate_tok_bf16, 16) ||
      (gate_tok_bf16 && gate_stride % 8) || !is_aligned(norm_w, 16) || !is_aligned(r_bf16, 16) || !is_aligned(h, 16) ||
      !is_aligned(h_s, fp4 ? 16 : 4) || !is_aligned(h_g, 4))
    return FP8BLK_ERR_ALIGN;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  NormParams p{};
  p.y = static_cast<const __nv_bfloat16*>(y_bf16);
  p.x = static_cast<const __nv_bfloat16*>(x_bf16);
  p.post_w = post_w;
  p.gate_col = gate_col;
  p.gate_tok = static_cast<const __nv_bfloat16*>(gate_tok_bf16);
  p.norm_w = norm_w;
  p.r = static_cast<__nv_bfloat16*>(r_bf16);
  p.h = h;
  p.h_s = h_s;
  p.h_g = h_g;
  p.y_stride = y_stride;
  p.x_stride = x_stride;
  p.gate_stride = gate_stride;
  p.ktiles = fp4 ? D / fp4_tile_cols(scale_fmt) : 0;
  p.residual_scale = residual_scale;
  p.eps = eps;
  p.inv_n = 1.0f / static_cast<float>(D);
  p.cols = static_cast<int>(D);
  p.ue8m0 = fp8 && scale_fmt_ue8m0(scale_fmt);
  const int units = static_cast<int>((D + 15) / 16);
  const int V = units > kMaxThreads ? 2 : 1;
  const int threads = ((units + V - 1) / V + 31) / 32 * 32;
  const void* kernel = !fp8 && !fp4               ? kernel_for<kOutBf16>(V)
                       : fp8                      ? kernel_for<kOutE4m3>(V)
                       : scale_fmt == kFp4E4M3    ? kernel_for<kOutFp4E4M3>(V)
                                                  : kernel_for<kOutFp4UE8M0>(V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T));
  cfg.blockDim = dim3(threads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {&p};
  return cuda_status(cudaLaunchKernelExC(&cfg, kernel, args));
}
