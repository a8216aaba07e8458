// Quantisation to microscaled 4-bit floats and back (fp4.cuh has the rules).
//
// fp4_quant: 16 columns to a thread and pass (an e4m3 block, half a ue8m0 block),
// read at once where the rows are aligned to 32 bytes. The row stays in registers
// as it was read between its amax and its codes (rows longer than that are read
// again). Short rows have a warp each. fp4_dequant: 16 columns to a thread. HBM
// bounds both, single rows launch latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kShortRows = 8;  // rows of a block where a warp has one

struct QuantParams {
  const void* x;
  uint2* q;
  uint8_t* s;
  float* g;
  int64_t rows, x_stride, ktiles;
  int units;    // K / 16
  int threads;  // of a row
  int wide;     // rows aligned to 32 bytes
  int early;    // the next kernel may start beside this one (inside a layer: what it reads ahead are weights)
};

__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = load_once16(p), b = load_once16(static_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// 16 columns as they are read.
template <typename T>
struct Unit;

template <>
struct Unit<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool wide) { load32(p, wide, w); }
  // The bits of the largest |x| as fp32.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};

template <>
struct Unit<float> {
  uint32_t w[16];
  __device__ __forceinline__ void load(const float* p, bool wide) {
    load32(p, wide, w);
    load32(p + 8, wide, w + 8);
  }
  __device__ __forceinline__ uint32_t amax() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2)  // (a NaN stays)
      asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(__uint_as_float(w[i])), "f"(__uint_as_float(w[i + 1])));
    return __float_as_uint(m) & 0x7FFFFFFFu;
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};

template <int FMT, typename T>
__device__ __forceinline__ void store_unit(const QuantParams& p, int64_t row, int unit, const Unit<T>& x, uint32_t amax,
                                           const RowScale& rs) {
  float2 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x.pair(i);
  fp4_store16<FMT>(v, amax, rs, row, unit, p.units, p.q, p.s, p.ktiles);
}

// P passes of p.threads units stay in registers.
template <typename T, int FMT, int P>
__global__ void __launch_bounds__(kMaxThreads) fp4_quant_kernel(const QuantParams p) {
  __shared__ uint32_t part[kMaxThreads / 32];
  if (p.early) griddep_launch_dependents();
  griddep_wait();
  const int n = p.threads, lane = threadIdx.x & 31;
  // (n is 32 where a block has several rows; a warp leaves as a whole)
  const int64_t row = blockDim.x == n ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kShortRows + (threadIdx.x >> 5);
  const int tid = blockDim.x == n ? threadIdx.x : lane;
  if (row >= p.rows) return;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  Unit<T> v[P];
  uint32_t am[P];
#pragma unroll
  for (int u = 0; u < P; ++u) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(v[u].w) / 4); ++i) v[u].w[i] = 0;
    if (tid + u * n < p.units) v[u].load(x + static_cast<int64_t>(tid + u * n) * 16, p.wide);
  }
#pragma unroll
  for (int u = 0; u < P; ++u) am[u] = v[u].amax();
  RowScale rs{};
  if constexpr (FMT == kFp4E4M3) {
    uint32_t m = am[0];
#pragma unroll
    for (int u = 1; u < P; ++u) m = max(m, am[u]);
    for (int i = tid + P * n; i < p.units; i += n) {
      Unit<T> w;
      w.load(x + static_cast<int64_t>(i) * 16, p.wide);
      m = max(m, w.amax());
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (n > 32) {
      if (lane == 0) part[tid >> 5] = m;
      __syncthreads();
      m = __reduce_max_sync(0xFFFFFFFFu, lane < n / 32 ? part[lane] : 0u);
    }
    rs = fp4_row_scale(m);
    if (tid == 0) p.g[row] = rs.g;
  }
#pragma unroll
  for (int u = 0; u < P; ++u)
    if ((tid & ~31) + u * n < p.units) store_unit<FMT>(p, row, tid + u * n, v[u], am[u], rs);
  for (int u = P; (tid & ~31) + u * n < p.units; ++u) {
    Unit<T> w{};
    if (tid + u * n < p.units) w.load(x + static_cast<int64_t>(tid + u * n) * 16, p.wide);
    store_unit<FMT>(p, row, tid + u * n, w, w.amax(), rs);
  }
}

template <typename T, int FMT>
const void* quant_kernel(int P) {
  return P == 1   ? reinterpret_cast<const void*>(fp4_quant_kernel<T, FMT, 1>)
         : P == 2 ? reinterpret_cast<const void*>(fp4_quant_kernel<T, FMT, 2>)
         : P == 4 ? reinterpret_cast<const void*>(fp4_quant_kernel<T, FMT, 4>)
                  : reinterpret_cast<const void*>(fp4_quant_kernel<T, FMT, 6>);
}

struct DequantParams {
  const uint2* q;
  const uint8_t* s;
  const float* g;
  uint4* out;
  int64_t rows, ktiles;
  int units;
};

// blockDim.x units of a row, blockDim.y rows.
template <int FMT>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const DequantParams p) {
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;
  float g = 1.0f;
  if constexpr (FMT == kFp4E4M3) g = p.g[row];
  for (int unit = blockIdx.y * blockDim.x + threadIdx.x; unit < p.units; unit += gridDim.y * blockDim.x) {
    const uint2 codes = load_once8(p.q + row * p.units + unit);
    float s;
    if constexpr (FMT == kFp4E4M3) {
      s = e4m3_value(p.s[fp4_scale_at(row, unit, p.ktiles)]);
    } else {
      const uint32_t e = p.s[fp4_scale_at(row, unit / 2, p.ktiles)];
      // 2^(e - 127): a subnormal for e = 0, NaN for e = 255
      s = e == 255 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(e ? e << 23 : 1u << 22);
    }
    uint32_t w[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float2 v[4];
      e2m1x8_values(half ? codes.y : codes.x, &v[0].x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = __fmul2_rn(v[j], make_float2(s, s));  // exact
        if constexpr (FMT == kFp4E4M3) v[j] = __fmul2_rn(v[j], make_float2(g, g));
        const __nv_bfloat162 b = __float22bfloat162_rn(v[j]);
        w[half * 4 + j] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    uint4* out = p.out + (row * p.units + unit) * 2;
    // (32-byte aligned: K is a multiple of 128, and out is checked)
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}

int launch(const void* kernel, dim3 grid, dim3 threads, void* params, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
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
                     int sm_count, bool early, cudaStream_t stream) {
  QuantParams p{};
  p.early = early;
  p.x = x;
  p.q = static_cast<uint2*>(q);
  p.s = static_cast<uint8_t*>(s);
  p.g = g;
  p.rows = M;
  p.x_stride = x_stride;
  p.ktiles = K / fp4_tile_cols(fmt);
  p.units = static_cast<int>(K / 16);
  p.wide = is_aligned(x, 32) && x_stride * (fp32 ? 4 : 2) % 32 == 0;
  // Up to 128 bytes of a row to a thread, which are under way together (4096 x 7168
  // bf16: 14.5 us; 64 bytes 15.8, 32 bytes 21; 18432 x 7168 fp32: 90, of 256 bytes
  // 95), as long as that leaves 24 warps to an SM (1407 x 2048 bf16: 3.5 us, of 128
  // bytes to a thread 4.2); more where the row is longer than 512 threads have.
  const auto warps = [&](int P) { return M * ((p.units + 32 * P - 1) / (32 * P)); };
  int P = 1;
  while (P < (fp32 ? 2 : 4) && p.units > 32 * P && warps(2 * P) >= 24 * sm_count) P *= 2;
  while (P < 6 && (p.units + P - 1) / P > kMaxThreads) P = P == 4 ? 6 : 2 * P;
  p.threads = ((p.units + P - 1) / P + 31) / 32 * 32;
  if (p.threads > kMaxThreads) p.threads = kMaxThreads;
  const bool several = p.threads == 32 && M > 2 * sm_count;
  const void* kernel = fp32 ? (fmt == kFp4E4M3 ? quant_kernel<float, kFp4E4M3>(P) : quant_kernel<float, kFp4UE8M0>(P))
                            : (fmt == kFp4E4M3 ? quant_kernel<__nv_bfloat16, kFp4E4M3>(P)
                                               : quant_kernel<__nv_bfloat16, kFp4UE8M0>(P));
  return launch(kernel, dim3(static_cast<unsigned>(several ? (M + kShortRows - 1) / kShortRows : M)),
                dim3(several ? 32 * kShortRows : p.threads), &p, stream);
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
  return fp4_quant_launch(x, is_fp32 == 1, x_stride, M, K, fmt, q, s, g, d->sm_count, false,
                          reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fp8blk_fp4_dequant(const void* q, const void* s, const float* g, int64_t M, int64_t K, int fmt,
                                  void* out_bf16, fp8blk_stream_t stream) {
  if (M < 0 || K < 0 || K % kBlock || M >= int64_t{1} << 31 || K >= int64_t{1} << 30) return FP8BLK_ERR_SHAPE;
  if (!fp4_fmt_valid(fmt)) return FP8BLK_ERR_ARG;
  if (M == 0 || K == 0) return FP8BLK_OK;
  if (!q || !s || !out_bf16 || (fmt == kFp4E4M3 && !g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(q, 16) || !is_aligned(s, 16) || !is_aligned(out_bf16, 32) || !is_aligned(g, 4)) return FP8BLK_ERR_ALIGN;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  DequantParams p{};
  p.q = static_cast<const uint2*>(q);
  p.s = static_cast<const uint8_t*>(s);
  p.g = g;
  p.out = static_cast<uint4*>(out_bf16);
  p.units = static_cast<int>(K / 16);
  p.ktiles = K / fp4_tile_cols(fmt);
  const void* kernel = fmt == kFp4E4M3 ? reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4E4M3>)
                                       : reinterpret_cast<const void*>(fp4_dequant_kernel<kFp4UE8M0>);
  p.rows = M;
  const int across = (p.units + 255) / 256;
  const int width = across > 1 ? ((p.units + across - 1) / across + 31) / 32 * 32 : p.units, rows = 256 / width;
  return launch(kernel, dim3(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>(across < 65535 ? across : 65535)),
                dim3(width, rows), &p, reinterpret_cast<cudaStream_t>(stream));
}
