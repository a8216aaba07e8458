// The seam between two blocks of a transformer layer: the block's output is
// normed (optionally), gated, added to the scaled residual, and the sum normed
// for the next block, whose product reads it in bf16, e4m3 or e2m1.
//
//   z = post_w ? y * rsqrt(mean(y^2) + eps) * post_w : y
//   r = residual_scale * x + gate * z          -> bf16
//   h = r * rsqrt(mean(r^2) + eps) * norm_w    -> bf16, or act_quant, or fp4_quant
//
// fp32 from the inputs to the one rounding of each output (the norm reads r
// before it is rounded). One block of threads to a token (or to token after token,
// below), 16 columns to a thread and unit (a quantisation block of e2m1, an eighth of one of e4m3), the row in
// registers from the first read to the last write. HBM bounds many tokens, launch
// and two block-wide sums a single one.
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
  const __nv_bfloat16* x;         // null: no residual
  const float* post_w;            // null: no norm of y
  const float* gate_col;          // null, or one factor per column
  const __nv_bfloat16* gate_tok;  // null, or one factor per token and column
  const float* norm_w;
  __nv_bfloat16* r;               // null: not written
  void* h;
  void* h_s;                      // e4m3: fp32 scales; e2m1: scale tiles
  float* h_g;                     // e2m1 with e4m3 scales: row scales
  int64_t y_stride, x_stride, gate_stride, ktiles;
  float residual_scale, eps, inv_n;
  int cols, units;                // units: ceil(cols / 16)
  int ahead;                      // tokens between a row and the one prefetched
  int ue8m0;
  int64_t rows;
  unsigned* err;
};

// 16 columns of a bf16 row, as they are read: at once where WIDE (all rows and
// factors aligned to 32 bytes, cols a multiple of 16), else by halves, the second
// where it is within `cols` (a multiple of 8). Columns past the row are zeros.
template <bool WIDE>
__device__ __forceinline__ void read16(const __nv_bfloat16* row, int unit, int cols, bool in, uint32_t* w) {
  const __nv_bfloat16* p = row + unit * 16;
  if constexpr (WIDE) {
    if (in) {
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p)
                   : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0;
    }
  } else {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a = in ? *reinterpret_cast<const uint4*>(p) : zero;
    const uint4 b = in && unit * 16 + 8 < cols ? *reinterpret_cast<const uint4*>(p + 8) : zero;
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// The same of fp32 factors (which stay in L1: every token reads them).
template <bool WIDE>
__device__ __forceinline__ void read16(const float* row, int unit, int cols, float2* v) {
  const float* p = row + unit * 16;
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[4 * h].x), "=f"(v[4 * h].y), "=f"(v[4 * h + 1].x), "=f"(v[4 * h + 1].y), "=f"(v[4 * h + 2].x),
                     "=f"(v[4 * h + 2].y), "=f"(v[4 * h + 3].x), "=f"(v[4 * h + 3].y)
                   : "l"(p + 8 * h)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = unit * 16 + 4 * i < cols ? reinterpret_cast<const float4*>(p)[i] : make_float4(0, 0, 0, 0);
      v[2 * i] = make_float2(a.x, a.y);
      v[2 * i + 1] = make_float2(a.z, a.w);
    }
  }
}

// Columns are worked on in pairs (packed fp32 multiplies and FMAs).
__device__ __forceinline__ float2 pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool WIDE>
__device__ __forceinline__ void write16(__nv_bfloat16* row, int unit, int cols, const float2* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(v[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  __nv_bfloat16* p = row + unit * 16;
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (unit * 16 + 8 < cols) reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A value combined over the block by f, the same in every thread: lanes, then
// warps in order. `at`: a place per warp, not used before.
template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T none, T* at, F f) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if (warps == 1) return v;
  if (lane == 0) at[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? at[lane] : none;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));  // at most 16 warps
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}

__device__ __forceinline__ float block_sum(float v, float* at) {
  return block_reduce(v, 0.0f, at, [](float a, float b) { return a + b; });
}

// Four sums over a warp at once: each of the first two exchanges halves the values
// that a lane goes on with, so lanes 8 k .. 8 k + 7 end with sum k.
__device__ __forceinline__ float warp_sum4(float4 v) {
  const int k = (threadIdx.x & 31) >> 3;
  float a = k & 2 ? v.z : v.x, b = k & 2 ? v.w : v.y;
  a += __shfl_xor_sync(0xFFFFFFFFu, k & 2 ? v.x : v.z, 16);
  b += __shfl_xor_sync(0xFFFFFFFFu, k & 2 ? v.y : v.w, 16);
  float s = k & 1 ? b : a;
  s += __shfl_xor_sync(0xFFFFFFFFu, k & 1 ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// The block's sums from those of its warps (at[4 warp + k], at most 16 warps).
__device__ __forceinline__ float4 warps_sum4(const float* at) {
  const int warps = blockDim.x >> 5, k = (threadIdx.x & 31) >> 3, w = threadIdx.x & 7;
  float s = (w < warps ? at[w * 4 + k] : 0.0f) + (w + 8 < warps ? at[(w + 8) * 4 + k] : 0.0f);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return make_float4(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 8), __shfl_sync(0xFFFFFFFFu, s, 16),
                     __shfl_sync(0xFFFFFFFFu, s, 24));
}

// 1 / sqrt(mean of v^2 + eps) over the block's row. Squares that overflow fp32 (a
// row near 2^60), or that vanish where eps does not hide it, are summed again
// with v times a power of two; the sum is the same in all threads, so they turn together.
// Not `in`: the thread's last unit is past the row and does not count (a zero there
// that was multiplied by an infinite factor is a NaN).
template <int P>
__device__ __forceinline__ float rms_factor(const float2 (&v)[P][8], bool in, float inv_n, float eps, float* at) {
  float2 two = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const float2 before = two;
#pragma unroll
    for (int i = 0; i < 8; ++i) two = __ffma2_rn(v[u][i], v[u][i], two);
    if (u == P - 1 && !in) two = before;
  }
  float sum = block_sum(two.x + two.y, at);
  const bool huge = sum == __uint_as_float(0x7F800000u);
  if (huge || (sum < 7.9e-31f && eps < 8.7e-19f)) {  // 2^-100, 2^-60
    const float s = __uint_as_float(huge ? (127u - 80u) << 23 : (127u + 60u) << 23);
    sum = 0.0f;
#pragma unroll
    for (int u = 0; u < P; ++u) {
      if (u == P - 1 && !in) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[u][i].x * s, v[u][i].x * s, fmaf(v[u][i].y * s, v[u][i].y * s, sum));
    }
    __syncthreads();  // every warp has read the first sums
    return inverse_root(fmaf(block_sum(sum, at), inv_n, eps * s * s)) * s;
  }
  return inverse_root(fmaf(sum, inv_n, eps));
}

// The act_quant scale of a block (block_scale's value: max(amax, 1e-4) / 448 by
// Markstein's correction: the IEEE quotient for every fp32 amax from 1e-4 on). h has
// passed several fp32 roundings, so its product with the scale's reciprocal takes the
// place of act_quant's exact quotient of a bf16 number: three more roundings, 2^-22 in
// all, and a value as near as that to a border between two codes may take either one
// (1 code in 1.5 million, as often as by the formula in fp32).
__device__ __forceinline__ float e4m3_scale(float amax, bool ue8m0) {
  float s = div_by_scale(fmaxf(amax, 1e-4f), 448.0f, 1.0f / 448.0f);
  if (ue8m0) {
    uint32_t b = __float_as_uint(s);
    if (b & 0x007FFFFFu) b = (b & 0x7F800000u) + 0x00800000u;
    s = __uint_as_float(b);
  }
  return s;
}

// A row's factor k goes onto its values after the columns' factors, where it is
// cheaper; before them where they might not stand without it (values near the ends
// of fp32's range).
template <int P>
__device__ __forceinline__ float apply_early(float2 (&v)[P][8], float k) {
  if (k > 1e-15f && k < 1e15f) return k;
#pragma unroll
  for (int u = 0; u < P; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], make_float2(k, k));
  return 1.0f;
}

// The largest of |v| of 16 columns. KEEP_NAN: a NaN is above all.
template <bool KEEP_NAN>
__device__ __forceinline__ float amax16(const float2* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (KEEP_NAN) asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v[i].x), "f"(v[i].y));
    else asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v[i].x), "f"(v[i].y));
  }
  return m;
}

// Asks for `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// r = s x + k1 v, in place of v.
template <int P>
__device__ __forceinline__ void add_residual(const NormParams& p, const uint32_t (&x)[P][8], float k1, float2 (&v)[P][8]) {
  const float2 scale2 = make_float2(p.residual_scale, p.residual_scale);
#pragma unroll
  for (int u = 0; u < P; ++u) {
    if (k1 != 1.0f)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], make_float2(k1, k1));
    if (p.x)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __ffma2_rn(pair(x[u][i]), scale2, v[u][i]);
  }
}

// A thread's parts of the sums of y^2 (given), v^2, x v and x^2 (`in`: as above).
template <int P>
__device__ __forceinline__ float4 row_sums(float2 yy, const float2 (&v)[P][8], const uint32_t (&x)[P][8], bool in) {
  float2 vv = make_float2(0.0f, 0.0f), xv = vv, xx = vv;
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const float2 vv_before = vv, xv_before = xv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 xf = pair(x[u][i]);
      vv = __ffma2_rn(v[u][i], v[u][i], vv);
      xv = __ffma2_rn(xf, v[u][i], xv);
      xx = __ffma2_rn(xf, xf, xx);
    }
    if (u == P - 1 && !in) vv = vv_before, xv = xv_before;
  }
  return make_float4(yy.x + yy.y, vv.x + vv.y, xv.x + xv.y, xx.x + xx.y);
}

// From the row's sums its residual, in place of v (y times its columns' factors, P units
// to a thread), and the factor of its norm: sum r^2 = s^2 sum x^2 + 2 s k1 sum x v +
// k1^2 sum v^2, unless the terms cancel (to less than a quarter) or leave fp32's range;
// then false, and r comes the long way, in the order of the formula.
template <int P, bool WIDE>
__device__ __forceinline__ bool both_norms(const NormParams& p, int64_t row, float4 sum, const uint32_t (&x)[P][8],
                                           float2 (&v)[P][8], float* k2, float* sum_y) {
  const int tid = threadIdx.x, n = blockDim.x;
  const float k1 = inverse_root(fmaf(sum.x, p.inv_n, p.eps)), s = p.residual_scale;
  const float a = s * s * sum.w, b = k1 * k1 * sum.y, all = a + b;
  const float rr = fmaf(2.0f * s * k1, sum.z, all);
  if (sum.x > 1e-20f && sum.x < 1e30f && sum.y < 1e30f && all > 1e-20f && rr < 1e30f && rr > 0.25f * all) {
    add_residual<P>(p, x, k1, v);
    *k2 = inverse_root(fmaf(rr, p.inv_n, p.eps));
    return true;
  }
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int unit = tid + u * n;
    uint32_t y[8];
    read16<WIDE>(p.y + row * p.y_stride, unit, p.cols, unit < p.units, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = pair(y[i]);
  }
  const float k = rms_factor<P>(v, true, p.inv_n, p.eps, sum_y);  // (zeros past the row)
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int unit = tid + u * n < p.units ? tid + u * n : 0;
    float2 w[8], g[8];
    read16<WIDE>(p.post_w, unit, p.cols, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(__fmul2_rn(v[u][i], make_float2(k, k)), w[i]);
    if (p.gate_col) {
      read16<WIDE>(p.gate_col, unit, p.cols, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], g[i]);
    }
    if (p.gate_tok) {
      uint32_t t[8];
      read16<WIDE>(p.gate_tok + row * p.gate_stride, unit, p.cols, true, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], pair(t[i]));
    }
  }
  add_residual<P>(p, x, 1.0f, v);
  return false;
}

template <int P, bool WIDE>
__device__ __forceinline__ void write_residual(const NormParams& p, int64_t row, const float2 (&v)[P][8]) {
  if (!p.r) return;
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int unit = static_cast<int>(threadIdx.x + u * blockDim.x);
    if (unit < p.units) write16<WIDE>(p.r + row * p.cols, unit, p.cols, v[u]);
  }
}

// h = k2 v, v being r times norm_w, in its type. `tops`: a place per warp.
template <int OUT, int P, bool WIDE>
__device__ __forceinline__ void write_h(const NormParams& p, int64_t row, float2 (&v)[P][8], float k2, uint32_t* tops) {
  const int tid = threadIdx.x, n = blockDim.x;
  const float2 k2k2 = make_float2(k2, k2);
  if constexpr (OUT == kOutBf16) {
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int unit = tid + u * n;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], k2k2);
      if (unit < p.units) write16<WIDE>(static_cast<__nv_bfloat16*>(p.h) + row * p.cols, unit, p.cols, v[u]);
    }
  } else if constexpr (OUT == kOutE4m3) {
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int unit = tid + u * n;
      if ((unit & ~31) >= p.units) continue;
      float m = amax16<false>(v[u]);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));  // 8 lanes: 128 columns
      if (unit >= p.units) continue;
      const float s = e4m3_scale(m * k2, p.ue8m0 != 0), f = k2 * inverse(s);
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = __fmul2_rn(v[u][2 * i], make_float2(f, f)), b = __fmul2_rn(v[u][2 * i + 1], make_float2(f, f));
        q[i] = e4m3x2(a.x, a.y) | (static_cast<uint32_t>(e4m3x2(b.x, b.y)) << 16);
      }
      reinterpret_cast<uint4*>(p.h)[row * p.units + unit] = make_uint4(q[0], q[1], q[2], q[3]);
      if ((tid & 7) == 0) static_cast<float*>(p.h_s)[row * (p.units / 8) + unit / 8] = s;
    }
  } else {
    uint32_t am[P], top = 0;
#pragma unroll
    for (int u = 0; u < P; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], k2k2);
      am[u] = __float_as_uint(amax16<true>(v[u])) & 0x7FFFFFFFu;
      top = max(top, am[u]);
    }
    RowScale rs{};
    if constexpr (OUT == kOutFp4E4M3) {
      rs = fp4_row_scale(block_reduce(top, 0u, tops,
                                      [](uint32_t a, uint32_t b) { return max(a, b); }));
      if (tid == 0) p.h_g[row] = rs.g;
    }
#pragma unroll
    for (int u = 0; u < P; ++u)
      if ((tid & ~31) + u * n < p.units)
        fp4_store16<OUT == kOutFp4E4M3 ? kFp4E4M3 : kFp4UE8M0>(v[u], am[u], rs, row, tid + u * n, p.units,
                                                               static_cast<uint2*>(p.h), static_cast<uint8_t*>(p.h_s),
                                                               p.ktiles);
  }
}

// A block to a token, P units to a thread. EARLY: norm_w is asked for with the rows
// (few tokens); otherwise where it is used, from L1, which keeps registers free
// for another block to an SM. It has what does not go from token to token, below: few
// tokens, y that is not normed (4099 x 7168 into bf16 36.1 us, HBM's rate), a gate by
// token (4099 x 7168 into e4m3 46.6, 4099 x 8192 into e2m1 58.2), e2m1 with row scales
// (4099 x 7168 48.5): with a post norm the blocks' arithmetic between their loads, not
// HBM, sets the time. (Tried on such a case, 4099 x 7168 into e4m3: next rows not
// prefetched 50.7 against 47.4; two units to a thread 55; rows through shared memory 49
// to 57.)
template <int OUT, int P, bool WIDE, bool EARLY>
__global__ void __maxnreg__(EARLY || P > 1 ? 128 : 72) residual_norm_kernel(const NormParams p) {
  constexpr int kWarps = kMaxThreads / 32;
  __shared__ float sums[4 * kWarps], sum_y[kWarps], sum_r[kWarps];
  __shared__ uint32_t tops[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, n = blockDim.x;
  const int64_t row = blockIdx.x;
  const bool has_x = p.x != nullptr, tok = p.gate_tok != nullptr;
  if (!EARLY && tid == 0 && row + p.ahead < gridDim.x) {
    // The rows that a block will read when this one's place is free again, into L2.
    const uint32_t bytes = static_cast<uint32_t>(p.cols) * 2;
    prefetch_l2(p.y + (row + p.ahead) * p.y_stride, bytes);
    if (has_x) prefetch_l2(p.x + (row + p.ahead) * p.x_stride, bytes);
    if (tok) prefetch_l2(p.gate_tok + (row + p.ahead) * p.gate_stride, bytes);
  }
  const bool last_in = tid + (P - 1) * n < p.units;
  uint32_t x[P][8];
  float2 v[P][8], ne[EARLY ? P : 1][8];
  float2 yy = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int unit = tid + u * n;
    const bool in = unit < p.units;
    uint32_t y[8], g[8];
    read16<WIDE>(p.y + row * p.y_stride, unit, p.cols, in, y);
    read16<WIDE>(p.x + row * p.x_stride, unit, p.cols, in && has_x, x[u]);
    if (tok) read16<WIDE>(p.gate_tok + row * p.gate_stride, unit, p.cols, in, g);
    if constexpr (EARLY) read16<WIDE>(p.norm_w, in ? unit : 0, p.cols, ne[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = pair(y[i]);
    if (p.post_w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) yy = __ffma2_rn(v[u][i], v[u][i], yy);
    }
    // v becomes y times its columns' factors.
    float2 w[8];
    if (p.post_w) {
      read16<WIDE>(p.post_w, in ? unit : 0, p.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], w[i]);
    }
    if (p.gate_col) {
      read16<WIDE>(p.gate_col, in ? unit : 0, p.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], w[i]);
    }
    if (tok) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], pair(g[i]));
    }
  }
  float k2 = 0.0f;
  bool known = false;
  if (p.post_w) {
    const float sum = warp_sum4(row_sums<P>(yy, v, x, last_in));
    if ((tid & 7) == 0) sums[(tid >> 5) * 4 + ((tid & 31) >> 3)] = sum;
    __syncthreads();
    known = both_norms<P, WIDE>(p, row, warps_sum4(sums), x, v, &k2, sum_y);
  } else {
    add_residual<P>(p, x, 1.0f, v);
  }
  write_residual<P, WIDE>(p, row, v);
  if (!known) k2 = rms_factor<P>(v, last_in, p.inv_n, p.eps, sum_r);
  k2 = apply_early<P>(v, k2);
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int unit = tid + u * n < p.units ? tid + u * n : 0;
    float2 w[8];
    if constexpr (!EARLY) read16<WIDE>(p.norm_w, unit, p.cols, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = __fmul2_rn(v[u][i], EARLY ? ne[u][i] : w[i]);
  }
  write_h<OUT, P, WIDE>(p, row, v, k2, tops);
}

// Many tokens whose y is normed, without a gate by token, into types that need nothing
// else of the whole row: a block keeps its columns' factors in registers and goes from row to row. The sums of the next row are under way
// (its warps arrive on a barrier per row, of four in turn: a warp that writes a row's
// sums has seen all warps' next but two, so they have read the ones four rows before)
// while this one is finished, and the one after it is being read.
template <int OUT>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_rows_kernel(const NormParams p) {
  constexpr int kWarps = kMaxThreads / 32;
  __shared__ float sums[4][4 * kWarps], sum_y[kWarps], sum_r[kWarps];
  __shared__ uint64_t summed[4];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&summed[i], blockDim.x >> 5);
    fence_barrier_init();
    abort_flag = 0;
  }
  __syncthreads();
  griddep_wait();
  const bool in = tid < p.units;
  const int unit = in ? tid : 0;
  float2 norm[8], factor[8];
  read16<true>(p.norm_w, unit, p.cols, norm);
  read16<true>(p.post_w, unit, p.cols, factor);
  if (p.gate_col) {
    float2 w[8];
    read16<true>(p.gate_col, unit, p.cols, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) factor[i] = __fmul2_rn(factor[i], w[i]);
  }
  // (zeros past the row times infinity would be none)
#pragma unroll
  for (int i = 0; i < 8; ++i) factor[i] = in ? factor[i] : make_float2(0.0f, 0.0f);
  const int64_t step = gridDim.x;
  uint32_t y[8], x_new[1][8], x[1][8];
  float2 v[1][8];
  auto load = [&](int64_t row) {
    read16<true>(p.y + row * p.y_stride, tid, p.cols, in && row < p.rows, y);
    read16<true>(p.x + row * p.x_stride, tid, p.cols, in && row < p.rows && p.x, x_new[0]);
    if (tid == 0 && row + step < p.rows) {
      prefetch_l2(p.y + (row + step) * p.y_stride, static_cast<uint32_t>(p.cols) * 2);
      if (p.x) prefetch_l2(p.x + (row + step) * p.x_stride, static_cast<uint32_t>(p.cols) * 2);
    }
  };
  // A row that has been read: v, x, and its warps' sums.
  auto begin = [&](float2 (&to)[1][8], uint32_t (&x_to)[1][8], int turn) {
    float2 yy = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      to[0][i] = pair(y[i]);
      yy = __ffma2_rn(to[0][i], to[0][i], yy);
      to[0][i] = __fmul2_rn(to[0][i], factor[i]);
      x_to[0][i] = x_new[0][i];
    }
    const float sum = warp_sum4(row_sums<1>(yy, to, x_to, true));
    if ((lane & 7) == 0) sums[turn & 3][(tid >> 5) * 4 + (lane >> 3)] = sum;
    __syncwarp();
    if (lane == 0) mbar_arrive(&summed[turn & 3]);
  };
  int64_t row = blockIdx.x;
  load(row);
  begin(v, x, 0);
  load(row + step);
  for (int turn = 0; row < p.rows; row += step, ++turn) {
    float2 v_next[1][8];
    uint32_t x_next[1][8];
    if (row + step < p.rows) {
      begin(v_next, x_next, turn + 1);
      load(row + 2 * step);
    }
    // A warp whose wait gave up ends here: its row's sums are not all there. (The block's barriers
    // count the threads that have not ended; the other warps' waits see the flag.)
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&summed[turn & 3], (turn >> 2) & 1, &abort_flag, p.err, kDevErrTimeoutEpilogue)))
      return;
    float k2;
    const bool known = both_norms<1, true>(p, row, warps_sum4(sums[turn & 3]), x, v, &k2, sum_y);
    write_residual<1, true>(p, row, v);
    if (!known) k2 = rms_factor<1>(v, in, p.inv_n, p.eps, sum_r);
    k2 = apply_early<1>(v, k2);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[0][i] = __fmul2_rn(v[0][i], norm[i]);
    write_h<OUT, 1, true>(p, row, v, k2, nullptr);  // (no OUT that needs the places)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[0][i] = v_next[0][i], x[0][i] = x_next[0][i];
  }
}

template <int OUT, bool WIDE>
const void* kernel_of(int P, bool early) {
  return P == 2  ? reinterpret_cast<const void*>(residual_norm_kernel<OUT, 2, WIDE, false>)
         : early ? reinterpret_cast<const void*>(residual_norm_kernel<OUT, 1, WIDE, true>)
                 : reinterpret_cast<const void*>(residual_norm_kernel<OUT, 1, WIDE, false>);
}

const void* rows_kernel(int out) {
  return out == kOutBf16   ? reinterpret_cast<const void*>(residual_norm_rows_kernel<kOutBf16>)
         : out == kOutE4m3 ? reinterpret_cast<const void*>(residual_norm_rows_kernel<kOutE4m3>)
                           : reinterpret_cast<const void*>(residual_norm_rows_kernel<kOutFp4UE8M0>);
}

template <int OUT>
const void* kernel_for(int P, bool wide, bool early) {
  return wide ? kernel_of<OUT, true>(P, early) : kernel_of<OUT, false>(P, early);
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
  p.ahead = d->sm_count;
  p.rows = T;
  p.err = d->err_word;
  p.units = static_cast<int>((D + 15) / 16);
  p.ue8m0 = fp8 && scale_fmt_ue8m0(scale_fmt);
  const auto wide_rows = [](const void* t, int64_t stride) { return !t || (is_aligned(t, 32) && stride % 16 == 0); };
  const bool wide = D % 16 == 0 && wide_rows(y_bf16, y_stride) && wide_rows(x_bf16, x_stride) &&
                    wide_rows(gate_tok_bf16, gate_stride) && wide_rows(r_bf16, D) && wide_rows(h, D) &&
                    is_aligned(norm_w, 32) && is_aligned(post_w, 32) && is_aligned(gate_col, 32);
  const int P = p.units > kMaxThreads ? 2 : 1;
  const bool early = T <= 2 * d->sm_count;
  const int threads = ((p.units + P - 1) / P + 31) / 32 * 32;
  // Blocks that go from row to row: where y is normed, the factors are the columns' alone,
  // nothing but the norms needs the whole row, and blocks of 128 registers to a thread
  // leave an SM twelve warps (with a gate by column, us: 4099 x 7168 into e4m3 42.1, a block
  // to a token 46.3; into bf16 38.0 and 46.4; into e2m1 with powers of two 44.4 and 46.4;
  // 4099 x 8192 into e4m3 42.1 and 51.9; 500 x 7168 8.2 and 8.5; 16000 x 1536 35.2 and 34.6;
  // with ten warps, 8000 x 5120 into e4m3, 69.0 and 58.7). E2m1 with row scales needs the
  // row's maximum besides (built so, 55.0 against 48.5).
  const int64_t places = kMaxThreads / threads;
  const bool rows = !early && post_w && !gate_tok_bf16 && wide && P == 1 && !(fp4 && scale_fmt == kFp4E4M3) &&
                    places * threads >= 384;
  const void* kernel = rows                    ? rows_kernel(fp8 ? kOutE4m3 : fp4 ? kOutFp4UE8M0 : kOutBf16)
                       : !fp8 && !fp4          ? kernel_for<kOutBf16>(P, wide, early)
                       : fp8                   ? kernel_for<kOutE4m3>(P, wide, early)
                       : scale_fmt == kFp4E4M3 ? kernel_for<kOutFp4E4M3>(P, wide, early)
                                               : kernel_for<kOutFp4UE8M0>(P, wide, early);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows && T > places * d->sm_count ? places * d->sm_count : T));
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
