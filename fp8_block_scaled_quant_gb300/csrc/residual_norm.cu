// The seam between two blocks of a transformer layer: the block's output is
// normed (optionally), gated, added to the scaled residual, and the sum normed
// for the next block, whose product reads it in bf16, e4m3 or e2m1.
//
//   z = post_w ? y * rsqrt(mean(y^2) + eps) * post_w : y
//   r = residual_scale * x + gate * z          -> bf16
//   h = r * rsqrt(mean(r^2) + eps) * norm_w    -> bf16, or act_quant, or fp4_quant
//
// fp32 from the inputs to the one rounding of each output (the norm reads r
// before it is rounded). One block of threads to a token, 8 columns to a thread
// and vector, so that a warp reads and writes whole lines; the row stays in
// registers from the first read to the last write. A few tokens have a block
// each, which reads its row from memory; launch and the block-wide sums bound
// them. More tokens than SMs go round over one block per SM: groups of its
// threads have a token each, whose rows come into shared memory by bulk copies
// while the group works on the one before; the columns' factors lie there too
// (read from L2 for each token they would be as many bytes as the token's rows).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

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
constexpr int kGroupThreads = 1024;       // of a block of groups
constexpr int kMaxGroups = kGroupThreads / 32;
constexpr int kSharedBytes = 224 * 1024;  // factors and slots of a block of groups

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
  int64_t rows, y_stride, x_stride, gate_stride, ktiles;
  float residual_scale, eps, inv_n;
  unsigned* err;
  int vecs;  // columns / 8
  int group, slots;  // blocks of groups: a group's threads and slots
  int ue8m0;
};

// Columns are worked on in pairs (packed fp32 multiplies and FMAs: half the instructions).
__device__ __forceinline__ void unpack8(const uint4& a, float2* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(v[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load8(const float* row, int vec, float2* v) {
  const float4* src = reinterpret_cast<const float4*>(row) + 2 * vec;
  const float4 a = __ldg(src), b = __ldg(src + 1);
  v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
}

// The threads that have a token: a block, or a group of a block's warps.
struct Group {
  int id, tid, n;  // which group, the thread in it, its threads

  __device__ __forceinline__ void sync() const {
    if (n == 32) __syncwarp();
    else named_barrier_sync(1 + id, n);
  }
  // Lanes, then warps in order: the same result in every thread. `at`: where the
  // warps' values meet, not used by the sum before.
  template <typename T, typename F>
  __device__ __forceinline__ T reduce(T v, T none, float* at, F f) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (n == 32) return v;
    T* w = reinterpret_cast<T*>(at);
    if ((tid & 31) == 0) w[tid >> 5] = v;
    sync();
    v = (tid & 31) < (n >> 5) ? w[tid & 31] : none;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
  __device__ __forceinline__ float sum(float v, float* at) const {
    return reduce(v, 0.0f, at, [](float a, float b) { return a + b; });
  }
};

// 1 / sqrt(a): the hardware's estimate and one Newton step, y (1 + (1 - a y^2) / 2).
__device__ __forceinline__ float root_inverse(float a) {
  const float y = rsqrtf(a), e = fmaf(-a * y, y, 1.0f);
  return fabsf(e) < 1.0f ? fmaf(0.5f * y, e, y) : y;  // (a = 0, infinity, NaN: as the estimate is)
}

// 1 / sqrt(mean of v^2 + eps) over the group's row. Squares that overflow fp32 (a
// row near 2^60), or that vanish where eps does not hide it, are summed again
// with v times a power of two; the sum is the same in all threads, so they turn
// together. each(f) calls f on the thread's pairs.
template <typename Each>
__device__ __forceinline__ float rms_factor(const Group& g, float inv_n, float eps, float* at, Each each) {
  float2 two = make_float2(0.0f, 0.0f);
  each([&](float2 v) { two = __ffma2_rn(v, v, two); });
  float sum = g.sum(two.x + two.y, at);
  const bool huge = sum == __uint_as_float(0x7F800000u);
  if (huge || (sum < 7.9e-31f && eps < 8.7e-19f)) {  // 2^-100, 2^-60
    const float s = __uint_as_float(huge ? (127u - 80u) << 23 : (127u + 60u) << 23);
    sum = 0.0f;
    each([&](float2 v) { sum = fmaf(v.x * s, v.x * s, fmaf(v.y * s, v.y * s, sum)); });
    g.sync();  // every warp has read the first sums
    return root_inverse(fmaf(g.sum(sum, at), inv_n, eps * s * s)) * s;
  }
  return root_inverse(fmaf(sum, inv_n, eps));
}

// The act_quant scale of a block (block_scale's value: max(amax, 1e-4) / 448 by
// Markstein's correction, exact), and its reciprocal to half a step or a little more.
// h has passed several fp32 roundings, so the product with the reciprocal takes
// the place of act_quant's exact quotient.
__device__ __forceinline__ float e4m3_scale(float amax, bool ue8m0) {
  float s = div_by_scale(fmaxf(amax, 1e-4f), 448.0f, 1.0f / 448.0f);
  if (ue8m0) {
    uint32_t b = __float_as_uint(s);
    if (b & 0x007FFFFFu) b = (b & 0x7F800000u) + 0x00800000u;
    s = __uint_as_float(b);
  }
  return s;
}

__device__ __forceinline__ float scale_inverse(float s) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.0f), r, r);
}

__device__ __forceinline__ uint4 load_vec(const __nv_bfloat16* row, int vec, bool in) {
  return in ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : make_uint4(0, 0, 0, 0);
}

// The factors of vector `vec`'s columns in z.
__device__ __forceinline__ void z_factors(const NormParams& p, int vec, float2* c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = make_float2(1.0f, 1.0f);
  if (p.post_w) load8(p.post_w, vec, c);
  if (p.gate_col) {
    float2 w[4];
    load8(p.gate_col, vec, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __fmul2_rn(c[i], w[i]);
  }
}

// h of a vector (in all lanes of a warp; those with vec >= p.vecs have zeros and store nothing), written as OUT says.
template <int OUT>
__device__ __forceinline__ void store_h(const NormParams& p, int64_t row, int vec, const float2* h, const RowScale& rs) {
  if constexpr (OUT == kOutBf16) {
    if (vec < p.vecs) reinterpret_cast<uint4*>(p.h)[row * p.vecs + vec] = pack8(h);
  } else if constexpr (OUT == kOutE4m3) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(h[i].x), fabsf(h[i].y)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));  // 16 lanes: 128 columns
    if (vec >= p.vecs) return;
    const float s = e4m3_scale(m, p.ue8m0 != 0), ri = scale_inverse(s);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = __fmul2_rn(h[i], make_float2(ri, ri));
      q[i] = e4m3x2(d.x, d.y);
    }
    reinterpret_cast<uint2*>(p.h)[row * p.vecs + vec] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    if ((threadIdx.x & 15) == 0) static_cast<float*>(p.h_s)[row * (p.vecs / 16) + vec / 16] = s;
  } else {
    fp4_store8<OUT == kOutFp4E4M3 ? kFp4E4M3 : kFp4UE8M0>(&h[0].x, amax8(&h[0].x), rs, row, vec, p.vecs,
                                                          static_cast<uint32_t*>(p.h), static_cast<uint8_t*>(p.h_s),
                                                          p.ktiles);
  }
}

// The scale of the row whose largest |h| in this thread is `top`.
__device__ __forceinline__ RowScale row_scale(const NormParams& p, const Group& g, int64_t row, uint32_t top, float* at) {
  const RowScale rs = fp4_row_scale(g.reduce(top, 0u, at, [](uint32_t a, uint32_t b) { return max(a, b); }));
  if (g.tid == 0) p.h_g[row] = rs.g;
  return rs;
}

// A block to a token, V vectors to a thread.
template <int OUT, int V>
__global__ void __launch_bounds__(kMaxThreads, 1) residual_norm_kernel(const NormParams p) {
  __shared__ float part[3][32];
  griddep_launch_dependents();
  griddep_wait();
  const Group g{0, static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x)};
  const int64_t row = blockIdx.x;
  const bool has_x = p.x != nullptr, tok = p.gate_tok != nullptr;
  uint4 y[V], x[V], gate[V];
  float2 v[V][4], c[V][4], nw[V][4];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int vec = g.tid + u * g.n;
    const bool in = vec < p.vecs;
    y[u] = load_vec(p.y + row * p.y_stride, vec, in);
    x[u] = load_vec(p.x + row * p.x_stride, vec, in && has_x);
    gate[u] = load_vec(p.gate_tok + row * p.gate_stride, vec, in && tok);
    z_factors(p, in ? vec : 0, c[u]);
    load8(p.norm_w, in ? vec : 0, nw[u]);
  }
#pragma unroll
  for (int u = 0; u < V; ++u) unpack8(y[u], v[u]);
  auto each = [&](auto f) {
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) f(v[u][i]);
  };
  // r = residual_scale x + v c, with c the factors of the column
  const float k1 = p.post_w ? rms_factor(g, p.inv_n, p.eps, part[0], each) : 1.0f;
  const float2 k1k1 = make_float2(k1, k1), scale2 = make_float2(p.residual_scale, p.residual_scale);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int vec = g.tid + u * g.n;
    if (vec >= p.vecs) continue;  // v is zeros
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[u][i] = __fmul2_rn(k1k1, c[u][i]);
    if (tok) {
      unpack8(gate[u], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[u][i] = __fmul2_rn(c[u][i], w[i]);
    }
    unpack8(x[u], w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[u][i] = __ffma2_rn(v[u][i], c[u][i], __fmul2_rn(w[i], scale2));
    if (p.r) reinterpret_cast<uint4*>(p.r)[row * p.vecs + vec] = pack8(v[u]);
  }
  const float k2 = rms_factor(g, p.inv_n, p.eps, part[1], each);
  const float2 k2k2 = make_float2(k2, k2);
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < V; ++u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[u][i] = __fmul2_rn(v[u][i], __fmul2_rn(k2k2, nw[u][i]));
    if constexpr (OUT == kOutFp4E4M3) top = max(top, amax8(&v[u][0].x));
  }
  RowScale rs{};
  if constexpr (OUT == kOutFp4E4M3) rs = row_scale(p, g, row, top, part[2]);
#pragma unroll
  for (int u = 0; u < V; ++u)
    if ((g.tid & ~31) + u * g.n < p.vecs) store_h<OUT>(p, row, g.tid + u * g.n, v[u], rs);
}

// A block to an SM, in groups of p.group threads with a token each at a time and
// p.slots slots of shared memory. A slot has the rows of y, x and the token's gate;
// r takes the place of y and x in fp32. Registers hold one vector, not the row:
// what a row of four vectors to a thread spilled went through the little L1 that
// the slots leave, and cost more than reading it from shared memory.
// Shared memory: [factors of z][norm_w] (each the first, then the second halves of
// the vectors' 8 numbers, so that a warp reads whole lines), [group][slot][row][vector].
template <int OUT>
__global__ void __launch_bounds__(kGroupThreads, 1) residual_norm_groups_kernel(const NormParams p) {
  __shared__ float parts[2][3][32];
  __shared__ uint64_t full[2 * kMaxGroups];
  extern __shared__ uint4 shared[];
  Group g;
  g.n = p.group;
  g.id = threadIdx.x / p.group;
  g.tid = threadIdx.x - g.id * g.n;
  float* part = &parts[0][0][0] + g.id * (g.n >> 5);
  const int64_t first = blockIdx.x + static_cast<int64_t>(g.id) * gridDim.x;
  const int64_t step = static_cast<int64_t>(blockDim.x / p.group) * gridDim.x;
  const bool has_x = p.x != nullptr, tok = p.gate_tok != nullptr;
  const int slot_vecs = p.vecs * (tok ? 3 : 2);
  float4* factors = reinterpret_cast<float4*>(shared);
  uint4* slots = shared + 4 * p.vecs + g.id * p.slots * slot_vecs;
  uint64_t* filled = full + g.id * p.slots;
  if (g.tid < p.slots) {
    mbar_init(&filled[g.tid], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t row_bytes = static_cast<uint32_t>(p.vecs) * 16;
  auto request = [&](int64_t row, int slot) {
    uint4* at = slots + slot * slot_vecs;
    mbar_arrive_expect_tx(&filled[slot], row_bytes * (1 + has_x + tok));
    bulk_load(at, p.y + row * p.y_stride, row_bytes, &filled[slot]);
    if (has_x) bulk_load(at + p.vecs, p.x + row * p.x_stride, row_bytes, &filled[slot]);
    if (tok) bulk_load(at + 2 * p.vecs, p.gate_tok + row * p.gate_stride, row_bytes, &filled[slot]);
  };
  __syncwarp();  // the group's first warp has made its barriers
  if (g.tid == 0)
    for (int s = 0; s < p.slots; ++s)
      if (first + s * step < p.rows) request(first + s * step, s);
  for (int vec = threadIdx.x; vec < p.vecs; vec += blockDim.x) {
    float2 c[4];
    z_factors(p, vec, c);
    factors[vec] = make_float4(c[0].x, c[0].y, c[1].x, c[1].y);
    factors[p.vecs + vec] = make_float4(c[2].x, c[2].y, c[3].x, c[3].y);
    load8(p.norm_w, vec, c);
    factors[2 * p.vecs + vec] = make_float4(c[0].x, c[0].y, c[1].x, c[1].y);
    factors[3 * p.vecs + vec] = make_float4(c[2].x, c[2].y, c[3].x, c[3].y);
  }
  __syncthreads();
  // 8 fp32 numbers of a vector kept as two halves.
  auto get8 = [&](const float4* halves, int vec, float2* c) {
    const float4 a = halves[vec], b = halves[p.vecs + vec];
    c[0] = make_float2(a.x, a.y), c[1] = make_float2(a.z, a.w);
    c[2] = make_float2(b.x, b.y), c[3] = make_float2(b.z, b.w);
  };
  auto put8 = [&](float4* halves, int vec, const float2* c) {
    halves[vec] = make_float4(c[0].x, c[0].y, c[1].x, c[1].y);
    halves[p.vecs + vec] = make_float4(c[2].x, c[2].y, c[3].x, c[3].y);
  };
  const float2 scale2 = make_float2(p.residual_scale, p.residual_scale);
  int turn = 0, slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t row = first; row < p.rows; row += step, turn ^= 96) {
    uint4* at = slots + slot * slot_vecs;
    float4* rf = reinterpret_cast<float4*>(at);
    // A wait that gave up (the error bit says so: the outputs are not valid) is the last one.
    if (ok) ok = mbar_wait(&filled[slot], phase, nullptr, p.err, kDevErrTimeoutProducer);
    float k1 = 1.0f;
    if (p.post_w)
      k1 = rms_factor(g, p.inv_n, p.eps, part + turn, [&](auto f) {
#pragma unroll 4
        for (int vec = g.tid; vec < p.vecs; vec += g.n) {
          float2 v[4];
          unpack8(at[vec], v);
#pragma unroll
          for (int i = 0; i < 4; ++i) f(v[i]);
        }
      });
    // r = residual_scale x + y c, with c the factors of the column
    const float2 k1k1 = make_float2(k1, k1);
    uint4* r_row = reinterpret_cast<uint4*>(p.r) + row * p.vecs;
#pragma unroll 2
    for (int vec = g.tid; vec < p.vecs; vec += g.n) {
      float2 v[4], c[4], w[4];
      unpack8(at[vec], v);
      get8(factors, vec, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __fmul2_rn(k1k1, c[i]);
      if (tok) {
        unpack8(at[2 * p.vecs + vec], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __fmul2_rn(c[i], w[i]);
      }
      if (has_x) {
        unpack8(at[p.vecs + vec], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ffma2_rn(v[i], c[i], __fmul2_rn(w[i], scale2));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(v[i], c[i]);
      }
      if (p.r) r_row[vec] = pack8(v);
      put8(rf, vec, v);
    }
    const float k2 = rms_factor(g, p.inv_n, p.eps, part + turn + 32, [&](auto f) {
#pragma unroll 4
      for (int vec = g.tid; vec < p.vecs; vec += g.n) {
        float2 v[4];
        get8(rf, vec, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f(v[i]);
      }
    });
    const float2 k2k2 = make_float2(k2, k2);
    auto h_of = [&](int vec, float2* v) {
      float2 w[4];
      get8(rf, vec, v);
      get8(factors + 2 * p.vecs, vec, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(v[i], __fmul2_rn(k2k2, w[i]));
    };
    RowScale rs{};
    if constexpr (OUT == kOutFp4E4M3) {
      uint32_t top = 0;
#pragma unroll 2
      for (int vec = g.tid; vec < p.vecs; vec += g.n) {
        float2 v[4];
        h_of(vec, v);
        top = max(top, amax8(&v[0].x));
      }
      rs = row_scale(p, g, row, top, part + turn + 64);
    }
#pragma unroll 2
    for (int vec = g.tid; (vec & ~31) < p.vecs; vec += g.n) {
      float2 v[4] = {};
      if (vec < p.vecs) h_of(vec, v);
      store_h<OUT>(p, row, vec, v, rs);
    }
    // The slot is the copies' again: after what all of the group did with it.
    fence_proxy_async_smem();
    g.sync();
    const int64_t later = row + p.slots * step;
    if (g.tid == 0 && ok && later < p.rows) request(later, slot);
    if (++slot == p.slots) slot = 0, phase ^= 1;
  }
  if (!ok && g.tid == 0) {  // the copies in flight land before the block ends
    for (int s = 0; s < p.slots; ++s) {
      mbar_wait(&filled[slot], phase, nullptr, p.err, kDevErrTimeoutDrain);
      if (++slot == p.slots) slot = 0, phase ^= 1;
    }
  }
}

template <int OUT>
const void* kernel_for(int v, bool groups) {
  return groups   ? reinterpret_cast<const void*>(residual_norm_groups_kernel<OUT>)
         : v == 1 ? reinterpret_cast<const void*>(residual_norm_kernel<OUT, 1>)
         : v == 2 ? reinterpret_cast<const void*>(residual_norm_kernel<OUT, 2>)
                  : reinterpret_cast<const void*>(residual_norm_kernel<OUT, 4>);
}

// Lets a kernel of groups have its shared memory: once per device and kind of output.
int allow_shared(const void* kernel, int device, int which) {
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices][4];
  static cudaError_t set[kMaxDevices][4];
  std::call_once(once[device][which], [&] {
    set[device][which] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
  });
  return cuda_status(set[device][which]);
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
  p.rows = T;
  p.err = d->err_word;
  p.vecs = static_cast<int>(D / 8);
  p.ue8m0 = fp8 && scale_fmt_ue8m0(scale_fmt);
  // Up to a token per SM: as many threads as there are vectors, up to 512. More:
  // four vectors to a thread (fewer in narrow rows), which then share the cost of
  // the sums; as many groups as their threads and slots leave room for.
  const bool groups = T > d->sm_count;
  const int V = groups ? 4 : p.vecs <= kMaxThreads ? 1 : p.vecs <= 2 * kMaxThreads ? 2 : 4;
  int threads = ((p.vecs + V - 1) / V + 31) / 32 * 32, shared = 0;
  int64_t blocks = T;
  if (groups) {
    const int factors = p.vecs * 64, slot = p.vecs * 16 * (gate_tok_bf16 ? 3 : 2);
    p.group = threads;
    p.slots = factors + 2 * slot <= kSharedBytes ? 2 : 1;
    int count = (kSharedBytes - factors) / (p.slots * slot);
    if (count > kGroupThreads / threads) count = kGroupThreads / threads;
    if (threads > 32 && count > 15) count = 15;  // a named barrier each
    const int64_t need = (T + d->sm_count - 1) / d->sm_count;
    if (count > need) count = static_cast<int>(need);
    threads *= count;
    shared = factors + count * p.slots * slot;
    blocks = d->sm_count;
  }
  const int out = !fp8 && !fp4 ? kOutBf16 : fp8 ? kOutE4m3 : scale_fmt == kFp4E4M3 ? kOutFp4E4M3 : kOutFp4UE8M0;
  const void* kernel = out == kOutBf16      ? kernel_for<kOutBf16>(V, groups)
                       : out == kOutE4m3    ? kernel_for<kOutE4m3>(V, groups)
                       : out == kOutFp4E4M3 ? kernel_for<kOutFp4E4M3>(V, groups)
                                            : kernel_for<kOutFp4UE8M0>(V, groups);
  if (groups) {
    if (int st = allow_shared(kernel, d->device, out)) return st;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {&p};
  return cuda_status(cudaLaunchKernelExC(&cfg, kernel, args));
}
