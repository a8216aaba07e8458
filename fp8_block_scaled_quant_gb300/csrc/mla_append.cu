// The latent cache append of a decode or prefill step ("Administrator &
// Developer Guide", 8.3: the MLA layer caches the normalised latent and the
// rotated key part; 1.2: RMSNorm and rotary embedding). Per token t, with
// position p = positions[t] and angle cosines / sines (c_i, s_i) of p:
//
//   latent  n = kv[t, 0:512] * rsqrt(mean(kv[t, 0:512]^2) + eps) * norm_w
//   key     r = rot(kv[t, 512:576])
//   cache[slots[t]] = bf16([n, r])
//   q_nope[t, h] = q[t, h, 0:128]          (a copy: the absorb GEMM's operand)
//   q_pe[t, h]   = bf16(rot(q[t, h, 128:192]))
//   rot: (a, b) = (v[2i], v[2i+1]) -> (a c_i - b s_i, a s_i + b c_i)
//
// A negative slot is a padding token: no cache row. A slot past the cache writes
// none either and sets an error bit; a position outside the table sets it too
// and is taken as 0 (row and queries are written, turned by that angle).
// fp32 with one rounding to bf16. One launch, one pass: every input byte
// is read once and every output byte written once, so HBM bounds long
// prompts and launch latency single tokens (measured: 6151 tokens of 128 heads,
// 621 MB, 104.6 us, 5.9 TB/s; one token 2.1 us, 129 tokens of 16 heads 2.4 us).
//
// Layout: a head's 192 columns are 24 vectors of 16 bytes, so 192 threads take
// eight heads of one token: thread i always has vector i % 24 of a head, and
// whether it copies (vectors 0-15) or rotates (16-23) and which four angles
// it needs do not change over its heads. A seventh warp takes the token's
// latent and key row. A block takes eight heads of a token, or 32 (four passes,
// their loads in flight together) where blocks of eight would be more than
// eight per SM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

constexpr int kC = 512, kR = 64, kRow = kC + kR;  // latent and rotary columns of a cache row
constexpr int kNope = 128, kHead = kNope + kR;    // columns of a query head
constexpr int kHeadVecs = kHead / 8;              // 24 vectors of 16 bytes
constexpr int kGroupHeads = 8;                    // heads per pass of a block
constexpr int kQThreads = kGroupHeads * kHeadVecs;
constexpr int kThreads = kQThreads + 32;
constexpr int kUnroll = 4;                        // passes whose loads are in flight together
constexpr unsigned kDevErrBadSlot = 1u << 8;

struct AppendParams {
  const __nv_bfloat16* kv;
  const __nv_bfloat16* q;
  const float* norm_w;
  const float2* rope;  // [max_pos][32] (cos, sin)
  const int64_t* positions;
  const int64_t* slots;
  __nv_bfloat16* cache;
  __nv_bfloat16* q_nope;
  __nv_bfloat16* q_pe;
  unsigned* err;
  int64_t kv_stride, q_stride, max_pos, num_slots;
  int H, groups_per_block;
  float eps;
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four pairs turned by the angles whose (cos, sin) are cs[0..3].
__device__ __forceinline__ uint4 rotate4(const uint4& v, const float2 (&cs)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2(w[i]);
    r[i] = pack2(__fsub_rn(__fmul_rn(x.x, cs[i].x), __fmul_rn(x.y, cs[i].y)),
                 __fadd_rn(__fmul_rn(x.x, cs[i].y), __fmul_rn(x.y, cs[i].x)));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The (cos, sin) of pairs 4 part .. 4 part + 3 at a position.
__device__ __forceinline__ void load_angles(const AppendParams& p, int64_t pos, int part, float2 (&cs)[4]) {
  const float4* src = reinterpret_cast<const float4*>(p.rope + pos * (kR / 2) + part * 4);
  const float4 a = __ldg(src), b = __ldg(src + 1);
  cs[0] = make_float2(a.x, a.y);
  cs[1] = make_float2(a.z, a.w);
  cs[2] = make_float2(b.x, b.y);
  cs[3] = make_float2(b.z, b.w);
}

__global__ void __launch_bounds__(kThreads) mla_append_kernel(const AppendParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  int64_t pos = p.positions[t];
  if (pos < 0 || pos >= p.max_pos) {
    if (tid == 0 && blockIdx.y == 0) atomicOr(p.err, kDevErrBadSlot);
    pos = 0;
  }
  if (tid < kQThreads) {
    if (!p.q) return;
    const int part = tid % kHeadVecs;
    float2 cs[4];
    if (part >= kNope / 8) load_angles(p, pos, part - kNope / 8, cs);
    const uint4* src = reinterpret_cast<const uint4*>(p.q + t * p.q_stride) + part;
    const int h0 = static_cast<int>(blockIdx.y) * p.groups_per_block * kGroupHeads + tid / kHeadVecs;
    const int h1 = min(p.H, (static_cast<int>(blockIdx.y) + 1) * p.groups_per_block * kGroupHeads);
    for (int h = h0; h < h1; h += kUnroll * kGroupHeads) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u * kGroupHeads < h1) v[u] = __ldcs(src + static_cast<int64_t>(h + u * kGroupHeads) * kHeadVecs);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t hu = h + u * kGroupHeads;
        if (hu >= h1) break;
        if (part < kNope / 8)
          reinterpret_cast<uint4*>(p.q_nope)[(t * p.H + hu) * (kNope / 8) + part] = v[u];
        else
          reinterpret_cast<uint4*>(p.q_pe)[(t * p.H + hu) * (kR / 8) + part - kNope / 8] = rotate4(v[u], cs);
      }
    }
    return;
  }
  if (blockIdx.y != 0) return;
  // The cache row, by one warp: lane l has latent vectors l and l + 32, lanes
  // 0-7 also key vector l.
  const int lane = tid - kQThreads;
  const int64_t slot = p.slots[t];
  if (slot < 0) return;  // a padding token
  if (slot >= p.num_slots) {
    if (lane == 0) atomicOr(p.err, kDevErrBadSlot);
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(p.kv + t * p.kv_stride);
  uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * kRow);
  const uint4 a[2] = {__ldcs(src + lane), __ldcs(src + 32 + lane)};
  if (lane < kR / 8) {
    float2 cs[4];
    load_angles(p, pos, lane, cs);
    dst[kC / 8 + lane] = rotate4(__ldcs(src + kC / 8 + lane), cs);
  }
  float sum = 0.f;
  float2 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4& v = a[i >> 2];
    const uint32_t w = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    x[i] = unpack2(w);
    sum = fmaf(x[i].x, x[i].x, fmaf(x[i].y, x[i].y, sum));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float r = __frsqrt_rn(sum * (1.0f / kC) + p.eps);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float4* wv = reinterpret_cast<const float4*>(p.norm_w) + (half * 32 + lane) * 2;
    const float4 w0 = __ldg(wv), w1 = __ldg(wv + 1);
    const float2* y = x + half * 4;
    dst[half * 32 + lane] =
        make_uint4(pack2(y[0].x * r * w0.x, y[0].y * r * w0.y), pack2(y[1].x * r * w0.z, y[1].y * r * w0.w),
                   pack2(y[2].x * r * w1.x, y[2].y * r * w1.y), pack2(y[3].x * r * w1.z, y[3].y * r * w1.w));
  }
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_mla_append(const void* kv_bf16, int64_t kv_stride, const float* norm_w, float eps,
                                 const void* q_bf16, int64_t q_stride, int64_t H, const float* rope, int64_t max_pos,
                                 const int64_t* positions, const int64_t* slots, int64_t T, void* cache_bf16,
                                 int64_t num_slots, void* q_nope_bf16, void* q_pe_bf16, fp8blk_stream_t stream) {
  const bool has_q = q_bf16 != nullptr;
  if (T < 0 || T > (int64_t{1} << 31) - 1 || max_pos < 1 || num_slots < 0 || kv_stride < kRow)
    return FP8BLK_ERR_SHAPE;
  if (has_q && (H < 1 || H > 1024 || q_stride < H * kHead)) return FP8BLK_ERR_SHAPE;
  if (!(eps >= 0.0f)) return FP8BLK_ERR_ARG;
  if (T == 0) return FP8BLK_OK;
  if (!kv_bf16 || !norm_w || !rope || !positions || !slots || (!cache_bf16 && num_slots > 0)) return FP8BLK_ERR_NULL;
  if (has_q && (!q_nope_bf16 || !q_pe_bf16)) return FP8BLK_ERR_NULL;
  if (!is_aligned(kv_bf16, 16) || kv_stride % 8 || !is_aligned(norm_w, 16) || !is_aligned(rope, 16) ||
      !is_aligned(positions, 8) || !is_aligned(slots, 8) || !is_aligned(cache_bf16, 16))
    return FP8BLK_ERR_ALIGN;
  if (has_q && (!is_aligned(q_bf16, 16) || q_stride % 8 || !is_aligned(q_nope_bf16, 16) || !is_aligned(q_pe_bf16, 16)))
    return FP8BLK_ERR_ALIGN;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  AppendParams p{};
  p.kv = static_cast<const __nv_bfloat16*>(kv_bf16);
  p.q = static_cast<const __nv_bfloat16*>(q_bf16);
  p.norm_w = norm_w;
  p.rope = reinterpret_cast<const float2*>(rope);
  p.positions = positions;
  p.slots = slots;
  p.cache = static_cast<__nv_bfloat16*>(cache_bf16);
  p.q_nope = static_cast<__nv_bfloat16*>(q_nope_bf16);
  p.q_pe = static_cast<__nv_bfloat16*>(q_pe_bf16);
  p.err = d->err_word;
  p.kv_stride = kv_stride;
  p.q_stride = q_stride;
  p.max_pos = max_pos;
  p.num_slots = num_slots;
  p.H = static_cast<int>(H);
  p.eps = eps;
  const int groups = has_q ? static_cast<int>((H + kGroupHeads - 1) / kGroupHeads) : 1;
  // Blocks of eight heads up to eight per SM, more heads to a block beyond: 128 heads
  // of 38 tokens 2.16 us in blocks of 8 and 2.0 in blocks of 32, of 76 tokens (at the
  // border) 2.76 and 2.80, of 152 4.6 and 3.0, of 2432 74.5 and 41.5; 16 heads of 304
  // tokens (half the border) 2.28 and 2.48.
  p.groups_per_block = T * groups <= 8 * d->sm_count ? 1 : kUnroll;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T),
                     static_cast<unsigned>((groups + p.groups_per_block - 1) / p.groups_per_block));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, mla_append_kernel, p));
}
