// Product of two matrices of microscaled 4-bit floats (fp4.cuh has the formats):
//
//   C[m, n] = bf16( ag[m] wg[n] sum over blocks b of sa[m, b] sw[n, b] sum_{k in b} a[m, k] w[n, k] )
//
// The block-scaled MMA applies sa and sw itself (products of e2m1 numbers and
// their scales, summed in fp32 in tensor memory), the epilogue the row scales.
//
// Two kernels. Few tokens: 128 weight rows are the MMA's M (tensor-memory lanes), 16,
// 32 or 64 tokens its columns; memory and latency bound it. Many tokens: tiles of CTA
// pairs, at the tensor cores' rate (below). In both, 256 of K make a stage: codes by
// TMA (128-byte rows, 128-byte swizzle), scale tiles in the order of their use, from
// shared into tensor memory by tcgen05.cp in the order of the MMAs.
//
// Every wait is bounded; a wait that gives up sets an error bit, and the CTA
// waits (bounded) for its own copies and MMAs, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "fp4.cuh"
#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {

bool fp4_fmt_valid(int fmt);
int fp4_quant_launch(const void* x, bool fp32, int64_t x_stride, int64_t M, int64_t K, int fmt, void* q, void* s, float* g,
                     int sm_count, bool early, cudaStream_t stream);

namespace {

// A sum is multiplied by its two row scales one after the other: their own product may
// leave fp32's range where the result does not (rows of small numbers: 0; rows of large
// ones and a sum of 0: NaN). Of the lane's scale, `first` is multiplied before the other
// scale and `last` after it, and one of them is 1: a scale below 1 goes first, where a sum
// (2^-20 at least) keeps 18 bits with the smallest of fp4_quant's scales, 2^-112; one
// above 1 goes last, when the product is as large only as the result. A NaN stays.
struct LaneScale {
  float first = 1.0f, last = 1.0f;
  __device__ __forceinline__ LaneScale() {}
  __device__ __forceinline__ explicit LaneScale(float g)
      : first(fabsf(g) <= 1.0f ? g : 1.0f), last(fabsf(g) <= 1.0f ? 1.0f : g) {}
};

constexpr int kStageK = 256;
constexpr int kLaneBytes = 128 * 128;  // 128 weight rows of a stage

struct Fp4Params {
  const uint8_t* w_s;
  const uint8_t* a_s;
  const float* w_g;
  const float* a_g;
  __nv_bfloat16* c;
  unsigned* err;
  const __nv_bfloat16* x;  // few tokens: the activations themselves, quantised by every CTA
  int64_t x_stride;
  int64_t M, N, ktiles;    // ktiles: scale tiles along K
  int ksteps;              // K / 64
  int stages_k;            // ceil(K / 256)
  int tiles_n, tiles_m;    // weight tiles; token tiles (pairs)
  int ksplit;              // few tokens: CTAs of a tile's cluster
  int stages;              // few tokens: slots of the ring
  int part_cols, part_vec; // few tokens: columns that a CTA of the cluster sums, and that it is sent at once
};

// ---- few tokens ------------------------------------------------------------------------
//
//   warp 0      weights: requested before the dependency wait as far as the ring goes
//   warp 1      MMA issuer: the weights' scales of those stages go to tensor memory
//               before the tokens are there; then a stage is four copies and four MMAs,
//               0.28 us (an MMA of 16 columns takes about 95 cycles, a copy 40)
//   warps 2-5   epilogue, a lane quarter each
//   warp 6      tokens, as codes; FUSE: none, warps 2-5 quantise the activations into
//               shared memory (one launch, and 1.5 us less than a kernel of its own)
//
// Few weight tiles are split over K by clusters of up to 8 CTAs. A CTA sends each
// column of its partial sums to the one that sums it (st.async on its mbarrier, no
// barrier of the cluster on the way; up to four columns at once, a store takes 0.06 us
// of a warp), which adds them in rank order.

constexpr int kFewThreads = 224;
constexpr int kMaxStages = 12;
constexpr int kFuseUnits = 4;  // units of 16 numbers that a quantising thread holds

template <int BN_, int FMT_, bool FUSE_>
struct Cfg {
  static constexpr int BN = BN_, FMT = FMT_;
  static constexpr bool FUSE = FUSE_;
  static constexpr int kTiles = FMT == kFp4E4M3 ? 4 : 2;  // scale tiles of a stage
  static constexpr int kSfBytes = kTiles * kScaleTile;
  static constexpr int kColAt = kLaneBytes + kSfBytes;    // the tokens' part of a stage
  static constexpr int kStageBytes = (kColAt + (FUSE ? 0 : BN * 128 + kSfBytes) + 1023) / 1024 * 1024;
  static constexpr int kColCodesAt = (kColAt + 1023) / 1024 * 1024;  // (a swizzled tile starts at 1024 bytes)
  static constexpr int kAccCols = BN < 32 ? 32 : BN;
  static constexpr int kSfCols = kTiles * 4;              // one operand's scales of a stage
  // FUSE: all of the CTA's tokens: codes, then scale tiles of 16 rows (256 bytes; a copy reads on into the next).
  static constexpr int kFuseCodes = BN * 128, kFuseScales = kTiles * 256;
  static constexpr int kBarBytes = (3 * kMaxStages + 3) * 8 + 16 + 64;
};

// Stage slots that half of tensor memory has room for.
constexpr int kFewTmemCols = 256;
template <class C>
constexpr int kMostStages = (kFewTmemCols - C::kAccCols) / C::kSfCols - 2 < kMaxStages
                                ? (kFewTmemCols - C::kAccCols) / C::kSfCols - 2
                                : kMaxStages;

__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

// mbar_wait for a barrier that other CTAs arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err,
                                                  unsigned code) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_wait_cluster(a, parity) ||
         (mbar_wait(bar, parity, abort, err, code) && mbar_try_wait_cluster(a, parity));
}

// V numbers (1, 2 or 4) into a CTA of the cluster; they complete on its barrier.
template <int V>
__device__ __forceinline__ void st_async(uint32_t addr, const uint32_t* v, uint32_t bar) {
  if constexpr (V == 4)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
                 : "memory");
  else if constexpr (V == 2)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
                 "r"(v[0]), "r"(v[1]), "r"(bar)
                 : "memory");
  else
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v[0]),
                 "r"(bar)
                 : "memory");
}

// The columns' sums of this lane's weight row, r[0..N), to their shares' CTAs. A
// share is `share` columns, a multiple of V; its part of this CTA: [share / V][128][V].
template <int V, int N>
__device__ __forceinline__ void send_columns(const uint32_t* r, int c0, int share, int ks, const float* part,
                                             const uint64_t* bar) {
#pragma unroll
  for (int i = 0; i < N; i += V) {
    const int c = c0 + i, to = c / share;
    if (to < ks)
      st_async<V>(map_to_rank(smem_u32(part + (c - to * share) * 128), static_cast<uint32_t>(to)), r + i,
                  map_to_rank(smem_u32(bar), static_cast<uint32_t>(to)));
  }
}

// The sums of a share's columns, parts [rank][share / V][128][V] in rank order, to
// put(column, sum).
template <int V, typename Put>
__device__ __forceinline__ void sum_columns(const float* parts, int ks, int share, int lane, const Put& put) {
  struct alignas(4 * V) Part {
    float v[V];
  };
  const Part* at = reinterpret_cast<const Part*>(parts) + lane;
  for (int g = 0; g < share; g += V, at += 128) {
    float sum[V] = {};
#pragma unroll 4
    for (int k = 0; k < ks; ++k) {
      const Part part = at[k * (share / V) * 128];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += part.v[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) put(g + i, sum[i]);
  }
}

template <class C>
__global__ void __launch_bounds__(kFewThreads, 2)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                    const Fp4Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const int ks = p.ksplit, rank = static_cast<int>(blockIdx.x) % ks;
  const int tile = static_cast<int>(blockIdx.x) / ks;
  const int tile_n = tile % p.tiles_n, tile_m = tile / p.tiles_n;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.stages_k) * rank / ks);
  const int n = static_cast<int>(static_cast<int64_t>(p.stages_k) * (rank + 1) / ks) - k0;  // stages of this CTA
  const int most_n = (p.stages_k + ks - 1) / ks;
  uint8_t* fused = smem + p.stages * C::kStageBytes;  // FUSE: codes, scales
  uint8_t* fused_s = fused + most_n * C::kFuseCodes;
  float* parts = reinterpret_cast<float*>(C::FUSE ? fused_s + most_n * C::kFuseScales + 256 : fused);  // [rank][column][128]
  uint64_t* full_w = reinterpret_cast<uint64_t*>(parts + (ks > 1 ? ks * p.part_cols * 128 : 0));
  uint64_t* full_t = full_w + kMaxStages;
  uint64_t* empty = full_t + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  uint64_t* tokens_ready = done + 1;
  uint64_t* parts_full = tokens_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(parts_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* row_top = tmem_slot + 4;  // FUSE: bits of the rows' largest |x|, [16]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m0 = static_cast<int64_t>(tile_m) * C::BN;
  const int cols = static_cast<int>(p.M - m0 < C::BN ? p.M - m0 : C::BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_w[s], 1);
      mbar_init(&full_t[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(tokens_ready, 4);
    mbar_init(parts_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    if (ks > 1) mbar_arrive_expect_tx(parts_full, static_cast<uint32_t>(ks * p.part_cols * 512));
  }
  if (C::FUSE && threadIdx.x >= 64 && threadIdx.x < 80) row_top[threadIdx.x - 64] = 0;
  if (warp == 6 && lane == 0) {
    tma_prefetch_desc(&map_w);
    if constexpr (!C::FUSE) tma_prefetch_desc(&map_a);
  }
  if (ks > 1) {
    // This CTA's barrier of partial sums is there (waited for before they are sent).
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  // No CTA waits for another of its cluster while it holds tensor memory or waits for
  // it (the arrival above is before the allocation, the release before the wait for the
  // sums): its columns may be another kernel's, whose cluster waits for this SM's.
  if (warp == 1) {
    tmem_alloc(tmem_slot, kFewTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // After the allocation: a CTA of the next kernel that came first to this SM's
  // tensor memory would hold it until this kernel ends.
  griddep_launch_dependents();

  const int ktiles = static_cast<int>(p.ktiles);
  // Bytes of the scale tiles of stage k: of all of them, or those that K has left.
  auto scale_bytes = [&](int k) {
    const int left = ktiles - k * C::kTiles;
    return static_cast<uint32_t>(left < C::kTiles ? left : C::kTiles) * kScaleTile;
  };
  bool finished = true;  // epilogue warps: the accumulator is complete
  const int q = warp & 3;  // lane quarter of an epilogue warp
  const int64_t row = static_cast<int64_t>(tile_n) * 128 + q * 32 + lane;
  LaneScale wg;
  float ag[C::BN < 32 ? 1 : C::BN / 32];
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(ag) / 4); ++i) ag[i] = 1.0f;

  if (warp == 0 || (!C::FUSE && warp == 6)) {
    const bool weights = warp == 0;
    if (!weights) griddep_wait();
    uint64_t* full = weights ? full_w : full_t;
    const uint8_t* scales = weights ? p.w_s + static_cast<int64_t>(tile_n) * ktiles * kScaleTile
                                    : p.a_s + m0 / 128 * ktiles * kScaleTile;
    const CUtensorMap* map = weights ? &map_w : &map_a;
    const int y = weights ? tile_n * 128 : static_cast<int>(m0);
    const uint32_t bytes = weights ? kLaneBytes : C::BN * 128;
    auto ask = [&](int i, int st) {
      uint8_t* at = smem + st * C::kStageBytes;
      const uint32_t sf = scale_bytes(k0 + i);
      mbar_arrive_expect_tx(&full[st], bytes + sf);
      tma_load_2d(weights ? at : at + C::kColCodesAt, map, &full[st], (k0 + i) * 128, y);
      bulk_load(weights ? at + kLaneBytes : at + C::kColCodesAt + C::BN * 128,
                scales + static_cast<int64_t>(k0 + i) * C::kSfBytes, sf, &full[st]);
    };
    // The first stages by a lane each, at once; the others in their turn.
    const int pre = n < p.stages ? n : p.stages;
    if (lane < pre) ask(lane, lane);
    __syncwarp();
    if (lane == 0) {
      int st = 0, i = pre;
      uint32_t phase = 0;
      for (; i < n; ++i) {
        if (!mbar_wait(&empty[st], phase, abort_flag, p.err, kDevErrTimeoutProducer)) break;
        ask(i, st);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
      if (i < n) {  // gave up: the copies in flight land before the CTA ends
        for (int j = i > p.stages ? i - p.stages : 0; j < i; ++j)
          mbar_wait(&full[j % p.stages], (j / p.stages) & 1, nullptr, p.err, kDevErrTimeoutDrain);
      }
    }
  } else if (warp == 1) {
    const bool leader = elect_one_sync();
    const uint32_t sf_w = tmem + C::kAccCols, sf_t = sf_w + static_cast<uint32_t>(p.stages * C::kSfCols);
    const uint32_t sf_first = static_cast<uint32_t>(m0 >> 5) & 3;  // a column holds the scales of 32 tokens
    auto all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.err, kDevErrTimeoutMma));
    };
    auto weight_scales = [&](int st) {
      const uint32_t at = smem_u32(smem + st * C::kStageBytes) + kLaneBytes;
      tc_fence_after_sync();
      if (leader) {
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
          tmem_cp_scales(sf_w + st * C::kSfCols + 4 * t, sdesc_scale_tile(at + t * kScaleTile));
      }
      __syncwarp();
    };
    // Where the tokens of stage i (slot st) are.
    auto token_codes = [&](int i, int st) {
      return C::FUSE ? smem_u32(fused + i * C::kFuseCodes) : smem_u32(smem + st * C::kStageBytes + C::kColCodesAt);
    };
    auto token_scales = [&](int i, int st) {
      const uint32_t at = C::FUSE ? smem_u32(fused_s + i * C::kFuseScales) : token_codes(i, st) + C::BN * 128;
      tc_fence_after_sync();
      if (leader) {
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
          tmem_cp_scales(sf_t + (i & 1) * C::kSfCols + 4 * t, sdesc_scale_tile(at + t * (C::FUSE ? 256 : kScaleTile)));
      }
      __syncwarp();
    };
    const int pre = n < p.stages ? n : p.stages;
    bool ok = true;
    for (int i = 0; ok && i < pre; ++i)
      if ((ok = all(&full_w[i], 0))) weight_scales(i);
    if (C::FUSE && ok) ok = all(tokens_ready, 0);
    int st = 0;
    uint32_t phase = 0;
    for (int i = 0; ok && i < n; ++i) {
      if (i >= pre) {
        if (!(ok = all(&full_w[st], phase))) break;
        weight_scales(st);
      }
      if (!C::FUSE && !(ok = all(&full_t[st], phase))) break;
      token_scales(i, st);
      const uint64_t ad = sdesc_kmajor_sw128(smem_u32(smem + st * C::kStageBytes)), bd = sdesc_kmajor_sw128(token_codes(i, st));
      const uint32_t sfa = sf_w + static_cast<uint32_t>(st * C::kSfCols), sfb = sf_t + static_cast<uint32_t>((i & 1) * C::kSfCols) + sf_first;
      const int left = p.ksteps - (k0 + i) * 4, steps = left < 4 ? left : 4;  // 2 or 4
      if (leader) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= steps) break;
          const int t = C::FMT == kFp4E4M3 ? j : j / 2;
          mma_fp4<C::FMT>(tmem, ad + 2 * j, bd + 2 * j,
                          idesc_fp4(128, C::BN, C::FMT, C::FMT == kFp4E4M3 ? 0 : 2 * (j & 1)), sfa + 4 * t, sfb + 4 * t,
                          i > 0 || j > 0 ? 1u : 0u);
        }
        if (i + p.stages < n) mma_commit(&empty[st]);
        if (i + 1 == n) mma_commit(done);
      }
      __syncwarp();
      if (++st == p.stages) st = 0, phase ^= 1;
    }
    if (!ok) __threadfence_block();  // the abort flag, before the epilogue is let go
    __syncwarp();
    if (leader) {
      if (!ok) mma_commit(done);
      mbar_wait(done, 0, nullptr, p.err, kDevErrTimeoutDrain);
    }
    __syncwarp();
  } else if (warp < 6) {
    griddep_wait();
    if constexpr (C::FUSE) {
      // Units of 16 numbers, row by row over the 128 threads; the row's largest first.
      const int t = threadIdx.x - 64, per_row = p.ksteps * 4, units = cols * per_row;
      const __nv_bfloat16* x = p.x + m0 * p.x_stride;
      uint32_t v[kFuseUnits][8];
#pragma unroll
      for (int u = 0; u < kFuseUnits; ++u) {
        const int i = t + u * 128;
        if (i >= units) break;
        const int m = i / per_row, unit = i - m * per_row;
        const uint4* src = reinterpret_cast<const uint4*>(x + m * p.x_stride + unit * 16);
        const uint4 a = src[0], b = src[1];
        v[u][0] = a.x, v[u][1] = a.y, v[u][2] = a.z, v[u][3] = a.w;
        v[u][4] = b.x, v[u][5] = b.y, v[u][6] = b.z, v[u][7] = b.w;
      }
      uint32_t am[kFuseUnits];
#pragma unroll
      for (int u = 0; u < kFuseUnits; ++u) {
        const int i = t + u * 128;
        if (i >= units) break;
        uint32_t m = v[u][0] & 0x7FFF7FFFu;
#pragma unroll
        for (int j = 1; j < 8; ++j) m = __vmaxu2(m, v[u][j] & 0x7FFF7FFFu);
        am[u] = max(m << 16, m & 0xFFFF0000u);
        if constexpr (C::FMT == kFp4E4M3) atomicMax(&row_top[i / per_row], am[u]);
      }
      __syncwarp();
      if constexpr (C::FMT == kFp4E4M3) named_barrier_sync(1, 128);
#pragma unroll
      for (int u = 0; u < kFuseUnits; ++u) {
        const int i = t + u * 128;
        if (i >= units) break;
        const int m = i / per_row, unit = i - m * per_row, stage = unit / 16 - k0;
        float mul;
        uint8_t code;
        if constexpr (C::FMT == kFp4E4M3) {
          code = fp4_block_scale_e4m3(am[u], fp4_row_scale(row_top[m]), &mul);
        } else {
          const int left = units - (i - lane);  // of this warp's units: a multiple of 8
          am[u] = max(am[u], __shfl_xor_sync(left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u, am[u], 1));
          code = fp4_block_scale_ue8m0(am[u], &mul);
        }
        if (stage < 0 || stage >= n) continue;
        float2 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = __fmul2_rn(make_float2(__uint_as_float(v[u][j] << 16), __uint_as_float(v[u][j] & 0xFFFF0000u)),
                            make_float2(mul, mul));
        const uint2 codes = mul == 0.0f ? make_uint2(0, 0) : make_uint2(e2m1x8(&y[0].x), e2m1x8(&y[4].x));
        const int in = unit & 15;  // the stage's 16 units are 128 bytes of the row, swizzled in chunks of 16
        *reinterpret_cast<uint2*>(fused + stage * C::kFuseCodes + m * 128 + (((in >> 1) ^ (m & 7)) << 4) + (in & 1) * 8) = codes;
        const int block = C::FMT == kFp4E4M3 ? in : in >> 1;
        if (C::FMT == kFp4E4M3 || (in & 1) == 0)
          fused_s[stage * C::kFuseScales + (block >> 2) * 256 + m * 16 + (block & 3)] = code;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tokens_ready);
    }
    // The scales of this lane's weight row and of the tokens (token 32 i + lane in ag[i]).
    if (p.w_g) {
      if (row < p.N) wg = LaneScale(p.w_g[row]);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(ag) / 4); ++i) {
        const int m = i * 32 + lane;
        if constexpr (C::FUSE) ag[i] = m < cols ? fp4_row_scale(row_top[m]).g : 0.0f;
        else ag[i] = m < cols ? p.a_g[m0 + m] : 0.0f;
      }
    }
    // (After a wait that gave up the MMA warp commits what it has: not all of K.)
    finished = mbar_wait(done, 0, nullptr, p.err, kDevErrTimeoutEpilogue) && *abort_flag == 0;
    tc_fence_after_sync();
  }
  __syncwarp();
  const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
  auto store = [&](int col, float v, float a) {
    v = v * wg.first * a * wg.last;  // (without row scales: all 1)
    if (row < p.N && finished) p.c[(m0 + col) * p.N + row] = __float2bfloat16(v);
  };
  constexpr int kStep = C::BN < 32 ? 16 : 32;
  if (warp >= 2 && warp < 6) {
    // The accumulator: lane = weight row, column = token.
    const float* mine = parts + (rank * p.part_cols * 128 + (q * 32 + lane) * p.part_vec);
    if (ks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int c0 = 0; c0 < C::BN; c0 += kStep) {
      if (c0 >= (ks == 1 ? cols : ks * p.part_cols)) break;
      uint32_t r[kStep];
      if constexpr (kStep == 16) tmem_ld_32x32b_x16(acc + c0, r);
      else tmem_ld_32x32b_x32(acc + c0, r);
      if (ks > 1) {
        if (!finished) {  // the CTAs that sum this part wait for it, and must not take it for a sum
#pragma unroll
          for (int i = 0; i < kStep; ++i) r[i] = 0x7FFFFFFFu;
        }
        if (p.part_vec == 4) send_columns<4, kStep>(r, c0, p.part_cols, ks, mine, parts_full);
        else if (p.part_vec == 2) send_columns<2, kStep>(r, c0, p.part_cols, ks, mine, parts_full);
        else send_columns<1, kStep>(r, c0, p.part_cols, ks, mine, parts_full);
        continue;
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const float a = __shfl_sync(0xFFFFFFFFu, ag[(c0 + i) / 32], i);
        if (c0 + i < cols) store(c0 + i, __uint_as_float(r[i]), a);
      }
    }
    if (ks > 1) {  // (the shares may reach past BN)
      const uint32_t zero[4] = {0, 0, 0, 0};
      for (int c = C::BN; c < ks * p.part_cols; c += p.part_vec) {
        if (p.part_vec == 4) send_columns<4, 4>(zero, c, p.part_cols, ks, mine, parts_full);
        else if (p.part_vec == 2) send_columns<2, 2>(zero, c, p.part_cols, ks, mine, parts_full);
        else send_columns<1, 1>(zero, c, p.part_cols, ks, mine, parts_full);
      }
    }
    tc_fence_before_sync();
    named_barrier_arrive(2, 160);
  }
  __syncwarp();
  if (warp == 1) {
    named_barrier_sync(2, 160);  // the accumulator has been read
    tc_fence_after_sync();
    tmem_dealloc(tmem, kFewTmemCols);
  }
  if (ks > 1) {
    if (warp < 2 || warp == 6) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // everything is sent
    if (warp >= 2 && warp < 6) {
      if (!mbar_wait_cluster(parts_full, 0, nullptr, p.err, kDevErrTimeoutEpilogue)) finished = false;
      auto put = [&](int c, float sum) {
        const int col = rank * p.part_cols + c;
        float a = ag[0];
#pragma unroll
        for (int i = 1; i < static_cast<int>(sizeof(ag) / 4); ++i) a = col / 32 == i ? ag[i] : a;
        a = __shfl_sync(0xFFFFFFFFu, a, col & 31);
        if (col < cols) store(col, sum, a);
      };
      if (p.part_vec == 4) sum_columns<4>(parts, ks, p.part_cols, q * 32 + lane, put);
      else if (p.part_vec == 2) sum_columns<2>(parts, ks, p.part_cols, q * 32 + lane, put);
      else sum_columns<1>(parts, ks, p.part_cols, q * 32 + lane, put);
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // no CTA ends before all that is sent to it
  }
}

// ---- CTA pairs -----------------------------------------------------------------------
//
// Many tokens: 256 tokens x 256 weight rows (128 or 384 where that makes better
// rounds) to a pair of CTAs (cta_group::2), tokens as tensor-memory lanes. Each CTA has
// 128 tokens and half of the weight rows, so a byte of either operand is fetched once
// per 256 products; both have the scales of all the tile's weight rows. The accumulator
// is single: the epilogue's eight warps take it out into registers, hand it back, and
// store from there while the next tile is summed. The MMAs bound it: 147 cycles for each
// 256 x 256 x 64 (128 by the nominal rate), tensor pipe 81 % active, the clock at 1.86
// GHz by power (4096 x 18432 x 7168: 155 us, 7.0 PFLOP/s; power-of-two scales, half the
// scale copies, 149). An SM takes 38 KB a stage from L2, 57 bytes a clock; tiles of 384
// rows, which take a sixth less for a product, need the same time for it.
//
//   warps 0, 2   producers: this CTA's codes and scales, completing on the leader's barriers
//   warp 1       MMA issuer (leader CTA); both allocate tensor memory
//   warps 4-11   epilogue: lane quarter warp % 4, the tile's second half from warp 8 on

constexpr int kPairThreads = 384;

template <int BN_, int FMT_>
struct PairCfg {
  static constexpr int BN = BN_, FMT = FMT_;
  static constexpr int kHalf = BN / 2;                           // weight rows of a CTA; columns of an epilogue half
  static constexpr int kMmas = BN > 256 ? 2 : 1;                 // side by side: an MMA has 256 columns at most
  static constexpr int kMmaN = BN / kMmas, kBox = kMmaN / 2;     // an MMA's columns, and its weight rows in a CTA
  static constexpr int kSfRows = BN / 128;                       // scale tile rows of the weights
  static constexpr int kTiles = FMT == kFp4E4M3 ? 4 : 2;
  static constexpr int kSfBytes = kTiles * kScaleTile;           // 128 rows of a stage
  static constexpr int kSfaAt = kLaneBytes + kHalf * 128, kSfbAt = kSfaAt + kSfBytes;
  static constexpr int kTxBytes = kSfbAt + kSfRows * kSfBytes;   // of one CTA
  static constexpr int kStageBytes = (kTxBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = BN == 128 ? 6 : BN == 256 ? 5 : 4;
  static constexpr int kSfStep = 4 + 4 * kSfRows;                // columns of 4 blocks' scales: tokens', weights'
  static constexpr int kSfCols = kTiles * kSfStep;
  static constexpr int kOutAt = kStages * kStageBytes;           // 8 warps x 4 KB
  static constexpr int kFactorsAt = kOutAt + 8 * 4096;           // the tile's weight row scales
  static constexpr int kBarsAt = kFactorsAt + BN * 4;
  static constexpr int kSmem = 1024 + kBarsAt + (2 * kStages + 3) * 8 + 8;
  static_assert(BN + 2 * kSfCols <= 512, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t pair_leader_addr(const void* local) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(cluster_ctarank() & ~1u));
  return a;
}

// A box into this CTA's shared memory, completing on the leader's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == kFp4E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// (Relaxed: what it hands over is tensor memory, ordered by the tcgen05 fences.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <class C>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_as, const __grid_constant__ CUtensorMap map_ws,
                         const __grid_constant__ CUtensorMap map_c, const Fp4Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarsAt);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  const int tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 16);  // the epilogue warps of both CTAs
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_as);
    tma_prefetch_desc(&map_ws);
    tma_prefetch_desc(&map_c);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  if (warp == 0 || warp == 2) {
    // Two producers: warp 0 the codes, warp 2 the scales (a thread that asks for
    // all five boxes of a stage takes longer than the stage's MMAs).
    const bool codes = warp == 0;
    if (lane == 0) {
      // A cursor over this pair's stages; every CTA asks for the operands of its own half.
      struct Cursor {
        int tile, k, st, y_a, y_w;
        uint32_t at, bar;
      };
      const uint32_t smem0 = smem_u32(smem), bar0 = pair_leader_addr(full);
      const int ktiles = static_cast<int>(p.ktiles);
      auto place = [&](Cursor& c) {  // at the head of a tile
        const int tm = c.tile % p.tiles_m, tn = c.tile / p.tiles_m;
        c.k = 0;
        c.y_a = codes ? tm * 256 + rank * 128 : (tm * 2 + rank) * ktiles;
        c.y_w = codes ? tn * C::BN + rank * C::kBox : tn * C::kSfRows * ktiles;
      };
      auto advance = [&](Cursor& c) {
        if (++c.st == C::kStages) c.st = 0, c.at = smem0, c.bar = bar0;
        else c.at += C::kStageBytes, c.bar += 8;
        if (++c.k == p.stages_k) {
          c.tile += pairs;
          place(c);
        }
      };
      auto weights = [&](const Cursor& c) {
        if (codes) {
          if (rank == 0) mbar_arrive_expect_tx(&full[c.st], 2 * C::kTxBytes);
#pragma unroll
          for (int m = 0; m < C::kMmas; ++m)
            tma_load_pair(c.at + kLaneBytes + m * C::kBox * 128, &map_w, c.bar, c.k * 128, c.y_w + m * C::kMmaN);
        } else {
#pragma unroll
          for (int r = 0; r < C::kSfRows; ++r)
            tma_load_pair(c.at + C::kSfbAt + r * C::kSfBytes, &map_ws, c.bar, 0, c.y_w + r * ktiles + c.k * C::kTiles);
        }
      };
      auto tokens = [&](const Cursor& c) {
        if (codes) tma_load_pair(c.at, &map_a, c.bar, c.k * 128, c.y_a);
        else tma_load_pair(c.at + C::kSfaAt, &map_as, c.bar, 0, c.y_a + c.k * C::kTiles);
      };
      const int total = ((tiles - pair + pairs - 1) / pairs) * p.stages_k;
      const int pre = total < C::kStages ? total : C::kStages;
      Cursor c{pair, 0, 0, 0, 0, smem0, bar0};
      place(c);
      const Cursor head = c;
      for (int i = 0; i < pre; ++i, advance(c)) weights(c);
      griddep_wait();
      c = head;
      int i = 0;
      uint32_t phase = 1;  // of the stages before they are filled again
      for (; i < total; ++i, advance(c)) {
        if (i >= pre) {
          if (!mbar_wait(&empty[c.st], phase, abort_flag, p.err, kDevErrTimeoutProducer)) break;
          weights(c);
        }
        tokens(c);
        if (c.st == C::kStages - 1) phase ^= 1;
      }
      // The MMAs have read the last stages (or, after a wait that gave up, the copies have landed).
      for (int j = i > C::kStages ? i - C::kStages : 0; j < i; ++j) {
        if (i == total) mbar_wait(&empty[j % C::kStages], (j / C::kStages) & 1, abort_flag, p.err, kDevErrTimeoutDrain);
        else if (rank == 0) mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1, nullptr, p.err, kDevErrTimeoutDrain);
      }
    }
  } else if (warp == 1 && rank == 0) {
    const bool leader = elect_one_sync();
    const uint32_t sf0 = tmem + C::BN;
    bool ok = true;
    int st = 0;
    uint32_t turn = 0, phase = 0, sf_turn = 0;
    for (int tile = pair; ok && tile < tiles; tile += pairs, turn ^= 1) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(acc_empty, turn ^ 1, abort_flag, p.err, kDevErrTimeoutMma))) break;
      tc_fence_after_sync();
      for (int k = 0; k < p.stages_k; ++k, sf_turn ^= 1) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], phase, abort_flag, p.err, kDevErrTimeoutMma))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t at = smem_u32(smem + st * C::kStageBytes);
        const uint64_t ad = sdesc_kmajor_sw128(at);
        const uint32_t sf = sf0 + sf_turn * C::kSfCols;
        const int left = p.ksteps - k * 4;
        if (leader) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= left) break;
            const int t = C::FMT == kFp4E4M3 ? j : j / 2;
            const uint32_t sfa = sf + static_cast<uint32_t>(C::kSfStep * t), sfb = sfa + 4;
            if (C::FMT == kFp4E4M3 || (j & 1) == 0) {
              tmem_cp_scales_pair(sfa, sdesc_scale_tile(at + C::kSfaAt + t * kScaleTile));
#pragma unroll
              for (int r = 0; r < C::kSfRows; ++r)
                tmem_cp_scales_pair(sfb + 4 * r, sdesc_scale_tile(at + C::kSfbAt + r * C::kSfBytes + t * kScaleTile));
            }
#pragma unroll
            for (int m = 0; m < C::kMmas; ++m)
              mma_fp4_pair<C::FMT>(tmem + m * C::kMmaN, ad + 2 * j,
                                   sdesc_kmajor_sw128(at + kLaneBytes + m * C::kBox * 128) + 2 * j,
                                   idesc_fp4(256, C::kMmaN, C::FMT, C::FMT == kFp4E4M3 ? 0 : 2 * (j & 1)), sfa,
                                   sfb + m * (C::kMmaN / 32), k > 0 || j > 0 ? 1u : 0u);
          }
          mma_commit_pair(&empty[st]);
          if (k + 1 == p.stages_k) mma_commit_pair(acc_full);
        }
        __syncwarp();
        if (++st == C::kStages) st = 0, phase ^= 1;
      }
    }
    // Every MMA issued has ended before tensor memory is released.
    if (leader) {
      mma_commit_pair(drain);
      mbar_wait(drain, 0, nullptr, p.err, kDevErrTimeoutDrain);
    }
    __syncwarp();
  } else if (warp >= 4) {
    griddep_wait();  // row scales of the tokens; the output may be the previous kernel's to read
    const int w = warp - 4, q = warp & 3, half = w >> 2;
    uint8_t* out = smem + C::kOutAt + w * 4096;
    float* factors = reinterpret_cast<float*>(smem + C::kFactorsAt + half * C::kHalf * 4);
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * C::kHalf);
    const uint32_t hand_back = pair_leader_addr(acc_empty);
    uint32_t turn = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles; tile += pairs, turn ^= 1) {
      const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
      const int64_t row = static_cast<int64_t>(tm) * 256 + rank * 128 + q * 32 + lane;
      const int64_t col0 = static_cast<int64_t>(tn) * C::BN + half * C::kHalf;
      LaneScale ag;
      if (p.a_g) {
        // The four warps of these columns bring their scales.
        named_barrier_sync(1 + half, 128);  // the tile before has been multiplied
        for (int in = q * 32 + lane; in < C::kHalf; in += 128) factors[in] = col0 + in < p.N ? p.w_g[col0 + in] : 0.0f;
        if (row < p.M) ag = LaneScale(p.a_g[row]);
        named_barrier_sync(1 + half, 128);
      }
      // (After a wait that gave up the warps still meet at their barriers, and store nothing.)
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, turn, abort_flag, p.err, kDevErrTimeoutEpilogue));
      if (!ok) continue;
      tc_fence_after_sync();
      // Two columns of this lane's row, times their scales, as bf16.
      auto two = [&](int col, uint32_t a, uint32_t b) {
        float2 v = make_float2(__uint_as_float(a), __uint_as_float(b));
        if (p.a_g) {
          v = __fmul2_rn(v, make_float2(ag.first, ag.first));
          v = __fmul2_rn(v, *reinterpret_cast<const float2*>(factors + col));
          v = __fmul2_rn(v, make_float2(ag.last, ag.last));
        }
        const __nv_bfloat162 t = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&t);
      };
      // All columns into registers (as bf16 where fp32 would take too many) and the
      // accumulator back to the MMAs, then 64 columns at a time through a swizzled box of 32 rows.
      constexpr bool kPack = C::kHalf > 128;
      uint32_t r[C::kHalf / 64][kPack ? 32 : 64];
#pragma unroll
      for (int h = 0; h < C::kHalf / 64; ++h) {
        if constexpr (kPack) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t t[32];
            tmem_ld_32x32b_x32(acc + h * 64 + c, t);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[h][c / 2 + i] = two(h * 64 + c + 2 * i, t[2 * i], t[2 * i + 1]);
          }
        } else {
          tmem_ld_32x32b_x64(acc + h * 64, r[h]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(hand_back);
#pragma unroll
      for (int h = 0; h < C::kHalf / 64; ++h) {
        if (lane == 0) bulk_wait_group_read0();  // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // eight columns
          uint32_t packed[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (kPack) packed[i] = r[h][c * 4 + i];
            else packed[i] = two(h * 64 + c * 8 + 2 * i, r[h][c * 8 + 2 * i], r[h][c * 8 + 2 * i + 1]);
          }
          *reinterpret_cast<uint4*>(out + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(packed[0], packed[1], packed[2], packed[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row < p.M && col0 + h * 64 < p.N) {  // (lane 0 has the box's first row)
          tma_store_2d(&map_c, out, static_cast<int>(col0 + h * 64), static_cast<int>(row));
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
    tc_fence_before_sync();
  }
  __syncthreads();
  cluster_sync();  // no CTA ends while its pair may still write into it
  if (warp == 1) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---- host --------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn fp4_map_encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &st) == cudaSuccess &&
        st == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(q);
  });
  return fn;
}

// Codes [rows, K / 2 bytes] in boxes of 128 bytes x box_rows, 128-byte swizzled.
bool make_code_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes, int box_rows) {
  EncodeTiledFn enc = fp4_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles [tiles, 512 bytes] in boxes of box_tiles.
bool make_scale_map(CUtensorMap* map, const void* base, uint64_t tiles, int box_tiles) {
  EncodeTiledFn enc = fp4_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {kScaleTile / 4, tiles};
  const cuuint64_t strides[1] = {kScaleTile};
  const cuuint32_t box[2] = {kScaleTile / 4, static_cast<cuuint32_t>(box_tiles)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output [rows, cols] in boxes of 64 columns x 32 rows, 128-byte swizzled.
bool make_out_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols) {
  EncodeTiledFn enc = fp4_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

template <class C>
int launch_pair(const DevInfo* d, const void* a, const void* w, int64_t K, Fp4Params p, cudaStream_t stream) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  std::call_once(once[d->device], [&] {
    set[d->device] = cudaFuncSetAttribute(fp4_gemm_pair_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (set[d->device] != cudaSuccess) return FP8BLK_ERR_CUDA;
  CUtensorMap ma, mw, mas, mws, mc;
  const uint64_t at = static_cast<uint64_t>((p.M + 127) / 128 * p.ktiles), wt = static_cast<uint64_t>((p.N + 127) / 128 * p.ktiles);
  if (!make_code_map(&ma, a, p.M, K / 2, 128) || !make_code_map(&mw, w, p.N, K / 2, C::kBox) ||
      !make_scale_map(&mas, p.a_s, at, C::kTiles) || !make_scale_map(&mws, p.w_s, wt, C::kTiles) ||
      !make_out_map(&mc, p.c, p.M, p.N))
    return FP8BLK_ERR_CUDA;
  p.tiles_m = static_cast<int>((p.M + 255) / 256);
  p.tiles_n = static_cast<int>((p.N + C::BN - 1) / C::BN);
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n, pairs = d->sm_count / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, fp4_gemm_pair_kernel<C>, ma, mw, mas, mws, mc, p));
}

// Whether a product's sizes fit the pair kernel's 32-bit tile coordinates and its
// output the vector stores.
bool pair_fits(const Fp4Params& p) {
  const int64_t tiles = (p.M + 255) / 256 * ((p.N + 127) / 128);
  return p.N % 8 == 0 && is_aligned(p.c, 16) && tiles * p.stages_k < int64_t{1} << 30 &&
         (p.M + 255) / 128 * p.ktiles < int64_t{1} << 30 && (p.N + 255) / 128 * p.ktiles < int64_t{1} << 30;
}

// Weight rows of a pair's tile. 128 where all tiles then run at once: twice the SMs
// bring the operands (us, 128 x 2112 x 7168 9.8, by 256 rows 11.3; 200 x 5120 x 7168 10.7
// and 11.6; in two rounds against one, 517 x 5120 x 7168, 17.7 and 12.9). Else 256, or 384
// where that leaves so many rounds fewer that they are shorter in all: a round of 256 is
// 0.35 us a stage and 0.55 to hand the accumulator over, of 384 0.51 and 1.3 (1024 x 7168 x
// 7168 19.4, by 256 22.4; 4096 x 7168 x 18432 140 and 143; 900 x 5120 x 1536 8.3 and 7.7;
// 4096 x 18432 x 7168 156 and 154).
int pair_columns(const DevInfo* d, const Fp4Params& p) {
  const int64_t pairs = d->sm_count / 2, tm = (p.M + 255) / 256, s = p.stages_k;
  auto rounds = [&](int bn) { return (tm * ((p.N + bn - 1) / bn) + pairs - 1) / pairs; };
  if (rounds(128) == 1) return 128;
  return rounds(384) * (51 * s + 130) + 100 < rounds(256) * (35 * s + 55) ? 384 : 256;
}

// CTAs of a tile's cluster, of two stages of K at least: as many as give every SM one,
// or one and a half where a CTA would have eight stages or more (8 tokens, us: 4096 x
// 4096 4.0 at one, 5.8 at one and a half; 4096 x 7168 5.6 and 5.9; 7168 x 7168 8.9 and
// 7.2; 7168 x 18432 20.7 and 15.6; without a split 8.8, 13.9, 14.6 and 35.2).
int few_split(int64_t tiles, int stages_k, int sm_count) {
  int64_t ks = sm_count / tiles;
  if (stages_k >= 8 * (ks < 1 ? 1 : ks)) ks = 3 * sm_count / 2 / tiles;
  if (ks > stages_k / 2) ks = stages_k / 2;
  return ks < 1 ? 1 : ks > 8 ? 8 : static_cast<int>(ks);
}

// Whether pairs multiply. Up to 32 tokens, where K is four stages or less and the weight
// rows are few (us: 32 x 2112 x 1024 3.8 and 4.7, but 32 x 2112 x 2048 4.9 and 4.2, 32 x
// 18432 x 1536 6.9 and 6.1). With more, unless splitting K saves more than the longer
// rows of partial sums cost (33 x 2112 x 7168 9.6 and 6.6, 48 x 5120 x 2048 5.7 and 6.1)
// and, from 49 on, the clusters take a part of the SMs, more of it the longer K is (128 x
// 1024 x 7168 9.9 and 7.0, 256 x 2112 x 7168 10.2 and 12.3, 100 x 1536 x 4096 7.1 and 7.1).
bool takes_pairs(const DevInfo* d, const Fp4Params& p) {
  if (p.M <= 32) return p.M > 16 && p.stages_k <= 4 && p.tiles_n <= 32;
  const int64_t tiles = p.tiles_n * ((p.M + 63) / 64);
  const int ks = few_split(tiles, p.stages_k, d->sm_count);
  if (6 * (p.stages_k - (p.stages_k + ks - 1) / ks) < (p.M < 64 ? p.M : 64) + 4) return true;
  return p.M > 48 && (5 * tiles > 2 * d->sm_count || 3 * tiles > 5 * p.stages_k);
}

// Whether a call's activations are quantised by the product's own CTAs (us, and by a
// kernel of their own): a token of up to 8192 numbers (1 x 24576 x 1536 4.9 and 6.6; 1 x
// 2112 x 7168 5.8 and 5.9; 1 x 1536 x 7168 5.1 and 5.5), or up to 4096 numbers of more
// (2 x 24576 x 1536 5.4 and 6.7; 2 x 10944 x 2048 5.4 and 5.9; 4 x 10944 x 2048, 8192
// numbers, 6.4 and 5.9; 5 x 7168 x 1536 5.6 and 5.1), where a CTA's share takes a corner
// of its shared memory. (In both formats each CTA converts all of K, with the 128 threads
// of its epilogue, and keeps its share. Powers of two need no more than the share, row
// scales the rows' maxima besides; neither is built.)
bool fuses(const DevInfo* d, int64_t M, int64_t N, int64_t K) {
  const int stages_k = static_cast<int>((K + kStageK - 1) / kStageK);
  const int ks = few_split((N + 127) / 128, stages_k, d->sm_count);
  return M <= 16 && M * K <= 128 * kFuseUnits * 16 / (M == 1 ? 1 : 2) && (stages_k + ks - 1) / ks <= 12;
}

template <class C>
int launch_few(const DevInfo* d, const CUtensorMap& mw, const CUtensorMap& ma, Fp4Params p, cudaStream_t stream) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  std::call_once(once[d->device], [&] {
    set[d->device] = cudaFuncSetAttribute(fp4_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  });
  if (set[d->device] != cudaSuccess) return FP8BLK_ERR_CUDA;
  const int64_t tiles = p.tiles_n * ((p.M + C::BN - 1) / C::BN);
  const int cols = static_cast<int>(p.M < C::BN ? p.M : C::BN);
  const int ks = few_split(tiles, p.stages_k, d->sm_count);
  if (tiles * ks >= int64_t{1} << 31) return FP8BLK_ERR_SHAPE;
  p.ksplit = ks;
  p.part_cols = (cols + ks - 1) / ks;
  p.part_vec = p.part_cols > 2 ? 4 : p.part_cols;
  p.part_cols = (p.part_cols + p.part_vec - 1) / p.part_vec * p.part_vec;
  // Two CTAs to an SM: an uneven last round is then spread, and the next product's CTAs
  // start beside this one's.
  const int most_n = (p.stages_k + ks - 1) / ks;
  const int other = 1024 + (C::FUSE ? most_n * (C::kFuseCodes + C::kFuseScales) + 256 : 0) +
                    (ks > 1 ? ks * p.part_cols * 512 : 0) + C::kBarBytes;
  p.stages = (113 * 1024 - other) / C::kStageBytes;
  if (p.stages > kMostStages<C>) p.stages = kMostStages<C>;
  if (p.stages > most_n) p.stages = most_n;
  if (p.stages < 1) return FP8BLK_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * ks));
  cfg.blockDim = dim3(kFewThreads);
  // (At least so much that no SM is given more CTAs than its tensor memory has columns for.)
  cfg.dynamicSmemBytes = other + p.stages * C::kStageBytes;
  if (cfg.dynamicSmemBytes < 78 * 1024) cfg.dynamicSmemBytes = 78 * 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, fp4_gemm_kernel<C>, mw, ma, p));
}

template <int FMT>
int run_fmt(const DevInfo* d, const void* a, const void* w, int64_t K, const Fp4Params& p, cudaStream_t stream) {
  CUtensorMap mw, ma;
  if (p.x) {
    if (!make_code_map(&mw, w, p.N, K / 2, 128)) return FP8BLK_ERR_CUDA;
    return launch_few<Cfg<16, FMT, true>>(d, mw, mw, p, stream);
  }
  if (takes_pairs(d, p) && pair_fits(p))
    switch (pair_columns(d, p)) {
      case 128: return launch_pair<PairCfg<128, FMT>>(d, a, w, K, p, stream);
      case 256: return launch_pair<PairCfg<256, FMT>>(d, a, w, K, p, stream);
      default: return launch_pair<PairCfg<384, FMT>>(d, a, w, K, p, stream);
    }
  const int bn = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  if (!make_code_map(&mw, w, p.N, K / 2, 128) || !make_code_map(&ma, a, p.M, K / 2, bn)) return FP8BLK_ERR_CUDA;
  switch (bn) {
    case 16: return launch_few<Cfg<16, FMT, false>>(d, mw, ma, p, stream);
    case 32: return launch_few<Cfg<32, FMT, false>>(d, mw, ma, p, stream);
    default: return launch_few<Cfg<64, FMT, false>>(d, mw, ma, p, stream);
  }
}

bool gemm_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && K % kBlock == 0 && M <= int64_t{1} << 28 && N <= int64_t{1} << 28 &&
         K <= int64_t{1} << 28;
}

// x: the activations where the product quantises them itself (else null, with a, a_s, a_g).
int gemm_checked(const DevInfo* d, const void* x, int64_t x_stride, const void* a, const void* a_s, const float* a_g,
                 const void* w, const void* w_s, const float* w_g, void* c, int64_t M, int64_t N, int64_t K, int fmt,
                 cudaStream_t stream) {
  Fp4Params p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.w_s = static_cast<const uint8_t*>(w_s);
  p.a_s = static_cast<const uint8_t*>(a_s);
  p.w_g = w_g;
  p.a_g = a_g;
  p.c = static_cast<__nv_bfloat16*>(c);
  p.err = d->err_word;
  p.M = M;
  p.N = N;
  p.ktiles = K / fp4_tile_cols(fmt);
  p.ksteps = static_cast<int>(K / 64);
  p.stages_k = static_cast<int>((K + kStageK - 1) / kStageK);
  p.tiles_n = static_cast<int>((N + 127) / 128);
  return fmt == kFp4E4M3 ? run_fmt<kFp4E4M3>(d, a, w, K, p, stream) : run_fmt<kFp4UE8M0>(d, a, w, K, p, stream);
}

// What the weight's side of a call has to be.
int check_weight(const void* w, const void* w_s, const float* w_g, const void* c, int fmt) {
  if (!w || !w_s || !c || (fmt == kFp4E4M3 && !w_g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(w, 16) || !is_aligned(w_s, 16) || !is_aligned(w_g, 4) || !is_aligned(c, 2)) return FP8BLK_ERR_ALIGN;
  return FP8BLK_OK;
}

size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_fp4_gemm(const void* a, const void* a_s, const float* a_g, const void* w, const void* w_s,
                               const float* w_g, void* c_bf16, int64_t M, int64_t N, int64_t K, int fmt,
                               fp8blk_stream_t stream) {
  if (!gemm_shape_ok(M, N, K)) return FP8BLK_ERR_SHAPE;
  if (!fp4_fmt_valid(fmt)) return FP8BLK_ERR_ARG;
  if (M == 0 || N == 0) return FP8BLK_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    if (!c_bf16) return FP8BLK_ERR_NULL;
    return cuda_status(cudaMemsetAsync(c_bf16, 0, static_cast<size_t>(M) * N * 2, s));
  }
  if (!a || !a_s || (fmt == kFp4E4M3 && !a_g)) return FP8BLK_ERR_NULL;
  if (!is_aligned(a, 16) || !is_aligned(a_s, 16) || !is_aligned(a_g, 4)) return FP8BLK_ERR_ALIGN;
  if (int st = check_weight(w, w_s, w_g, c_bf16, fmt)) return st;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  if (fmt == kFp4UE8M0) a_g = w_g = nullptr;
  return gemm_checked(d, nullptr, 0, a, a_s, a_g, w, w_s, w_g, c_bf16, M, N, K, fmt, s);
}

// Workspace of the linear layer: [codes M K / 2][scale tiles][row scales 4 M], each part 256-byte aligned.
extern "C" size_t fp8blk_fp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt) {
  if (!gemm_shape_ok(M, N, K) || !fp4_fmt_valid(fmt)) return 0;
  return align256(static_cast<size_t>(M) * (K / 2)) + align256(static_cast<size_t>(fp4_scale_bytes(M, K, fmt))) +
         align256(static_cast<size_t>(M) * 4);
}

extern "C" int fp8blk_fp4_linear(const void* x_bf16, int64_t x_stride, const void* w, const void* w_s, const float* w_g,
                                 void* y_bf16, int64_t M, int64_t N, int64_t K, int fmt, void* workspace,
                                 size_t workspace_bytes, fp8blk_stream_t stream) {
  if (!gemm_shape_ok(M, N, K) || x_stride < K) return FP8BLK_ERR_SHAPE;
  if (!fp4_fmt_valid(fmt)) return FP8BLK_ERR_ARG;
  if (M == 0 || N == 0) return FP8BLK_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    if (!y_bf16) return FP8BLK_ERR_NULL;
    return cuda_status(cudaMemsetAsync(y_bf16, 0, static_cast<size_t>(M) * N * 2, s));
  }
  if (!x_bf16) return FP8BLK_ERR_NULL;
  if (!is_aligned(x_bf16, 16) || x_stride % 8) return FP8BLK_ERR_ALIGN;
  if (int st = check_weight(w, w_s, w_g, y_bf16, fmt)) return st;
  if (!workspace) return FP8BLK_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return FP8BLK_ERR_ALIGN;
  if (workspace_bytes < fp8blk_fp4_linear_workspace_bytes(M, N, K, fmt)) return FP8BLK_ERR_WORKSPACE;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  const bool rows = fmt == kFp4E4M3;
  if (fuses(d, M, N, K))
    return gemm_checked(d, x_bf16, x_stride, nullptr, nullptr, nullptr, w, w_s, rows ? w_g : nullptr, y_bf16, M, N, K, fmt, s);
  uint8_t* q = static_cast<uint8_t*>(workspace);
  uint8_t* qs = q + align256(static_cast<size_t>(M) * (K / 2));
  float* g = reinterpret_cast<float*>(qs + align256(static_cast<size_t>(fp4_scale_bytes(M, K, fmt))));
  if (int st = fp4_quant_launch(x_bf16, false, x_stride, M, K, fmt, q, qs, g, d->sm_count, true, s)) return st;
  return gemm_checked(d, nullptr, 0, q, qs, rows ? g : nullptr, w, w_s, rows ? w_g : nullptr, y_bf16, M, N, K, fmt, s);
}
