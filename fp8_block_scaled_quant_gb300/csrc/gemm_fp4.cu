// Product of two matrices of microscaled 4-bit floats (fp4.cuh has the formats):
//
//   C[m, n] = bf16( ag[m] wg[n] sum over blocks b of sa[m, b] sw[n, b] sum_{k in b} a[m, k] w[n, k] )
//
// The block-scaled MMA applies sa and sw itself (products of e2m1 numbers and
// their scales, summed in fp32 in tensor memory), the epilogue the row scales.
//
// Kernel: 128 weight rows are the MMA's M (tensor-memory lanes), BN tokens its
// columns, 256 of K to a stage: codes by TMA (128-byte rows, 128-byte swizzle),
// scale tiles by bulk copies, from there into tensor memory by tcgen05.cp in the
// order of the MMAs that use them. Few weight tiles are split over K by clusters
// of up to 8 CTAs, whose partial sums meet in shared memory in rank order.
//
//   warp 0      producer: weights of the first stages before the dependency wait
//   warp 1      MMA issuer
//   warps 2-5   epilogue, a lane quarter each
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
                     int sm_count, cudaStream_t stream);

namespace {

constexpr int kStageK = 256;
constexpr int kLaneBytes = 128 * 128;  // 128 weight rows of a stage
constexpr int kThreads = 192;

struct Fp4Params {
  const uint8_t* w_s;
  const uint8_t* a_s;
  const float* w_g;
  const float* a_g;
  __nv_bfloat16* c;
  unsigned* err;
  int64_t M, N, ktiles;  // ktiles: scale tiles along K
  int ksteps;            // K / 64
  int stages_k;          // ceil(K / 256)
  int tiles_n, tiles_m;  // weight tiles; token tiles (pairs)
  int ksplit;            // CTAs of a tile's cluster
};

template <int BN_, int FMT_>
struct Cfg {
  static constexpr int BN = BN_, FMT = FMT_;
  static constexpr int kTiles = FMT == kFp4E4M3 ? 4 : 2;  // scale tiles of a stage
  static constexpr int kColBytes = BN * 128;
  static constexpr int kSfBytes = kTiles * kScaleTile;
  static constexpr int kStageBytes = (kLaneBytes + kColBytes + 2 * kSfBytes + 1023) / 1024 * 1024;
  // Two CTAs to an SM (113 KB each): the work of an uneven last round is then
  // spread, and one CTA's start and end lie beside the other's stream.
  static constexpr int kStages = 112 * 1024 / kStageBytes;
  static constexpr int kAccCols = BN < 32 ? 32 : BN;
  static constexpr int kSfCols = 2 * kTiles * 4;  // both operands' scales of a stage
  static constexpr int kTmemCols = kAccCols + 2 * kSfCols <= 128 ? 128 : 256;
  static constexpr int kBarBytes = (2 * kStages + 1) * 8 + 8;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes;
  static_assert(kAccCols + 2 * kSfCols <= kTmemCols, "tensor memory");
  static_assert(BN * 128 * 4 <= kStages * kStageBytes, "the partial sums lie where the stages were");
};

template <class C>
__global__ void __launch_bounds__(kThreads, 2)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                    const Fp4Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ks = p.ksplit, rank = static_cast<int>(blockIdx.x) % ks;
  const int tile = static_cast<int>(blockIdx.x) / ks;
  const int tile_n = tile % p.tiles_n, tile_m = tile / p.tiles_n;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.stages_k) * rank / ks);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.stages_k) * (rank + 1) / ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_a);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // After the allocation: a CTA of the next kernel that came first to this SM's
  // tensor memory would hold it until this kernel ends.
  griddep_launch_dependents();

  bool finished = true;  // epilogue warps: the accumulator is complete
  if (warp == 0) {
    if (lane == 0) {
      // Scale tiles of stage k: all of them, or those that K has left.
      auto tiles_of = [&](int k) {
        const int64_t left = p.ktiles - static_cast<int64_t>(k) * C::kTiles;
        return static_cast<uint32_t>(left < C::kTiles ? left : C::kTiles);
      };
      auto weights = [&](int st, int k) {
        uint8_t* at = smem + st * C::kStageBytes;
        const uint32_t sf = tiles_of(k) * kScaleTile;
        mbar_arrive_expect_tx(&full[st], kLaneBytes + C::kColBytes + 2 * sf);
        tma_load_2d(at, &map_w, &full[st], k * 128, tile_n * 128);
        bulk_load(at + kLaneBytes + C::kColBytes,
                  p.w_s + (static_cast<int64_t>(tile_n) * p.ktiles + static_cast<int64_t>(k) * C::kTiles) * kScaleTile, sf,
                  &full[st]);
      };
      auto tokens = [&](int st, int k) {
        uint8_t* at = smem + st * C::kStageBytes;
        tma_load_2d(at + kLaneBytes, &map_a, &full[st], k * 128, tile_m * C::BN);
        const int64_t row_tile = static_cast<int64_t>(tile_m) * C::BN / 128;
        bulk_load(at + kLaneBytes + C::kColBytes + C::kSfBytes,
                  p.a_s + (row_tile * p.ktiles + static_cast<int64_t>(k) * C::kTiles) * kScaleTile,
                  tiles_of(k) * kScaleTile, &full[st]);
      };
      const int n = k1 - k0, pre = n < C::kStages ? n : C::kStages;
      for (int i = 0; i < pre; ++i) weights(i, k0 + i);
      griddep_wait();
      int issued = 0;
      for (; issued < n; ++issued) {
        const int st = issued % C::kStages;
        if (issued >= pre) {
          if (!mbar_wait(&empty[st], ((issued / C::kStages) & 1) ^ 1, abort_flag, p.err, kDevErrTimeoutProducer)) break;
          weights(st, k0 + issued);
        }
        tokens(st, k0 + issued);
      }
      if (issued < n) {  // gave up: the copies in flight land before the CTA ends
        for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
          mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, nullptr, p.err, kDevErrTimeoutDrain);
      }
    }
  } else if (warp == 1) {
    const bool leader = elect_one_sync();
    const uint32_t sf0 = tmem + C::kAccCols;
    bool ok = true;
    for (int i = 0; i < k1 - k0; ++i) {
      const int st = i % C::kStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (i / C::kStages) & 1, abort_flag, p.err, kDevErrTimeoutMma))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t at = smem_u32(smem + st * C::kStageBytes);
      const uint64_t ad = sdesc_kmajor_sw128(at), bd = sdesc_kmajor_sw128(at + kLaneBytes);
      const uint32_t sw = at + kLaneBytes + C::kColBytes;
      const uint32_t sf = sf0 + static_cast<uint32_t>((i & 1) * C::kSfCols);
      const int left = p.ksteps - (k0 + i) * 4, steps = left < 4 ? left : 4;  // 2 or 4
      if (leader) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= steps) break;
          const int t = C::FMT == kFp4E4M3 ? j : j / 2;
          const uint32_t sfa = sf + static_cast<uint32_t>(8 * t), sfb = sfa + 4;
          if (C::FMT == kFp4E4M3 || (j & 1) == 0) {
            tmem_cp_scales(sfa, sdesc_scale_tile(sw + t * kScaleTile));
            tmem_cp_scales(sfb, sdesc_scale_tile(sw + C::kSfBytes + t * kScaleTile));
          }
          mma_fp4<C::FMT>(tmem, ad + 2 * j, bd + 2 * j,
                          idesc_fp4(128, C::BN, C::FMT, C::FMT == kFp4E4M3 ? 0 : 2 * (j & 1)), sfa, sfb,
                          i > 0 || j > 0 ? 1u : 0u);
        }
        mma_commit(&empty[st]);
        if (i + 1 == k1 - k0) mma_commit(done);
      }
      __syncwarp();
    }
    if (leader) {
      if (!ok) mma_commit(done);
      mbar_wait(done, 0, nullptr, p.err, kDevErrTimeoutDrain);
    }
    __syncwarp();
  } else {
    griddep_wait();
    finished = mbar_wait(done, 0, nullptr, p.err, kDevErrTimeoutEpilogue);
    tc_fence_after_sync();
  }

  __syncwarp();
  // The accumulator: lane = weight row, column = token.
  const int q = warp & 3;  // lane quarter of an epilogue warp
  const int64_t row = static_cast<int64_t>(tile_n) * 128 + q * 32 + lane;
  const int64_t m0 = static_cast<int64_t>(tile_m) * C::BN;
  const int cols = static_cast<int>(p.M - m0 < C::BN ? p.M - m0 : C::BN);
  const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16);
  float* part = reinterpret_cast<float*>(smem);  // [BN][128]
  float wg = 1.0f;
  if (warp >= 2 && p.w_g && row < p.N) wg = __ldg(p.w_g + row);
  auto store = [&](int col, float v) {
    const int64_t m = m0 + col;
    if (p.a_g) v *= wg * __ldg(p.a_g + m);
    if (row < p.N) p.c[m * p.N + row] = __float2bfloat16(v);
  };
  if (ks == 1) {
    if (warp >= 2) {
      constexpr int kStep = C::BN < 32 ? 16 : 32;
      for (int c = 0; c < cols; c += kStep) {
        uint32_t r[kStep];
        if constexpr (kStep == 16) tmem_ld_32x32b_x16(at + c, r);
        else tmem_ld_32x32b_x32(at + c, r);
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if (c + i < cols && finished) store(c + i, __uint_as_float(r[i]));
      }
      tc_fence_before_sync();
    }
  } else {
    if (warp >= 2) {
      constexpr int kStep = C::BN < 32 ? 16 : 32;
      for (int c = 0; c < cols; c += kStep) {
        uint32_t r[kStep];
        if constexpr (kStep == 16) tmem_ld_32x32b_x16(at + c, r);
        else tmem_ld_32x32b_x32(at + c, r);
#pragma unroll
        for (int i = 0; i < kStep; ++i) part[(c + i) * 128 + q * 32 + lane] = __uint_as_float(r[i]);
      }
      tc_fence_before_sync();
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
      // Four columns at a time, so that 4 ks loads are under way together.
      const int c1 = cols * (rank + 1) / ks;
      for (int c = cols * rank / ks; c < c1; c += 4) {
        float v[4][8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i][k] = k < ks && c + i < c1
                          ? ld_shared_cluster_f32(part + (c + i) * 128 + q * 32 + lane, static_cast<uint32_t>(k))
                          : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float sum = v[i][0];
#pragma unroll
          for (int k = 1; k < 8; ++k) sum += v[i][k];
          if (finished && c + i < c1) store(c + i, sum);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA ends while another reads its sums
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---- CTA pairs -----------------------------------------------------------------------
//
// Many tokens: 256 tokens x 256 weight rows to a pair of CTAs (cta_group::2), tokens
// as tensor-memory lanes. Each CTA has 128 tokens and half of the weight rows, so a
// byte of either operand is fetched once per 256 products; both have the scales of
// all 256 weight rows. One accumulator of 256 columns: the epilogue's eight warps
// take it out in bf16 registers, hand it back, and store from there while the next
// tile is summed.
//
//   warps 0, 2   producers: this CTA's codes and scales, completing on the leader's barriers
//   warp 1       MMA issuer (leader CTA); both allocate tensor memory
//   warps 4-11   epilogue: lane quarter warp % 4, columns 128 (warp >= 8) on

constexpr int kPairThreads = 384;
constexpr int kPairN = 256;

template <int FMT_>
struct PairCfg {
  static constexpr int FMT = FMT_;
  static constexpr int kTiles = FMT == kFp4E4M3 ? 4 : 2;
  static constexpr int kSfBytes = kTiles * kScaleTile;           // 128 rows of a stage
  static constexpr int kSfaAt = 2 * kLaneBytes, kSfbAt = kSfaAt + kSfBytes;
  static constexpr int kTxBytes = kSfbAt + 2 * kSfBytes;         // of one CTA
  static constexpr int kStageBytes = (kTxBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = 5;
  static constexpr int kSfCols = kTiles * 12;                    // 4 for the tokens, 8 for the weights
  static constexpr int kOutAt = kStages * kStageBytes;           // 8 warps x 4 KB
  static constexpr int kFactorsAt = kOutAt + 8 * 4096;           // the tile's 256 weight row scales
  static constexpr int kBarsAt = kFactorsAt + kPairN * 4;
  static constexpr int kSmem = 1024 + kBarsAt + (2 * kStages + 3) * 8 + 8;
  static_assert(kPairN + 2 * kSfCols <= 512, "tensor memory");
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

// mbar_wait for a barrier that threads of both CTAs arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err,
                                                  unsigned code) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_wait_cluster(a, parity) ||
         (mbar_wait(bar, parity, abort, err, code) && mbar_try_wait_cluster(a, parity));
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
        c.y_w = codes ? tn * kPairN + rank * 128 : tn * 2 * ktiles;
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
          tma_load_pair(c.at + kLaneBytes, &map_w, c.bar, c.k * 128, c.y_w);
        } else {
          tma_load_pair(c.at + C::kSfbAt, &map_ws, c.bar, 0, c.y_w + c.k * C::kTiles);
          tma_load_pair(c.at + C::kSfbAt + C::kSfBytes, &map_ws, c.bar, 0, c.y_w + ktiles + c.k * C::kTiles);
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
    const uint32_t sf0 = tmem + kPairN;
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
        const uint64_t ad = sdesc_kmajor_sw128(at), bd = sdesc_kmajor_sw128(at + kLaneBytes);
        const uint32_t sf = sf0 + sf_turn * C::kSfCols;
        const int left = p.ksteps - k * 4;
        if (leader) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= left) break;
            const int t = C::FMT == kFp4E4M3 ? j : j / 2;
            const uint32_t sfa = sf + static_cast<uint32_t>(12 * t), sfb = sfa + 4;
            if (C::FMT == kFp4E4M3 || (j & 1) == 0) {
              tmem_cp_scales_pair(sfa, sdesc_scale_tile(at + C::kSfaAt + t * kScaleTile));
              tmem_cp_scales_pair(sfb, sdesc_scale_tile(at + C::kSfbAt + t * kScaleTile));
              tmem_cp_scales_pair(sfb + 4, sdesc_scale_tile(at + C::kSfbAt + C::kSfBytes + t * kScaleTile));
            }
            mma_fp4_pair<C::FMT>(tmem, ad + 2 * j, bd + 2 * j,
                                 idesc_fp4(256, kPairN, C::FMT, C::FMT == kFp4E4M3 ? 0 : 2 * (j & 1)), sfa, sfb,
                                 k > 0 || j > 0 ? 1u : 0u);
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
    float* factors = reinterpret_cast<float*>(smem + C::kFactorsAt + half * 512);
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * 128);
    const uint32_t hand_back = pair_leader_addr(acc_empty);
    uint32_t turn = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles; tile += pairs, turn ^= 1) {
      const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
      const int64_t row = static_cast<int64_t>(tm) * 256 + rank * 128 + q * 32 + lane;
      const int64_t col0 = static_cast<int64_t>(tn) * kPairN + half * 128;
      float ag = 1.0f;
      if (p.a_g) {
        // The four warps of these columns bring 32 of their scales each.
        const int64_t c = col0 + q * 32 + lane;
        const float wg = c < p.N ? __ldg(p.w_g + c) : 0.0f;
        if (row < p.M) ag = __ldg(p.a_g + row);
        named_barrier_sync(1 + half, 128);  // the tile before has been multiplied
        factors[q * 32 + lane] = wg;
        named_barrier_sync(1 + half, 128);
      }
      // (After a wait that gave up the warps still meet at their barriers, and store nothing.)
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, turn, abort_flag, p.err, kDevErrTimeoutEpilogue));
      if (!ok) continue;
      tc_fence_after_sync();
      uint32_t packed[64];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + c * 32, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f[4] = {1.0f, 1.0f, 1.0f, 1.0f};
          if (p.a_g) {
            const float4 g4 = *reinterpret_cast<const float4*>(factors + c * 32 + i * 4);
            f[0] = ag * g4.x, f[1] = ag * g4.y, f[2] = ag * g4.z, f[3] = ag * g4.w;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[4 * i + 2 * j]) * f[2 * j],
                                                           __uint_as_float(r[4 * i + 2 * j + 1]) * f[2 * j + 1]);
            packed[c * 16 + i * 2 + j] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(hand_back);
      // 64 columns at a time through a swizzled box of 32 rows.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (lane == 0) bulk_wait_group_read0();  // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(out + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(packed[h * 32 + c * 4], packed[h * 32 + c * 4 + 1], packed[h * 32 + c * 4 + 2],
                         packed[h * 32 + c * 4 + 3]);
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

template <int FMT>
int launch_pair(const DevInfo* d, const void* a, const void* w, int64_t K, Fp4Params p, cudaStream_t stream) {
  using C = PairCfg<FMT>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  std::call_once(once[d->device], [&] {
    set[d->device] = cudaFuncSetAttribute(fp4_gemm_pair_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (set[d->device] != cudaSuccess) return FP8BLK_ERR_CUDA;
  CUtensorMap ma, mw, mas, mws, mc;
  const uint64_t at = static_cast<uint64_t>((p.M + 127) / 128 * p.ktiles), wt = static_cast<uint64_t>((p.N + 127) / 128 * p.ktiles);
  if (!make_code_map(&ma, a, p.M, K / 2, 128) || !make_code_map(&mw, w, p.N, K / 2, 128) ||
      !make_scale_map(&mas, p.a_s, at, C::kTiles) || !make_scale_map(&mws, p.w_s, wt, C::kTiles) ||
      !make_out_map(&mc, p.c, p.M, p.N))
    return FP8BLK_ERR_CUDA;
  p.tiles_m = static_cast<int>((p.M + 255) / 256);
  p.tiles_n = static_cast<int>((p.N + kPairN - 1) / kPairN);
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
  const int64_t tiles = (p.M + 255) / 256 * ((p.N + kPairN - 1) / kPairN);
  return p.N % 8 == 0 && is_aligned(p.c, 16) && tiles * p.stages_k < int64_t{1} << 30 &&
         (p.M + 255) / 128 * p.ktiles < int64_t{1} << 30 && (p.N + 255) / 128 * p.ktiles < int64_t{1} << 30;
}

template <class C>
int launch_swapped(const DevInfo* d, const CUtensorMap& mw, const CUtensorMap& ma, Fp4Params p, cudaStream_t stream) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  std::call_once(once[d->device], [&] {
    set[d->device] = cudaFuncSetAttribute(fp4_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (set[d->device] != cudaSuccess) return FP8BLK_ERR_CUDA;
  const int64_t tiles = p.tiles_n * ((p.M + C::BN - 1) / C::BN);
  int ks = 1;
#ifdef FP4_KS
  while (ks < FP4_KS && ks < p.stages_k) ++ks;
#else
  while (ks < 8 && ks < p.stages_k && tiles * (ks + 1) <= 2 * d->sm_count) ++ks;
#endif
  if (tiles * ks >= int64_t{1} << 31) return FP8BLK_ERR_SHAPE;
  p.ksplit = ks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * ks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
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
#ifndef FP4_PAIR_MIN
#define FP4_PAIR_MIN 256
#endif
  if (p.M >= FP4_PAIR_MIN && pair_fits(p)) return launch_pair<FMT>(d, a, w, K, p, stream);
  const int bn = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  CUtensorMap mw, ma;
  if (!make_code_map(&mw, w, p.N, K / 2, 128) || !make_code_map(&ma, a, p.M, K / 2, bn)) return FP8BLK_ERR_CUDA;
  switch (bn) {
    case 16: return launch_swapped<Cfg<16, FMT>>(d, mw, ma, p, stream);
    case 32: return launch_swapped<Cfg<32, FMT>>(d, mw, ma, p, stream);
    case 64: return launch_swapped<Cfg<64, FMT>>(d, mw, ma, p, stream);
    default: return launch_swapped<Cfg<128, FMT>>(d, mw, ma, p, stream);
  }
}

bool gemm_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && K % kBlock == 0 && M <= int64_t{1} << 28 && N <= int64_t{1} << 28 &&
         K <= int64_t{1} << 28;
}

int gemm_checked(const DevInfo* d, const void* a, const void* a_s, const float* a_g, const void* w, const void* w_s,
                 const float* w_g, void* c, int64_t M, int64_t N, int64_t K, int fmt, cudaStream_t stream) {
  Fp4Params p{};
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
  return gemm_checked(d, a, a_s, a_g, w, w_s, w_g, c_bf16, M, N, K, fmt, s);
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
  uint8_t* q = static_cast<uint8_t*>(workspace);
  uint8_t* qs = q + align256(static_cast<size_t>(M) * (K / 2));
  float* g = reinterpret_cast<float*>(qs + align256(static_cast<size_t>(fp4_scale_bytes(M, K, fmt))));
  if (int st = fp4_quant_launch(x_bf16, false, x_stride, M, K, fmt, q, qs, g, d->sm_count, s)) return st;
  const bool rows = fmt == kFp4E4M3;
  return gemm_checked(d, q, qs, rows ? g : nullptr, w, w_s, rows ? w_g : nullptr, y_bf16, M, N, K, fmt, s);
}
