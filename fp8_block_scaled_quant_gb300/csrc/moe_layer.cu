// A whole mixture-of-experts layer for up to 32 tokens in one kernel
// ("Administrator & Developer Guide", 8.4: the Gate, the routed experts, the
// shared experts; 6.3 and 6.4: FP8 Linears). Per token t:
//
//   logits = x gate_w^T (fp32 sums), ids e_j and weights g_j by the gate rule,
//   (xq, xs) = act_quant(x),
//   h1 = w1_e xq, h3 = w3_e xq   (block-scaled, fp32 sums),
//   u  = silu(h1) h3 in fp32, (uq, us) = act_quant(u),
//   y[t] = bf16( sum_j g_j w2_{e_j} uq_j + sum over shared experts s of w2_s uq_s ).
//
// Between the two roundings that FP8 Linears make (act_quant of x and of u)
// everything is fp32 and y is rounded once; the chained kernels round h1, h3,
// silu, u and each expert's output to bf16.
//
// What bounds it: the weights. Each expert that a token reaches is read once
// (44 MB of codes for 7168 x 2048), whatever the number of its tokens, so the
// floor is those bytes at HBM rate. The kernel is built to keep that stream
// from stopping:
//   - One CTA per SM, one launch (cooperative: CTAs meet at two barriers). Per
//     CTA a producer warp keeps 160 KB of weight tiles in flight by TMA (128 rows x
//     one K block, 16 KB), a warp issues the MMAs, four promote and finish.
//   - The gate decides what the routed weights are, but not the shared ones: the
//     CTA's share of the shared experts streams through while the gate is computed
//     by the warps that do not stream.
//   - w2 does not depend on u, only its use does: the ring runs on from phase 1
//     into w2 before the barrier between them.
//   - Phase 1 lays its units (expert, 128 rows of w1 and the same of w3) end to
//     end, K block by K block, and phase 2 its row tiles of w2, over all experts
//     and K blocks; each CTA has the same number of K blocks of either. Where a
//     unit or a row tile is cut between CTAs, the one that finishes last adds the
//     parts in CTA order (in warps of their own, while the stream goes on): one
//     order of every sum. A unit's 128 rows are one block
//     of u, quantised where the unit is finished.
//
// The products are tcgen05 MMAs with 128 weight rows as M and the tokens as N = 16
// or 32 (all tokens for every expert: idle columns cost nothing): 156 or 160
// cycles for a 16 KB tile (measured, 105 bytes a cycle and SM; HBM brings 23).
// Each K block has its own accumulators in tensor memory (eight sets), promoted
// as acc += D * (a_s w_s) by the thread that owns the row. Warp-level FP8 MMAs on
// the same stream, which are carried out as conversions and half-precision MMAs,
// ran the SM's issue slots full: 846 us where these took 538 for 32 tokens of
// 5120 x 1536 x 160.
//
// Measured (GPU time): one token of 7168 x 2048, 256 experts, 8 and a shared one
// reached: 83-85 us for 400 MB, 4.8 TB/s over the call, 6.1 to 6.6 of a copy's 6.7 in the
// two phases; 14 us go by before the routed weights can be asked for (x read,
// logits, the CTAs' meeting, the gate), 6 between the phases, 3 after them. 16
// tokens of it that reach 78 experts 542 us, 6.35 TB/s; 32 tokens of 5120 x 1536,
// 160 experts (112 reached), 492 us, 5.4 TB/s; 5 tokens of 2048 x 1408, 64 experts,
// 67.1 us, 3.6 TB/s. Two token-column widths share 128 registers a thread: the
// wider one spills 604 bytes. For all of 1 to 32 tokens it is ahead of the chain of
// gate product, gate, act_quant and grouped GEMMs (1.6 times for one token of 7168
// x 2048, 1.13 for 32).
//
// Every wait is bounded (2 s): on expiry an error bit is set, waits return at
// once from then on, and the control flow, whose loops are finite, runs out.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "block_rule.cuh"
#include "fp8blk.h"
#include "gate.cuh"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {

int gate_shape_status(const float* bias, int64_t T, int64_t E, int64_t n_groups, int64_t topk_groups, int64_t topk,
                      int score_func, float route_scale);

namespace {

constexpr int kMaxTokens = 32;
constexpr int kMaxShared = 8;
constexpr int kMaxActive = 256 + kMaxShared;
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 192;             // SMs a device may have
constexpr int kMaxDim = 8192, kMaxInter = 16384;
constexpr int kGateVecs = 4;              // 16-byte vectors of a gate row per thread
constexpr int kStages = 10;               // weight tiles in flight
constexpr int kTileBytes = 128 * 128;
constexpr int kSets = 8;                  // accumulator sets in tensor memory
// Streaming roles: finishers are warps 4-7, closers 8-11. All but producer,
// issuer and finishers compute the gate first (0, 3, 8-15).
constexpr int kProducer = 2, kIssuer = 1, kFinisher = 4, kCloser = 8;
constexpr int kGaters = 10;
// Up to here the closers load eight parts at a time, more tokens' two: one token of
// 5120 x 1536 x 160 57.6 us against 61.5, four tokens the same either way.
constexpr int kFewTokens = 4;
constexpr unsigned kDevErrTimeoutLayer = 1u << 9;

// Shared memory: weight tiles, token tiles, token scales, barriers, tables.
__host__ __device__ constexpr int off_tok() { return kStages * kTileBytes; }
__host__ __device__ constexpr int off_scl(int n) { return off_tok() + kStages * n * 128; }
__host__ __device__ constexpr int off_bar(int n) { return off_scl(n) + kStages * n * 4; }
constexpr int kCuts = 6;                  // cut units and tiles of a CTA: two per range
constexpr int kNumBars = 3 * kStages + 2 * kSets + kCuts + 2;
__host__ __device__ constexpr int off_act(int n) { return (off_bar(n) + kNumBars * 8 + 8 + 15) / 16 * 16; }
__host__ __device__ constexpr int off_mask(int n) { return off_act(n) + kMaxActive * 4; }
__host__ __device__ constexpr int off_sel(int n) { return off_mask(n) + kMaxActive * 4; }  // ids, weights; scratch before
__host__ __device__ constexpr int off_scan(int n) { return off_sel(n) + 2 * kMaxTokens * 32 * 4; }
__host__ __device__ constexpr int off_red(int n) { return off_scan(n) + 64 * 4; }          // [4][n][4] row maxima
__host__ __device__ constexpr int off_bias(int n) { return off_red(n) + 4 * n * 4 * 4; }
__host__ __device__ constexpr int layer_smem(int n) { return 1024 + off_bias(n) + 256 * 4; }
static_assert(layer_smem(32) <= 232448, "shared memory per CTA");
static_assert(off_red(16) % 16 == 0 && off_red(32) % 16 == 0 && off_scl(16) % 16 == 0, "16-byte reads");

struct LayerParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* gate_w;
  const float* gate_bias;
  const float* w1_s;
  const float* w3_s;
  const float* w2_s;
  __nv_bfloat16* y;
  int32_t* topk_idx;    // may be null
  float* topk_w;        // may be null
  unsigned* counters;   // [0..1] barrier arrivals, [2] tokens gated, [3] CTAs done, [16..31] row tiles, a byte each; zero between calls
  unsigned* unit_parts;  // [unit] parts so far; zeroed before the first barrier
  float* logits;        // [T][E]
  int* ids;             // [T][k], where the grid shares the gate
  float* weights;
  uint8_t* xq;          // [T][dim]
  float* xs;            // [dim / 128][N]
  uint8_t* uq;          // [active expert][T][inter], rows of routed tokens
  float* us;            // [active expert][inter / 128][N]: scale * gate weight
  float* part;          // [CTA][range][it starts the unit][h1, h3][T][128]
  float* part2;         // [CTA][it starts the tile][T][128]
  unsigned* err;
  int T, dim, inter, E, ns, k, groups, kept, sigmoid, normalize, ue8m0, max_units;
  float route_scale;
};

// The bounded wait, its slow part out of line (the loops that call it stay
// small in the instruction cache). Returns at once after an abort.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 63u) == 0) {
      if (abort && *abort) return;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        if (abort) *abort = 1;
        atomicOr(err, kDevErrTimeoutLayer);
        return;
      }
    }
  }
}

__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint32_t a = smem_u32(bar);
  if (!mbar_try_wait(a, parity)) wait_slow(a, parity, abort, err);
}

// `bytes` (a multiple of 16) from global to shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Orders this thread's generic accesses, to any memory, before async-proxy ones.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// N consecutive tensor-memory columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(taddr, r); }

// Quantises one 128-element block, four elements per lane; returns its scale.
__device__ __forceinline__ float quant_block(const float (&v)[4], bool ue8m0, int lane, uint8_t* q) {
  float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const float sc = block_scale(amax, ue8m0);
  const uint32_t lo = e4m3x2(__fdiv_rn(v[0], sc), __fdiv_rn(v[1], sc));
  const uint32_t hi = e4m3x2(__fdiv_rn(v[2], sc), __fdiv_rn(v[3], sc));
  reinterpret_cast<uint32_t*>(q)[lane] = lo | (hi << 16);
  return sc;
}

// First block of part c of G when n blocks are split evenly, and the part of
// block x. (n * G stays below 2^32: at most 264 experts x 128 x 64 K blocks and
// 192 CTAs.)
__device__ __forceinline__ int even(int n, int c, int G) {
  return static_cast<int>(static_cast<uint32_t>(n) * static_cast<uint32_t>(c) / static_cast<uint32_t>(G));
}
__device__ __forceinline__ int part_of(int n, int x, int G) {
  return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(G) - 1u) / static_cast<uint32_t>(n));
}

// h1 (and, of kTwo, h3) += the parts 0, 1, ..., of which each has [h1, h3][T][128]
// of this thread's row: U parts are loaded together, tokens mk < 2^J of them.
template <int U, int J, bool kTwo, int N, class F>
__device__ __forceinline__ void add_parts(float (&h1)[N], float (&h3)[N], int parts, int T, uint32_t mk, F part) {
#pragma unroll 1
  for (int i = 0; i < parts; i += U) {
    float a[U][J], b[U][kTwo ? J : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* v = part(min(i + u, parts - 1));
      const uint32_t want = i + u < parts ? mk : 0u;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        a[u][j] = (want >> j) & 1u ? __ldcg(v + j * 128) : 0.f;
        if (kTwo) b[u][kTwo ? j : 0] = (want >> j) & 1u ? __ldcg(v + (T + j) * 128) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        h1[j] += a[u][j];
        if (kTwo) h3[j] += b[u][kTwo ? j : 0];
      }
  }
}

__device__ __forceinline__ float silu_mul(float h1, float h3) { return h1 / (1.0f + expf(-h1)) * h3; }

// Ids and weights of token m by one warp, into the pair tables.
__device__ __noinline__ void gate_of_token(const LayerParams& p, const float* bias, int m, int lane, bool store,
                                           int* sel_e, float* sel_w) {
  const int v = p.E / 32;
  float xl[8], bl[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xl[i] = i < v ? __ldcg(p.logits + static_cast<size_t>(m) * p.E + lane * v + i) : 0.f;
    bl[i] = i < v ? bias[lane * v + i] : 0.f;
  }
  int e;
  float w;
  gate_warp<8>(xl, bl, p.gate_bias != nullptr, v, p.groups, p.kept, p.k, p.sigmoid, p.route_scale, p.normalize, lane,
               &e, &w);
  if (lane < p.k) {
    e = min(max(e, 0), p.E - 1);
    sel_e[m * p.k + lane] = e;
    sel_w[m * p.k + lane] = w;
    if (store && p.topk_idx) p.topk_idx[m * p.k + lane] = e;
    if (store && p.topk_w) p.topk_w[m * p.k + lane] = w;
  }
}

// The phases that copies were given on kStages barriers: which barriers, and the
// parity of the last one of each.
struct Armed {
  uint32_t used, parity;
  __host__ __device__ __forceinline__ void arm(int s) {
    parity ^= used & (1u << s);
    used |= 1u << s;
  }
};

template <int N>  // token columns
__global__ void __launch_bounds__(kThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map3,
                     const __grid_constant__ CUtensorMap map2, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_u, const __grid_constant__ LayerParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  float* scl = reinterpret_cast<float*>(smem + off_scl(N));  // [stage][N] token scales
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + off_bar(N));
  uint64_t* tok_full = full + kStages;
  uint64_t* empty = tok_full + kStages;
  uint64_t* set_full = empty + kStages;
  uint64_t* set_empty = set_full + kSets;
  uint64_t* cut_stored = set_empty + kSets;  // this CTA's part of its i-th cut unit or tile is in memory
  uint64_t* tables = cut_stored + kCuts;     // the gate's tables are there
  uint64_t* drain = tables + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* act = reinterpret_cast<int*>(smem + off_act(N));              // active experts, shared ones first
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + off_mask(N));  // their tokens
  int* sel_e = reinterpret_cast<int*>(smem + off_sel(N));
  float* sel_w = reinterpret_cast<float*>(sel_e + kMaxTokens * 32);
  int* scan = reinterpret_cast<int*>(smem + off_scan(N));            // [16] active; [32] all active
  float* red = reinterpret_cast<float*>(smem + off_red(N));
  float* bias = reinterpret_cast<float*>(smem + off_bias(N));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, c = blockIdx.x;
  const int Kb1 = p.dim / 128, Kb2 = p.inter / 128;  // K blocks; Kb2 is also the units of an expert
  const uint32_t all_tokens = p.T == 32 ? 0xFFFFFFFFu : (1u << p.T) - 1u;

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&tok_full[i], 1);
      mbar_init(&empty[i], 5);  // the MMAs and the four finishers
    }
    for (int i = 0; i < kSets; ++i) {
      mbar_init(&set_full[i], 1);
      mbar_init(&set_empty[i], 4);
    }
    for (int i = 0; i < kCuts; ++i) mbar_init(&cut_stored[i], 4);
    mbar_init(tables, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&map1);
    tma_prefetch_desc(&map3);
    tma_prefetch_desc(&map2);
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_u);
  }
  if (tid < p.ns) {
    act[tid] = p.E + tid;
    mask[tid] = all_tokens;
  }
  if (tid < p.E) bias[tid] = p.gate_bias ? __ldg(p.gate_bias + tid) : 0.f;
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // The gate rows of this CTA's experts. The experts share the warps, each with a slice of
  // K: warp's vectors v0, v0 + step, ... of its expert's row.
  const int per_cta = min((p.E + G - 1) / G, kWarps);  // experts at a time
  const int wpe = kWarps / per_cta;                    // warps of an expert
  const int v0 = warp % wpe * 32 + lane, step = wpe * 32, vecs = p.dim / 8;
  uint4 gate_row[kGateVecs];
  auto load_gate = [&](int e) {
#pragma unroll
    for (int i = 0; i < kGateVecs; ++i)
      gate_row[i] = e < p.E && warp < per_cta * wpe && v0 + i * step < vecs
                        ? __ldg(reinterpret_cast<const uint4*>(p.gate_w + static_cast<size_t>(e) * p.dim) + v0 + i * step)
                        : make_uint4(0u, 0u, 0u, 0u);
  };
  load_gate(c + warp / wpe * G);

  // A cursor walks this CTA's K blocks of a range of units (the shared ones,
  // the routed ones), K laid end to end.
  struct Cursor {
    int a, blk, kb, left;  // active expert, its 128-row block, K block; K blocks left
  };
  auto cursor = [&](int first, int blocks) {
    const int q0 = even(blocks, c, G), q1 = even(blocks, c + 1, G), u = q0 / Kb1;
    return Cursor{first + u / Kb2, u % Kb2, q0 % Kb1, q1 - q0};
  };
  auto advance = [&](Cursor& k) {
    --k.left;
    if (++k.kb == Kb1) {
      k.kb = 0;
      if (++k.blk == Kb2) {
        k.blk = 0;
        ++k.a;
      }
    }
  };
  const int shared_blocks = p.ns * Kb2 * Kb1;
  // ---- producer (one lane): weight tiles, then the tokens' codes and scales that
  // go with them, when those exist.
  const bool producer = warp == kProducer && lane == 0;
  const uint64_t policy = l2_policy_evict_first();  // weights are read once
  int issued = 0;                                   // tiles
  auto load_tile = [&](const CUtensorMap* map, int x, int y) {
    const int s = issued % kStages;
    if (issued >= kStages) wait(&empty[s], (issued / kStages - 1) & 1, abort_flag, p.err);
    if (*abort_flag) return;
    mbar_arrive_expect_tx(&full[s], kTileBytes);
    tma_load_2d_hint(smem + s * kTileBytes, map, &full[s], x, y, policy);
    ++issued;
  };
  Armed tokens_armed{0, 0};
  auto load_tokens = [&](int s, const CUtensorMap* map, int x, int y, const float* scales) {
    if (*abort_flag) return;
    tokens_armed.arm(s);
    mbar_arrive_expect_tx(&tok_full[s], N * 128 + N * 4);
    tma_load_2d(smem + off_tok() + s * N * 128, map, &tok_full[s], x, y);
    bulk_load(scl + s * N, scales, N * 4, &tok_full[s]);
  };
  auto load_unit = [&](const Cursor& k) {  // one K block: w1's tile, w3's tile
    const int y = ((k.a < p.ns ? p.E + k.a : act[k.a]) * Kb2 + k.blk) * 128;
    load_tile(&map1, k.kb * 128, y);
    load_tile(&map3, k.kb * 128, y);
  };
  Cursor ahead = cursor(0, shared_blocks);
  // K blocks asked for before the gate: their 64 KB a CTA are on their way while
  // the CTAs meet; more (half the ring's stages, 160 KB) hold the meeting's atomics
  // up: 86.0 us for one token of 7168 x 2048 x 256 where two blocks take 84.5.
  const int early = min(2, ahead.left);
  auto first_tiles = [&] {
    if (producer)
#pragma unroll 1
      for (int q = 0; q < early; ++q) {
        load_unit(ahead);
        advance(ahead);
      }
  };

  // Waits until counter i has `goal` arrivals.
  auto arrived = [&](int i, unsigned goal) {
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t spin = 0;; ++spin) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.counters + i) : "memory");
      if (v >= goal) break;
      if ((spin & 63u) == 63u) {
        if (*abort_flag) break;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(p.err, kDevErrTimeoutLayer);
          break;
        }
      }
    }
    __threadfence();
  };
  // Grid barrier i: every CTA's threads have arrived, their global writes are visible.
  // (`meanwhile` runs between a CTA's arrival and the wait.)
  auto grid_barrier = [&](int i, auto meanwhile) {
    __threadfence();
    __syncthreads();
    meanwhile();
    if (tid == 0) {
      atomicAdd(p.counters + i, 1u);
      arrived(i, static_cast<unsigned>(G));
    }
    __syncthreads();
  };

  // Phase 0: x quantised and the logits formed, both spread over the grid. A
  // CTA's experts share its warps, each with a slice of K.
#pragma unroll 1
  for (int i = warp * G + c; i < p.T * Kb1; i += G * kWarps) {
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x) + static_cast<size_t>(i) * 32 + lane);
    const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                        __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
    const float s = quant_block(v, p.ue8m0 != 0, lane, p.xq + static_cast<size_t>(i) * 128);
    if (lane == 0) p.xs[i % Kb1 * N + i / Kb1] = s;
  }
  fence_proxy_async_all();  // TMA reads these
  for (int i = c * kThreads + tid; i < p.max_units; i += G * kThreads) p.unit_parts[i] = 0;
  // The shared experts' stream starts when the gate's operands are here (its
  // copies, asked for earlier, made the logits wait 4 us behind them).
  {
    float* sums = sel_w;  // [warp][columns]
#pragma unroll 1
    for (int e0 = c; e0 < p.E; e0 += per_cta * G) {
      // (The row's K is at most kGateVecs passes, see kMaxDim.) Four tokens' vectors
      // are loaded together: a token at a time was 1700 cycles each, a load's way
      // and a reduction's.
#pragma unroll 1
      for (int m0 = 0; m0 < p.T; m0 += 4) {
        uint4 xv[4][kGateVecs];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int i = 0; i < kGateVecs; ++i)
            xv[m][i] = m0 + m < p.T && v0 + i * step < vecs
                           ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(m0 + m) * p.dim) + v0 + i * step)
                           : make_uint4(0u, 0u, 0u, 0u);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kGateVecs; ++i) {
          const uint32_t aw[4] = {gate_row[i].x, gate_row[i].y, gate_row[i].z, gate_row[i].w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t bw[4] = {xv[m][i].x, xv[m][i].y, xv[m][i].z, xv[m][i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[m] = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(bw[q] << 16), acc[m]);
              acc[m] = fmaf(__uint_as_float(aw[q] & 0xFFFF0000u), __uint_as_float(bw[q] & 0xFFFF0000u), acc[m]);
            }
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int m = 0; m < 4; ++m) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (lane == m && m0 + m < p.T) sums[warp * N + m0 + m] = acc[m];
      }
      __syncthreads();
      for (int i = tid; i < per_cta * p.T; i += kThreads) {
        const int k = i / p.T, m = i % p.T;
        float v = 0.f;
        for (int w = 0; w < wpe; ++w) v += sums[(k * wpe + w) * N + m];
        if (e0 + k * G < p.E) p.logits[static_cast<size_t>(m) * p.E + e0 + k * G] = v;
      }
      __syncthreads();
      if (e0 + per_cta * G < p.E) load_gate(e0 + per_cta * G + warp / wpe * G);
    }
  }
  tc_fence_before_sync();
  grid_barrier(0, first_tiles);
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // The gate, then the tables: active experts in order (shared ones first) and
  // their tokens. Every CTA gates up to kGaters tokens for itself, a warp each
  // (one token of 5120 x 1536 x 160 57.6 us, 61.0 by the other way). Of more, a
  // CTA gates one and all read the results: one round and an exchange instead of
  // rounds (24 tokens 415 us against 421).
  if (warp == 0 || warp == 3 || warp >= kCloser) {
    const int gw = warp == 0 ? 0 : warp == 3 ? 1 : warp - kCloser + 2, gt = gw * 32 + lane;
    auto meet = [&] { named_barrier_sync(4, kGaters * 32); };
    if (p.T <= kGaters) {
      if (gw < p.T) gate_of_token(p, bias, gw, lane, c == 0, sel_e, sel_w);
    } else {
      if (gw == 0) {
#pragma unroll 1
        for (int m = c; m < p.T; m += G) {
          gate_of_token(p, bias, m, lane, true, p.ids, p.weights);
          __threadfence();
          __syncwarp();
          if (lane == 0) atomicAdd(p.counters + 2, 1u);
        }
        if (lane == 0) arrived(2, static_cast<unsigned>(p.T));
      }
      meet();
      for (int i = gt; i < p.T * p.k; i += kGaters * 32) {
        sel_e[i] = min(max(__ldcg(p.ids + i), 0), p.E - 1);
        sel_w[i] = __ldcg(p.weights + i);
      }
    }
    uint32_t* tokens_of = reinterpret_cast<uint32_t*>(bias);  // by expert id; the bias has been used
    meet();
    if (gt < p.E) tokens_of[gt] = 0;
    meet();
    for (int i = gt; i < p.T * p.k; i += kGaters * 32) atomicOr(&tokens_of[sel_e[i]], 1u << (i / p.k));
    meet();
    const uint32_t my_tokens = gt < p.E ? tokens_of[gt] : 0;
    const unsigned have = __ballot_sync(0xFFFFFFFFu, my_tokens != 0);
    if (lane == 0) scan[gw] = __popc(have);
    meet();
    int a0 = p.ns;
#pragma unroll
    for (int w = 0; w < kGaters; ++w) a0 += w < gw ? scan[w] : 0;
    if (my_tokens) {
      const int a = a0 + __popc(have & ((1u << lane) - 1u));
      act[a] = gt;
      mask[a] = my_tokens;
    }
    if (gt == kGaters * 32 - 1) scan[32] = a0 + __popc(have);
    meet();
    if (gt == 0) mbar_arrive(tables);
  }
  // What follows from the tables, learnt by each role when it needs it. Items of
  // phase 2: K blocks of row tiles of w2, expert by expert.
  struct Item {
    int tile, a, kb;
  };
  int nact = 0, routed_blocks = 0, tile_blocks = 0, blocks2 = 0, q2 = 0, n2 = 0;
  Item first_item{0, 0, 0};
  auto learn = [&] {
    wait(tables, 0, abort_flag, p.err);
    nact = *abort_flag ? p.ns : scan[32];
    routed_blocks = (nact - p.ns) * Kb2 * Kb1;
    tile_blocks = nact * Kb2;
    blocks2 = p.dim / 128 * tile_blocks;
    q2 = even(blocks2, c, G);
    n2 = even(blocks2, c + 1, G) - q2;
    if (n2 > 0) first_item = Item{q2 / tile_blocks, q2 / Kb2 % nact, q2 % Kb2};
  };
  auto gate_weight = [&](int a, int m) {
    if (a < p.ns) return 1.0f;
    float w = 0.f;
    for (int j = 0; j < p.k; ++j)
      if (sel_e[m * p.k + j] == act[a]) w = sel_w[m * p.k + j];
    return w;
  };
  constexpr uint32_t kIdesc = idesc_e4m3_f32(128, N);
  // Streaming positions, alike in every role: tiles and K blocks so far.
  int tile = 0, kblock = 0;
  uint32_t tok_phase = 0;  // bit s: phase of tok_full[s]
  auto tok_parity = [&](int s) {
    const uint32_t ph = (tok_phase >> s) & 1;
    tok_phase ^= 1u << s;
    return ph;
  };
  // One K block's MMAs: `tiles` weight tiles against its tokens, into set
  // kblock % kSets. The whole warp calls it.
  auto multiply = [&](int tiles) {
    const int set = kblock % kSets, s0 = tile % kStages;
    if (kblock >= kSets) wait(&set_empty[set], (kblock / kSets - 1) & 1, abort_flag, p.err);
    wait(&tok_full[s0], tok_parity(s0), abort_flag, p.err);
    const uint64_t bd = sdesc_kmajor_sw128(smem_u32(smem + off_tok() + s0 * N * 128));
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int s = (tile + t) % kStages;
      wait(&full[s], ((tile + t) / kStages) & 1, abort_flag, p.err);
      __syncwarp();
      tc_fence_after_sync();
      if (!__any_sync(0xFFFFFFFFu, *abort_flag != 0) && elect_one_sync()) {
        const uint64_t ad = sdesc_kmajor_sw128(smem_u32(smem + s * kTileBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_e4m3(tmem + (set * 2 + t) * N, ad + 2 * k, bd + 2 * k, kIdesc, k > 0);
        if (t == tiles - 1) {
          for (int q = 0; q < tiles; ++q) mma_commit(&empty[(tile + q) % kStages]);
          mma_commit(&set_full[set]);
        }
      }
      __syncwarp();
    }
    tile += tiles;
    ++kblock;
  };
  // The finishers' side: the tokens' scales of the K block and its `tiles` products.
  const int row = (warp & 3) * 32 + lane;  // of the 128 weight rows: finishers and closers
  const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  auto products_ready = [&] {
    const int s0 = tile % kStages;
    wait(&tok_full[s0], tok_parity(s0), abort_flag, p.err);
    wait(&set_full[kblock % kSets], (kblock / kSets) & 1, abort_flag, p.err);
    __syncwarp();
    tc_fence_after_sync();
  };
  // The parts of cut units and tiles. The finishers store this CTA's and go on;
  // the closers count it in, and where it was the last of its unit add them up.
  int cuts = 0;
  auto part_stored = [&] {
    __threadfence();
    __syncwarp();
    if (lane == 0) mbar_arrive(&cut_stored[cuts]);
    ++cuts;
  };
  // (`count` holds a counter of `parts` in `field` << shift.)
  auto last_part = [&](unsigned* count, unsigned field, int shift, unsigned parts) {
    wait(&cut_stored[cuts], 0, abort_flag, p.err);
    ++cuts;
    __threadfence();
    named_barrier_sync(3, 128);
    if (warp == kCloser && lane == 0) {
      const bool last = ((atomicAdd(count, 1u << shift) >> shift) & field) == parts - 1;
      if (last) atomicSub(count, parts << shift);
      scan[48] = last;
      __threadfence();
    }
    named_barrier_sync(3, 128);
    const bool last = scan[48] != 0;
    named_barrier_sync(3, 128);  // before scan[48] is written again
    return last;
  };
  // u of a finished unit for its tokens, by 128 threads (one per row): the rows
  // are one block of u. `group` 0: finishers, 1: closers; they alternate between
  // two halves of their maxima.
  int flips = 0;
  auto quantise_unit = [&](float (&h1)[N], const float (&h3)[N], int a, int blk, uint32_t mk, int group, int r) {
    float* top = red + (group * 2 + (flips & 1)) * N * 4;
    ++flips;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if ((mk >> j) & 1u) {
        h1[j] = silu_mul(h1[j], h3[j]);
        float m = fabsf(h1[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0) top[j * 4 + (warp & 3)] = m;
      }
    }
    named_barrier_sync(2 + group, 128);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if ((mk >> j) & 1u) {
        const float4 m = *reinterpret_cast<const float4*>(top + j * 4);
        const float sc = block_scale(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)), p.ue8m0 != 0);
        p.uq[(static_cast<size_t>(a) * p.T + j) * p.inter + blk * 128 + r] =
            static_cast<uint8_t>(e4m3x2(__fdiv_rn(h1[j], sc), 0.f));
        if (r == j) p.us[(a * Kb2 + blk) * N + j] = sc * gate_weight(a, j);
      }
    }
  };
  // acc += (product t of the K block) * (token scale * ws), for tokens in mk.
  auto promote = [&](float (&acc)[N], int t, float ws, uint32_t mk) {
    uint32_t d[N];
    tmem_ld_cols(t_lane + (kblock % kSets * 2 + t) * N, d);
    const float4* sc = reinterpret_cast<const float4*>(scl + tile % kStages * N);
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 v = sc[j / 4];
      if ((mk >> j) & 1u) acc[j] = fmaf(__uint_as_float(d[j]), v.x * ws, acc[j]);
      if ((mk >> (j + 1)) & 1u) acc[j + 1] = fmaf(__uint_as_float(d[j + 1]), v.y * ws, acc[j + 1]);
      if ((mk >> (j + 2)) & 1u) acc[j + 2] = fmaf(__uint_as_float(d[j + 2]), v.z * ws, acc[j + 2]);
      if ((mk >> (j + 3)) & 1u) acc[j + 3] = fmaf(__uint_as_float(d[j + 3]), v.w * ws, acc[j + 3]);
    }
  };
  auto products_done = [&](int tiles) {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&set_empty[kblock % kSets]);
      for (int q = 0; q < tiles; ++q) mbar_arrive(&empty[(tile + q) % kStages]);
    }
    tile += tiles;
    ++kblock;
  };

  // ---- phase 1 -------------------------------------------------------------------
  auto next_item = [&](Item& k) {
    if (++k.kb == Kb2) {
      k.kb = 0;
      if (++k.a == nact) {
        k.a = 0;
        ++k.tile;
      }
    }
  };
  auto load_item = [&](const Item& k) { load_tile(&map2, k.kb * 128, act[k.a] * p.dim + k.tile * 128); };
  Item item_ahead = first_item;
  int early2 = 0, phase1_tiles = 0;
  if (producer) {
    fence_proxy_async_all();
    Cursor k = cursor(0, shared_blocks);
#pragma unroll 1
    for (int q = 0; q < early; ++q) {
      load_tokens(2 * q, &map_x, k.kb * 128, 0, p.xs + k.kb * N);
      advance(k);
    }
#pragma unroll 1
    for (int range = 0; range < 2; ++range) {
      if (range) {
        learn();
        ahead = cursor(p.ns, routed_blocks);
      }
#pragma unroll 1
      for (; ahead.left > 0; advance(ahead)) {
        const int s = issued % kStages;
        load_unit(ahead);
        load_tokens(s, &map_x, ahead.kb * 128, 0, p.xs + ahead.kb * N);
      }
    }
    phase1_tiles = issued;
    early2 = min(kStages, n2);  // w2 tiles asked for before u is quantised
    item_ahead = first_item;
#pragma unroll 1
    for (int q = 0; q < early2; ++q) {
      load_item(item_ahead);
      next_item(item_ahead);
    }
  } else if (warp == kIssuer) {
#pragma unroll 1
    for (int range = 0; range < 2; ++range) {
      if (range) learn();
      const int blocks = range ? routed_blocks : shared_blocks;
#pragma unroll 1
      for (int q = even(blocks, c + 1, G) - even(blocks, c, G); q > 0; --q) multiply(2);
    }
  } else if (warp >= kFinisher && warp < kFinisher + 4) {
#pragma unroll 1
    for (int range = 0; range < 2; ++range) {
      if (range) learn();
      Cursor at = range ? cursor(p.ns, routed_blocks) : cursor(0, shared_blocks);
#pragma unroll 1
      while (at.left > 0) {
        // One unit, or this CTA's part of it.
        const int a = at.a, blk = at.blk, from = at.kb, n = min(at.left, Kb1 - from);
        const uint32_t mk = mask[a];
        const float* s1 = p.w1_s + (act[a] * Kb2 + blk) * Kb1 + from;
        const float* s3 = p.w3_s + (s1 - p.w1_s);
        float acc1[N], acc3[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc1[j] = acc3[j] = 0.f;
        float w1s = __ldg(s1), w3s = __ldg(s3);
#pragma unroll 1
        for (int q = 0; q < n; ++q) {
          const float w1n = q + 1 < n ? __ldg(s1 + q + 1) : 0.f, w3n = q + 1 < n ? __ldg(s3 + q + 1) : 0.f;
          products_ready();
          promote(acc1, 0, w1s, 0xFFFFFFFFu);
          promote(acc3, 1, w3s, 0xFFFFFFFFu);
          products_done(2);
          w1s = w1n;
          w3s = w3n;
          advance(at);
        }
        if (n == Kb1) {
          quantise_unit(acc1, acc3, a, blk, mk, 0, row);
        } else {
          float* t = p.part + static_cast<size_t>((c * 2 + range) * 2 + (from == 0 ? 1 : 0)) * 2 * p.T * 128 + row;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if ((mk >> j) & 1u) {
              t[j * 128] = acc1[j];
              t[(p.T + j) * 128] = acc3[j];
            }
          part_stored();
        }
      }
    }
    fence_proxy_async_all();  // TMA reads uq and us
  } else if (warp >= kCloser && warp < kCloser + 4) {
#pragma unroll 1
    for (int range = 0; range < 2; ++range) {
      if (range) learn();
      const int blocks = range ? routed_blocks : shared_blocks, first = range ? p.ns : 0;
      const int q0 = even(blocks, c, G), q1 = even(blocks, c + 1, G);
#pragma unroll 1
      for (int q = q0; q < q1;) {
        const int u = q / Kb1, end = (u + 1) * Kb1;
        const bool whole = q == u * Kb1 && end <= q1;
        q = end;
        if (whole) continue;
        const int a = first + u / Kb2, blk = u % Kb2;
        const uint32_t mk = mask[a];
        // (With fewer K blocks than CTAs some CTAs have none, the others one.)
        const int c0 = part_of(blocks, u * Kb1, G), c1 = part_of(blocks, end - 1, G);
        const int parts = blocks >= G ? c1 - c0 + 1 : Kb1;
        if (!last_part(p.unit_parts + a * Kb2 + blk, 0xFFFFFFFFu, 0, parts)) continue;
        auto part = [&](int i) {
          const int k = blocks >= G ? c0 + i : part_of(blocks, u * Kb1 + i, G);
          return p.part + static_cast<size_t>((k * 2 + range) * 2 + (i == 0 ? 1 : 0)) * 2 * p.T * 128 + row;
        };
        float h1[N], h3[N];
#pragma unroll
        for (int j = 0; j < N; ++j) h1[j] = h3[j] = 0.f;
        if (N == 16 && p.T <= kFewTokens)
          add_parts<8, kFewTokens, true>(h1, h3, parts, p.T, mk, part);
        else
          add_parts<N == 16 ? 2 : 1, N, true>(h1, h3, parts, p.T, mk, part);
        quantise_unit(h1, h3, a, blk, mk, 1, row);
      }
    }
    fence_proxy_async_all();
  }
  __syncwarp();
  grid_barrier(1, [] {});

  // ---- phase 2 -------------------------------------------------------------------
  if (producer) {
    fence_proxy_async_all();
    Item k = first_item;
#pragma unroll 1
    for (int q = 0; q < early2; ++q) {
      load_tokens((phase1_tiles + q) % kStages, &map_u, k.kb * 128, k.a * p.T, p.us + (k.a * Kb2 + k.kb) * N);
      next_item(k);
    }
#pragma unroll 1
    for (int q = early2; q < n2; ++q) {
      const int s = issued % kStages;
      load_item(item_ahead);
      load_tokens(s, &map_u, item_ahead.kb * 128, item_ahead.a * p.T, p.us + (item_ahead.a * Kb2 + item_ahead.kb) * N);
      next_item(item_ahead);
    }
  } else if (warp == kIssuer) {
#pragma unroll 1
    for (int q = 0; q < n2; ++q) multiply(1);
  } else if (warp >= kFinisher && warp < kFinisher + 4) {
    Item at = first_item;
    int left = n2;
#pragma unroll 1
    while (left > 0) {
      // One row tile, or this CTA's part of it.
      const int from = at.a * Kb2 + at.kb, n = min(left, tile_blocks - from), tl = at.tile;
      left -= n;
      float acc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
      auto scale_of = [&](const Item& k) { return __ldg(p.w2_s + (act[k.a] * (p.dim / 128) + k.tile) * Kb2 + k.kb); };
      float ws = scale_of(at);
#pragma unroll 1
      for (int q = 0; q < n; ++q) {
        const uint32_t mk = mask[at.a];
        next_item(at);
        const float wn = q + 1 < n ? scale_of(at) : 0.f;
        products_ready();
        promote(acc, 0, ws, mk);  // columns of other tokens hold nothing of theirs
        products_done(1);
        ws = wn;
      }
      __nv_bfloat16* y = p.y + tl * 128 + row;
      if (n == tile_blocks) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j < p.T) y[static_cast<size_t>(j) * p.dim] = __float2bfloat16_rn(acc[j]);
      } else {
        float* t = p.part2 + static_cast<size_t>(c * 2 + (from == 0 ? 1 : 0)) * p.T * 128 + row;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (j < p.T) t[j * 128] = acc[j];
        part_stored();
      }
    }
  } else if (warp >= kCloser && warp < kCloser + 4) {
#pragma unroll 1
    for (int q = q2; q < q2 + n2;) {
      const int tl = q / tile_blocks, end = (tl + 1) * tile_blocks;
      const bool whole = q == tl * tile_blocks && end <= q2 + n2;
      q = end;
      if (whole) continue;
      const int c0 = part_of(blocks2, tl * tile_blocks, G), c1 = part_of(blocks2, end - 1, G);
      const int parts = blocks2 >= G ? c1 - c0 + 1 : tile_blocks;
      // (At most 192 parts: a byte per tile.)
      if (!last_part(p.counters + 16 + tl / 4, 0xFFu, tl % 4 * 8, parts)) continue;
      auto part = [&](int i) {
        const int k = blocks2 >= G ? c0 + i : part_of(blocks2, tl * tile_blocks + i, G);
        return p.part2 + static_cast<size_t>(k * 2 + (i == 0 ? 1 : 0)) * p.T * 128 + row;
      };
      float acc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
      if (N == 16 && p.T <= kFewTokens)
        add_parts<8, kFewTokens, false>(acc, acc, parts, p.T, all_tokens, part);
      else
        add_parts<N == 16 ? 4 : 2, N, false>(acc, acc, parts, p.T, all_tokens, part);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j < p.T) p.y[static_cast<size_t>(j) * p.dim + tl * 128 + row] = __float2bfloat16_rn(acc[j]);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    // (No role sets it any more.) Copies and MMAs in flight are waited for
    // (bounded) before the CTA ends.
    if (producer) {
#pragma unroll 1
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        wait(&full[i % kStages], (i / kStages) & 1, nullptr, p.err);
#pragma unroll 1
      for (int s = 0; s < kStages; ++s)
        if ((tokens_armed.used >> s) & 1u) wait(&tok_full[s], (tokens_armed.parity >> s) & 1, nullptr, p.err);
    }
    if (warp == kIssuer) {
      if (elect_one_sync()) mma_commit(drain);
      __syncwarp();
      wait(drain, 0, nullptr, p.err);
      __syncwarp();
    }
  }
  if (warp == kIssuer) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  // The last CTA to leave zeroes the counters for the next call. (After a wait
  // that gave up, in whichever CTA, the row tiles' may hold a part of a count.)
  if (tid == 0 && atomicAdd(p.counters + 3, 1u) == static_cast<unsigned>(G) - 1u)
    for (int i = 0; i < 32; ++i) p.counters[i] = 0;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn layer_map_encoder() {
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

// e4m3 rows x cols, boxes of 128 columns x box_rows, 128-byte swizzled; rows past
// the end read as zeros.
bool make_code_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn enc = layer_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

struct LayerSizes {
  int64_t active;  // experts at most
  int cols;        // token columns
  size_t logits, ids, weights, xq, xs, uq, us, units, part, part2, total;
};

LayerSizes layer_sizes(int64_t T, int64_t dim, int64_t inter, int64_t E, int64_t topk, int64_t ns) {
  LayerSizes z{};
  z.active = (T * topk < E ? T * topk : E) + ns;
  z.cols = T <= 16 ? 16 : 32;
  z.logits = 256;
  z.ids = z.logits + align256(static_cast<size_t>(T) * E * 4);
  z.weights = z.ids + align256(static_cast<size_t>(T) * topk * 4);
  z.xq = z.weights + align256(static_cast<size_t>(T) * topk * 4);
  z.xs = z.xq + align256(static_cast<size_t>(T) * dim);
  z.uq = z.xs + align256(static_cast<size_t>(dim / 128) * z.cols * 4);
  z.us = z.uq + align256(static_cast<size_t>(z.active) * T * inter);
  z.units = z.us + align256(static_cast<size_t>(z.active) * (inter / 128) * z.cols * 4);
  z.part = z.units + align256(static_cast<size_t>(z.active) * (inter / 128) * 4);
  z.part2 = z.part + static_cast<size_t>(kMaxCtas) * 4 * 2 * T * 128 * 4;
  z.total = z.part2 + static_cast<size_t>(kMaxCtas) * 2 * T * 128 * 4;
  return z;
}

bool layer_shape_ok(int64_t T, int64_t dim, int64_t inter, int64_t E, int64_t topk, int64_t ns) {
  return T >= 0 && T <= kMaxTokens && dim >= 128 && dim <= kMaxDim && dim % 128 == 0 && inter >= 128 &&
         inter <= kMaxInter && inter % 128 == 0 && E >= 32 && E <= 256 && E % 32 == 0 && topk >= 1 && topk <= 32 &&
         ns >= 0 && ns <= kMaxShared;
}

template <int N>
int layer_launch(const DevInfo* d, const CUtensorMap& m1, const CUtensorMap& m3, const CUtensorMap& m2,
                 const CUtensorMap& mx, const CUtensorMap& mu, const LayerParams& p, cudaStream_t stream) {
  static bool attr_done[64] = {};
  auto kern = moe_layer_kernel<N>;
  if (d->device >= 64 || !attr_done[d->device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, layer_smem(N)) != cudaSuccess)
      return FP8BLK_ERR_CUDA;
    if (d->device < 64) attr_done[d->device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d->sm_count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = layer_smem(N);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, m1, m3, m2, mx, mu, p));
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_moe_layer_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t dim, int64_t inter,
                                                   int64_t n_shared) {
  if (!layer_shape_ok(T, dim, inter, E, topk, n_shared)) return 0;
  return layer_sizes(T, dim, inter, E, topk, n_shared).total;
}

extern "C" int fp8blk_moe_layer(const void* x_bf16, const void* gate_w_bf16, const float* gate_bias,
                                const void* w1_e4m3, const float* w1_s, const void* w3_e4m3, const float* w3_s,
                                const void* w2_e4m3, const float* w2_s, void* y_bf16, int64_t T, int64_t topk,
                                int64_t E, int64_t dim, int64_t inter, int64_t n_shared, int64_t n_groups,
                                int64_t topk_groups, int score_func, float route_scale, int normalize, int scale_fmt,
                                int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                                fp8blk_stream_t stream) {
  if (!scale_fmt_valid(scale_fmt)) return FP8BLK_ERR_ARG;
  if (int st = gate_shape_status(gate_bias, T, E, n_groups, topk_groups, topk, score_func, route_scale)) return st;
  if (!layer_shape_ok(T, dim, inter, E, topk, n_shared)) return FP8BLK_ERR_SHAPE;
  if (T == 0) return FP8BLK_OK;
  if (!x_bf16 || !gate_w_bf16 || !w1_e4m3 || !w1_s || !w3_e4m3 || !w3_s || !w2_e4m3 || !w2_s || !y_bf16)
    return FP8BLK_ERR_NULL;
  if (!is_aligned(x_bf16, 16) || !is_aligned(gate_w_bf16, 16) || !is_aligned(w1_e4m3, 16) ||
      !is_aligned(w3_e4m3, 16) || !is_aligned(w2_e4m3, 16) || !is_aligned(y_bf16, 2) || !is_aligned(w1_s, 4) ||
      !is_aligned(w3_s, 4) || !is_aligned(w2_s, 4) || !is_aligned(gate_bias, 4) || !is_aligned(topk_idx, 4) ||
      !is_aligned(topk_w, 4))
    return FP8BLK_ERR_ALIGN;
  if (!workspace) return FP8BLK_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return FP8BLK_ERR_ALIGN;
  const LayerSizes z = layer_sizes(T, dim, inter, E, topk, n_shared);
  if (workspace_bytes < z.total) return FP8BLK_ERR_WORKSPACE;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  if (d->sm_count > kMaxCtas) return FP8BLK_ERR_SHAPE;
  // The gate product keeps its share of an expert's row in registers.
  const int64_t per_cta = (E + d->sm_count - 1) / d->sm_count;
  if (per_cta > kWarps || dim / 8 > kWarps / per_cta * 32 * kGateVecs) return FP8BLK_ERR_SHAPE;
  LayerParams p{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.x = static_cast<const __nv_bfloat16*>(x_bf16);
  p.gate_w = static_cast<const __nv_bfloat16*>(gate_w_bf16);
  p.gate_bias = gate_bias;
  p.w1_s = w1_s;
  p.w3_s = w3_s;
  p.w2_s = w2_s;
  p.y = static_cast<__nv_bfloat16*>(y_bf16);
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.counters = reinterpret_cast<unsigned*>(ws);
  p.logits = reinterpret_cast<float*>(ws + z.logits);
  p.ids = reinterpret_cast<int*>(ws + z.ids);
  p.weights = reinterpret_cast<float*>(ws + z.weights);
  p.xq = ws + z.xq;
  p.xs = reinterpret_cast<float*>(ws + z.xs);
  p.uq = ws + z.uq;
  p.us = reinterpret_cast<float*>(ws + z.us);
  p.unit_parts = reinterpret_cast<unsigned*>(ws + z.units);
  p.max_units = static_cast<int>(z.active * (inter / 128));
  p.part = reinterpret_cast<float*>(ws + z.part);
  p.part2 = reinterpret_cast<float*>(ws + z.part2);
  p.err = d->err_word;
  p.T = static_cast<int>(T);
  p.dim = static_cast<int>(dim);
  p.inter = static_cast<int>(inter);
  p.E = static_cast<int>(E);
  p.ns = static_cast<int>(n_shared);
  p.k = static_cast<int>(topk);
  p.groups = static_cast<int>(n_groups);
  p.kept = static_cast<int>(topk_groups);
  p.sigmoid = score_func == FP8BLK_SCORE_SIGMOID;
  p.normalize = normalize != 0;
  p.ue8m0 = scale_fmt_ue8m0(scale_fmt);
  p.route_scale = route_scale;
  const uint64_t K = static_cast<uint64_t>(E + n_shared);
  CUtensorMap m1, m3, m2, mx, mu;
  if (!make_code_map(&m1, w1_e4m3, K * inter, dim, 128) || !make_code_map(&m3, w3_e4m3, K * inter, dim, 128) ||
      !make_code_map(&m2, w2_e4m3, K * dim, inter, 128) || !make_code_map(&mx, p.xq, T, dim, z.cols) ||
      !make_code_map(&mu, p.uq, static_cast<uint64_t>(z.active) * T, inter, z.cols))
    return FP8BLK_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return z.cols == 16 ? layer_launch<16>(d, m1, m3, m2, mx, mu, p, cs) : layer_launch<32>(d, m1, m3, m2, mx, mu, p, cs);
}
