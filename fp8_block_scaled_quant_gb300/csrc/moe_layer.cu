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
//   - One CTA per SM, one launch (cooperative: CTAs meet at three barriers).
//     Each of the CTA's sixteen warps owns 12 KB of shared memory and streams
//     and multiplies its own share of the weights: nothing but the phases'
//     ends makes warps wait for one another, so one warp's latencies hide
//     behind fifteen others. (A producer warp with stages that all sixteen
//     warps multiplied together, then met to add up, ran at 3.9 TB/s.)
//   - The gate decides what the routed weights are, but not the shared ones:
//     every warp asks for its share of the shared experts first, then x is
//     quantised and the gate computed.
//   - w2 does not depend on u, only its use does: a warp that is done with
//     its part of phase 1 asks for its first w2 tiles before the barriers.
//   - Phase 1 splits (expert, 8 rows of w1 and the same 8 of w3) evenly over
//     the CTAs, and a CTA's units, K laid end to end, evenly over its warps; a
//     unit cut between warps is added up in warp order. Phase 2 gives each CTA
//     the same rows of every expert's w2, and its (expert, K block) pairs round
//     robin to the warps: the sum over experts stays in registers. No atomics
//     on values, one order of every sum.
//
// The products are warp-level FP8 MMAs (m16n8k32): tokens are the 8 columns,
// so one MMA serves up to 8 tokens at the cost of one. In phase 1 rows 0-7 of
// an MMA tile are w1's and rows 8-15 w3's, so one lane ends with h1 and h3 of
// the same element. Each K block's product is promoted as acc += D * (a_s w_s).
// A tcgen05.mma with so few columns takes about 130 cycles for 4 KB of weights,
// 31 bytes a cycle, hardly the HBM rate of one SM (23); the warp MMAs take 64.
// Operand fragments as in the decode GEMM: lane (g, t) reads bytes [32 t, 32 t +
// 32) of a K block for row g, MMA j of the block takes bytes [8 j, 8 j + 8) of
// those, the same for both operands.
//
// Columns. In phase 1 they are an expert's tokens, closely packed (one tile of 8
// columns serves nearly every routed expert). In phase 2, whose accumulators
// run over the experts, they are the tokens 0-7, 8-15, ... themselves, and a
// tile without any token of the expert is skipped.
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
constexpr int kMaxRows = kMaxTokens * (32 + kMaxShared);  // (token, expert) pairs
constexpr int kWarps = 16;
constexpr int kMaxCtas = 192;                             // SMs a device may have
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroups = 4;                             // 16-row groups of w2 per CTA
constexpr int kMaxDim = 8192, kMaxInter = 16384;
constexpr int kWarpRing = 12288;                          // a warp's weight tiles
constexpr int kSlots = 3;                                 // at most
constexpr int kChunk = 2;                                 // K blocks of a phase-1 slot
constexpr int kSlot1 = kChunk * 2 * 1024;                 // 8 rows of w1 and of w3
constexpr int kGateVecs = 4;                              // 16-byte vectors of a gate row per thread

// Shared memory: rings, barriers, then the routing tables.
constexpr int kOffBar = kWarps * kWarpRing;
constexpr int kOffAct = kOffBar + kWarps * kSlots * 8 + 16;
constexpr int kOffMask = kOffAct + kMaxActive * 4;
constexpr int kOffBase = kOffMask + kMaxActive * 4;
constexpr int kOffRowW = kOffBase + (kMaxActive + 1) * 4;
constexpr int kOffRowT = kOffRowW + kMaxRows * 4;
constexpr int kOffSel = kOffRowT + kMaxRows;              // ids, weights of the pairs; scratch before
constexpr int kOffScan = kOffSel + 2 * kMaxTokens * 32 * 4;
constexpr int kLayerSmem = 1024 + kOffScan + 48 * 4;
static_assert(kLayerSmem <= 232448, "shared memory per CTA");

struct LayerParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* gate_w;
  const float* gate_bias;
  const float* w1_s;
  const float* w3_s;
  const float* w2_s;
  __nv_bfloat16* y;
  int32_t* topk_idx;  // may be null
  float* topk_w;      // may be null
  unsigned* counters;  // [0..2] barrier arrivals, [3] CTAs done; zero between calls
  float* logits;      // [T][E]
  uint8_t* xq;        // [T][dim]
  float* xs;          // [T][dim / 128]
  float* u;           // [rows][inter]
  uint8_t* uq;        // [rows][inter]
  float* us;          // [rows][inter / 128]
  float* part;        // [CTA][warp][4][16 rows x columns] sums of units cut between warps
  unsigned* err;
  int T, dim, inter, E, ns, k, groups, kept, sigmoid, normalize, ue8m0;
  float route_scale;
  int r2, slots2;  // rows of w2 per CTA at most, ring slots of that size
};

constexpr unsigned kDevErrTimeoutLayer = 1u << 9;

__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// d += A (16 x 32, rows) * B (32 x 8, columns), e4m3 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bounded wait, its slow part out of line (the loops that call it stay
// small enough for the instruction cache).
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

// Quantises one 128-element block, four elements per lane; lane 0 stores the scale.
__device__ __forceinline__ void quant_block(const float (&v)[4], bool ue8m0, int lane, uint8_t* q, float* s) {
  float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const float sc = block_scale(amax, ue8m0);
  const uint32_t lo = e4m3x2(__fdiv_rn(v[0], sc), __fdiv_rn(v[1], sc));
  const uint32_t hi = e4m3x2(__fdiv_rn(v[2], sc), __fdiv_rn(v[3], sc));
  reinterpret_cast<uint32_t*>(q)[lane] = lo | (hi << 16);
  if (lane == 0) *s = sc;
}

// First unit of part c of G when n units are split evenly (n * c stays below
// 2^31: at most 264 experts x 2048 units x 192 CTAs).
__device__ __forceinline__ int even(int n, int c, int G) {
  return static_cast<int>(static_cast<uint32_t>(n) * static_cast<uint32_t>(c) / static_cast<uint32_t>(G));
}

// First routed unit of CTA c, such that shared and routed units together are
// split evenly (`us` shared units are split evenly by themselves).
__device__ __forceinline__ int routed_start(int us, int ur, int c, int G) {
  if (ur < 2 * G) return even(ur, c, G);
  return even(us + ur, c, G) - even(us, c, G);
}

// The B fragment of one K block for 8 columns and the columns' scales.
struct Frag {
  uint4 b0, b1;
  float s0, s1;
};

// One K block of a 16-row tile: rows g of `lo` and of `hi` (128-byte swizzled
// rows of 128 bytes), promoted into acc with the rows' weight scales.
__device__ __forceinline__ void block_product(const uint8_t* lo, const uint8_t* hi, const Frag& f, float wlo, float whi,
                                              int g, int t4, float (&acc)[4]) {
  uint4 al[2], ah[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = g * 128 + (((2 * t4 + h) ^ g) << 4);
    al[h] = *reinterpret_cast<const uint4*>(lo + at);
    ah[h] = *reinterpret_cast<const uint4*>(hi + at);
  }
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  mma_16x8x32(d, al[0].x, ah[0].x, al[0].y, ah[0].y, f.b0.x, f.b0.y);
  mma_16x8x32(d, al[0].z, ah[0].z, al[0].w, ah[0].w, f.b0.z, f.b0.w);
  mma_16x8x32(d, al[1].x, ah[1].x, al[1].y, ah[1].y, f.b1.x, f.b1.y);
  mma_16x8x32(d, al[1].z, ah[1].z, al[1].w, ah[1].w, f.b1.z, f.b1.w);
  acc[0] = fmaf(d[0], f.s0 * wlo, acc[0]);
  acc[1] = fmaf(d[1], f.s1 * wlo, acc[1]);
  acc[2] = fmaf(d[2], f.s0 * whi, acc[2]);
  acc[3] = fmaf(d[3], f.s1 * whi, acc[3]);
}

__device__ __forceinline__ float silu_mul(float h1, float h3) { return h1 / (1.0f + expf(-h1)) * h3; }

// Ids and weights of token m by one warp, into the pair tables.
__device__ __noinline__ void gate_of_token(const LayerParams& p, int m, int lane, bool store, int* sel_e, float* sel_w) {
  const int v = p.E / 32;
  float xl[8], bl[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xl[i] = i < v ? __ldcg(p.logits + static_cast<size_t>(m) * p.E + lane * v + i) : 0.f;
    bl[i] = i < v && p.gate_bias ? __ldg(p.gate_bias + lane * v + i) : 0.f;
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

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map3,
                     const __grid_constant__ CUtensorMap map2, const __grid_constant__ LayerParams p) {
  constexpr int kCols = 8 * NT;
  constexpr int kTile = 16 * kCols;  // sums of a 16-row tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + kWarps * kSlots * 8);
  int* act = reinterpret_cast<int*>(smem + kOffAct);             // active experts, shared ones first
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + kOffMask);  // tokens; by expert id until sorted
  int* base = reinterpret_cast<int*>(smem + kOffBase);           // first (token, expert) row; one past the last
  float* row_w = reinterpret_cast<float*>(smem + kOffRowW);      // gate weight of each row
  uint8_t* row_t = smem + kOffRowT;                              // token of each row
  int* sel_e = reinterpret_cast<int*>(smem + kOffSel);
  float* sel_w = reinterpret_cast<float*>(sel_e + kMaxTokens * 32);
  int* scan = reinterpret_cast<int*>(smem + kOffScan);  // [16] active, [16] rows, active experts, rows

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = gridDim.x, c = blockIdx.x;
  const int Kb1 = p.dim / 128, Kb2 = p.inter / 128;
  const int chunks = (Kb1 + kChunk - 1) / kChunk;  // phase-1 slots of a unit
  const int upe = p.inter / 8;                     // units of an expert
  const int d0 = even(p.dim / 8, c, G) * 8, d1 = even(p.dim / 8, c + 1, G) * 8;  // this CTA's rows of w2
  const int ngroups = (d1 - d0 + 15) / 16;
  const uint32_t all_tokens = p.T == 32 ? 0xFFFFFFFFu : (1u << p.T) - 1u;
  uint8_t* ring = smem + warp * kWarpRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar) + warp * kSlots;
  uint32_t phase = 0;  // bit s: phase of slot s

  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  if (tid == 0) *abort_flag = 0;
  __syncwarp();

  // The gate rows of this CTA's experts, asked for before the weight stream
  // fills the memory's queues. The experts share the warps, each with a slice of
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

  // This warp's phase-1 slots: first of the shared units, then of the routed
  // ones, each a range of chunks of the CTA's units. A cursor walks a range.
  struct Cursor {
    int a, rb, ck, left;  // active expert, its 8-row block, chunk of K; chunks left
  };
  auto cursor = [&](int first, int u0, int q0, int q1) {
    const int u = u0 + q0 / chunks;
    return Cursor{first + u / upe, u % upe, q0 % chunks, q1 - q0};
  };
  auto advance = [&](Cursor& k, int n) {
    k.left -= n;
    k.ck += n;
    if (k.ck == chunks) {
      k.ck = 0;
      if (++k.rb == upe) {
        k.rb = 0;
        ++k.a;
      }
    }
  };
  const int us0 = even(p.ns * upe, c, G), us1 = even(p.ns * upe, c + 1, G);
  const int sq0 = even((us1 - us0) * chunks, warp, kWarps), sq1 = even((us1 - us0) * chunks, warp + 1, kWarps);
  const uint64_t policy = l2_policy_evict_first();  // weights are read once
  int put = 0;                                      // the slot that the next copy goes to
  Cursor ahead = cursor(0, us0, sq0, sq1);          // of the copies
  auto issue1 = [&] {
    if (elect_one_sync()) {
      const int y = (ahead.a < p.ns ? p.E + ahead.a : act[ahead.a]) * p.inter + ahead.rb * 8, z = ahead.ck * kChunk;
      uint8_t* dst = ring + put * kSlot1;
      mbar_arrive_expect_tx(&full[put], kSlot1);
      tma_load_3d_hint(dst, &map1, &full[put], 0, y, z, policy);
      tma_load_3d_hint(dst + kSlot1 / 2, &map3, &full[put], 0, y, z, policy);
    }
    __syncwarp();
    put = put + 1 == kSlots ? 0 : put + 1;
    advance(ahead, 1);
  };
#pragma unroll 1
  for (int q = 0; q < kSlots && ahead.left > 0; ++q) issue1();

  // Grid barrier i: every CTA's threads have arrived, their global writes are visible.
  auto grid_barrier = [&](int i) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      atomicAdd(p.counters + i, 1u);
      const uint64_t t0 = global_timer_ns();
#pragma unroll 1
      for (uint32_t spin = 0;; ++spin) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.counters + i) : "memory");
        if (v >= static_cast<unsigned>(G)) break;
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
    }
    __syncthreads();
  };

  // Phase 0: x quantised and the logits formed, both spread over the grid. A
  // CTA's experts share its warps, each with a slice of K.
#pragma unroll 1
  for (int i = c * kWarps + warp; i < p.T * Kb1; i += G * kWarps) {
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x) + static_cast<size_t>(i) * 32 + lane);
    const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                        __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
    quant_block(v, p.ue8m0 != 0, lane, p.xq + static_cast<size_t>(i) * 128, p.xs + i);
  }
  {
    float* sums = sel_w;  // [warp][columns]
#pragma unroll 1
    for (int e0 = c; e0 < p.E; e0 += per_cta * G) {
      float acc[kCols];
#pragma unroll
      for (int m = 0; m < kCols; ++m) acc[m] = 0.f;
      // (The row's K is at most kGateVecs passes, see kMaxDim.)
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
        if (m < p.T) {
          const uint4* xv = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(m) * p.dim) + v0;
#pragma unroll
          for (int i = 0; i < kGateVecs; ++i)
            if (v0 + i * step < vecs) {
              const uint4 b = __ldg(xv + i * step);
              const uint32_t aw[4] = {gate_row[i].x, gate_row[i].y, gate_row[i].z, gate_row[i].w};
              const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                acc[m] = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(bw[q] << 16), acc[m]);
                acc[m] = fmaf(__uint_as_float(aw[q] & 0xFFFF0000u), __uint_as_float(bw[q] & 0xFFFF0000u), acc[m]);
              }
            }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
          if (lane == 0) sums[warp * kCols + m] = acc[m];
        }
      }
      __syncthreads();
      for (int i = tid; i < per_cta * p.T; i += kThreads) {
        const int k = i / p.T, m = i % p.T;
        float v = 0.f;
        for (int w = 0; w < wpe; ++w) v += sums[(k * wpe + w) * kCols + m];
        if (e0 + k * G < p.E) p.logits[static_cast<size_t>(m) * p.E + e0 + k * G] = v;
      }
      __syncthreads();
      if (e0 + per_cta * G < p.E) load_gate(e0 + per_cta * G + warp / wpe * G);
    }
  }
  grid_barrier(0);

  // The gate, by every CTA for itself, then the tables: tokens of each expert,
  // active experts in order (shared ones first), their rows.
#pragma unroll 1
  for (int m = warp; m < p.T; m += kWarps) gate_of_token(p, m, lane, c == 0, sel_e, sel_w);
  uint32_t* tokens_of = reinterpret_cast<uint32_t*>(base);  // by expert id, until the scan
  for (int e = tid; e < p.E; e += kThreads) tokens_of[e] = 0;
  __syncthreads();
  const int pairs = p.T * p.k;
  for (int i = tid; i < pairs; i += kThreads) atomicOr(&tokens_of[sel_e[i]], 1u << (i / p.k));
  __syncthreads();
  const uint32_t my_tokens = tid < p.E ? tokens_of[tid] : 0;
  const unsigned have = __ballot_sync(0xFFFFFFFFu, my_tokens != 0);
  int upto = __popc(my_tokens);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) {
    scan[warp] = __popc(have);
    scan[16 + warp] = upto;
  }
  __syncthreads();  // every thread has its tokens: base may be written
  int a0 = p.ns, r0 = p.ns * p.T;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    a0 += w < warp ? scan[w] : 0;
    r0 += w < warp ? scan[16 + w] : 0;
  }
  if (tid < p.ns) {
    act[tid] = p.E + tid;
    mask[tid] = all_tokens;
    base[tid] = tid * p.T;
  }
  for (int i = tid; i < p.ns * p.T; i += kThreads) {
    row_w[i] = 1.0f;
    row_t[i] = static_cast<uint8_t>(i % p.T);
  }
  if (my_tokens) {
    const int a = a0 + __popc(have & ((1u << lane) - 1u));
    const int r = r0 + upto - __popc(my_tokens);
    act[a] = tid;
    mask[a] = my_tokens;
    base[a] = r;
    int k = r;
    for (uint32_t left = my_tokens; left; left &= left - 1, ++k) {
      const int m = __ffs(left) - 1;
      row_t[k] = static_cast<uint8_t>(m);
      float w = 0.f;
      for (int j = 0; j < p.k; ++j)
        if (sel_e[m * p.k + j] == tid) w = sel_w[m * p.k + j];
      row_w[k] = w;
    }
  }
  if (tid == kThreads - 1) {
    scan[32] = a0 + __popc(have);
    scan[33] = r0 + upto;
  }
  __syncthreads();
  const int nact = scan[32], nrows = scan[33];
  const int routed_units = (nact - p.ns) * upe;
  const int ur0 = routed_start(p.ns * upe, routed_units, c, G), ur1 = routed_start(p.ns * upe, routed_units, c + 1, G);
  const int rq0 = even((ur1 - ur0) * chunks, warp, kWarps), rq1 = even((ur1 - ur0) * chunks, warp + 1, kWarps);
  bool ahead_routed = false;
  auto issue_next = [&] {  // the next copy, if any: the shared range's, then the routed one's
    if (ahead.left == 0 && !ahead_routed) {
      ahead = cursor(p.ns, ur0, rq0, rq1);
      ahead_routed = true;
    }
    if (ahead.left > 0 && !*abort_flag) issue1();
  };
#pragma unroll 1
  for (int q = min(kSlots, sq1 - sq0); q < kSlots; ++q) issue_next();

  // Phase 1: u = silu(w1 x) (w3 x).
  auto store_u = [&](int a, int rb, int cnt, int nt, const float (&v)[4]) {
    // Lane (g, t4) has columns 2 t4, 2 t4 + 1 of row g: h1 and h3.
    const int col = nt * 8 + 2 * t4;
    float* dst = p.u + static_cast<size_t>(base[a] + col) * p.inter + rb * 8 + g;
    if (col < cnt) dst[0] = silu_mul(v[0], v[2]);
    if (col + 1 < cnt) dst[p.inter] = silu_mul(v[1], v[3]);
  };
  int take = 0;  // the slot that is multiplied next
#pragma unroll 1
  for (int range = 0; range < 2; ++range) {
    Cursor at = range ? cursor(p.ns, ur0, rq0, rq1) : cursor(0, us0, sq0, sq1);
#pragma unroll 1
    while (at.left > 0) {
      // One unit, or the part of it that falls to this warp.
      const int n = min(at.left, chunks - at.ck);
      const int cnt = __popc(mask[at.a]), rows0 = base[at.a];
      const float* s1 = p.w1_s + static_cast<size_t>((act[at.a] * upe + at.rb) / 16) * Kb1;
      const float* s3 = p.w3_s + (s1 - p.w1_s);
      // Column tile 0's tokens: this lane's operand row and the two columns it scales.
      const bool c0 = g < cnt, c1 = 2 * t4 < cnt, c2 = 2 * t4 + 1 < cnt;
      const uint8_t* x0 = p.xq + static_cast<size_t>(c0 ? row_t[rows0 + g] : 0) * p.dim + t4 * 32;
      const float* xs1 = p.xs + (c1 ? row_t[rows0 + 2 * t4] : 0) * Kb1;
      const float* xs2 = p.xs + (c2 ? row_t[rows0 + 2 * t4 + 1] : 0) * Kb1;
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int kb0 = (at.ck + j) * kChunk;
        Frag f[kChunk];
        float wlo[kChunk], whi[kChunk];
#pragma unroll
        for (int h = 0; h < kChunk; ++h) {
          const int kb = min(kb0 + h, Kb1 - 1);  // past K: the weights are zeros
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          f[h].b0 = c0 ? __ldcg(reinterpret_cast<const uint4*>(x0 + kb * 128)) : zero;
          f[h].b1 = c0 ? __ldcg(reinterpret_cast<const uint4*>(x0 + kb * 128) + 1) : zero;
          f[h].s0 = c1 ? __ldcg(xs1 + kb) : 0.f;
          f[h].s1 = c2 ? __ldcg(xs2 + kb) : 0.f;
          wlo[h] = __ldg(s1 + kb);
          whi[h] = __ldg(s3 + kb);
        }
        const uint8_t* w = ring + take * kSlot1;
        wait(&full[take], (phase >> take) & 1, abort_flag, p.err);
        phase ^= 1u << take;
        take = take + 1 == kSlots ? 0 : take + 1;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kChunk; ++h)
          block_product(w + h * 1024, w + kSlot1 / 2 + h * 1024, f[h], wlo[h], whi[h], g, t4, acc[0]);
#pragma unroll
        for (int nt = 1; nt < NT; ++nt) {
          if (nt * 8 >= cnt) break;
#pragma unroll
          for (int h = 0; h < kChunk; ++h) {
            const int kb = min(kb0 + h, Kb1 - 1), col = nt * 8 + g, cs = nt * 8 + 2 * t4;
            Frag x;
            x.b0 = x.b1 = make_uint4(0u, 0u, 0u, 0u);
            if (col < cnt) {
              const uint4* src = reinterpret_cast<const uint4*>(p.xq + static_cast<size_t>(row_t[rows0 + col]) * p.dim +
                                                                kb * 128 + t4 * 32);
              x.b0 = __ldcg(src);
              x.b1 = __ldcg(src + 1);
            }
            x.s0 = cs < cnt ? __ldcg(p.xs + row_t[rows0 + cs] * Kb1 + kb) : 0.f;
            x.s1 = cs + 1 < cnt ? __ldcg(p.xs + row_t[rows0 + cs + 1] * Kb1 + kb) : 0.f;
            block_product(w + h * 1024, w + kSlot1 / 2 + h * 1024, x, wlo[h], whi[h], g, t4, acc[nt]);
          }
        }
        __syncwarp();
        issue_next();
      }
      if (n == chunks) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (nt * 8 < cnt) store_u(at.a, at.rb, cnt, nt, acc[nt]);
      } else {  // sums of a cut unit: [range][it starts here]
        float4* t = reinterpret_cast<float4*>(p.part + ((static_cast<size_t>(c) * kWarps + warp) * 4 + range * 2 +
                                                        (at.ck == 0 ? 1 : 0)) * kTile) + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (nt * 8 < cnt) t[nt * 32] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
      }
      advance(at, n);
    }
  }

  // The first w2 tiles. Item i is K block i % Kb2 of active expert i / Kb2; this
  // warp has items warp, warp + 16, ...
  struct Item {
    int a, kb;
  };
  auto next_item = [&](Item& k) {
    k.kb += kWarps;
    while (k.kb >= Kb2) {
      k.kb -= Kb2;
      ++k.a;
    }
  };
  Item item_ahead{warp / Kb2, warp % Kb2};
  put = 0;
  auto issue2 = [&] {
    if (item_ahead.a >= nact || *abort_flag) return;
    if (elect_one_sync()) {
      mbar_arrive_expect_tx(&full[put], static_cast<uint32_t>(p.r2) * 128);
      tma_load_3d_hint(ring + put * p.r2 * 128, &map2, &full[put], 0, act[item_ahead.a] * p.dim + d0, item_ahead.kb,
                       policy);
    }
    __syncwarp();
    put = put + 1 == p.slots2 ? 0 : put + 1;
    next_item(item_ahead);
  };
#pragma unroll 1
  for (int q = 0; q < p.slots2; ++q) issue2();

  // Units cut between warps: warp w adds up units w, w + 16, ... of the CTA.
  __syncthreads();
#pragma unroll 1
  for (int range = 0; range < 2; ++range) {
    const int u0 = range ? ur0 : us0, n = (range ? ur1 : us1) - u0, total = n * chunks;
#pragma unroll 1
    for (int k = warp; k < n; k += kWarps) {
      // The warp of chunk x is the largest w with even(total, w) <= x.
      const int w0 = ((k * chunks + 1) * kWarps - 1) / total;
      const int w1 = ((k + 1) * chunks * kWarps - 1) / total;
      if (w0 == w1) continue;
      const int u = u0 + k, a = (range ? p.ns : 0) + u / upe, cnt = __popc(mask[a]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= cnt) break;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int w = w0; w <= w1; ++w) {
          const int from = even(total, w, kWarps);
          if (from == even(total, w + 1, kWarps)) continue;  // fewer chunks than warps: this one has none
          const float4 x = __ldcg(reinterpret_cast<const float4*>(
                                      p.part + ((static_cast<size_t>(c) * kWarps + w) * 4 + range * 2 +
                                                (from <= k * chunks ? 1 : 0)) * kTile) +
                                  nt * 32 + lane);
          v[0] += x.x;
          v[1] += x.y;
          v[2] += x.z;
          v[3] += x.w;
        }
        store_u(a, u % upe, cnt, nt, v);
      }
    }
  }
  grid_barrier(1);
#pragma unroll 1
  for (int i = c * kWarps + warp; i < nrows * Kb2; i += G * kWarps) {
    const float4 raw = __ldcg(reinterpret_cast<const float4*>(p.u) + static_cast<size_t>(i) * 32 + lane);
    const float v[4] = {raw.x, raw.y, raw.z, raw.w};
    quant_block(v, p.ue8m0 != 0, lane, p.uq + static_cast<size_t>(i) * 128, p.us + i);
  }
  grid_barrier(2);

  // Phase 2: this CTA's rows of every active expert's w2, weighted and summed
  // over the experts in the accumulators.
  float acc[kMaxGroups][NT][4];
#pragma unroll
  for (int q = 0; q < kMaxGroups; ++q)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[q][nt][0] = acc[q][nt][1] = acc[q][nt][2] = acc[q][nt][3] = 0.f;
  // Weight-scale rows of the groups' low and high halves within an expert.
  int slo[kMaxGroups], shi[kMaxGroups];
#pragma unroll
  for (int q = 0; q < kMaxGroups; ++q) {
    slo[q] = (d0 + q * 16) / 128 * Kb2;
    shi[q] = (d0 + q * 16 + 8) / 128 * Kb2;
  }
  const bool odd = ((d1 - d0) & 8) != 0;  // the last group has no high half
  take = 0;
#pragma unroll 1
  for (Item it{warp / Kb2, warp % Kb2}; it.a < nact; next_item(it)) {
    const int a = it.a, kb = it.kb;
    const uint32_t mk = mask[a];
    const int r_base = base[a];
    const float* ws = p.w2_s + static_cast<size_t>(act[a]) * (p.dim / 128) * Kb2 + kb;
    auto frag = [&](int nt) {
      Frag f;
      f.b0 = f.b1 = make_uint4(0u, 0u, 0u, 0u);
      f.s0 = f.s1 = 0.f;
      const int m = nt * 8 + g, m2 = nt * 8 + 2 * t4;
      const int r = r_base + __popc(mk & ((1u << m) - 1u)), r2 = r_base + __popc(mk & ((1u << m2) - 1u));
      if ((mk >> m) & 1u) {
        const uint4* src = reinterpret_cast<const uint4*>(p.uq + static_cast<size_t>(r) * p.inter + kb * 128 + t4 * 32);
        f.b0 = __ldcg(src);
        f.b1 = __ldcg(src + 1);
      }
      const int r3 = r2 + ((mk >> m2) & 1u);
      if ((mk >> m2) & 1u) f.s0 = __ldcg(p.us + r2 * Kb2 + kb) * row_w[r2];
      if ((mk >> (m2 + 1)) & 1u) f.s1 = __ldcg(p.us + r3 * Kb2 + kb) * row_w[r3];
      return f;
    };
    float wlo[kMaxGroups], whi[kMaxGroups];
#pragma unroll
    for (int q = 0; q < kMaxGroups; ++q) {
      wlo[q] = q < ngroups ? __ldg(ws + slo[q]) : 0.f;
      whi[q] = q < ngroups && !(odd && q == ngroups - 1) ? __ldg(ws + shi[q]) : 0.f;
    }
    Frag f0;
    if (NT == 1) f0 = frag(0);
    const uint8_t* w = ring + take * p.r2 * 128;
    wait(&full[take], (phase >> take) & 1, abort_flag, p.err);
    phase ^= 1u << take;
    take = take + 1 == p.slots2 ? 0 : take + 1;
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1 && !((mk >> (nt * 8)) & 0xFFu)) continue;
      const Frag f = NT == 1 ? f0 : frag(nt);
#pragma unroll
      for (int q = 0; q < kMaxGroups; ++q)
        if (q < ngroups) {
          // A last group of 8 rows takes them twice; the second copy has scale 0.
          const uint8_t* lo = w + q * 2048;
          block_product(lo, odd && q == ngroups - 1 ? lo : lo + 1024, f, wlo[q], whi[q], g, t4, acc[q][nt]);
        }
    }
    __syncwarp();
    issue2();
  }
  __syncthreads();
  // Every warp's copies have landed and are used: the rings hold the warps'
  // sums [warp][row][columns] now (a copy still in flight after a wait that
  // gave up is waited for first).
  if (*abort_flag) {
    for (int i = 0; i < kSlots; ++i) wait(&full[i], (phase >> i) & 1, nullptr, p.err);
    __syncthreads();
  }
  float* sums = reinterpret_cast<float*>(smem);
  const int rows2 = ngroups * 16;
#pragma unroll
  for (int q = 0; q < kMaxGroups; ++q)
    if (q < ngroups)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* t = sums + (warp * rows2 + q * 16 + g) * kCols + nt * 8 + 2 * t4;
        *reinterpret_cast<float2*>(t) = make_float2(acc[q][nt][0], acc[q][nt][1]);
        *reinterpret_cast<float2*>(t + 8 * kCols) = make_float2(acc[q][nt][2], acc[q][nt][3]);
      }
  __syncthreads();
  for (int i = tid; i < (d1 - d0) * p.T; i += kThreads) {
    const int m = i / (d1 - d0), r = i % (d1 - d0);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[(w * rows2 + r) * kCols + m];
    p.y[static_cast<size_t>(m) * p.dim + d0 + r] = __float2bfloat16_rn(v);
  }
  // The last CTA to leave zeroes the counters for the next call.
  if (tid == 0 && atomicAdd(p.counters + 3, 1u) == static_cast<unsigned>(G) - 1u) {
    p.counters[0] = p.counters[1] = p.counters[2] = 0;
    p.counters[3] = 0;
  }
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

// An e4m3 weight [N, K] as (128 bytes of a K block, row, K block), read in
// boxes of `rows` x kb blocks, 128-byte swizzled; blocks past K read as zeros.
bool make_weight_map(CUtensorMap* map, const void* w, uint64_t N, uint64_t K, uint32_t rows, uint32_t kb) {
  EncodeTiledFn enc = layer_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {128, N, K / 128};
  const cuuint64_t strides[2] = {K, 128};
  const cuuint32_t box[3] = {128, rows, kb};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

struct LayerSizes {
  size_t logits, xq, xs, u, uq, us, part, total;
};

LayerSizes layer_sizes(int64_t T, int64_t dim, int64_t inter, int64_t E, int64_t topk, int64_t ns) {
  LayerSizes z{};
  const size_t rows = static_cast<size_t>(T) * (topk + ns);
  z.logits = 256;
  z.xq = z.logits + align256(static_cast<size_t>(T) * E * 4);
  z.xs = z.xq + align256(static_cast<size_t>(T) * dim);
  z.u = z.xs + align256(static_cast<size_t>(T) * (dim / 128) * 4);
  z.uq = z.u + align256(rows * inter * 4);
  z.us = z.uq + align256(rows * inter);
  z.part = z.us + align256(rows * (inter / 128) * 4);
  const size_t cols = T <= 8 ? 8 : T <= 16 ? 16 : 32;
  z.total = z.part + static_cast<size_t>(kMaxCtas) * kWarps * 4 * 16 * cols * 4;
  return z;
}

bool layer_shape_ok(int64_t T, int64_t dim, int64_t inter, int64_t E, int64_t topk, int64_t ns) {
  return T >= 0 && T <= kMaxTokens && dim >= 128 && dim <= kMaxDim && dim % 128 == 0 && inter >= 128 &&
         inter <= kMaxInter && inter % 128 == 0 && E >= 32 && E <= 256 && E % 32 == 0 && topk >= 1 && topk <= 32 &&
         ns >= 0 && ns <= kMaxShared;
}

template <int NT>
int layer_launch(const DevInfo* d, const CUtensorMap& m1, const CUtensorMap& m3, const CUtensorMap& m2,
                 const LayerParams& p, cudaStream_t stream) {
  static bool attr_done[64] = {};
  auto kern = moe_layer_kernel<NT>;
  if (d->device >= 64 || !attr_done[d->device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLayerSmem) != cudaSuccess)
      return FP8BLK_ERR_CUDA;
    if (d->device < 64) attr_done[d->device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d->sm_count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kLayerSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, m1, m3, m2, p));
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
  // Phase 2 keeps a CTA's rows of w2 in its accumulators.
  if ((dim / 8 + d->sm_count - 1) / d->sm_count > 2 * kMaxGroups || d->sm_count > kMaxCtas) return FP8BLK_ERR_SHAPE;
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
  p.xq = ws + z.xq;
  p.xs = reinterpret_cast<float*>(ws + z.xs);
  p.u = reinterpret_cast<float*>(ws + z.u);
  p.uq = ws + z.uq;
  p.us = reinterpret_cast<float*>(ws + z.us);
  p.part = reinterpret_cast<float*>(ws + z.part);
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
  p.r2 = static_cast<int>((dim / 8 + d->sm_count - 1) / d->sm_count) * 8;
  p.slots2 = kWarpRing / (p.r2 * 128);
  if (p.slots2 > kSlots) p.slots2 = kSlots;
  const uint64_t K = static_cast<uint64_t>(E + n_shared);
  CUtensorMap m1, m3, m2;
  if (!make_weight_map(&m1, w1_e4m3, K * inter, dim, 8, kChunk) ||
      !make_weight_map(&m3, w3_e4m3, K * inter, dim, 8, kChunk) ||
      !make_weight_map(&m2, w2_e4m3, K * dim, inter, static_cast<uint32_t>(p.r2), 1))
    return FP8BLK_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return T <= 8    ? layer_launch<1>(d, m1, m3, m2, p, cs)
         : T <= 16 ? layer_launch<2>(d, m1, m3, m2, p, cs)
                   : layer_launch<4>(d, m1, m3, m2, p, cs);
}
