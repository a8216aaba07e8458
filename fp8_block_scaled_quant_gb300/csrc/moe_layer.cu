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
//     Each of the CTA's sixteen warps owns 12.5 KB of shared memory and streams
//     and multiplies its own share of the weights, 2 KB (16 rows of a K block)
//     at a time, three such slots in flight (cp.async), the tokens' codes and all
//     scales in the slot beside them: nothing but the phases' ends makes warps
//     wait for one another, so one warp's latencies hide behind fifteen others.
//     (Stages that all warps multiplied together ran at 3.9 TB/s; the same slots
//     by TMA cost a warp 400 cycles a copy to issue; operands by plain loads wait
//     behind the stream, 20 us of 100 for one token.)
//   - The gate decides what the routed weights are, but not the shared ones:
//     every warp asks for its share of the shared experts as soon as the gate's
//     operands are here, and the gate is computed meanwhile.
//   - w2 does not depend on u, only its use does: a warp's slots run on from
//     its part of phase 1 into w2 before the barriers between them.
//   - Phase 1 lays its units (expert, 8 rows of w1 and the same 8 of w3) end to
//     end, K block by K block, and gives every warp of the GPU the same number
//     of K blocks; the parts of a unit cut between warps are added in warp order
//     where u is quantised. Phase 2 gives each CTA the same rows of every
//     expert's w2, and its (expert, K block) pairs round robin to the warps: the
//     sum over experts stays in registers. No atomics on values, one order of
//     every sum.
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
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

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
constexpr int kSlots = 4;                                 // slots of a warp
constexpr int kOffTok = 2048;                             // after 16 weight rows x 128 bytes: 8 tokens' codes
constexpr int kOffScl = 3072;                             // 8 token scales, 2 weight scales
constexpr int kSlot = 3200;
constexpr int kWarpRing = kSlots * kSlot;
constexpr int kGateVecs = 4;                              // 16-byte vectors of a gate row per thread

// Shared memory: the rings, then the routing tables.
constexpr int kOffAct = kWarps * kWarpRing + 16;
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
  float* part;        // [warp of the grid][range][it starts the unit][16 rows x columns]: sums of cut units
  unsigned* err;
  int T, dim, inter, E, ns, k, groups, kept, sigmoid, normalize, ue8m0;
  float route_scale;
  const uint8_t* w1;  // weights
  const uint8_t* w3;
  const uint8_t* w2;
};

constexpr unsigned kDevErrTimeoutLayer = 1u << 9;

// 16 bytes from global to shared memory, past the L1 cache.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_plain(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's `N` latest groups of copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d += A (16 x 32, rows) * B (32 x 8, columns), e4m3 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The same for large n (a K block count times a warp index).
__device__ __forceinline__ int even_wide(int n, int c, int G) {
  return static_cast<int>(static_cast<int64_t>(n) * c / G);
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
    moe_layer_kernel(const __grid_constant__ LayerParams p) {
  constexpr int kCols = 8 * NT;
  constexpr int kTile = 16 * kCols;  // sums of a 16-row tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kWarps * kWarpRing);
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
  const int upe = p.inter / 8;                     // units of an expert
  const int d0 = even(p.dim / 8, c, G) * 8, d1 = even(p.dim / 8, c + 1, G) * 8;  // this CTA's rows of w2
  const int ngroups = (d1 - d0 + 15) / 16;
  const uint32_t all_tokens = p.T == 32 ? 0xFFFFFFFFu : (1u << p.T) - 1u;
  uint8_t* ring = smem + warp * kWarpRing;
  if (tid == 0) *abort_flag = 0;

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

  // This warp's slots: K blocks of the shared units, then of the routed ones
  // (each range of units, K laid end to end, split evenly over the grid's
  // warps), then its w2 items, 16 rows at a time. A cursor walks a range.
  struct Cursor {
    int a, rb, kb, left;  // active expert, its 8-row block, K block; K blocks left
  };
  const int gw = c * kWarps + warp, W = G * kWarps;
  auto cursor = [&](int first, int blocks) {
    const int q0 = even_wide(blocks, gw, W), q1 = even_wide(blocks, gw + 1, W), u = q0 / Kb1;
    return Cursor{first + u / upe, u % upe, q0 % Kb1, q1 - q0};
  };
  auto advance = [&](Cursor& k) {
    --k.left;
    if (++k.kb == Kb1) {
      k.kb = 0;
      if (++k.rb == upe) {
        k.rb = 0;
        ++k.a;
      }
    }
  };
  const int shared_blocks = p.ns * upe * Kb1;
  // Item i of phase 2 is K block i % Kb2 of active expert i / Kb2; this warp has
  // items warp, warp + 16, ...
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
  // Copies: lane l has 16 bytes l % 8 of rows l / 8 and l / 8 + 4 of a slot's low
  // and high eight weight rows and of its eight tokens; chunk j of row r goes to
  // chunk j ^ r. Lanes 0-9 also have a scale each.
  const uint64_t policy = l2_policy_evict_first();  // weights are read once
  const int lane_row = lane >> 3, lane_byte = (lane & 7) * 16;
  const uint32_t ring_addr = smem_u32(ring);
  const uint32_t lane_dst = lane_row * 128 + (((lane & 7) ^ lane_row) << 4);
  int put = 0;  // the slot that the next copy goes to
  auto copy_weights = [&](const uint8_t* lo, const uint8_t* hi, int64_t pitch, bool has_hi) {
    const uint32_t dst = ring_addr + put * kSlot + lane_dst, dst4 = ring_addr + put * kSlot + (lane_dst ^ 64) + 512;
    copy16(dst, lo, policy);
    copy16(dst4, lo + 4 * pitch, policy);
    if (has_hi) {
      copy16(dst + 1024, hi, policy);
      copy16(dst4 + 1024, hi + 4 * pitch, policy);
    }
  };
  // What the tokens bring to a slot: codes of two of them, one scale.
  const uint8_t *tok0 = nullptr, *tok1 = nullptr;
  const float* scl = nullptr;
  auto copy_operands = [&](int slot) {
    const uint32_t at = ring_addr + slot * kSlot;
    if (tok0) copy16_plain(at + kOffTok + lane_dst, tok0);
    if (tok1) copy16_plain(at + kOffTok + (lane_dst ^ 64) + 512, tok1);
    if (scl) copy4(at + kOffScl + lane * 4, scl);
  };
  auto open_operands = [&](const Cursor& k) {
    const int cnt = __popc(mask[k.a]), rows0 = base[k.a];
    tok0 = lane_row < cnt ? p.xq + row_t[rows0 + lane_row] * p.dim + k.kb * 128 + lane_byte : nullptr;
    tok1 = lane_row + 4 < cnt ? p.xq + row_t[rows0 + lane_row + 4] * p.dim + k.kb * 128 + lane_byte : nullptr;
    const int srow = (act[k.a] * upe + k.rb) / 16 * Kb1 + k.kb;
    scl = lane < min(cnt, 8) ? p.xs + row_t[rows0 + lane] * Kb1 + k.kb
          : lane == 8        ? p.w1_s + srow
          : lane == 9        ? p.w3_s + srow
                             : nullptr;
  };
  Cursor ahead = cursor(0, shared_blocks);  // of the copies
  const uint8_t *src1 = nullptr, *src3 = nullptr;
  bool fresh = true;  // the sources are not the cursor's unit's yet
  auto copy_unit = [&](bool operands) {  // the slot at `ahead`
    if (fresh || ahead.kb == 0) {
      const int64_t row =
          static_cast<int64_t>(ahead.a < p.ns ? p.E + ahead.a : act[ahead.a]) * p.inter + ahead.rb * 8 + lane_row;
      const int64_t off = row * p.dim + ahead.kb * 128 + lane_byte;
      src1 = p.w1 + off;
      src3 = p.w3 + off;
      if (operands) open_operands(ahead);
      fresh = false;
    }
    copy_weights(src1, src3, p.dim, true);
    src1 += 128;
    src3 += 128;
    if (operands) {
      copy_operands(put);
      if (tok0) tok0 += 128;
      if (tok1) tok1 += 128;
      if (scl) ++scl;
    }
    put = put + 1 == kSlots ? 0 : put + 1;
    advance(ahead);
  };

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
  for (int i = warp * G + c; i < p.T * Kb1; i += G * kWarps) {
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x) + static_cast<size_t>(i) * 32 + lane);
    const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                        __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
    quant_block(v, p.ue8m0 != 0, lane, p.xq + static_cast<size_t>(i) * 128, p.xs + i);
  }
  // The shared experts' stream starts when the gate's operands are here (its
  // copies, asked for earlier, made the logits wait 4 us behind them).
  const int early = min(kSlots - 1, ahead.left);
  auto first_copies = [&] {
#pragma unroll 1
    for (int q = 0; q < early; ++q) {
      copy_unit(false);
      copy_commit();
    }
  };
  if (c >= p.E) first_copies();
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
      if (e0 == c) first_copies();
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
  const int routed_blocks = (nact - p.ns) * upe * Kb1;
  // The next slot's copies, one group: the shared units', the routed units',
  // w2's. Operands of w2 come with them once u is quantised.
  int stage = 0, group_ahead = 0, early2 = 0;
  const int nact2 = ngroups > 0 ? nact : 0;  // a CTA without rows of w2 has no items
  bool have_u = false;
  Item item_ahead{warp / Kb2, warp % Kb2};
  const uint8_t* src2 = nullptr;
  const int sblk = d0 / 128 * Kb2, sblk2 = (d1 - 1) / 128 * Kb2;  // the CTA's rows lie in one or two 128-row blocks
  auto open_item = [&](const Item& k) {
    const uint32_t mk = mask[k.a];
    const int m0 = NT == 1 ? 0 : (__ffs(mk) - 1) & ~7;  // its lowest column tile
    auto row_of = [&](int m) { return base[k.a] + __popc(mk & ((1u << m) - 1u)); };
    const int ma = m0 + lane_row, mb = ma + 4, ms = m0 + (lane & 7);
    tok0 = (mk >> ma) & 1u ? p.uq + static_cast<size_t>(row_of(ma)) * p.inter + k.kb * 128 + lane_byte : nullptr;
    tok1 = (mk >> mb) & 1u ? p.uq + static_cast<size_t>(row_of(mb)) * p.inter + k.kb * 128 + lane_byte : nullptr;
    const int srow = act[k.a] * (p.dim / 128) * Kb2 + k.kb;
    scl = lane < 8 ? ((mk >> ms) & 1u ? p.us + row_of(ms) * Kb2 + k.kb : nullptr)
          : lane == 8 ? p.w2_s + srow + sblk
          : lane == 9 ? p.w2_s + srow + sblk2
                      : nullptr;
  };
  auto copy_next = [&] {
    if (ahead.left == 0 && stage == 0) {
      stage = 1;
      ahead = cursor(p.ns, routed_blocks);
      fresh = true;
    }
    if (ahead.left > 0) {
      copy_unit(true);
    } else if (item_ahead.a < nact2) {
      if (group_ahead == 0) {
        src2 = p.w2 + (static_cast<int64_t>(act[item_ahead.a]) * p.dim + d0 + lane_row) * p.inter +
               item_ahead.kb * 128 + lane_byte;
        if (have_u) {
          open_item(item_ahead);
          copy_operands(put);
        }
      }
      copy_weights(src2, src2 + 8 * static_cast<int64_t>(p.inter), p.inter, d0 + group_ahead * 16 + 8 < d1);
      put = put + 1 == kSlots ? 0 : put + 1;
      early2 += have_u ? 0 : 1;
      src2 += 16 * static_cast<int64_t>(p.inter);
      if (++group_ahead == ngroups) {
        group_ahead = 0;
        next_item(item_ahead);
      }
    }
    copy_commit();
  };
  // Operands of the slots that were asked for before x was quantised.
  {
    Cursor k = cursor(0, shared_blocks);
#pragma unroll 1
    for (int q = 0; q < early; ++q) {
      open_operands(k);
      copy_operands(q);
      advance(k);
    }
    copy_commit();
    fresh = true;
  }
#pragma unroll 1
  for (int q = early; q < kSlots - 1; ++q) copy_next();
  copy_wait<0>();
  int take = 0;  // the slot that is multiplied next
  auto slot_ready = [&] {
    copy_wait<kSlots - 2>();
    __syncwarp();
    const uint8_t* w = ring + take * kSlot;
    take = take + 1 == kSlots ? 0 : take + 1;
    return w;
  };
  // Column 8-tile's fragment and scales of a slot.
  auto slot_frag = [&](const uint8_t* w) {
    Frag f;
    const uint8_t* x = w + kOffTok + g * 128;
    f.b0 = *reinterpret_cast<const uint4*>(x + (((2 * t4) ^ g) << 4));
    f.b1 = *reinterpret_cast<const uint4*>(x + (((2 * t4 + 1) ^ g) << 4));
    const float2 sc = *reinterpret_cast<const float2*>(w + kOffScl + t4 * 8);
    f.s0 = sc.x;
    f.s1 = sc.y;
    return f;
  };

  // Phase 1: u = silu(w1 x) (w3 x).
  auto store_u = [&](int a, int rb, int cnt, int nt, const float (&v)[4]) {
    // Lane (g, t4) has columns 2 t4, 2 t4 + 1 of row g: h1 and h3.
    const int col = nt * 8 + 2 * t4;
    float* dst = p.u + static_cast<size_t>(base[a] + col) * p.inter + rb * 8 + g;
    if (col < cnt) dst[0] = silu_mul(v[0], v[2]);
    if (col + 1 < cnt) dst[p.inter] = silu_mul(v[1], v[3]);
  };
#pragma unroll 1
  for (int range = 0; range < 2; ++range) {
    Cursor at = range ? cursor(p.ns, routed_blocks) : cursor(0, shared_blocks);
    if (at.left == 0) continue;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
    int from = at.kb, cnt = __popc(mask[at.a]);  // the unit's first K block here, its tokens
#pragma unroll 1
    while (true) {
      const uint8_t* w = slot_ready();
      const float2 ws = *reinterpret_cast<const float2*>(w + kOffScl + 32);
      block_product(w, w + 1024, slot_frag(w), ws.x, ws.y, g, t4, acc[0]);
#pragma unroll
      for (int nt = 1; nt < NT; ++nt) {
        if (nt * 8 >= cnt) break;
        const int rows0 = base[at.a], col = nt * 8 + g, cs = nt * 8 + 2 * t4;
        Frag x;
        x.b0 = x.b1 = make_uint4(0u, 0u, 0u, 0u);
        if (col < cnt) {
          const uint4* src = reinterpret_cast<const uint4*>(p.xq + row_t[rows0 + col] * p.dim + at.kb * 128 + t4 * 32);
          x.b0 = __ldcg(src);
          x.b1 = __ldcg(src + 1);
        }
        x.s0 = cs < cnt ? __ldcg(p.xs + row_t[rows0 + cs] * Kb1 + at.kb) : 0.f;
        x.s1 = cs + 1 < cnt ? __ldcg(p.xs + row_t[rows0 + cs + 1] * Kb1 + at.kb) : 0.f;
        block_product(w, w + 1024, x, ws.x, ws.y, g, t4, acc[nt]);
      }
      copy_next();
      const Cursor now = at;
      advance(at);
      if (at.kb == 0 || at.left == 0) {
        if (from == 0 && at.kb == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (nt * 8 < cnt) store_u(now.a, now.rb, cnt, nt, acc[nt]);
        } else {
          float4* t = reinterpret_cast<float4*>(p.part + (static_cast<size_t>(gw) * 4 + range * 2 + (from == 0 ? 1 : 0)) *
                                                             kTile) + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (nt * 8 < cnt) t[nt * 32] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
        if (at.left == 0) break;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
        from = 0;
        cnt = __popc(mask[at.a]);
      }
    }
  }
  grid_barrier(1);
  // u by 128-column blocks of a row, four elements per lane: stored by the warp
  // that had all of a unit's K, else added up from its parts; then quantised.
#pragma unroll 1
  for (int i = warp * G + c; i < nrows * Kb2; i += W) {
    const int row = i / Kb2, kb = i % Kb2;
    int lo = 0, hi = nact - 1;  // the active expert of the row: the last whose base is not past it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (base[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    const int col = row - base[lo], range = lo < p.ns ? 0 : 1, blocks = range ? routed_blocks : shared_blocks;
    const int unit = (lo - (range ? p.ns : 0)) * upe + kb * 16 + lane / 2;
    // The warp of K block x of a range is the largest w with even(blocks, w) <= x.
    const int w0 = static_cast<int>((static_cast<int64_t>(unit * Kb1 + 1) * W - 1) / blocks);
    const int w1 = static_cast<int>((static_cast<int64_t>((unit + 1) * Kb1) * W - 1) / blocks);
    float v[4];
    if (w0 == w1) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(p.u) + static_cast<size_t>(i) * 32 + lane);
      v[0] = u.x;
      v[1] = u.y;
      v[2] = u.z;
      v[3] = u.w;
    } else {
      float h1[4] = {0.f, 0.f, 0.f, 0.f}, h3[4] = {0.f, 0.f, 0.f, 0.f};
      const int in_tile = ((col >> 3) * 32 + (lane & 1) * 16 + ((col & 7) >> 1)) * 4 + (col & 1);
#pragma unroll 1
      for (int w = w0; w <= w1; w += 4) {
        float a[4][4], b[4][4];  // four parts' loads in flight together
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* t = p.part + (static_cast<size_t>(w + k) * 4 + range * 2 + (w + k == w0 ? 1 : 0)) * kTile + in_tile;
          // (With fewer K blocks than warps some warps have none.)
          const bool there = w + k <= w1 && (blocks >= W || even_wide(blocks, w + k, W) < even_wide(blocks, w + k + 1, W));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            a[k][r] = there ? __ldcg(t + r * 16) : 0.f;
            b[k][r] = there ? __ldcg(t + r * 16 + 2) : 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            h1[r] += a[k][r];
            h3[r] += b[k][r];
          }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = silu_mul(h1[r], h3[r]);
    }
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
  const int rows_in_first = (d0 / 128 + 1) * 128 - d0;  // rows of the CTA's first 128-row block
  const bool odd = ((d1 - d0) & 8) != 0;                // the last group has no high half
  // Operands of the slots that were asked for before u was quantised.
  have_u = true;
  Item it{warp / Kb2, warp % Kb2};
  {
    Item k = it;
    int slot = take;
#pragma unroll 1
    for (int q = 0; q < early2; q += ngroups) {
      open_item(k);
      copy_operands(slot);
      slot = (slot + ngroups) % kSlots;
      next_item(k);
    }
    copy_commit();
    copy_wait<0>();
  }
#pragma unroll 1
  while (it.a < nact2) {
    const uint32_t mk = mask[it.a];
    const int r_base = base[it.a], lowest = NT == 1 ? 0 : (__ffs(mk) - 1) >> 3;
    Frag f0, more[NT > 1 ? NT - 1 : 1];  // column tiles' fragments, for all groups
    float wa = 0.f, wb = 0.f;
    if constexpr (NT > 1) {
#pragma unroll
      for (int nt = 1; nt < NT; ++nt) {
        if (nt == lowest || !((mk >> (nt * 8)) & 0xFFu)) continue;
        Frag& f = more[nt - 1];
        f.b0 = f.b1 = make_uint4(0u, 0u, 0u, 0u);
        f.s0 = f.s1 = 0.f;
        const int m = nt * 8 + g, m2 = nt * 8 + 2 * t4;
        const int r = r_base + __popc(mk & ((1u << m) - 1u)), r2 = r_base + __popc(mk & ((1u << m2) - 1u));
        if ((mk >> m) & 1u) {
          const uint4* src =
              reinterpret_cast<const uint4*>(p.uq + static_cast<size_t>(r) * p.inter + it.kb * 128 + t4 * 32);
          f.b0 = __ldcg(src);
          f.b1 = __ldcg(src + 1);
        }
        const int r3 = r2 + ((mk >> m2) & 1u);
        if ((mk >> m2) & 1u) f.s0 = __ldcg(p.us + r2 * Kb2 + it.kb) * row_w[r2];
        if ((mk >> (m2 + 1)) & 1u) f.s1 = __ldcg(p.us + r3 * Kb2 + it.kb) * row_w[r3];
      }
    }
#pragma unroll
    for (int q = 0; q < kMaxGroups; ++q)
      if (q < ngroups) {
        const uint8_t* w = slot_ready();
        if (q == 0) {
          // The item's first slot carries the lowest tile's operands. Columns
          // without a token have zero codes: their sums go on for other experts.
          f0 = slot_frag(w);
          const int m = lowest * 8 + g, m2 = lowest * 8 + 2 * t4;
          const int r2 = r_base + __popc(mk & ((1u << m2) - 1u));
          if (!((mk >> m) & 1u)) f0.b0 = f0.b1 = make_uint4(0u, 0u, 0u, 0u);
          f0.s0 = (mk >> m2) & 1u ? f0.s0 * row_w[r2] : 0.f;
          f0.s1 = (mk >> (m2 + 1)) & 1u ? f0.s1 * row_w[r2 + ((mk >> m2) & 1u)] : 0.f;
          const float2 ws = *reinterpret_cast<const float2*>(w + kOffScl + 32);
          wa = ws.x;
          wb = ws.y;
        }
        const float wlo = q * 16 < rows_in_first ? wa : wb, whi = q * 16 + 8 < rows_in_first ? wa : wb;
        // A last group of 8 rows takes them twice; the second copy is not stored.
        const uint8_t* hi = odd && q == ngroups - 1 ? w : w + 1024;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT > 1 && !((mk >> (nt * 8)) & 0xFFu)) continue;
          const Frag& f = nt == 0 || nt == lowest ? f0 : more[nt > 0 ? nt - 1 : 0];
          block_product(w, hi, f, wlo, whi, g, t4, acc[q][nt]);
        }
        copy_next();
      }
    next_item(it);
  }
  copy_wait<0>();
  __syncthreads();
  // The rings hold the warps' sums [warp][row][columns] now.
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
  z.total = z.part + static_cast<size_t>(kMaxCtas) * kWarps * 4 * 16 * cols * 4;  // a tile is 16 rows x cols floats
  return z;
}

bool layer_shape_ok(int64_t T, int64_t dim, int64_t inter, int64_t E, int64_t topk, int64_t ns) {
  return T >= 0 && T <= kMaxTokens && dim >= 128 && dim <= kMaxDim && dim % 128 == 0 && inter >= 128 &&
         inter <= kMaxInter && inter % 128 == 0 && E >= 32 && E <= 256 && E % 32 == 0 && topk >= 1 && topk <= 32 &&
         ns >= 0 && ns <= kMaxShared;
}

template <int NT>
int layer_launch(const DevInfo* d, const LayerParams& p, cudaStream_t stream) {
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
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
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
  p.w1 = static_cast<const uint8_t*>(w1_e4m3);
  p.w3 = static_cast<const uint8_t*>(w3_e4m3);
  p.w2 = static_cast<const uint8_t*>(w2_e4m3);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return T <= 8    ? layer_launch<1>(d, p, cs)
         : T <= 16 ? layer_launch<2>(d, p, cs)
                   : layer_launch<4>(d, p, cs);
}
