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
//     A producer warp feeds a ring of 32 KB stages by TMA; sixteen warps
//     multiply.
//   - The gate decides what the routed weights are, but not the shared ones:
//     the producer starts on its share of the shared experts while the other
//     warps quantise x, form the logits and run the gate.
//   - w2 does not depend on u, only its use does: the ring fills with w2
//     tiles while the CTAs wait for the last u and quantise it.
//   - Phase 1 splits (expert, 8 rows of w1 and the same 8 of w3) evenly over
//     the CTAs, phase 2 gives each CTA the same rows of every expert's w2: the
//     sum over experts stays in its registers, without atomics or partial
//     outputs, in one order.
//
// The products are warp-level FP8 MMAs (m16n8k32): tokens are the 8 columns,
// so one MMA serves an expert's up to 8 tokens at the cost of one, and a stage
// of 16 rows x 16 K blocks gives every warp one K block. In phase 1 rows 0-7
// of an MMA tile are w1's and rows 8-15 w3's, so one lane ends with h1 and h3 of
// the same element. Each K block's product is promoted as acc += D * (a_s w_s).
// A tcgen05.mma with so few columns takes about 130 cycles for 4 KB of weights,
// 31 bytes a cycle, hardly the HBM rate of one SM (23); the warp MMAs take 64.
// Operand fragments as in the decode GEMM: lane (g, t) reads bytes [32 t, 32 t +
// 32) of a K block for row g, MMA j of the block takes bytes [8 j, 8 j + 8) of
// those, the same for both operands.
//
// Token columns are tokens 0-7, 8-15, ... themselves (a tile of 8 columns
// without any token of the expert is skipped): no gathering, and in phase 2 the
// columns mean the same token for every expert.
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
constexpr int kWarps = 16;                                // multiplying warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kStageBytes = 2 * 8 * 128 * kWarps;         // two boxes of 8 rows x 16 K blocks
constexpr int kMaxGroups = 4;                             // 16-row groups of w2 per CTA
constexpr int kMaxDim = 8192, kMaxInter = 16384;

constexpr int kTables = kMaxActive * 12 + kMaxRows * 4 + 64;
constexpr int kLayerSmemLimit = 232448;

// Partial sums of a 16-row tile: [warp][row][columns], padded so that a warp's
// stores of 8 rows hit different banks.
__host__ __device__ constexpr int part_width(int nt) { return 8 * nt + (nt > 1 ? 8 : 0); }
__host__ __device__ constexpr int part_floats(int nt) { return kWarps * 16 * part_width(nt); }
__host__ __device__ constexpr int ring_stages(int nt) {
  return (kLayerSmemLimit - 1024 - kTables - 2 * part_floats(nt) * 4 - 256) / kStageBytes;
}

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
  unsigned* err;
  int T, dim, inter, E, ns, k, groups, kept, sigmoid, normalize, ue8m0;
  float route_scale;
  int kb1, st1;  // K blocks per stage and stages per unit, phase 1
  int kb2, st2;  // the same, phase 2
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

// First unit of CTA c of G when n units are split evenly.
__device__ __forceinline__ int even(int n, int c, int G) {
  return static_cast<int>(static_cast<int64_t>(n) * c / G);
}

// First routed unit of CTA c, such that shared and routed units together are
// split evenly (`us` shared units are split evenly by themselves).
__device__ __forceinline__ int routed_start(int us, int ur, int c, int G) {
  if (ur < 2 * G) return even(ur, c, G);
  return even(us + ur, c, G) - even(us, c, G);
}

// The B fragments of one K block for NT column tiles, its activation scales,
// and the weight scales of the low and high rows.
template <int NT>
struct Frag {
  uint4 b[NT][2];
  float s[NT][2];
  float wlo, whi;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map3,
                     const __grid_constant__ CUtensorMap map2, const LayerParams p) {
  constexpr int kStages = ring_stages(NT);
  constexpr int W = part_width(NT);
  constexpr int kCols = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  float* part = reinterpret_cast<float*>(ring + kStages * kStageBytes);  // [2][part_floats]
  int* act = reinterpret_cast<int*>(part + 2 * part_floats(NT));         // active experts, shared ones first
  uint32_t* mask = reinterpret_cast<uint32_t*>(act + kMaxActive);        // their tokens
  int* base = reinterpret_cast<int*>(mask + kMaxActive);                 // their first (token, expert) row
  float* wrow = reinterpret_cast<float*>(base + kMaxActive);             // gate weight of each row
  int* misc = reinterpret_cast<int*>(wrow + kMaxRows);                   // active experts, rows
  uint64_t* full = reinterpret_cast<uint64_t*>(misc + 16);
  uint64_t* empty = full + kStages;
  uint64_t* routed = empty + kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(routed + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, c = blockIdx.x;
  const int Kb1 = p.dim / 128, Kb2 = p.inter / 128;
  const int upe = p.inter / 8;  // phase-1 units of an expert
  const int shared_units = p.ns * upe;
  const int d0 = even(p.dim / 8, c, G) * 8, d1 = even(p.dim / 8, c + 1, G) * 8;  // this CTA's rows of w2
  const int ngroups = (d1 - d0 + 15) / 16;
  const uint32_t all_tokens = p.T == 32 ? 0xFFFFFFFFu : (1u << p.T) - 1u;

  if (tid == 0) {
    *abort_flag = 0;
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(routed, 1);
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ---- producer ---------------------------------------------------------------
    int n = 0;  // stages issued
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_first();  // weights are read once
      tma_prefetch_desc(&map1);
      tma_prefetch_desc(&map3);
      tma_prefetch_desc(&map2);
      auto issue = [&](const CUtensorMap* mlo, int ylo, const CUtensorMap* mhi, int yhi, int z, int nkb) {
        const int s = n % kStages;
        if (n >= kStages) wait(&empty[s], ((n / kStages) - 1) & 1, abort_flag, p.err);
        if (*abort_flag) return;
        uint8_t* dst = ring + s * kStageBytes;
        const uint32_t bytes = static_cast<uint32_t>(nkb) * 1024;
        mbar_arrive_expect_tx(&full[s], mhi ? 2 * bytes : bytes);
        tma_load_3d_hint(dst, mlo, &full[s], 0, ylo, z, policy);
        if (mhi) tma_load_3d_hint(dst + bytes, mhi, &full[s], 0, yhi, z, policy);
        ++n;
      };
      auto units = [&](int u0, int u1, bool shared) {
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
          const int e = shared ? p.E + u / upe : act[p.ns + u / upe];
          const int y = e * p.inter + (u % upe) * 8;
#pragma unroll 1
          for (int st = 0; st < p.st1; ++st) issue(&map1, y, &map3, y, st * p.kb1, p.kb1);
        }
      };
      units(even(shared_units, c, G), even(shared_units, c + 1, G), true);
      wait(routed, 0, abort_flag, p.err);
      if (!*abort_flag) {
        const int nact = misc[0], ur = (nact - p.ns) * upe;
        units(routed_start(shared_units, ur, c, G), routed_start(shared_units, ur, c + 1, G), false);
#pragma unroll 1
        for (int a = 0; a < nact; ++a)
#pragma unroll 1
          for (int st = 0; st < p.st2; ++st)
#pragma unroll 1
            for (int g = 0; g < ngroups; ++g) {
              const int y = act[a] * p.dim + d0 + g * 16;
              issue(&map2, y, d0 + g * 16 + 8 < d1 ? &map2 : nullptr, y + 8, st * p.kb2, p.kb2);
            }
      }
      // No copy may be in flight when the CTA exits.
#pragma unroll 1
      for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
        wait(&full[i % kStages], (i / kStages) & 1, nullptr, p.err);
    }
    __syncwarp();
  } else {
    // ---- the multiplying warps ----------------------------------------------------
    const int g = lane >> 2, t4 = lane & 3;
    auto sync_warps = [&] { named_barrier_sync(1, kWarps * 32); };
    // Grid barrier i: every CTA's warps have arrived, their global writes are visible.
    auto grid_barrier = [&](int i) {
      __threadfence();
      sync_warps();
      if (tid == 0) {
        atomicAdd(p.counters + i, 1u);
        const uint64_t t0 = global_timer_ns();
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
      sync_warps();
    };

    // Phase 0: x quantised and the logits formed, both spread over the grid.
#pragma unroll 1
    for (int i = c * kWarps + warp; i < p.T * Kb1; i += G * kWarps) {
      const uint2 raw = reinterpret_cast<const uint2*>(p.x)[static_cast<size_t>(i) * 32 + lane];
      const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                          __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)};
      quant_block(v, p.ue8m0 != 0, lane, p.xq + static_cast<size_t>(i) * 128, p.xs + i);
    }
#pragma unroll 1
    for (int e = c; e < p.E; e += G) {
      float acc[kCols];
#pragma unroll
      for (int m = 0; m < kCols; ++m) acc[m] = 0.f;
      const uint4* wv = reinterpret_cast<const uint4*>(p.gate_w + static_cast<size_t>(e) * p.dim);
#pragma unroll 1
      for (int v = tid; v < p.dim / 8; v += kWarps * 32) {
        const uint4 a = __ldg(wv + v);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int m = 0; m < kCols; ++m) {
          if (m < p.T) {
            const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(m) * p.dim) + v);
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[m] = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(bw[q] << 16), acc[m]);
              acc[m] = fmaf(__uint_as_float(aw[q] & 0xFFFF0000u), __uint_as_float(bw[q] & 0xFFFF0000u), acc[m]);
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
        if (lane == 0) part[warp * kCols + m] = acc[m];
      }
      sync_warps();
      if (tid < p.T) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += part[w * kCols + tid];
        p.logits[static_cast<size_t>(tid) * p.E + e] = s;
      }
      sync_warps();
    }
    grid_barrier(0);

    // The gate, by every CTA for itself: ids and weights of all tokens, in the
    // part buffer until they are sorted by expert.
    int* sel_e = reinterpret_cast<int*>(part);
    float* sel_w = part + kMaxTokens * 32;
#pragma unroll 1
    for (int m = warp; m < p.T; m += kWarps) {
      const int v = p.E / 32;
      float xl[8], bl[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xl[i] = i < v ? __ldcg(p.logits + static_cast<size_t>(m) * p.E + lane * v + i) : 0.f;
        bl[i] = i < v && p.gate_bias ? __ldg(p.gate_bias + lane * v + i) : 0.f;
      }
      int e;
      float w;
      gate_warp<8>(xl, bl, p.gate_bias != nullptr, v, p.groups, p.kept, p.k, p.sigmoid, p.route_scale, p.normalize,
                   lane, &e, &w);
      if (lane < p.k) {
        e = min(max(e, 0), p.E - 1);
        sel_e[m * p.k + lane] = e;
        sel_w[m * p.k + lane] = w;
        if (c == 0 && p.topk_idx) p.topk_idx[m * p.k + lane] = e;
        if (c == 0 && p.topk_w) p.topk_w[m * p.k + lane] = w;
      }
    }
    sync_warps();
    // Experts' token masks (thread e for expert e), then the active list by a
    // scan over the 8 warps that hold experts.
    uint32_t my_mask = 0;
    if (tid < p.E)
#pragma unroll 1
      for (int i = 0; i < p.T * p.k; ++i)
        if (sel_e[i] == tid) my_mask |= 1u << (i / p.k);
    const unsigned have = __ballot_sync(0xFFFFFFFFu, my_mask != 0);
    int rows = __popc(my_mask);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, rows, o);
      if (lane >= o) rows += v;
    }
    int* wsum = reinterpret_cast<int*>(part) + 2 * kMaxTokens * 32;  // [16] active, [16] rows
    if (lane == 31) {
      wsum[warp] = __popc(have);
      wsum[16 + warp] = rows;
    }
    if (tid < p.ns) {
      act[tid] = p.E + tid;
      mask[tid] = all_tokens;
      base[tid] = tid * p.T;
    }
#pragma unroll 1
    for (int i = tid; i < p.ns * p.T; i += kWarps * 32) wrow[i] = 1.0f;
    sync_warps();
    int a0 = p.ns, r0 = p.ns * p.T;
    for (int w = 0; w < warp; ++w) {
      a0 += wsum[w];
      r0 += wsum[16 + w];
    }
    if (my_mask) {
      const int a = a0 + __popc(have & ((1u << lane) - 1u));
      const int r = r0 + rows - __popc(my_mask);
      act[a] = tid;
      mask[a] = my_mask;
      base[a] = r;
#pragma unroll 1
      for (int i = 0; i < p.T * p.k; ++i)
        if (sel_e[i] == tid) wrow[r + __popc(my_mask & ((1u << (i / p.k)) - 1u))] = sel_w[i];
    }
    if (tid == kWarps * 32 - 1) {
      misc[0] = a0 + __popc(have);
      misc[1] = r0 + rows;
    }
    sync_warps();
    const int nact = misc[0], nrows = misc[1];
    if (tid == 0) mbar_arrive(routed);

    int n = 0;  // stages consumed
    // The fragments of K block kb for active expert a; `rows` maps a token to
    // its row of the quantised activations.
    auto load_frag = [&](Frag<NT>& f, const uint8_t* q, const float* s, int K, int Kb, int a, int kb, bool by_row,
                         const float* slo, const float* shi) {
      const uint32_t mk = mask[a];
      const int bs = base[a];
      auto row_of = [&](int m) { return by_row ? bs + __popc(mk & ((1u << m) - 1u)) : m; };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int m = nt * 8 + g, m2 = nt * 8 + 2 * t4;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if ((mk >> m) & 1u) {
          const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<size_t>(row_of(m)) * K + kb * 128 + t4 * 32);
          f.b[nt][0] = __ldcg(src);
          f.b[nt][1] = __ldcg(src + 1);
        } else {
          f.b[nt][0] = f.b[nt][1] = zero;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f.s[nt][i] = 0.f;
          if ((mk >> (m2 + i)) & 1u) {
            const int r = row_of(m2 + i);
            f.s[nt][i] = __ldcg(s + static_cast<size_t>(r) * Kb + kb) * (by_row ? wrow[r] : 1.0f);
          }
        }
      }
      f.wlo = __ldg(slo);
      f.whi = __ldg(shi);
    };
    // One stage: this warp's K block (the warp-th) of 16 rows, promoted into acc.
    auto multiply = [&](const Frag<NT>& f, uint32_t mk, int nkb, bool mine, float (&acc)[NT][4]) {
      const int s = n % kStages;
      wait(&full[s], (n / kStages) & 1, abort_flag, p.err);
      if (mine) {
        const uint8_t* lo = ring + s * kStageBytes + warp * 1024 + g * 128;
        const uint8_t* hi = lo + nkb * 1024;
        uint4 al[2], ah[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          al[h] = *reinterpret_cast<const uint4*>(lo + (((2 * t4 + h) ^ g) << 4));
          ah[h] = *reinterpret_cast<const uint4*>(hi + (((2 * t4 + h) ^ g) << 4));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT > 1 && !((mk >> (nt * 8)) & 0xFFu)) continue;
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16x8x32(d, al[0].x, ah[0].x, al[0].y, ah[0].y, f.b[nt][0].x, f.b[nt][0].y);
          mma_16x8x32(d, al[0].z, ah[0].z, al[0].w, ah[0].w, f.b[nt][0].z, f.b[nt][0].w);
          mma_16x8x32(d, al[1].x, ah[1].x, al[1].y, ah[1].y, f.b[nt][1].x, f.b[nt][1].y);
          mma_16x8x32(d, al[1].z, ah[1].z, al[1].w, ah[1].w, f.b[nt][1].z, f.b[nt][1].w);
          acc[nt][0] = fmaf(d[0], f.s[nt][0] * f.wlo, acc[nt][0]);
          acc[nt][1] = fmaf(d[1], f.s[nt][1] * f.wlo, acc[nt][1]);
          acc[nt][2] = fmaf(d[2], f.s[nt][0] * f.whi, acc[nt][2]);
          acc[nt][3] = fmaf(d[3], f.s[nt][1] * f.whi, acc[nt][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      ++n;
    };
    // This warp's sums of a 16-row tile into part buffer `buf`.
    auto put = [&](const float (&acc)[NT][4], float* buf) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* q = buf + (warp * 16 + g) * W + nt * 8 + 2 * t4;
        *reinterpret_cast<float2*>(q) = make_float2(acc[nt][0], acc[nt][1]);
        *reinterpret_cast<float2*>(q + 8 * W) = make_float2(acc[nt][2], acc[nt][3]);
      }
    };

    // Phase 1: u = silu(w1 x) (w3 x), unit by unit (8 rows of an expert).
    int nb = 0;  // units so far: which part buffer
    auto phase1 = [&](int u0, int u1, int first) {
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        const int a = first + u / upe, e = act[a], rb = u % upe;
        const uint32_t mk = mask[a];
        const size_t srow = static_cast<size_t>((static_cast<int64_t>(e) * p.inter + rb * 8) / 128) * Kb1;
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll 1
        for (int st = 0; st < p.st1; ++st) {
          const int kb = st * p.kb1 + warp;
          const bool mine = warp < p.kb1 && kb < Kb1;
          Frag<NT> f;
          if (mine) load_frag(f, p.xq, p.xs, p.dim, Kb1, a, kb, false, p.w1_s + srow + kb, p.w3_s + srow + kb);
          multiply(f, mk, p.kb1, mine, acc);
        }
        float* buf = part + (nb & 1) * part_floats(NT);
        ++nb;
        put(acc, buf);
        sync_warps();
        // kCols x 8 elements, 8 / NT threads each, summed in warp order within a
        // thread and then across the threads.
        constexpr int kTpo = 8 / NT;
        const int o = tid / kTpo, q = tid % kTpo;
        const int m = o / 8, r = o % 8;
        float h1 = 0.f, h3 = 0.f;
        for (int w = q; w < p.kb1; w += kTpo) {
          h1 += buf[(w * 16 + r) * W + m];
          h3 += buf[(w * 16 + r + 8) * W + m];
        }
#pragma unroll
        for (int of = kTpo / 2; of > 0; of >>= 1) {
          h1 += __shfl_xor_sync(0xFFFFFFFFu, h1, of);
          h3 += __shfl_xor_sync(0xFFFFFFFFu, h3, of);
        }
        if (q == 0 && ((mk >> m) & 1u)) {
          const int row = base[a] + __popc(mk & ((1u << m) - 1u));
          p.u[static_cast<size_t>(row) * p.inter + rb * 8 + r] = h1 / (1.0f + expf(-h1)) * h3;
        }
      }
    };
    phase1(even(shared_units, c, G), even(shared_units, c + 1, G), 0);
    const int ur = (nact - p.ns) * upe;
    phase1(routed_start(shared_units, ur, c, G), routed_start(shared_units, ur, c + 1, G), p.ns);
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
#pragma unroll 1
    for (int a = 0; a < nact; ++a) {
      const uint32_t mk = mask[a];
      const int e = act[a];
#pragma unroll 1
      for (int st = 0; st < p.st2; ++st) {
        const int kb = st * p.kb2 + warp;
        const bool mine = warp < p.kb2 && kb < Kb2;
        Frag<NT> f;
        if (mine) load_frag(f, p.uq, p.us, p.inter, Kb2, a, kb, true, p.w2_s, p.w2_s);
#pragma unroll
        for (int q = 0; q < kMaxGroups; ++q) {
          if (q < ngroups) {
            if (mine) {
              const int64_t row = static_cast<int64_t>(e) * p.dim + d0 + q * 16;
              const int64_t last = static_cast<int64_t>(e) * p.dim + d1 - 1;
              f.wlo = __ldg(p.w2_s + row / 128 * Kb2 + kb);
              f.whi = __ldg(p.w2_s + (row + 8 < last ? row + 8 : last) / 128 * Kb2 + kb);
            }
            multiply(f, mk, p.kb2, mine, acc[q]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kMaxGroups; ++q) {
      if (q < ngroups) {
        float* buf = part + (nb & 1) * part_floats(NT);
        ++nb;
        put(acc[q], buf);
        sync_warps();
        if (tid < 16 * kCols) {
          const int m = tid / 16, r = tid % 16;
          float s = 0.f;
          for (int w = 0; w < p.kb2; ++w) s += buf[(w * 16 + r) * W + m];
          if (m < p.T && d0 + q * 16 + r < d1)
            p.y[static_cast<size_t>(m) * p.dim + d0 + q * 16 + r] = __float2bfloat16_rn(s);
        }
      }
    }
  }
  __syncthreads();
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
// boxes of 8 rows x kb blocks, 128-byte swizzled; blocks past K read as zeros.
bool make_weight_map(CUtensorMap* map, const void* w, uint64_t N, uint64_t K, uint32_t kb) {
  EncodeTiledFn enc = layer_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {128, N, K / 128};
  const cuuint64_t strides[2] = {K, 128};
  const cuuint32_t box[3] = {128, 8, kb};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

struct LayerSizes {
  size_t logits, xq, xs, u, uq, us, total;
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
  z.total = z.us + align256(rows * (inter / 128) * 4);
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
  static_assert(ring_stages(NT) >= 3, "ring depth");
  constexpr int kSmem = 1024 + ring_stages(NT) * kStageBytes + 2 * part_floats(NT) * 4 + kTables +
                        (2 * ring_stages(NT) + 1) * 8 + 16;
  static_assert(kSmem <= kLayerSmemLimit, "shared memory per CTA");
  static bool attr_done[64] = {};
  auto kern = moe_layer_kernel<NT>;
  if (d->device >= 64 || !attr_done[d->device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return FP8BLK_ERR_CUDA;
    if (d->device < 64) attr_done[d->device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d->sm_count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
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
  if ((dim / 8 + d->sm_count - 1) / d->sm_count > 2 * kMaxGroups) return FP8BLK_ERR_SHAPE;
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
  // Stages of at most 16 K blocks, as even as they divide.
  const int Kb1 = p.dim / 128, Kb2 = p.inter / 128;
  p.st1 = (Kb1 + kWarps - 1) / kWarps;
  p.kb1 = (Kb1 + p.st1 - 1) / p.st1;
  p.st2 = (Kb2 + kWarps - 1) / kWarps;
  p.kb2 = (Kb2 + p.st2 - 1) / p.st2;
  const uint64_t K = static_cast<uint64_t>(E + n_shared);
  CUtensorMap m1, m3, m2;
  if (!make_weight_map(&m1, w1_e4m3, K * inter, dim, p.kb1) || !make_weight_map(&m3, w3_e4m3, K * inter, dim, p.kb1) ||
      !make_weight_map(&m2, w2_e4m3, K * dim, inter, p.kb2))
    return FP8BLK_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return T <= 8    ? layer_launch<1>(d, m1, m3, m2, p, cs)
         : T <= 16 ? layer_launch<2>(d, m1, m3, m2, p, cs)
                   : layer_launch<4>(d, m1, m3, m2, p, cs);
}
