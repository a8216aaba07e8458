// The MoE gate of one token, by one warp: shared by the gate and route
// kernels and the few-token layer.
// Per token ("Administrator & Developer Guide", 8.4 and 3.3; "Repository
// overview" MoE data flow): scores s from the logits (sigmoid, or softmax over
// the E experts), selection keys z = s + bias (z = s without a bias); with G > 1
// groups of E/G consecutive experts a group scores its largest z (no bias) or
// the sum of its two largest (bias), and only the TG best groups' experts stay
// eligible; the K best eligible z give the experts in descending order (ties:
// lower index); the weights are their s, divided by the sum of the K when
// `normalize`, times route_scale.
//
// One warp per token. Lane l holds experts [l V, l V + V) (E = 32 V), so a
// group is a run of 32 / G whole lanes: group maxima and top-two pairs merge
// with shuffles inside that run. Each top-k round is a warp argmax: the largest
// order-preserving bits of z, then the lowest index that has them.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace fp8blk {

// Order-preserving bits of a float.
__device__ __forceinline__ uint32_t gate_order(float z) {
  const uint32_t u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The smaller number, or NaN where one of the two is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float c;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// The lowest lane that has the warp's largest key.
__device__ __forceinline__ int warp_argmax_lane(uint32_t key) {
  const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key);
  return __ffs(__ballot_sync(0xFFFFFFFFu, key == best)) - 1;
}

// The gate of one token, computed by one warp from its logits: lane l holds
// x[i] = logit of expert l v + i for i < v <= V (E = 32 v experts; v = V where
// the caller knows it at compile time; x[i] past v is any finite number), and the
// experts' biases likewise. Lane
// j < K ends with the expert of slot j in *out_idx and its weight (normalised,
// times route_scale) in *out_w.
template <int V>
__device__ __forceinline__ void gate_warp(float (&x)[V], const float (&bias)[V], bool has_bias, int v, int G, int TG,
                                          int K, int sigmoid, float route_scale, int normalize, int lane, int* out_idx,
                                          float* out_w) {
  float s[V], z[V];
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = __frcp_rn(__fadd_rn(1.0f, expf(-x[i])));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < v) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < v) {
        x[i] = expf(__fsub_rn(x[i], m));
        sum = __fadd_rn(sum, x[i]);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, o));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < v) s[i] = __fdiv_rn(x[i], sum);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = has_bias ? __fadd_rn(s[i], bias[i]) : s[i];

  // Group selection: a lane is eligible while its group is kept.
  bool eligible = true;
  if (G > 1) {
    const int lpg = 32 / G;  // lanes per group (G divides 32)
    float a = -INFINITY, b = -INFINITY;  // this lane's two largest z
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float zi = i < v ? z[i] : -INFINITY;
      b = fmaxf(b, min_nan(a, zi));  // (fminf of a NaN and the largest would be the largest)
      a = fmaxf(a, zi);
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) {  // merge the pairs of the group's lanes
      const float a2 = __shfl_xor_sync(0xFFFFFFFFu, a, o);
      const float b2 = __shfl_xor_sync(0xFFFFFFFFu, b, o);
      const float hi = fmaxf(a, a2);
      b = fmaxf(fminf(a, a2), fmaxf(b, b2));
      a = hi;
    }
    const float gscore = has_bias ? __fadd_rn(a, b) : a;
    const int shift = __ffs(lpg) - 1, g = lane >> shift;  // lpg is a power of two
    bool kept = false;
    for (int r = 0; r < TG; ++r) {
      // A group's lanes agree, and lanes are in group order: ties go to the lower.
      if (warp_argmax_lane(kept ? 0u : gate_order(gscore)) >> shift == g) kept = true;
    }
    eligible = kept;
  }

  // Top-k experts among the eligible lanes' z. Each lane puts its keys in
  // descending order (equal ones in expert order) and offers the first; the lane
  // whose offer wins takes it out. A round is then an argmax and a move: scores
  // are fetched for all slots at once afterwards.
  uint32_t key[V];
  int at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = i < v && eligible ? gate_order(z[i]) : 0u;
    at[i] = i;
  }
#pragma unroll
  for (int r = 0; r < V; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < V; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t k = key[i];
      const int a = at[i];
      key[i] = swap ? key[i + 1] : k;
      key[i + 1] = swap ? k : key[i + 1];
      at[i] = swap ? at[i + 1] : a;
      at[i + 1] = swap ? a : at[i + 1];
    }
  int my_idx = 0;
#pragma unroll 1
  for (int j = 0; j < K; ++j) {
    // Lanes are in expert order: ties go to the lower expert.
    const int owner = warp_argmax_lane(key[0]);
    const int e = __shfl_sync(0xFFFFFFFFu, lane * v + at[0], owner);
    if (lane == j) my_idx = e;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) {
        key[i] = key[i + 1];
        at[i] = at[i + 1];
      }
      key[V - 1] = 0u;
    }
  }
  const int from = my_idx / v, which = my_idx - from * v;
  float my_s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float si = __shfl_sync(0xFFFFFFFFu, s[i], from);
    if (which == i) my_s = si;
  }
  float sum = 0.0f;
  if (normalize)
#pragma unroll 4
    for (int j = 0; j < K; ++j) sum = __fadd_rn(sum, __shfl_sync(0xFFFFFFFFu, my_s, j));
  *out_idx = my_idx;
  *out_w = __fmul_rn(normalize ? __fdiv_rn(my_s, sum) : my_s, route_scale);
}

}  // namespace fp8blk
