// Attention of single query tokens over a paged latent cache whose first
// `prefix_len` keys are shared by the whole batch ("Administrator & Developer
// Guide", 8.3, attn_impl "absorb": scores are q_nope' c + q_pe k_pe on the
// latent cache, the output stays in the latent space for wkv_b's v rows).
// Per request b and head h, with x = [q[b, h], q_pe[b, h]] (576 columns) and
// cache rows c_j over the prefix's keys and then the request's own:
//
//   s_j = scale * <x, c_j>,   a = softmax(s),   out = sum_j a_j c_j[0:512].
//
// Rows and keys. A tile is 128 query rows (rows are (b, h) flattened) against
// 128 keys. The prefix is the same for all rows, so its tiles hold rows of
// any requests: it is read once per 128 rows instead of once per request. A
// request's own keys meet that request's rows alone. Where H is a multiple
// of 128 a row tile belongs to one request and prefix and own keys form one
// item, one running softmax over both; otherwise prefix row tiles and the
// requests' own keys are items of their own, joined at the end (a row never
// meets another request's keys: 0 * Inf in the product would leak them).
//
// Work split. The items' key tiles, laid end to end, are cut into equal
// ranges, one per CTA pair: one long sequence and a ragged batch fill the GPU
// alike. Where a range cuts an item, each part leaves its unnormalised sum,
// maximum and weight sum in the workspace, and a second kernel joins each
// row's parts in key order: no atomics, the same bits every run. Lengths are
// read on the device.
//
// The pair. The fp32 output of 128 rows x 512 columns would fill an SM's whole
// tensor memory, so two SMs share a tile (cta_group::2, M = 128): each holds
// 64 rows, as 128 lanes x 256 columns (lanes 64-127 hold the upper half of
// each MMA's columns), and two 64-column score buffers beside it. Each SM's
// shared memory holds its 64 query rows, half the tile's keys (all 576
// columns) as the B operand of the scores, half the columns of all 128 keys
// as the MN-major B operand of the output, and its rows' weights P in bf16.
// The tensor cores run this M = 128 pair shape at their full rate (measured:
// 4090 multiply-adds per clock and SM; a single SM's M = 64 runs at half).
//
// Softmax. Four warps per CTA, a thread per (row, key half): base-2 exponents
// in fp32, the running maximum raised only when a tile's maximum passes it by
// more than 8 (weights stay below 2^8, so the fp32 sums lose nothing and the
// output is rescaled in tensor memory on few tiles). P is rounded to bf16, the
// type the tensor cores take next to bf16 keys; the weight sum adds the
// rounded weights, so equal keys give exactly their mean. Keys past the end
// are masked by position, not by value, and their rows are overwritten with
// zeros before the output product, so whatever an unused cache row holds, NaN
// included, stays out. The logarithm of the sum, where asked for,
// comes from a second sum of the weights before their rounding.
//
// What bounds it, measured (GPU time): 64 requests of 128 heads behind 32768
// shared keys take 328 us, 1.8 PFLOP/s of the 1.94 that a library GEMM reaches:
// the tensor cores (369 us a call in long runs). 32 requests of 128 heads
// with up to 8191 own keys take 48.2 us, of which HBM needs 25.5 and the products
// 20, side by side; first loads (6 us) and join (7 us) leave 9 us unexplained.
// Where a call is short the chain of latencies is all there is: 24.0 us for one
// request of 128 heads and 32768 keys are 5 us of launch, plan and first loads, 6
// us of tiles, 2 us for 20 MB of parts to L2, 1.7 us between the kernels and 5 us
// to read the parts back; 61 requests of 16 heads behind 2011 keys take 21.2 us,
// one short request 7.5. (One kernel whose CTAs meet at a barrier and join with
// their own seven warps, loading the parts into registers, took 29.6 us for that
// one long request where two kernels took 27.)
//
// Every wait is bounded (2 s): on expiry roles leave their loops, in-flight
// copies are waited for (bounded), tensor memory is freed, an error bit set.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "fp8blk.h"
#include "host.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

constexpr int kC = 512, kR = 64, kRow = kC + kR;
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr int kSlab = 64 * 128;             // 64 rows x 64 bf16, 128-byte swizzled
constexpr int kQSlabs = kRow / 64;          // 9 slabs of 64 columns
constexpr int kKGroups = 3;                 // key slabs signalled three at a time
constexpr int kGroupBytes = 3 * kSlab;
// Keys of a value chunk, 256 columns each: with 32 the twice as many waits and
// commits cost the large case 342 us against 322; pages of 16 rows lose 0.4 us of 21.
constexpr int kVRows = 64;
constexpr int kVChunks = kTileKeys / kVRows;
constexpr int kVSlab = kVRows * 128;        // kVRows keys x 64 columns
constexpr int kVChunk = 4 * kVSlab;
constexpr int kOffQ = 0;
constexpr int kOffP = kOffQ + kQSlabs * kSlab;
constexpr int kOffK = kOffP + 2 * kSlab;
constexpr int kOffV = kOffK + kQSlabs * kSlab;
constexpr int kOffRed = kOffV + kVChunks * kVChunk;  // [2][2][64] row maxima, then sums
constexpr int kOffBar = kOffRed + 2 * 2 * 64 * 4;
constexpr int kNumBars = 2 + 2 * kKGroups + 2 * kVChunks + 4 + 4 + 3;
static_assert(kNumBars <= 32, "a lane of a warp initialises each");
constexpr int kAttnSmem = 1024 + kOffBar + kNumBars * 8 + 32;
static_assert(kAttnSmem <= 232448, "shared memory per CTA");

// Warps: 0-3 softmax (warp w: tensor-memory lanes 32 w ..), 4 keys, 5
// queries and values, 6 the scores' MMAs, 7 the output's.
constexpr int kAttnThreads = 256;
constexpr int kMaxPairs = 96;
constexpr uint32_t kTmemS = 256;            // columns 0-255: output; 256-383: two score buffers
constexpr float kRaise = 8.0f;              // log2 by which a tile's maximum must pass the running one
constexpr unsigned kDevErrTimeoutMla = 1u << 6;
constexpr unsigned kDevErrBadSlot = 1u << 8;

// Division of 0 <= n < 2^30 by a constant d of the launch, 1 <= d <= 2^20: with
// 2^(L-1) < d <= 2^L and mul = floor(2^(30+L) / d) + 1, mul d exceeds 2^(30+L) by
// at most 2^L, so n mul / 2^(30+L) passes n / d by less than 1 / d.
struct Divisor {
  uint32_t mul, shift;
};

__host__ Divisor divisor(int64_t d) {
  uint32_t l = 0;
  while ((int64_t{1} << l) < d) ++l;
  return {static_cast<uint32_t>((uint64_t{1} << (30 + l)) / static_cast<uint64_t>(d) + 1), 30 + l};
}

__host__ __device__ __forceinline__ int div_by(int n, const Divisor& d) {
  return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.mul >> d.shift);
}

struct AttnParams {
  const __nv_bfloat16* cache;
  const int* prefix_pages;
  const int* table;        // [B][table_stride]
  const int* lens;         // [B]
  __nv_bfloat16* out;      // [B H][512]
  float* lse;              // [B H] or null
  float4* part_o;          // per part [128 column quads][rows of the item]: a warp's rows are contiguous
  float4* part_ml;         // [part rows] (maximum in log2 units, sum of the rounded weights, of the fp32 weights)
  int* plan;               // [0] units, [1] pairs in use, [2 + i] first unit of item i (items + 1 entries)
  unsigned* err;
  Divisor by_page, by_per, by_pairs;  // page size, row tiles per request, pairs of the launch
  int B, H, P, page, per, num_pages, table_stride, max_own;
  int total_rows;          // cache rows: the out-of-range row coordinate
  int prefix_tiles, prefix_items, items, own_rows;
  int merged;              // H % 128 == 0: prefix and own keys in one item
  int kbox, vbox;          // rows of a TMA box of keys / values
  int kslabs, vslabs;      // and its 64-column slabs (several where a box has a slab's rows)
  int direct;              // no item can be cut or share a row: no join
  float scale_log2;
};

struct Item {
  int row0, nrows;   // flattened query rows
  int pt, tiles;     // prefix tiles, all tiles
  int b, len;        // the request whose own keys follow the prefix tiles
};

__device__ __forceinline__ int own_len(const AttnParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.max_own);
}

__device__ __forceinline__ Item get_item(const AttnParams& p, int i) {
  Item it;
  if (p.merged) {
    it.row0 = i * kTileRows;
    it.nrows = kTileRows;
    it.b = div_by(i, p.by_per);
    it.pt = p.prefix_tiles;
  } else if (i < p.prefix_items) {
    it.row0 = i * kTileRows;
    it.nrows = min(kTileRows, p.B * p.H - it.row0);
    it.b = -1;
    it.pt = p.prefix_tiles;
  } else {
    const int k = i - p.prefix_items;
    it.b = div_by(k, p.by_per);
    it.row0 = it.b * p.H + (k - it.b * p.per) * kTileRows;
    it.nrows = min(kTileRows, (it.b + 1) * p.H - it.row0);
    it.pt = 0;
  }
  it.len = it.b >= 0 ? own_len(p, it.b) : 0;
  it.tiles = it.pt + (it.len + kTileKeys - 1) / kTileKeys;
  return it;
}

// What an item costs beside its tiles (queries loaded, rows stored), in tiles:
// the split's units are its tiles after that many units without one. (32 ragged
// requests x 128 heads: 50.9 us with none, 47.9 with one, 49.0 with two; 61 x 16
// rows 21.4, 21.3, 22.8.)
constexpr int kItemCost = 1;

struct Span {
  int t0, t1, units;  // tiles, and the units they took from the pair's range
};

// The tiles of an item of `tiles` in its units [v0, v0 + left).
__device__ __forceinline__ Span span_of(int tiles, int v0, int left) {
  const int v1 = min(tiles > 0 ? tiles + kItemCost : 0, v0 + left);
  return {max(v0 - kItemCost, 0), max(v1 - kItemCost, 0), v1 - v0};
}

__device__ __forceinline__ int item_tiles(const AttnParams& p, int i) {
  if (!p.merged && i < p.prefix_items) return p.prefix_tiles;
  const int len = own_len(p, div_by(i - p.prefix_items, p.by_per));
  return (p.merged ? p.prefix_tiles : 0) + (len + kTileKeys - 1) / kTileKeys;
}

__device__ __forceinline__ int item_units(const AttnParams& p, int i) {
  const int n = item_tiles(p, i);
  return n > 0 ? n + kItemCost : 0;
}

// First row of the parts of item i written by pair q: item-major, 128 rows
// apart from one pair to the next, so parts never overlap.
__host__ __device__ __forceinline__ int64_t part_row(int merged, int prefix_items, int own_rows, int i, int q) {
  const int64_t base = merged || i < prefix_items
                           ? static_cast<int64_t>(i) * kTileRows
                           : static_cast<int64_t>(prefix_items) * kTileRows +
                                 static_cast<int64_t>(i - prefix_items) * own_rows;
  return base + static_cast<int64_t>(q) * kTileRows;
}

// First unit of pair q of `launched` (by_pairs divides by that many): units q /
// launched rounded down, without 64-bit products. Fewer units than pairs go to a
// pair each, and the pairs past the last unit start at the end: their ranges, and
// every range of a batch without any key, are empty.
__host__ __device__ __forceinline__ int unit_of_pair(const Divisor& by_pairs, int units, int launched, int q) {
  if (units < launched) return q < units ? q : units;
  const int each = div_by(units, by_pairs);
  return each * q + div_by((units - each * launched) * q, by_pairs);
}

// The pair whose range holds unit u: the largest q with units q / pairs <= u,
// that is units q < (u + 1) pairs. An estimate, then put right.
__device__ __forceinline__ int pair_of_unit(int units, int pairs, int u) {
  const int64_t x = static_cast<int64_t>(u + 1) * pairs;
  int q = static_cast<int>(__fdividef(static_cast<float>(u + 1) * static_cast<float>(pairs), static_cast<float>(units)));
  while (static_cast<int64_t>(units) * (q + 1) < x) ++q;
  while (static_cast<int64_t>(units) * q >= x) --q;
  return q;
}

// ---- instructions of the CTA pair ----------------------------------------------

__device__ __forceinline__ uint32_t map_to_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

// Arrives on an mbarrier of any CTA of the cluster (shared::cluster address).
// What it orders are tensor-memory accesses, by the tcgen05 fences around it, or
// nothing but a count: no release of memory.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// The same for shared memory written before it (made visible to the async proxy
// by the writers' proxy fences): the thread that waits issues MMAs whose operands
// are read in this CTA, so the release is of cluster scope, restricted to this
// CTA's shared memory. (A release of cluster scope over all memory stalls the
// warp for about 800 cycles here: 64 x 128 rows, 32768 shared keys 482 us; an
// arrival of CTA scope, which orders nothing between the two, 325; this one,
// with the acquires below, 328.)
__device__ __forceinline__ void mbar_publish_cluster(uint32_t addr) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_cluster(addr);
}

// The bounded wait of every role, out of line: the roles' loops have to stay
// in the instruction cache together (with inlined waits and unrolled tile loops
// the kernel was 131 KB, and every role ran five times slower on fetches).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint64_t t0 = global_timer_ns();
  bool ok = false;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) {
      ok = true;
      break;
    }
    if ((i & 63u) == 0) {
      if (abort && *abort) break;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        if (abort) *abort = 1;
        atomicOr(err, kDevErrTimeoutMla);
        break;
      }
    }
  }
  return ok;
}

__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_wait(a, parity) || wait_slow(a, parity, abort, err);
}

// The same for a phase that threads of both CTAs arrive in.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_wait_cluster(a, parity) || (wait_slow(a, parity, abort, err) && mbar_try_wait_cluster(a, parity));
}

// The same for a whole warp: true in all lanes or in none.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err) {
  const uint32_t a = smem_u32(bar);
  bool ok = mbar_try_wait(a, parity);
  if (!__all_sync(0xFFFFFFFFu, ok)) ok = __all_sync(0xFFFFFFFFu, ok || wait_slow(a, parity, abort, err));
  return ok;
}

// Tiled load (column in a slab, row, slab) into this CTA's shared memory; the
// bytes complete on the mbarrier at shared::cluster address `bar`, in this CTA
// or its pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y, int slab) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(slab)
      : "memory");
}

// Asks for `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// D (+)= A B^T over the pair for one K = 16 slice; issued by one thread of CTA 0.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Arrives on `bar` in both CTAs when the MMAs issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// bf16 x bf16 -> f32, A K-major, B K-major or MN-major, M x N over the pair.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The cache row of key `key`, whose page is `pg`, or the out-of-range row
// where that is not one of the cache's pages.
__device__ __forceinline__ int entry_row(const AttnParams& p, int pg, int key) {
  if (pg < 0 || pg >= p.num_pages) {
    atomicOr(p.err, kDevErrBadSlot);
    return p.total_rows;
  }
  return pg * p.page + key - div_by(key, p.by_page) * p.page;
}

// Value chunks of a tile that hold keys.
__device__ __forceinline__ int chunks_of(int key0, int limit) { return min(kVChunks, (limit - key0 + kVRows - 1) / kVRows); }

// Items [lo, hi) of thread `tid` of `n`.
__device__ __forceinline__ int split(int items, int tid, int n) {
  return static_cast<int>(static_cast<int64_t>(items) * tid / n);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttnThreads, 1)
    mla_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_qpe,
                         const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + kKGroups;
  uint64_t* v_full = k_empty + kKGroups;
  uint64_t* v_empty = v_full + kVChunks;
  uint64_t* s_full = v_empty + kVChunks;  // [2]
  uint64_t* s_empty = s_full + 2;         // [2]
  uint64_t* p_full = s_empty + 2;
  uint64_t* pv_done = p_full + 1;
  uint64_t* o_empty = pv_done + 1;
  uint64_t* red_bar = o_empty + 1;
  uint64_t* v_end = red_bar + 1;  // this CTA's part of the chunk that holds the end of the keys
  uint64_t* drain = v_end + 1;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* start = reinterpret_cast<int*>(tmem_slot + 2);  // first item, first unit in it, unit count

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x) >> 1;
  const int npairs_max = static_cast<int>(gridDim.x) >> 1;

  if (warp == 0) {
    // A lane per barrier. Arrivals: the softmax warps of both CTAs, of one, or one.
    uint64_t* bar = q_full + lane;
    const bool both = bar == s_empty || bar == s_empty + 1 || bar == p_full || bar == o_empty;
    const bool values = bar >= v_full && bar < v_full + kVChunks;  // a value warp of each CTA
    if (lane < kNumBars) mbar_init(bar, both ? 8 : bar == red_bar ? 4 : values ? 2 : 1);
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 128) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_qpe);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  griddep_wait();

  // The plan: every CTA sums the items' tiles (thread-contiguous ranges, then
  // a scan over the threads) and finds the item its range starts in. Warp 6 is
  // not waited for: it allocates tensor memory.
  if (warp < 6) {
    constexpr int kPlanners = 192;
    int* sums = reinterpret_cast<int*>(red);
    const int lo = split(p.items, tid, kPlanners), hi = split(p.items, tid + 1, kPlanners);
    int own = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) own += item_units(p, i);
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    if (tid == 0) start[0] = start[1] = 0;  // where the range is empty
    named_barrier_sync(1, kPlanners);
    int at = upto - own, units = 0;
#pragma unroll
    for (int w = 0; w < kPlanners / 32; ++w) {
      const int v = sums[w];
      at += w < warp ? v : 0;
      units += v;
    }
    const int u0 = unit_of_pair(p.by_pairs, units, npairs_max, pair);
    const int u1 = unit_of_pair(p.by_pairs, units, npairs_max, pair + 1);
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
      const int n = hi - lo == 1 ? own : item_units(p, i);
      if (u0 < u1 && u0 >= at && u0 < at + n) {
        start[0] = i;
        start[1] = u0 - at;
      }
      if (blockIdx.x == 0) p.plan[2 + i] = at;
      at += n;
    }
    if (tid == 0) start[2] = u1 - u0;
    if (blockIdx.x == 0 && tid == 0) {
      p.plan[0] = units;
      p.plan[1] = min(npairs_max, units);
      p.plan[2 + p.items] = units;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // Barriers initialised and tensor memory allocated in both CTAs.
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int nunits = start[2];
  const int item0 = start[0], unit0 = start[1];

  if (warp == 4 || warp == 5) {
    // ---- loads: keys (warp 4), queries and values (warp 5) -------------------
    const bool is_k = warp == 4;
    uint32_t n = 0, seg = 0;
    int left = nunits, i = item0, v0 = unit0;
    bool ok = true;
    const uint32_t bars = map_to_cta(smem_u32(is_k ? k_full : v_full), 0);
    const uint32_t dst0 = smem_u32(smem + (is_k ? kOffK : kOffV));
    const int rows = is_k ? p.kbox : 16;   // keys per looked-up page entry
    uint32_t vphase = 0, ends = 0;         // bit c: phase of value chunk c; uses of v_end
    const int mine = is_k ? static_cast<int>(rank) * 64 : 0;
    const bool looks = lane * rows < (is_k ? 64 : kTileKeys);
#pragma unroll 1
    while (ok && left > 0 && i < p.items) {
      const Item it = get_item(p, i);
      const Span in = span_of(it.tiles, v0, left);
      const int t0 = in.t0, t1 = in.t1;
      left -= in.units;
      // Lane l's page entry of tile t: that of its l-th `rows` keys. Entries are
      // loaded two tiles ahead and become cache rows when they are needed.
      auto first_key = [&](int t) { return (t < it.pt ? t : t - it.pt) * kTileKeys; };
      auto page_entry = [&](int t) {
        const bool pre = t < it.pt;
        const int key = first_key(t) + mine + lane * rows;
        const int limit = pre ? p.P : it.len;
        if (t >= t1 || !looks || key >= limit) return -1;
        const int* pages = pre ? p.prefix_pages : p.table + static_cast<int64_t>(it.b) * p.table_stride;
        return __ldg(pages + div_by(key, p.by_page));
      };
      auto row_of = [&](int t, int entry) {
        const int key = first_key(t) + mine + lane * rows;
        return looks && t < t1 && key < (t < it.pt ? p.P : it.len) ? entry_row(p, entry, key) : p.total_rows;
      };
      int entry1 = page_entry(t0), entry2 = page_entry(t0 + 1);
      // (The first by the value warp, beside the first keys; later ones, whose
      // wait would hold the values up, by the key warp.)
      if (t1 > t0 && is_k == (seg > 0)) {
        if (seg > 0) ok = wait_warp(q_empty, (seg - 1) & 1, abort_flag, p.err);
        if (!ok) break;
        if (elect_one_sync()) {
          if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * kQSlabs * kSlab);
          const uint32_t bar = map_to_cta(smem_u32(q_full), 0);
          const int y = it.row0 + static_cast<int>(rank) * 64;
          tma_load_pair(smem_u32(smem + kOffQ), &map_q, bar, y, 0);
          tma_load_pair(smem_u32(smem + kOffQ + kC / 64 * kSlab), &map_qpe, bar, y, 0);
        }
        __syncwarp();
      }
      if (t1 > t0) ++seg;
      int y_next = row_of(t0, entry1);
      entry1 = entry2;
#pragma unroll 1
      for (int t = t0; ok && t < t1; ++t, ++n) {
        const bool pre = t < it.pt;
        const int key0 = first_key(t);
        const int limit = pre ? p.P : it.len;
        const int y16 = y_next;
        y_next = row_of(t + 1, entry1);
        entry1 = page_entry(t + 2);
        if (is_k) {
          // This CTA's 64 keys, in boxes of kbox keys x 64 columns.
          const int nbox = 64 / p.kbox;
#pragma unroll 1
          for (int g = 0; g < kKGroups; ++g) {
            if (n > 0) ok = wait_warp(&k_empty[g], (n - 1) & 1, abort_flag, p.err);
            if (!ok) break;
            if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&k_full[g], 2 * kGroupBytes);
            __syncwarp();
            if (lane < nbox) {  // box `lane`: its rows are this lane's
              const uint32_t dst = dst0 + g * kGroupBytes + lane * p.kbox * 128;
              tma_load_pair(dst, &map_k, bars + g * 8, y16, 3 * g);
              if (p.kslabs == 1) {
                tma_load_pair(dst + kSlab, &map_k, bars + g * 8, y16, 3 * g + 1);
                tma_load_pair(dst + 2 * kSlab, &map_k, bars + g * 8, y16, 3 * g + 2);
              }
            }
            __syncwarp();
          }
          if (t + 1 >= it.pt) {
            // Keys that no other pair reads come from HBM: ask for the next tile's
            // while this one is loaded (32 requests x 128 heads, own keys: 53.4 us
            // without, 51.4 with; asked for by every pair, a shared prefix's keys
            // cost more than they give: 61 x 16 rows 22.7 us against 21.4).
            // A box's rows are one piece of memory.
            if (lane < 64 / p.kbox && y_next < p.total_rows)
              bulk_prefetch_l2(p.cache + static_cast<int64_t>(y_next) * kRow, static_cast<uint32_t>(p.kbox * kRow * 2));
            __syncwarp();
          }
        } else {
          // All 128 keys, this CTA's columns: of output columns [256 j, 256 j + 256)
          // the half 128 rank .. + 128, as slabs 2 j and 2 j + 1 of each chunk.
          // The chunk that holds the end completes on a barrier of this CTA; its
          // rows past the end are zeroed here before the MMA thread hears of it.
          // (Out-of-range rows of the copy itself took up to 44 copies, 3.5 us.)
          // Chunks past the end are neither loaded nor multiplied.
#pragma unroll 1
          for (int c = 0; c < chunks_of(key0, limit); ++c) {
            const int keys = limit - (key0 + c * kVRows);
            const uint32_t dst = dst0 + c * kVChunk;
            const uint32_t full = bars + c * 8;
            const uint32_t bar = keys < kVRows ? map_to_cta(smem_u32(v_end), rank) : full;
            ok = wait_warp(&v_empty[c], ((vphase >> c) & 1) ^ 1, abort_flag, p.err);
            if (!ok) break;
            if (elect_one_sync()) {
              if (keys < kVRows)
                mbar_arrive_expect_tx(v_end, kVChunk);
              else if (rank == 0)
                mbar_arrive_expect_tx(&v_full[c], 2 * kVChunk);
              else
                mbar_arrive_cluster(full);
            }
            __syncwarp();
#pragma unroll 1
            for (int q = 0; q < kVRows; q += p.vbox) {
              const int y = __shfl_sync(0xFFFFFFFFu, y16, kVRows / 16 * c + (q >> 4));
              if (elect_one_sync()) {
                const uint32_t to = dst + q * 128;
                const int slab = static_cast<int>(rank) * 2;
                tma_load_pair(to, &map_v, bar, y, slab);
                tma_load_pair(to + 2 * kVSlab, &map_v, bar, y, slab + 4);
                if (p.vslabs == 1) {
                  tma_load_pair(to + kVSlab, &map_v, bar, y, slab + 1);
                  tma_load_pair(to + 3 * kVSlab, &map_v, bar, y, slab + 5);
                }
              }
              __syncwarp();
            }
            if (keys < kVRows) {
              ok = wait_warp(v_end, ends & 1, abort_flag, p.err);
              if (!ok) {
                wait_slow(smem_u32(v_end), ends & 1, nullptr, p.err);  // the copies in flight
                break;
              }
              ++ends;
#pragma unroll 1
              for (int e = keys * 8 + lane; e < kVRows * 8; e += 32)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                  *reinterpret_cast<uint4*>(smem + kOffV + c * kVChunk + s * kVSlab + e * 16) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_publish_cluster(full);
            }
            vphase ^= 1u << c;
          }
        }
      }
      ++i;
      v0 = 0;
    }
    if (*abort_flag && rank == 0) {
      // Copies of both CTAs complete on this CTA's barriers: wait for the last
      // phase each was armed for.
      if (seg > 0) wait_slow(smem_u32(q_full), (seg - 1) & 1, nullptr, p.err);
      if (is_k) {
#pragma unroll 1
        for (int g = 0; g < kKGroups; ++g)
          if (n > 0) wait_slow(smem_u32(&k_full[g]), (n - 1) & 1, nullptr, p.err);
      } else {
#pragma unroll 1
        for (int c = 0; c < kVChunks; ++c)
          if (n > 0) wait_slow(smem_u32(&v_full[c]), ((vphase >> c) & 1) ^ 1, nullptr, p.err);
      }
    }
  } else if (warp >= 6) {
    // ---- MMA (CTA 0 issues for the pair): scores (warp 6), output (warp 7) ----
    // One thread of each warp runs its whole role: votes and elections around each
    // of a tile's waits leave the tensor cores idle between products (64 x 128
    // rows, 32768 shared keys: 407 us against 358). Two roles, so that an item's
    // last output product is not queued behind the next item's first scores (61 x
    // 16 rows: 21.4 us with one thread for both, 20.9).
    const bool scores = warp == 6;
    if (rank == 0 && elect_one_sync()) {
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false), kIdO = idesc_bf16(128, 256, true);
      uint32_t n = 0, seg = 0;
      int left = nunits, i = item0, v0 = unit0;
      bool ok = true;
      if (scores) {
        const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + kOffQ)), kd = sdesc_kmajor_sw128(smem_u32(smem + kOffK));
#pragma unroll 1
        while (ok && left > 0 && i < p.items) {
          const Item it = get_item(p, i);
          const Span in = span_of(it.tiles, v0, left);
          left -= in.units;
          if (in.t1 > in.t0) ok = wait_one(q_full, seg++ & 1, abort_flag, p.err);
#pragma unroll 1
          for (int t = in.t0; ok && t < in.t1; ++t, ++n) {
            const uint32_t buf = n & 1, d = tmem + kTmemS + buf * 64;
            if (n > 1) ok = wait_cluster(&s_empty[buf], ((n >> 1) - 1) & 1, abort_flag, p.err);
#pragma unroll 1
            for (int g = 0; ok && g < kKGroups; ++g) {
              ok = wait_one(&k_full[g], n & 1, abort_flag, p.err);
              if (!ok) break;
              tc_fence_after_sync();
              const uint64_t ad = qd + static_cast<uint32_t>(g) * (kGroupBytes >> 4);
              const uint64_t bd = kd + static_cast<uint32_t>(g) * (kGroupBytes >> 4);
#pragma unroll
              for (int k = 0; k < 12; ++k)
                mma_bf16_pair(d, ad + (k >> 2) * (kSlab >> 4) + 2 * (k & 3), bd + (k >> 2) * (kSlab >> 4) + 2 * (k & 3),
                              kIdS, g > 0 || k > 0 ? 1u : 0u);
              mma_commit_pair(&k_empty[g]);
              if (g == kKGroups - 1) {
                mma_commit_pair(&s_full[buf]);
                if (t == in.t1 - 1) mma_commit_pair(q_empty);
              }
            }
          }
          ++i;
          v0 = 0;
        }
      } else {
        const uint64_t pd = sdesc_kmajor_sw128(smem_u32(smem + kOffP));
        const uint64_t vd = sdesc_mn_sw128(smem_u32(smem + kOffV), kVSlab);
        uint32_t vphase = 0;
#pragma unroll 1
        while (ok && left > 0 && i < p.items) {
          const Item it = get_item(p, i);
          const Span in = span_of(it.tiles, v0, left);
          left -= in.units;
          if (in.t1 > in.t0 && seg++ > 0) ok = wait_cluster(o_empty, (seg - 2) & 1, abort_flag, p.err);
#pragma unroll 1
          for (int t = in.t0; ok && t < in.t1; ++t, ++n) {
            const bool pre = t < it.pt;
            const int keys = (pre ? p.P : it.len) - (pre ? t : t - it.pt) * kTileKeys;
            const int chunks = chunks_of(0, keys);
            ok = wait_cluster(p_full, n & 1, abort_flag, p.err);
#pragma unroll 2
            for (int c = 0; ok && c < chunks; ++c) {
              ok = wait_one(&v_full[c], (vphase >> c) & 1, abort_flag, p.err);
              // (The end of the keys: zeros stored by both CTAs.)
              if (ok && keys < (c + 1) * kVRows) ok = wait_cluster(&v_full[c], (vphase >> c) & 1, abort_flag, p.err);
              if (!ok) break;
              tc_fence_after_sync();
              const uint64_t ad = pd + static_cast<uint32_t>(c) * (kSlab >> 4);
              const uint64_t bd = vd + static_cast<uint32_t>(c) * (kVChunk >> 4);
#pragma unroll
              for (int h = 0; h < kVRows / 16; ++h)  // 16 keys
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  mma_bf16_pair(tmem + j * 128, ad + 2 * h, bd + j * (2 * kVSlab >> 4) + h * (2048 >> 4), kIdO,
                                t == in.t0 && c == 0 && h == 0 ? 0u : 1u);
              mma_commit_pair(&v_empty[c]);
              if (c == chunks - 1) mma_commit_pair(pv_done);
              vphase ^= 1u << c;
            }
          }
          ++i;
          v0 = 0;
        }
      }
      if (!ok) {  // let the MMAs in flight finish before tensor memory is freed
        mma_commit_pair(drain + (scores ? 0 : 1));
        wait_slow(smem_u32(drain + (scores ? 0 : 1)), 0, nullptr, p.err);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax and stores ---------------------------------------------------
    if (p.direct && rank == 0) {
      // Nothing joins the rows later: those without any key become zeros here.
#pragma unroll 1
      for (int e = pair; e < p.items; e += npairs_max) {
        if (item_tiles(p, e)) continue;
        const Item z = get_item(p, e);
#pragma unroll 1
        for (int k = tid; k < z.nrows * (kC / 8); k += 128)
          reinterpret_cast<uint4*>(p.out + z.row0 * static_cast<int64_t>(kC))[k] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse)
          for (int k = tid; k < z.nrows; k += 128) p.lse[z.row0 + k] = -INFINITY;
      }
    }
    const int row = (warp & 1) * 32 + lane;   // of this CTA's 64
    const int kh = warp >> 1;                 // key half of the scores, column half of the output
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t leader_p = map_to_cta(smem_u32(p_full), 0), leader_o = map_to_cta(smem_u32(o_empty), 0);
    uint8_t* prow = smem + kOffP + kh * kSlab + row * 128;
    uint32_t n = 0, nred = 0;
    int left = nunits, i = item0, v0 = unit0;
    bool ok = true;
    // Both threads of a row give a value; returns the partner's (bounded wait:
    // the four warps meet on an mbarrier).
    auto exchange = [&](float v) {
      float* r = red + (nred & 1) * 128;
      r[kh * 64 + row] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(red_bar);
      ok = ok && wait_warp(red_bar, nred & 1, abort_flag, p.err);
      ++nred;
      return r[(kh ^ 1) * 64 + row];
    };
#pragma unroll 1
    while (ok && left > 0 && i < p.items) {
      const Item it = get_item(p, i);
      const Span in = span_of(it.tiles, v0, left);
      const int t0 = in.t0, t1 = in.t1;
      left -= in.units;
      const int rt = static_cast<int>(rank) * 64 + row;  // row of the tile
      const bool have = rt < it.nrows;
      float m = -INFINITY, l = 0.f, lx = 0.f;  // running maximum, sums of rounded and of fp32 weights
#pragma unroll 1
      for (int t = t0; ok && t < t1; ++t, ++n) {
        const bool pre = t < it.pt;
        const int key0 = (pre ? t : t - it.pt) * kTileKeys;
        const int valid = have ? (pre ? p.P : it.len) - key0 - kh * 64 : 0;  // keys of this half that count
        const uint32_t buf = n & 1;
        ok = wait_warp(&s_full[buf], (n >> 1) & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t s[64];
        tmem_ld_32x32b_x64(t_lane + kTmemS + buf * 64, s);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_u32(&s_empty[buf]), 0));
        if (valid < 64) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j >= valid) s[j] = 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]));
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        mt = fmaxf(mt, exchange(mt)) * p.scale_log2;
        if (!ok) break;
        float fix = 1.f;
        bool raised = false;
        if (mt > m + kRaise) {
          raised = m != -INFINITY;  // a row without keys so far has no output to rescale
          fix = ex2(m - mt);
          m = mt;
        }
        const bool rescale = __any_sync(0xFFFFFFFFu, raised);
        l *= fix;
        lx *= fix;
        const float mu = m == -INFINITY ? 0.f : m;
        uint32_t w[32];
        float sum[4] = {0.f, 0.f, 0.f, 0.f}, sx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float a = ex2(fmaf(__uint_as_float(s[2 * j]), p.scale_log2, -mu));
          const float b = ex2(fmaf(__uint_as_float(s[2 * j + 1]), p.scale_log2, -mu));
          const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
          w[j] = *reinterpret_cast<const uint32_t*>(&r);
          sum[2 * (j & 1)] += __uint_as_float(w[j] << 16);
          sum[2 * (j & 1) + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
          sx[2 * (j & 1)] += a;
          sx[2 * (j & 1) + 1] += b;
        }
        lx += (sx[0] + sx[1]) + (sx[2] + sx[3]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // The previous tile's output product has read P and written the output.
        if (n > 0) {
          ok = wait_warp(pv_done, (n - 1) & 1, abort_flag, p.err);
          if (!ok) break;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(prow + ((c ^ (row & 7)) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        if (rescale && t > t0) {
          tc_fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_lane + c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fix);
            tmem_st_32x32b_x32(t_lane + c, o);
          }
          tmem_wait_st();
          tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_publish_cluster(leader_p);
      }
      if (ok && t1 > t0) {
        const float lt = l + exchange(l);
        const float lxt = lx + exchange(lx);
        ok = ok && wait_warp(pv_done, (n - 1) & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after_sync();
        const bool cut = t0 > 0 || t1 < it.tiles || (!p.merged && p.prefix_tiles > 0);
        const int64_t r = it.row0 + rt;
        // Rows leave through this warp's quarter of the P buffer (its readers are
        // done), 128 bytes of 32 rows at a time, so that stores cover whole
        // lines: 16-byte chunk j of row r sits at chunk j ^ (r % 8).
        uint8_t* stage = smem + kOffP + warp * 4096;
        const int r0 = static_cast<int>(rank) * 64 + (warp & 1) * 32;  // tile row of lane 0
        auto store_rows = [&](const uint32_t (&v)[32], uint8_t* dst, int64_t pitch) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int rr = q * 4 + (lane >> 3);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane ^ rr) & 7) << 4));
            if (r0 + rr < it.nrows) *reinterpret_cast<uint4*>(dst + rr * pitch + (lane & 7) * 16) = x;
          }
          __syncwarp();
        };
        if (!cut) {
          const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;  // NaN stays NaN
          uint8_t* dst = reinterpret_cast<uint8_t*>(p.out + (it.row0 + r0) * static_cast<int64_t>(kC) + kh * 128);
#pragma unroll 1
          for (int c = 0; c < 256; c += 64) {
            uint32_t o[64], v[32];
            tmem_ld_32x32b_x64(t_lane + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv,
                                                              __uint_as_float(o[2 * e + 1]) * inv);
              v[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            store_rows(v, dst + ((c >> 7) * 256 + (c & 127)) * 2, kC * 2);
          }
          if (have && kh == 0 && p.lse) p.lse[r] = m * 0.69314718055994531f + logf(lxt);
        } else {
          const int64_t pr = part_row(p.merged, p.prefix_items, p.own_rows, i, pair);
          const int pitch = it.b >= 0 && !p.merged ? p.own_rows : kTileRows;
          float4* dst = p.part_o + pr * (kC / 4) + rt;
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_lane + c, o);
            if (have) {
              float4* q = dst + ((c >> 7) * 64 + kh * 32 + (c & 127) / 4) * pitch;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                q[j * pitch] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                           __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
            }
          }
          if (have && kh == 0) p.part_ml[pr + rt] = make_float4(m, lt, lxt, 0.f);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_o);
      }
      ++i;
      v0 = 0;
    }
  }

  griddep_launch_dependents();  // not earlier: the join's waiting CTAs would share the SMs
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 6) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of each query row, in item and key order: with weights
// 2^(m_k - max m), out = sum w_k O_k / sum w_k l_k. A lane has one row and Q
// quads of columns (a warp's 32 rows of a quad are contiguous in a part); U
// parts are loaded together, then added under a running maximum. S warps share
// a row's parts and meet in shared memory in warp order. The fewer the rows,
// the more parts each has and the more warps they need: <1, 8, 6> up to 256 rows,
// <4, 2, 4> up to 2048, <8, 1, 3> beyond. Whole calls, heads of 128: 256 rows of
// 38 parts 25.1 us with the first, 29.3 with the second; 512 rows 34.2 and 30.9;
// 1024 rows 42.3 with the second, 46.4 with the third; 2048 rows 44.5 with
// either; 2560 rows 51.5 and 49.5. Rows whose one item was not cut were stored by
// the attention kernel; rows without any key become zeros.
template <int Q, int S, int U>
__global__ void __launch_bounds__(S > 1 ? S * 32 : 128) mla_join_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.B * p.H;
  const int r = static_cast<int>(blockIdx.x) * 32 + lane;
  const int quad = (S > 1 ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) * 4 + warp) * Q;
  const int slot = S > 1 ? warp : 0;
  const int rc = min(r, rows - 1), b = rc / p.H, h = rc - b * p.H;
  const int units = p.plan[0], pairs = p.plan[1];
  // Up to two items hold the row's keys: the prefix's (or both together) and
  // its own. Per item: parts, first part's row and quad-0 address, quad pitch.
  int n[2] = {0, 0};
  int64_t at[2] = {0, 0};
  int local[2], pitch[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int item = -1;
    if (k == 0 && (p.merged || p.prefix_tiles > 0)) item = rc / kTileRows;
    if (k == 1 && !p.merged) item = p.prefix_items + b * p.per + h / kTileRows;
    local[k] = k == 0 ? r % kTileRows : h % kTileRows;
    pitch[k] = k == 0 ? kTileRows : p.own_rows;
    if (item < 0) continue;
    const int a = p.plan[2 + item], e = p.plan[3 + item];
    if (e <= a) continue;
    const int q0 = pair_of_unit(units, pairs, a + kItemCost);  // the first tile's
    n[k] = pair_of_unit(units, pairs, e - 1) - q0 + 1;
    at[k] = part_row(p.merged, p.prefix_items, p.own_rows, item, q0);
  }
  const int parts = r < rows ? n[0] + n[1] : 0;
  const bool stored = r >= rows || (parts == 1 && (p.merged || p.prefix_tiles == 0));
  if (__all_sync(0xFFFFFFFFu, stored) && S == 1) return;
  const int todo = stored ? 0 : parts;
  constexpr int kStride = kTileRows * (kC / 4);  // from a part to the next pair's, in vectors
  float m = -INFINITY, l = 0.f, lx = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int c = 0; c < Q; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = slot; k0 < todo; k0 += S * U) {
    float4 ml[U], v[U][Q];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * S, g = k < n[0] ? 0 : 1, kk = k - (g ? n[0] : 0);
      ml[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < Q; ++c) v[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < todo) {
        ml[u] = p.part_ml[at[g] + static_cast<int64_t>(kk) * kTileRows + local[g]];
        const float4* src = p.part_o + at[g] * (kC / 4) + static_cast<int64_t>(kk) * kStride +
                            static_cast<int64_t>(quad) * pitch[g] + local[g];
#pragma unroll
        for (int c = 0; c < Q; ++c) v[u][c] = __ldcg(src + c * pitch[g]);
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float w0 = ex2(m - mu);
    m = mn;
    l *= w0;
    lx *= w0;
#pragma unroll
    for (int c = 0; c < Q; ++c) acc[c] = make_float4(acc[c].x * w0, acc[c].y * w0, acc[c].z * w0, acc[c].w * w0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = ex2(ml[u].x - mu);
      l = fmaf(ml[u].y, w, l);
      lx = fmaf(ml[u].z, w, lx);
#pragma unroll
      for (int c = 0; c < Q; ++c) {
        acc[c].x = fmaf(v[u][c].x, w, acc[c].x);
        acc[c].y = fmaf(v[u][c].y, w, acc[c].y);
        acc[c].z = fmaf(v[u][c].z, w, acc[c].z);
        acc[c].w = fmaf(v[u][c].w, w, acc[c].w);
      }
    }
  }
  float mm = m;
  if constexpr (S > 1) {
    __shared__ float red_s[S][3][32];
    __shared__ float4 acc_s[S - 1][Q][32];
    red_s[warp][0][lane] = m;
    red_s[warp][1][lane] = l;
    red_s[warp][2][lane] = lx;
    if (warp > 0)
#pragma unroll
      for (int c = 0; c < Q; ++c) acc_s[warp - 1][c][lane] = acc[c];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 1; k < S; ++k) mm = fmaxf(mm, red_s[k][0][lane]);
    const float mz = mm == -INFINITY ? 0.f : mm;
    const float w0 = ex2(m - mz);
    l *= w0;
    lx *= w0;
#pragma unroll
    for (int c = 0; c < Q; ++c) acc[c] = make_float4(acc[c].x * w0, acc[c].y * w0, acc[c].z * w0, acc[c].w * w0);
#pragma unroll
    for (int k = 1; k < S; ++k) {
      const float w = ex2(red_s[k][0][lane] - mz);
      l = fmaf(red_s[k][1][lane], w, l);
      lx = fmaf(red_s[k][2][lane], w, lx);
#pragma unroll
      for (int c = 0; c < Q; ++c) {
        const float4 o = acc_s[k - 1][c][lane];
        acc[c] = make_float4(fmaf(o.x, w, acc[c].x), fmaf(o.y, w, acc[c].y), fmaf(o.z, w, acc[c].z),
                             fmaf(o.w, w, acc[c].w));
      }
    }
  }
  if (stored) return;
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
  uint2 o[Q];
#pragma unroll
  for (int c = 0; c < Q; ++c) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv),
                         y = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    o[c] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  uint2* dst = reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(r) * kC) + quad;
  if constexpr (Q % 2 == 0) {
#pragma unroll
    for (int c = 0; c < Q; c += 2)
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(o[c].x, o[c].y, o[c + 1].x, o[c + 1].y);
  } else {
#pragma unroll
    for (int c = 0; c < Q; ++c) dst[c] = o[c];
  }
  if (quad == 0 && p.lse)
    p.lse[r] = l == 0.f ? -INFINITY : mm * 0.69314718055994531f + logf(lx);
}

// ---- host --------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn attention_map_encoder() {
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

// bf16 rows x cols as (64 columns, row, slab): boxes of 64 columns x box_rows
// x box_slabs, 128-byte swizzled, a slab's rows together.
bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, int box_rows, int box_slabs) {
  EncodeTiledFn enc = attention_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, rows, cols / 64};
  const cuuint64_t strides[2] = {cols * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_slabs)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

struct AttnSizes {
  bool merged;
  int64_t prefix_items, items, own_rows, part_rows;
  size_t plan_bytes, ml_bytes, o_bytes;
};

AttnSizes attention_sizes(int64_t B, int64_t H, int64_t P) {
  AttnSizes z{};
  z.merged = H % kTileRows == 0;
  z.own_rows = H < kTileRows ? H : kTileRows;
  const int64_t per = (H + kTileRows - 1) / kTileRows;
  z.prefix_items = !z.merged && P > 0 ? (B * H + kTileRows - 1) / kTileRows : 0;
  z.items = z.merged ? B * per : z.prefix_items + B * per;
  z.part_rows = part_row(z.merged, static_cast<int>(z.prefix_items), static_cast<int>(z.own_rows),
                         static_cast<int>(z.items), kMaxPairs);
  z.plan_bytes = align256(static_cast<size_t>(z.items + 3) * 4);
  z.ml_bytes = align256(static_cast<size_t>(z.part_rows) * 16);
  z.o_bytes = static_cast<size_t>(z.part_rows) * kC * 4;
  return z;
}

bool attention_shape_ok(int64_t B, int64_t H, int64_t P) {
  return B >= 0 && H >= 1 && H <= 1024 && P >= 0 && P <= (int64_t{1} << 30) && B <= (int64_t{1} << 20) &&
         B * H <= (int64_t{1} << 24);
}

// CTA pairs that run at once (one CTA per SM).
int resident_pairs(const DevInfo* d) {
  static int cached[64] = {};
  if (d->device < 64 && cached[d->device]) return cached[d->device];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d->sm_count / 2 * 2));
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kAttnSmem;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, mla_attention_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = d->sm_count / 2;
  }
  if (n > kMaxPairs) n = kMaxPairs;
  if (d->device < 64) cached[d->device] = n;
  return n;
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_mla_attention_workspace_bytes(int64_t B, int64_t H, int64_t prefix_len) {
  if (!attention_shape_ok(B, H, prefix_len)) return 0;
  const AttnSizes z = attention_sizes(B, H, prefix_len);
  return z.plan_bytes + z.ml_bytes + z.o_bytes;
}

extern "C" int fp8blk_mla_attention(const void* q_bf16, const void* q_pe_bf16, int64_t B, int64_t H,
                                    const void* cache_bf16, int64_t num_pages, int64_t page_size,
                                    const int32_t* prefix_pages, int64_t prefix_len, const int32_t* block_table,
                                    int64_t table_stride, const int32_t* lens, float scale, void* out_bf16, float* lse,
                                    void* workspace, size_t workspace_bytes, fp8blk_stream_t stream) {
  if (!attention_shape_ok(B, H, prefix_len)) return FP8BLK_ERR_SHAPE;
  if (page_size < 16 || page_size % 16 || num_pages < 0 || table_stride < 0 ||
      num_pages * page_size > (int64_t{1} << 31) - 129 || table_stride * page_size > (int64_t{1} << 30) ||
      page_size > (int64_t{1} << 20))
    return FP8BLK_ERR_SHAPE;
  if (!(scale > 0.0f) || scale > 1e30f) return FP8BLK_ERR_ARG;
  if (B == 0) return FP8BLK_OK;
  if (!q_bf16 || !q_pe_bf16 || !lens || !out_bf16 || (num_pages > 0 && !cache_bf16) ||
      (prefix_len > 0 && !prefix_pages) || (table_stride > 0 && !block_table))
    return FP8BLK_ERR_NULL;
  if (!is_aligned(q_bf16, 16) || !is_aligned(q_pe_bf16, 16) || !is_aligned(cache_bf16, 16) ||
      !is_aligned(out_bf16, 16) || !is_aligned(lens, 4) || !is_aligned(prefix_pages, 4) ||
      !is_aligned(block_table, 4) || !is_aligned(lse, 4))
    return FP8BLK_ERR_ALIGN;
  if (!workspace) return FP8BLK_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return FP8BLK_ERR_ALIGN;
  const AttnSizes z = attention_sizes(B, H, prefix_len);
  if (workspace_bytes < z.plan_bytes + z.ml_bytes + z.o_bytes) return FP8BLK_ERR_WORKSPACE;
  // The tile counts stay below 2^30.
  const int64_t most = (prefix_len + kTileKeys - 1) / kTileKeys * (z.merged ? z.items : z.prefix_items) +
                       (table_stride * page_size / kTileKeys + 1) * (z.items - z.prefix_items) + kItemCost * z.items;
  if (most >= int64_t{1} << 30) return FP8BLK_ERR_SHAPE;
  const DevInfo* d;
  if (int st = current_device(&d)) return st;
  static bool attr_done[64] = {};
  if (d->device >= 64 || !attr_done[d->device]) {
    if (cudaFuncSetAttribute(mla_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem) !=
        cudaSuccess)
      return FP8BLK_ERR_CUDA;
    if (d->device < 64) attr_done[d->device] = true;
  }
  AttnParams p{};
  p.cache = static_cast<const __nv_bfloat16*>(cache_bf16);
  p.prefix_pages = prefix_pages;
  p.table = block_table;
  p.lens = lens;
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float4*>(ws + z.plan_bytes);
  p.part_o = reinterpret_cast<float4*>(ws + z.plan_bytes + z.ml_bytes);
  p.err = d->err_word;
  p.B = static_cast<int>(B);
  p.H = static_cast<int>(H);
  p.P = static_cast<int>(prefix_len);
  p.page = static_cast<int>(page_size);
  p.per = static_cast<int>((H + kTileRows - 1) / kTileRows);
  p.by_page = divisor(page_size);
  p.by_per = divisor(p.per);
  p.by_pairs = divisor(resident_pairs(d));
  p.num_pages = static_cast<int>(num_pages);
  p.table_stride = static_cast<int>(table_stride);
  p.max_own = static_cast<int>(table_stride * page_size);
  p.total_rows = static_cast<int>(num_pages * page_size);
  p.prefix_tiles = static_cast<int>((prefix_len + kTileKeys - 1) / kTileKeys);
  p.prefix_items = static_cast<int>(z.prefix_items);
  p.items = static_cast<int>(z.items);
  p.own_rows = static_cast<int>(z.own_rows);
  p.merged = z.merged ? 1 : 0;
  p.kbox = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  p.vbox = page_size % kVRows == 0 ? kVRows : page_size % 32 == 0 ? 32 : 16;
  p.kslabs = p.kbox == 64 ? 3 : 1;
  p.vslabs = p.vbox == kVRows ? 2 : 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.direct = (z.merged || p.prefix_tiles == 0) && p.prefix_tiles + (p.max_own + kTileKeys - 1) / kTileKeys <= 1;
  // A cache without pages is never read: its maps describe one row of q.
  const void* cbase = num_pages > 0 ? cache_bf16 : q_bf16;
  const uint64_t crows = num_pages > 0 ? static_cast<uint64_t>(num_pages * page_size) : 1;
  const uint64_t ccols = num_pages > 0 ? kRow : kC;
  CUtensorMap mq, mqp, mk, mv;
  if (!make_bf16_map(&mq, q_bf16, static_cast<uint64_t>(B * H), kC, 64, kC / 64) ||
      !make_bf16_map(&mqp, q_pe_bf16, static_cast<uint64_t>(B * H), kR, 64, 1) ||
      !make_bf16_map(&mk, cbase, crows, ccols, p.kbox, p.kslabs) ||
      !make_bf16_map(&mv, cbase, crows, ccols, p.vbox, p.vslabs))
    return FP8BLK_ERR_CUDA;
  if (num_pages == 0) p.total_rows = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * resident_pairs(d)));
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kAttnSmem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (int st = cuda_status(cudaLaunchKernelEx(&cfg, mla_attention_kernel, mq, mqp, mk, mv, p))) return st;
  if (p.direct) return FP8BLK_OK;
  const int64_t rows = B * H;
  const int variant = rows <= 256 ? 0 : rows <= 2048 ? 1 : 2;
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3(static_cast<unsigned>((rows + 31) / 32), variant == 0 ? kC / 4 : variant == 1 ? kC / 16 : kC / 128);
  join.blockDim = dim3(variant == 0 ? 256 : variant == 1 ? 64 : 128);
  join.stream = cfg.stream;
  join.attrs = attr;
  join.numAttrs = 1;
  return cuda_status(variant == 0   ? cudaLaunchKernelEx(&join, mla_join_kernel<1, 8, 6>, p)
                     : variant == 1 ? cudaLaunchKernelEx(&join, mla_join_kernel<4, 2, 4>, p)
                                    : cudaLaunchKernelEx(&join, mla_join_kernel<8, 1, 3>, p));
}
