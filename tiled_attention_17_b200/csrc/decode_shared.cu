// Paged decode of a batch whose sequences share long prefixes: the prefix of a
// group of sequences is read and multiplied once for all of them.
//
// Softmax over a sequence's keys splits exactly into softmax over the group's
// prefix and softmax over the keys the sequence has of its own, joined by their
// log-sum-exp (FlashAttention optimisation article, section 3.2.2).  Decode
// alone reads every key once per sequence and is bound by those bytes.  Over a
// shared prefix the queries of the whole group meet each key, so the prefix is
// a matrix product: rows are (sequence, query head of one KV head) pairs, 128
// to a tile, and a K/V tile of 128 keys is read once for up to 256 rows.
//
// Own keys go through the tensor cores too, with the products transposed (S^T =
// K Q^T, O^T = V^T P^T: keys, then columns of d, on the 128 rows and 16 columns of
// queries).  The dot products of the paged decode are bound by instructions at
// such short lengths: 48 us against 10 us of bytes for 64 sequences of about 256
// own tokens, 104 us against 8 us with groups of 8 heads at d = 64.
//
// Measured (B200, whole call, L2 cold): 64 sequences, 32 + 8 heads of 128, 8000
// shared and up to 512 own tokens 42 us (the bytes alone 15); 96 sequences in 6
// groups, 32 + 4 heads of 64, 5000 shared and up to 1024 own tokens 45 us (12);
// 256 sequences behind 30000 tokens 162 us, 188 in a long run, whose power holds the
// SM clock at 1.64 GHz instead of 1.97 (products 77).  The time
// goes to the start (6 us: plan, tensor memory, first tiles), the steps, and the
// join (7 us).  A step with two row tiles, 128 keys, takes 3800 cycles, of which
// tensor pipe 2600 (products of 64 keys are bound by the reads of Q from shared
// memory) and exponentials 2050: neither role waits for the other any more.
//
// Two kernels, the second a programmatic dependent of the first:
//   shared_attend_kernel   all products, cut evenly over the SMs
//   shared_combine_kernel  joins a row's partials by their log-sum-exp
//
// Work.  An item is a group's prefix or a sequence's own keys; a unit is (item,
// KV head, block of 256 query rows); its steps are 128-key tiles.  All units'
// steps are laid end to end, each as long as its cost (more with more than 128
// rows), and CTA c of n takes the steps that start in
// [c L, (c + 1) L), L = ceil(total / n): equal shares whatever the groups' sizes
// and lengths, at the price of partial results per CTA and unit it touches.
// The (c, unit) pairs met along the line are monotone in both, so slot
// c + unit holds a pair's partials without a table.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"
#include "tiledattn_internal.h"

namespace ta {
namespace {

constexpr int kTile = 128;           // query rows and keys of a tile
constexpr int kUnitRows = 2 * kTile;
// warp 0 plans, 1 and 12 issue the products of row tile 0 and 1, 2 copies queries and K, 3 copies V, 4-7 and 8-11 are
// the softmax warpgroups of row tile 0 and 1
constexpr int kThreads = 416;
constexpr int kSoftmaxWarp0 = 4, kMmaWarp1 = 12;
constexpr float kRescaleLog2 = 8.0f;   // the stale-max margin of the prefill kernel
// Cost of a step with two row tiles, and with one.  Measured 2.33 us (256 samples
// behind 30000 shared tokens: both tiles' softmax; 3800 cycles at the 1.64 GHz of a
// long run) and 1.36 us (their own tokens, segments of one or two steps: latency);
// at 2 : 1 the last CTA ended 17% after the median.  All of these are of d = 128 and 4
// heads a group, and are used for every layout: at d = 64 a wide step has half the
// products and the same exponentials, and its own costs were not measured.
// A further unit with wide steps costs a CTA some 4 us more than the steps (its
// partial is 128 KB, and the pipeline starts again): without a cost of its own the
// CTAs with two of them ended 25% after the median of a small batch.
constexpr int kWideCost = 5, kNarrowCost = 3, kWideStart = 8;
// Cycles between the row tiles' first softmax of a wide segment (why: where it is waited).  With and without, us a call
// of a long run: d = 128, 4 heads a group, 6 groups of 64 sequences behind 4000 tokens 80.1 / 85.0, 64 behind 8000 43.4 /
// 43.7, 256 behind 30000 183.0 / 183.6; d = 64, 8 heads, within 0.3% (96 behind 5000 32.9 / 32.9, 256 behind 20000 133.0 /
// 132.5, 40 groups of 32 behind 1000 123.9 / 123.8), and so are segments of a single wide step (20 groups of 64 behind 112
// tokens, d = 128, 144.3 / 144.3).
constexpr int kApart = 1000;

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// mbar_wait with its bounded loop out of line: the attend kernel waits at some
// thirty places, and its roles share one instruction cache.
__device__ __noinline__ bool wait_loop(uint32_t bar, uint32_t parity, unsigned* status, volatile int* abort_flag) {
  return mbar_wait(bar, parity, status, abort_flag);
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, unsigned* status, volatile int* abort_flag) {
  const bool ok = mbar_try_wait(bar, parity) || wait_loop(bar, parity, status, abort_flag);
  return __all_sync(0xffffffffu, ok);   // one answer for the warp
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Eight, or four, 32-bit columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
// Largest of a value over the warp (one instruction on sm_100a).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// One group's prefix or one sequence's own keys, ranges checked.
struct Item {
  long long x0;   // its place on the line of costs
  int unit0;      // units of its kind before it
  int first, n;   // first sequence, number of sequences (own keys: 1)
  int base;       // first key of its first tile (the start of a page)
  int lo, end;    // its keys: [base + lo, end); none if end <= base
  int group;      // own keys: the group whose prefix the sequence uses, or -1
};

// What the combine kernel needs of the plan.
struct __align__(16) GroupPlan {
  long long x0;
  int unit0, first, n, tiles, pad[2];
};
struct __align__(16) SeqPlan {
  long long x0;   // of its own keys
  int tiles, group;
};

__host__ __device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
__host__ __device__ __forceinline__ int blocks_of(int n, int G) { return (n * G + kUnitRows - 1) / kUnitRows; }   // of rows
__host__ __device__ __forceinline__ int cost_of(int n, int G) { return n * G > kTile ? kWideCost : kNarrowCost; }   // of a step
// A unit's length on the line: what it costs to start, then its steps.
__host__ __device__ __forceinline__ int start_of(int cost) { return cost == kWideCost ? kWideStart : 0; }
__host__ __device__ __forceinline__ long long unit_cost(int tiles, int cost) {
  return tiles > 0 ? static_cast<long long>(tiles) * cost + start_of(cost) : 0;
}

struct SharedArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* group_offsets;
  const int32_t* prefix_lens;
  int page_size, page_shift, g_shift;   // page_size = 1 << page_shift, G = 1 << g_shift
  int num_seqs, num_groups, Hq, Hkv, G, max_pages, num_pages_total, n_ctas, max_own;
  float scale, scale_log2;
  // workspace
  unsigned* status;       // the call's status word (written by the combine kernel)
  unsigned* cta_status;   // [n_ctas]
  long long* per_cta;     // cost of one CTA's share
  GroupPlan* groups;      // [num_groups]
  SeqPlan* seqs;          // [num_seqs]
  float* pre_o;           // [slots][D / 4][256][4] normalised prefix partials
  float* pre_lse;         // [slots][256]
  float* own_o;           // [slots][2][G][D] normalised partials of own keys
  float* own_lse;         // [slots][2][G]
};

// Item i: a group's prefix (i < groups) or the own keys of sequence i - groups;
// beyond the last sequence one without keys.  x0 and unit0 are left open.
__device__ __forceinline__ Item describe_item(const SharedArgs& a, int groups, int i, bool& bad) {
  const int cap = a.max_pages * a.page_size;
  Item r = {};
  r.group = -1;
  if (i < groups) {
    const int len = __ldg(a.prefix_lens + i);
    r.first = __ldg(a.group_offsets + i);
    r.n = __ldg(a.group_offsets + i + 1) - r.first;
    if (r.n > 0) {   // a group without sequences shares nothing, whatever its length
      r.end = min(max(len, 0), cap);
      bad = bad || r.end != len;
    }
  } else if (i - groups < a.num_seqs) {
    const int s = i - groups, raw = __ldg(a.seq_lens + s);
    int len = min(max(raw, 0), cap), start = 0;
    int lo = 0, hi = groups;   // the first group whose end lies behind s
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.group_offsets + mid + 1) <= s) lo = mid + 1;
      else hi = mid;
    }
    if (lo < groups && __ldg(a.group_offsets + lo) <= s) {
      // a sequence shorter than its group's prefix does not use it: all its keys are its own
      const int prefix = min(max(__ldg(a.prefix_lens + lo), 0), cap);
      if (prefix > 0 && len >= prefix) {
        start = prefix;
        r.group = lo;
      }
    }
    bad = bad || raw != len || len - start > a.max_own;
    len = min(len, start + a.max_own);
    r.first = s;
    r.n = 1;
    r.base = start & ~(a.page_size - 1);
    r.lo = start - r.base;
    r.end = len > start ? len : r.base;
  }
  return r;
}

// 32 items, one a lane, with their costs and places: base and base_u are those of
// the first; moved on to the next 32.  (Out of line: called from three places,
// none of them hot.  A CTA's first call takes 2.5 us, L2 cold or warm: the loads are
// a few dependent ones, most of it is the first fetch of the instructions, so the
// plan divides by shifts and products.)
struct Window {
  Item it;
  long long cost;
};
__device__ __noinline__ Window load_window(const SharedArgs& a, int groups, int w, long long& base, int& base_u,
                                           bool& bad) {
  const int lane = threadIdx.x & 31, i = w * 32 + lane;
  Window r;
  r.it = describe_item(a, groups, i, bad);
  if (r.it.end > r.it.base)   // its first pages' table entries, soon wanted by the CTA that starts there
    prefetch_l2(a.block_table + static_cast<size_t>(r.it.first) * a.max_pages + (r.it.base >> a.page_shift));
  const int tiles = tiles_of(r.it.end - r.it.base);
  const int units = tiles > 0 ? blocks_of(r.it.n, a.G) * a.Hkv : 0, own_units = i < groups ? units : 0;
  r.cost = units * unit_cost(tiles, cost_of(r.it.n, a.G));
  long long sum = r.cost;
  int sum_u = own_units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, sum, o);
    const int y = __shfl_up_sync(0xffffffffu, sum_u, o);
    if (lane >= o) {
      sum += x;
      sum_u += y;
    }
  }
  r.it.x0 = base + sum - r.cost;
  r.it.unit0 = i < groups ? base_u + sum_u - own_units : r.it.first * a.Hkv;
  base += __shfl_sync(0xffffffffu, sum, 31);
  base_u += __shfl_sync(0xffffffffu, sum_u, 31);
  return r;
}

// x / cost rounded up, x >= 0: the high half of a product with 2^66 / 5 or 2^65 / 3 rounded up, exact for 64 bits.
static_assert(kWideCost == 5 && kNarrowCost == 3, "the reciprocals below");
__device__ __forceinline__ long long steps_in(long long x, int cost) {
  const unsigned long long u = static_cast<unsigned long long>(x) + static_cast<unsigned>(cost - 1);
  const bool wide = cost == kWideCost;
  return static_cast<long long>(__umul64hi(u, wide ? 0xCCCCCCCCCCCCCCCDull : 0xAAAAAAAAAAAAAAABull) >> (wide ? 2 : 1));
}
// Steps of a unit that start in CTA c's share (which reaches into the unit):
// [j0, j1) of `tiles`, x0 the unit's place on the line, `cost` a step's.  None
// where the share ends before the first, or begins inside the last.
__device__ __forceinline__ void unit_share(long long x0, int tiles, int cost, long long per, int c, int& j0, int& j1) {
  const long long a = per * c - x0 - start_of(cost);
  j0 = a <= 0 ? 0 : static_cast<int>(steps_in(a, cost));
  const long long e = a + per <= 0 ? 0 : steps_in(a + per, cost);
  j1 = e < tiles ? static_cast<int>(e) : tiles;
}

// ---------------------------------------------------------------------------
// Attend
// ---------------------------------------------------------------------------
// A segment: the steps of one unit that one CTA takes.  The producer describes
// each to the other roles through a ring in shared memory.  Rows up to 128
// ("narrow"): steps alternate between the two row tiles of the CTA, which both
// hold the same query rows, so two softmax warpgroups work on two key tiles at
// once; each tile's steps give a partial of their own.  More rows ("wide"):
// both tiles take every step, each with its own rows.
struct __align__(16) Segment {
  uint32_t g0;     // ring position of its first key tile
  int tiles;       // steps; 0 ends the work
  int wide;        // 1: two row tiles in every step
  int tile_first;  // narrow: the row tile of step 0
  int rows;        // query rows of the unit (1..256)
  int lo, hi;      // keys, counted from its first key tile: [lo, hi)
  int slot;        // of its partials: >= 0 prefix, ~slot own keys
  int hkv, seq;    // KV head, first sequence of the query rows
  int row, page0;  // block-table row, its first page
  int qslot;       // own keys: where in the query buffers its rows are (in 8 rows)
  int pad[3];
  int pages[kTile / 8];   // physical pages of its first key tile, -1 past the keys
};
static_assert(sizeof(Segment) == 128, "16-byte loads");
constexpr int kSegments = 4;   // ring depth
// Query loads of a row tile that may be outstanding: a segment is described
// only when the one kSegments before it has been taken up by every role, so
// more than kSegments of them cannot be.
constexpr uint32_t kQLoads = 8;
// Own keys have at most 8 query rows.  Their loads go round 8 places of 8 rows in
// the first half of a query buffer, so the loads of the next segments need not
// wait for the products of this one; the second half takes the weights of two
// steps (prefixes come first on the line, so no whole query tile follows).
constexpr int kQSlots = 8, kOwnP = 64 * 128, kOwnPBytes = 4096;
constexpr int kOwnCols = 16;   // columns of the own-keys products: 8 rows of queries, and 8 that do not count

constexpr int kMaxWindows = (2 * 65535 + 31) / 32;   // of 32 items

template <int D>
struct AttendLayout {
  static constexpr int kChunks = D / 64;               // 128-byte swizzle rows along d
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kChunkBytes = kTile * 128;
  // ring depths: K tiles are free once their scores are formed, V tiles only
  // after the softmax, so V gets the one that is left of 227 KB
  static constexpr int kKStages = D == 128 ? 2 : 4, kVStages = D == 128 ? 3 : 6;
  // A tile's arrival has a barrier of its own number, from a ring longer than the
  // slots.  A wait sees its phase's parity only, so whoever waits for tile g must
  // know that tile g - R, the one before on that barrier, has landed; a row tile that
  // takes every other step never waits for the steps between.  It has seen K tile
  // g - 2 or a later one (V: g - 4, scores run ahead of the products), and copies go
  // out in order, each after the release of the tile one slot ring before: all up to
  // g - 2 - kKStages (g - 4 - kVStages) have landed.
  static constexpr int kKBars = D == 128 ? 4 : 8, kVBars = D == 128 ? 8 : 16;
  static_assert(kKBars >= kKStages + 2 && kVBars >= kVStages + 4, "a barrier's phase before has completed");
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kSeg = kV + kVStages * kTileBytes;
  static constexpr int kRed = kSeg + kSegments * static_cast<int>(sizeof(Segment));   // [row tile][2][4 warps][8] floats
  static constexpr int kBar = kRed + 2 * 2 * 4 * 8 * 4;
  // k_full, v_full, k_empty, v_empty; per row tile: s_full[2], p_ready[2], o_free, o_done[2], exchange, own s_full[2], q_full[]; segment full, empty;
  // mma_done, windows read
  static constexpr int kNumBars = kKBars + kVBars + kKStages + kVStages + 20 + 2 * kQLoads + 2 * kSegments + 2;
  static constexpr int kMisc = kBar + kNumBars * 8;     // tmem base, abort flag, status word; line's cost, CTA's share
  // slack to align the base to 1024 B; with d = 64 the own-keys product reads 64 rows it does not need, 1 KB on
  static constexpr int kAlloc = kMisc + 32 + 1024 + (D == 64 ? 1024 : 0);
  static_assert(kAlloc <= 232448, "shared memory of one CTA");
  static_assert(kMaxWindows * 12 <= kKStages * kTileBytes, "the plan's windows overlay the K ring");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kTmS0 = 0, kTmS1 = 128, kTmO0 = 256, kTmO1 = 256 + D;
};

// kG: query rows own keys are worked on with, Hq / Hkv rounded up to 4 or 8.
template <int D, int kG>
__global__ void __launch_bounds__(kThreads, 1)
    shared_attend_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                         const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ SharedArgs a) {
  using L = AttendLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::kQ, sK = sbase + L::kK, sV = sbase + L::kV;
  constexpr uint32_t KS = L::kKStages, VS = L::kVStages, KB = L::kKBars, VB = L::kVBars;
  const uint32_t bar0 = sbase + L::kBar, bar_t = bar0 + 8u * (KB + VB + KS + VS), bar_s = bar_t + 8u * (20 + 2 * kQLoads);
  auto BAR_KF = [&](uint32_t g) { return bar0 + 8u * (g % KB); };          // of tile g
  auto BAR_VF = [&](uint32_t g) { return bar0 + 8u * (KB + g % VB); };
  auto BAR_KE = [&](uint32_t s) { return bar0 + 8u * (KB + VB + s); };     // of slot s
  auto BAR_VE = [&](uint32_t s) { return bar0 + 8u * (KB + VB + KS + s); };
  auto BAR_SF = [&](int t, int h) { return bar_t + 8u * (2 * t + h); };
  auto BAR_PR = [&](int t, uint32_t h) { return bar_t + 8u * (4 + 2 * t + h); };
  auto BAR_OF = [&](int t) { return bar_t + 8u * (8 + t); };
  auto BAR_OD = [&](int t, uint32_t h) { return bar_t + 8u * (10 + 2 * t + (h & 1u)); };
  auto BAR_X = [&](int t) { return bar_t + 8u * (14 + t); };
  auto BAR_SO = [&](int t, uint32_t k) { return bar_t + 8u * (16 + 2 * t + (k & 1u)); };
  auto BAR_QF = [&](int t, uint32_t load) { return bar_t + 8u * (20 + t * kQLoads + load % kQLoads); };
  auto BAR_GF = [&](uint32_t e) { return bar_s + 8u * e; };
  auto BAR_GE = [&](uint32_t e) { return bar_s + 8u * (kSegments + e); };
  const uint32_t BAR_FIN = bar_s + 8u * 2 * kSegments, BAR_GO = BAR_FIN + 8u;
  Segment* ring = reinterpret_cast<Segment*>(smem + L::kSeg);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  unsigned* status = reinterpret_cast<unsigned*>(smem + L::kMisc + 8);   // this CTA's
  long long* line = reinterpret_cast<long long*>(smem + L::kMisc + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_launch_dependents();   // the combine kernel waits for this grid before it reads anything
  // the plan's inputs on their way into L2 while barriers and tensor memory are set up (32 numbers a line)
#pragma unroll 1
  for (int i = threadIdx.x * 32; i < a.num_seqs; i += kThreads * 32) prefetch_l2(a.seq_lens + i);
#pragma unroll 1
  for (int i = threadIdx.x * 32; i < a.num_groups; i += kThreads * 32) {
    prefetch_l2(a.group_offsets + i);
    prefetch_l2(a.prefix_lens + i);
  }
  // ---- setup
  if (threadIdx.x == 0) {
    for (uint32_t b = 0; b < KB + VB; ++b) mbar_init(bar0 + 8u * b, 1);
    for (uint32_t s = 0; s < KS + VS; ++s) mbar_init(BAR_KE(s), 2);   // both row tiles' warps (narrow: twice by the one that takes the step)
    for (int t = 0; t < 2; ++t) {
      for (uint32_t u = 0; u < kQLoads; ++u) mbar_init(BAR_QF(t, u), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(BAR_SF(t, h), 1);
        mbar_init(BAR_PR(t, h), 128);
      }
      mbar_init(BAR_OF(t), 128);
      mbar_init(BAR_OD(t, 0), 1);
      mbar_init(BAR_OD(t, 1), 1);
      mbar_init(BAR_X(t), 4);   // one lane of each softmax warp
      mbar_init(BAR_SO(t, 0), 1);
      mbar_init(BAR_SO(t, 1), 1);
    }
    for (uint32_t e = 0; e < kSegments; ++e) {
      mbar_init(BAR_GF(e), 1);
      mbar_init(BAR_GE(e), 4 + 256);   // the MMA and copying warps and every softmax thread
    }
    mbar_init(BAR_FIN, 2);
    mbar_init(BAR_GO, 1);
    *abort_flag = 0;
    *status = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmQ1);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  // ---- plan.  Every CTA counts the whole line for itself: the arrays are a few
  // numbers a sequence, and a kernel of its own for them cost 8 us.
  // Groups that decrease or leave the batch might overlap: then none is used.
  bool bad = false;
#pragma unroll 1
  for (int g = threadIdx.x; g < a.num_groups; g += kThreads) {
    const int lo = __ldg(a.group_offsets + g), hi = __ldg(a.group_offsets + g + 1);
    bad = bad || lo < 0 || hi < lo || hi > a.num_seqs;
  }
  tc_fence_before();
  const bool ignore = __syncthreads_or(bad);
  const int groups = ignore ? 0 : a.num_groups, n_items = groups + a.num_seqs, n_windows = (n_items + 31) / 32;
  long long* wx = reinterpret_cast<long long*>(smem + L::kK);   // cost, then place, of each window of 32 items
  int* wu = reinterpret_cast<int*>(wx + kMaxWindows);
#pragma unroll 1
  for (int w = warp; w < n_windows; w += kThreads / 32) {
    long long cost = 0;
    int units = 0;
    load_window(a, groups, w, cost, units, bad);
    if (lane == 0) {
      wx[w] = cost;
      wu[w] = units;
    }
  }
  if (bad) atomicOr(status, kDevBadSeqLen);
  __syncthreads();
  if (warp == 0) {   // sums before each window
    long long base = 0;
    int base_u = 0;
#pragma unroll 1
    for (int w0 = 0; w0 < n_windows; w0 += 32) {
      const int w = w0 + lane;
      const long long c = w < n_windows ? wx[w] : 0;
      const int u = w < n_windows ? wu[w] : 0;
      long long sum = c;
      int sum_u = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o);
        const int y = __shfl_up_sync(0xffffffffu, sum_u, o);
        if (lane >= o) {
          sum += x;
          sum_u += y;
        }
      }
      if (w < n_windows) {
        wx[w] = base + sum - c;
        wu[w] = base_u + sum_u - u;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
      base_u += __shfl_sync(0xffffffffu, sum_u, 31);
    }
    if (lane == 0) {
      long long per = base <= UINT32_MAX - a.n_ctas
                          ? (static_cast<unsigned>(base) + a.n_ctas - 1) / static_cast<unsigned>(a.n_ctas)
                          : (base + a.n_ctas - 1) / a.n_ctas;
      if (per < kWideCost) per = kWideCost;   // a share inside a unit holds the start of a step at least
      line[0] = base;
      line[1] = per;
      if (blockIdx.x == 0) *a.per_cta = per;
    }
  }
  fence_proxy_async_smem();   // the windows' memory becomes the K ring
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long per = line[1];
  if (warp == kThreads / 32 - 2) {
    // The combine kernel's tables, 32 items of them by every n_ctas-th CTA (lane k
    // holds the place of the CTA's k-th window; read before the K ring fills).
    const int mine = static_cast<int>(blockIdx.x) + lane * a.n_ctas;
    const long long at = mine < n_windows ? wx[mine] : 0;
    const int at_u = mine < n_windows ? wu[mine] : 0;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR_GO);
    __syncwarp();
#pragma unroll 1
    for (int k = 0, w = static_cast<int>(blockIdx.x); w < n_windows; ++k, w += a.n_ctas) {
      long long base = __shfl_sync(0xffffffffu, at, k);
      int base_u = __shfl_sync(0xffffffffu, at_u, k);
      const Item it = load_window(a, groups, w, base, base_u, bad).it;
      const int i = w * 32 + lane, tiles = tiles_of(it.end - it.base);
      if (i < groups) {
        const GroupPlan g = {it.x0, it.unit0, it.first, it.n, tiles, {0, 0}};
        a.groups[i] = g;
      } else if (i < n_items) {
        const SeqPlan q = {it.x0, tiles, it.group};
        a.seqs[it.first] = q;
      }
    }
  }

  if (warp < kSoftmaxWarp0 || warp == kMmaWarp1) {
    if (warp == 0) {
      // ======================= planner: describes the CTA's segments, up to kSegments ahead =======================
      const long long begin = per * blockIdx.x, end = min(line[0], begin + per);
      const int per_tile = kTile >> a.page_shift;
      // where the walk is: window of items (one a lane, `work` those left in it), item, unit of it and the unit's place
      int w = 0, base_u = 0;
      long long base = 0;
      Window win = {};
      Item it = {};
      uint32_t work = 0;
      int unit = 0, tiles = 0, blocks = 1, cost = 1;
      bool own = false;
      long long ux = end;
      auto enter = [&](int lane_of) {   // the item of a lane of the window
        it.x0 = __shfl_sync(0xffffffffu, win.it.x0, lane_of);
        it.unit0 = __shfl_sync(0xffffffffu, win.it.unit0, lane_of);
        it.first = __shfl_sync(0xffffffffu, win.it.first, lane_of);
        it.n = __shfl_sync(0xffffffffu, win.it.n, lane_of);
        it.base = __shfl_sync(0xffffffffu, win.it.base, lane_of);
        it.lo = __shfl_sync(0xffffffffu, win.it.lo, lane_of);
        it.end = __shfl_sync(0xffffffffu, win.it.end, lane_of);
        work &= ~((2u << lane_of) - 1u);   // items behind it
        own = w * 32 + lane_of >= groups;
        tiles = tiles_of(it.end - it.base);
        blocks = blocks_of(it.n, a.G);
        cost = cost_of(it.n, a.G);
        unit = 0;
        ux = it.x0;
      };
      auto next_window = [&]() {
        win = load_window(a, groups, w, base, base_u, bad);
        work = __ballot_sync(0xffffffffu, win.cost > 0);
      };
      if (begin < end) {
        int lo = 0, n = n_windows;   // the last window that starts at or before `begin`: a 32-way search
#pragma unroll 1
        while (n > 1) {
          const int step = (n + 31) / 32, at = lane * step;
          const uint32_t le = __ballot_sync(0xffffffffu, at < n && wx[lo + at] <= begin);
          const int k = 31 - __clz(le);
          lo += k * step;
          n = min(step, n - k * step);
        }
        w = lo;
        base = wx[w];
        base_u = wu[w];
        next_window();
        // and in it the last item with work that does
        enter(31 - __clz(__ballot_sync(0xffffffffu, win.cost > 0 && win.it.x0 <= begin)));
        const long long length = unit_cost(tiles, cost), in = begin - ux;
        unit = static_cast<int>(in <= UINT32_MAX ? static_cast<unsigned>(in) / static_cast<unsigned>(length) : in / length);
        ux += unit * length;
      }
      auto advance = [&]() {   // to the next unit, if the share reaches it
        ux += unit_cost(tiles, cost);
        if (ux < end && ++unit == blocks * a.Hkv) {
          while (work == 0) {
            ++w;
            next_window();
          }
          enter(__ffs(work) - 1);
        }
      };
      uint32_t g0 = 0;
      int turn = 0;   // row tile that takes the next narrow step
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        int j0 = 0, j1 = 0;
#pragma unroll 1
        while (ux < end) {
          unit_share(ux, tiles, cost, per, static_cast<int>(blockIdx.x), j0, j1);
          if (j0 < j1) break;   // else the share only touches the unit
          advance();
        }
        const bool done = j0 >= j1;
        Segment sg = {};
        int pg = -1;
        if (!done) {
          const int head = blocks == 1 ? unit : static_cast<int>(static_cast<unsigned>(unit) / static_cast<unsigned>(blocks));
          const int row0 = (unit - head * blocks) * kUnitRows;
          const bool is_own = own;   // advance() moves on
          sg.g0 = g0;
          sg.tiles = j1 - j0;
          sg.rows = min(kUnitRows, it.n * a.G - row0);
          sg.wide = sg.rows > kTile;
          sg.tile_first = turn;
          sg.lo = j0 == 0 ? it.lo : 0;
          sg.hi = it.end - it.base - j0 * kTile;
          const int slot = static_cast<int>(blockIdx.x) + it.unit0 + unit;
          sg.slot = is_own ? ~slot : slot;
          sg.hkv = head;
          sg.seq = it.first + (row0 >> a.g_shift);
          sg.row = it.first;
          sg.page0 = (it.base >> a.page_shift) + j0 * per_tile;
          sg.qslot = is_own ? static_cast<int>(n % kQSlots) : 0;
          g0 += sg.tiles;
          if (!sg.wide) turn ^= sg.tiles & 1;
          const bool mine = lane < per_tile && lane * a.page_size < sg.hi;
          if (mine) pg = __ldg(a.block_table + static_cast<size_t>(sg.row) * a.max_pages + sg.page0 + lane);
          advance();   // while the table entries are under way
          if (mine && (pg < 0 || pg >= a.num_pages_total)) {   // read as page 0, flagged
            atomicOr(status, kDevBadBlockTable);
            pg = 0;
          }
        }
        const uint32_t e = n % kSegments;
        if (n >= kSegments && !wait_all(BAR_GE(e), (n / kSegments - 1) & 1u, status, abort_flag)) break;
        if (n == 0) {
          fence_proxy_async_smem();   // this warp's reads of the windows, before copies into the K ring
          if (!wait_all(BAR_GO, 0, status, abort_flag)) break;
        }
        if (lane < kTile / 8) ring[e].pages[lane] = pg;
        if (lane == 0) {
          const int4* src = reinterpret_cast<const int4*>(&sg);
          int4* dst = reinterpret_cast<int4*>(&ring[e]);
          dst[0] = src[0];
          dst[1] = src[1];
          dst[2] = src[2];
          dst[3] = src[3];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_GF(e));
        if (done) break;
      }
    } else if (warp == 2 || warp == 3) {
      // ======================= copying warps: 2 queries and K, 3 V (lane p: page p of a key tile) =======================
      const bool is_v = warp == 3;
      const int per_tile = kTile >> a.page_shift;
      const uint32_t page_bytes = static_cast<uint32_t>(a.page_size) * D * 2;
      const uint32_t stages = is_v ? VS : KS, data = is_v ? sV : sK;
      const uint32_t full0 = is_v ? BAR_VF(0) : BAR_KF(0), bars = is_v ? VB : KB, empty0 = is_v ? BAR_VE(0) : BAR_KE(0);
      const CUtensorMap* tm = is_v ? &tmV : &tmK;
      uint32_t slot = 0, use = 0, g = 0;   // ring slot of the next tile, how often the ring went round, tiles copied
      uint32_t qn[2] = {0, 0};      // loads into each query buffer
      uint32_t qlast[2] = {0, 0};   // ring position of the last step that reads each
      bool qown[2] = {false, false};
      bool ok = true;
#pragma unroll 1
      for (uint32_t n = 0; ok; ++n) {
        const uint32_t e = n % kSegments;
        if (!(ok = wait_all(BAR_GF(e), (n / kSegments) & 1u, status, abort_flag))) break;
        const Segment& sg = ring[e];
        const int tiles = sg.tiles, hkv = sg.hkv, hi = sg.hi, seq = sg.seq, wide = sg.wide, tile_first = sg.tile_first;
        const uint32_t g0 = sg.g0;
        const bool own = sg.slot < 0;
        const uint32_t qoff = static_cast<uint32_t>(sg.qslot) * 1024u;
        const int32_t* row = a.block_table + static_cast<size_t>(sg.row) * a.max_pages + sg.page0;
        int pg = lane < kTile / 8 ? sg.pages[lane] : -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR_GE(e));
        if (tiles == 0) break;
        // queries: narrow segments of several steps keep the same rows in both buffers
#pragma unroll 1
        for (int t = 0; t < 2 && !is_v; ++t) {
          if (!wide && tiles == 1 && t != tile_first) continue;
          // A whole tile, or rows after one, wait until the scores of the last step that reads the buffer are formed:
          // where that step's K slot has not been waited for since, its release says so.
          if (qn[t] > 0 && !(own && qown[t]) && qlast[t] + KS >= g0 &&
              !(ok = wait_all(BAR_KE(qlast[t] % KS), (qlast[t] / KS) & 1u, status, abort_flag)))
            break;
          const uint32_t bar = BAR_QF(t, qn[t]);
          ++qn[t];
          const int last = wide ? tiles - 1 : tiles - 1 - ((tile_first + tiles - 1 + t) & 1);
          qlast[t] = g0 + static_cast<uint32_t>(last);
          qown[t] = own;
          if (lane == 0) {
            const uint32_t dst = sQ + t * L::kTileBytes + qoff;
            if (own) {   // one sequence: its G rows
              mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a.G) * D * 2);
              for (int c = 0; c < L::kChunks; ++c)
                tma_load_4d(dst + c * L::kChunkBytes, &tmQ1, bar, 0, hkv * a.G, seq, c);
            } else {
              mbar_arrive_expect_tx(bar, L::kTileBytes);
              tma_load_4d(dst, &tmQ, bar, 0, hkv * a.G, seq + (wide ? t * (kTile / a.G) : 0), 0);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        // key tiles.  A page arrives in one copy in the 128-byte swizzle: K as [8-row
        // group][64-column chunk][8 rows][128 B], V as [chunk][page rows][128 B].
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          int pg_next = -1;   // under way before the wait
          const int p = (j + 1) * per_tile + lane;
          const bool more = j + 1 < tiles && lane < per_tile && static_cast<long long>(p) * a.page_size < hi;
          if (more) pg_next = __ldg(row + p);
          if (!(ok = wait_all(empty0 + 8u * slot, (use & 1u) ^ 1u, status, abort_flag))) break;
          const uint32_t bar = full0 + 8u * (g % bars);
          const uint32_t live = __ballot_sync(0xffffffffu, pg >= 0);
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(live)) * page_bytes);
          __syncwarp();
          if (pg >= 0) {
            const uint32_t at = data + slot * L::kTileBytes + static_cast<uint32_t>(lane) * page_bytes;
            tma_load_5d(at, tm, bar, 0, 0, 0, is_v ? hkv : 0, is_v ? pg : pg * a.Hkv + hkv);
          }
          ++g;
          if (++slot == stages) {
            slot = 0;
            ++use;
          }
          if (more && (pg_next < 0 || pg_next >= a.num_pages_total)) {   // read as page 0, flagged
            atomicOr(status, kDevBadBlockTable);
            pg_next = 0;
          }
          pg = pg_next;
        }
      }
      // drain: no copy into this CTA's shared memory may still be in flight at exit
      if (lane == 0) {
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
#pragma unroll 1
          for (uint32_t u = qn[t] > kQLoads ? qn[t] - kQLoads : 0u; u < qn[t]; ++u)
            mbar_wait(BAR_QF(t, u), (u / kQLoads) & 1u, nullptr, nullptr, kWaitLimitNs);
#pragma unroll 1
        for (uint32_t k = g > stages ? g - stages : 0u; k < g; ++k)   // the last fill of each slot
          mbar_wait(full0 + 8u * (k % bars), (k / bars) & 1u, nullptr, nullptr, kWaitLimitNs);
      }
      __syncwarp();
    } else {
      // ======================= MMA issuers, one warp per row tile (whole warp; the elected lane issues) ===========
      // Each tile's chain - scores, softmax, product with V, next scores - is a
      // string of waits and issues of some hundred cycles each; from one warp the
      // two tiles' chains add up (a narrow step took 2.4 us), from two they overlap.
      const int t = __shfl_sync(0xffffffffu, warp == kMmaWarp1 ? 1 : 0, 0);
      const bool leader = elect_one_sync();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kTile, kTile / 2, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kTile, D, true);
      const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t tS = tbase + (t ? L::kTmS1 : L::kTmS0), tO = tbase + (t ? L::kTmO1 : L::kTmO0);
      constexpr bool kTwo = L::kChunks == 2;
      constexpr uint64_t kTileStep = L::kTileBytes >> 4;
      const uint64_t dQ = smem_desc_sw128(sQ + (t ? L::kTileBytes : 0), 16, 1024);
      const uint64_t dK = smem_desc_sw128(sK, 16, L::kChunks * 1024);   // 8-row groups hold every chunk
      const int ps = a.page_size;
      const uint64_t dV = kTwo ? smem_desc_sw128(sV, static_cast<uint32_t>(ps) * 128u, ps >= 16 ? 1024u : 2048u)
                               : smem_desc_sw128(sV, L::kChunkBytes, 1024);
      // page-major V: 16-key step kk starts at byte 2048 (kk + (kk & vmask))
      const int vmask = ~(max(ps / 16, 1) - 1);
      bool ok = true;
      uint32_t steps_t = 0, used = 0;   // steps and segments of this row tile: S/P/o_done and Q/O barrier phases
#pragma unroll 1
      for (uint32_t n = 0; ok; ++n) {
        const uint32_t e = n % kSegments;
        if (!(ok = wait_all(BAR_GF(e), (n / kSegments) & 1u, status, abort_flag))) break;
        // broadcasts tell the compiler that the values are the same in all lanes: the
        // descriptors made of them stay in uniform registers
        const uint32_t g0 = __shfl_sync(0xffffffffu, ring[e].g0, 0);
        const int tiles = __shfl_sync(0xffffffffu, ring[e].tiles, 0);
        const int wide = __shfl_sync(0xffffffffu, ring[e].wide, 0);
        const int tile_first = __shfl_sync(0xffffffffu, ring[e].tile_first, 0);
        const int own = __shfl_sync(0xffffffffu, ring[e].slot, 0) < 0, qslot = __shfl_sync(0xffffffffu, ring[e].qslot, 0);
        if (leader) mbar_arrive(BAR_GE(e));
        __syncwarp();
        if (tiles == 0) break;
        const int stride = wide ? 1 : 2, first = wide ? 0 : (t ^ tile_first) & 1;
        if (first >= tiles) continue;
        if (!(ok = wait_all(BAR_QF(t, used), (used / kQLoads) & 1u, status, abort_flag))) break;
        if (own) {
          // Few query rows: the products are taken with keys (S^T = K Q^T) and columns of
          // d (O^T = V^T P^T) on the tensor memory's lanes and the queries on its columns.
          // Every softmax thread then has one key and a handful of weights, and
          // the products are an eighth as wide.  P^T comes from shared memory.
          const uint64_t dP = smem_desc_sw128(sQ + t * L::kTileBytes + kOwnP, 16, 1024);
          // with d = 64 rows 64..127 of V^T repeat others and are not read back
          const uint64_t dVt = kTwo ? dV : smem_desc_sw128(sV, 1024, 1024);
          constexpr uint32_t idesc_s = idesc_bf16_f32(kTile, kOwnCols, false);
          constexpr uint32_t idesc_o = idesc_bf16_f32(kTile, kOwnCols, false) | (1u << 15);   // A is d-major
          // Scores run one step ahead of the products with V, into the next segments (two
          // places for S^T and P^T), so the softmax finds its scores ready.
          uint32_t gs = g0, k = 0, pg = 0, pused = 0;   // segment's ring position; steps; the due product's step and segment
          int j = first, left = tiles;
          uint64_t dQs = dQ + static_cast<uint64_t>(qslot * 64);
          bool sfirst = true, pfirst = false;
          while (true) {
            const bool have = j < left;
            const uint32_t g = gs + static_cast<uint32_t>(j);
            if (have) {
              const uint32_t ks = g % KS;
              if (!(ok = wait_all(BAR_KF(g), (g / KB) & 1u, status, abort_flag))) break;
              tc_fence_after();
              if (leader) {
                const uint64_t a0 = dK + ks * kTileStep;
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                  mma_ss(tS + (k & 1u) * kOwnCols, a0 + (c >> 2) * (1024 >> 4) + (c & 3) * 2,
                         dQs + (c >> 2) * (L::kChunkBytes >> 4) + (c & 3) * 2, idesc_s, c != 0 ? 1u : 0u);
                mma_commit(BAR_SO(t, k));
                mma_commit(BAR_KE(ks));
                mbar_arrive(BAR_KE(ks));
              }
              __syncwarp();
            }
            if (k > 0) {   // the product of the step before, by now the softmax may be a step further: two barriers in turn
              const uint32_t vs = pg % VS;
              if (!(ok = wait_all(BAR_VF(pg), (pg / VB) & 1u, status, abort_flag))) break;
              if (pfirst && pused > 0 && !(ok = wait_all(BAR_OF(t), (pused - 1) & 1u, status, abort_flag))) break;
              if (!(ok = wait_all(BAR_PR(t, (k - 1) & 1u), (steps_t + ((k - 1) >> 1)) & 1u, status, abort_flag))) break;
              tc_fence_after();
              if (leader) {
                const uint64_t a0 = dVt + vs * kTileStep, b0 = dP + ((k & 1u) ^ 1u) * (kOwnPBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                  const uint32_t off = kTwo ? static_cast<uint32_t>((kk + (kk & vmask)) << 11) : kk * 2048u;
                  mma_ss(tO, a0 + static_cast<uint64_t>(off >> 4), b0 + (kk >> 2) * (kOwnCols * 128 >> 4) + (kk & 3) * 2,
                         idesc_o, (!pfirst || kk > 0) ? 1u : 0u);
                }
                mma_commit(BAR_OD(t, k - 1));
                mma_commit(BAR_VE(vs));
                mbar_arrive(BAR_VE(vs));
              }
              __syncwarp();
            }
            if (!have) break;
            pg = g;
            pfirst = sfirst;
            pused = used;
            sfirst = false;
            ++k;
            j += 2;
            while (j >= left) {   // the next segment with steps of this row tile
              ++n;
              const uint32_t en = n % kSegments;
              if (!(ok = wait_all(BAR_GF(en), (n / kSegments) & 1u, status, abort_flag))) break;
              gs = __shfl_sync(0xffffffffu, ring[en].g0, 0);
              left = __shfl_sync(0xffffffffu, ring[en].tiles, 0);
              j = (t ^ __shfl_sync(0xffffffffu, ring[en].tile_first, 0)) & 1;
              dQs = dQ + static_cast<uint64_t>(__shfl_sync(0xffffffffu, ring[en].qslot, 0) * 64);
              __syncwarp();
              if (leader) mbar_arrive(BAR_GE(en));
              if (left == 0) break;
              if (j < left) {
                ++used;
                sfirst = true;
                ok = wait_all(BAR_QF(t, used), (used / kQLoads) & 1u, status, abort_flag);
              }
            }
            if (!ok) break;
          }
          break;   // prefixes come first: no segment is left
        }
        // A step goes in two halves of 64 keys, each with its own scores and weights
        // in tensor memory: the scores of one half are formed while the softmax is at
        // the other, and the next step's as soon as the product that reads the weights
        // in their place is complete.  (Complete, not issued: products into different
        // accumulators are not ordered.)
        auto scores = [&](uint32_t g, int h) {   // S_t[h] = Q_t K[64 h ..]^T
          if (leader) {
            const uint64_t b0 = dK + (g % KS) * kTileStep + static_cast<uint64_t>(h) * (L::kChunks * 512);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              mma_ss(tS + h * 64, dQ + (c >> 2) * (L::kChunkBytes >> 4) + (c & 3) * 2,
                     b0 + (c >> 2) * (1024 >> 4) + (c & 3) * 2, idesc_qk, c != 0 ? 1u : 0u);
            mma_commit(BAR_SF(t, h));
            if (h == 1) {
              mma_commit(BAR_KE(g % KS));   // K's release also frees the query tile after a segment's last step
              if (!wide) mbar_arrive(BAR_KE(g % KS));
            }
          }
          __syncwarp();
        };
        uint32_t gs = g0 + static_cast<uint32_t>(first);   // ring position of the next scores
        int q = 0;                                         // halves of them formed
        int j = first - stride;                            // step of the products
        while (true) {
          const bool more = j + stride < tiles;
          const uint32_t g = gs - static_cast<uint32_t>(stride), vs = g % VS;
          q = 0;
          if (j >= 0 && !(ok = wait_all(BAR_VF(g), (g / VB) & 1u, status, abort_flag))) break;
          // the first product of a segment overwrites O_t: the epilogue before must have read it
          if (j == first && used > 0 && !(ok = wait_all(BAR_OF(t), (used - 1) & 1u, status, abort_flag))) break;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (j >= 0) {   // O_t += P_t[h] V[64 h ..]
              if (!(ok = wait_all(BAR_PR(t, h), steps_t & 1u, status, abort_flag))) break;
              tc_fence_after();
              if (leader) {
                const uint64_t b0 = dV + vs * kTileStep;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const int kk = h * 4 + c;
                  const uint32_t off = kTwo ? static_cast<uint32_t>((kk + (kk & vmask)) << 11) : kk * 2048u;
                  mma_ts(tO, tS + h * 64 + c * 8, b0 + static_cast<uint64_t>(off >> 4), idesc_pv,
                         (j > first || kk > 0) ? 1u : 0u);
                }
                mma_commit(BAR_OD(t, h));
              }
              __syncwarp();
              if (!(ok = wait_all(BAR_OD(t, h), steps_t & 1u, status, abort_flag))) break;
            }
            // the next step's scores: of this half if K is there, else both later
            if (more) {
              const uint32_t kf = BAR_KF(gs), kph = (gs / KB) & 1u;
              bool there = q > 0;   // known since the half before
              if (!there)
                there = h == 0 ? __all_sync(0xffffffffu, mbar_try_wait(kf, kph)) : (ok = wait_all(kf, kph, status, abort_flag));
              if (!ok) break;
              if (there) {
                tc_fence_after();
#pragma unroll 1
                for (; q <= h; ++q) scores(gs, q);
              }
            }
          }
          if (!ok) break;
          if (j >= 0) {
            if (leader) {
              mma_commit(BAR_VE(vs));
              if (!wide) mbar_arrive(BAR_VE(vs));
            }
            __syncwarp();
            ++steps_t;
          }
          if (!more) break;
          j += stride;
          gs += static_cast<uint32_t>(stride);
        }
        if (!ok) break;
        ++used;
      }
      // no commit may still be pending when the CTA exits
      if (leader) mma_commit(BAR_FIN);
      __syncwarp();
      mbar_wait_warp(BAR_FIN, 0, nullptr, nullptr);
    }
  } else {
    // ======================= softmax warpgroups (one thread per query row) =======================
    const int t = (warp - kSoftmaxWarp0) / 4;
    const int quarter = warp & 3, lane_row = quarter * 32 + lane;   // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + (t == 0 ? L::kTmS0 : L::kTmS1) + lane_off;
    const uint32_t tO = tmem + (t == 0 ? L::kTmO0 : L::kTmO1) + lane_off;
    const float c2 = a.scale_log2;
    bool ok = true;
    uint32_t steps_t = 0, held0 = 0, held1 = 0, exchanges = 0, own_k = 0;   // S/P and o_done phases; own-keys steps
    // Products with V complete in turn on two barriers (halves of a step; own keys:
    // every other step).  The scores of a half are formed when the product before on
    // the same barrier is complete, so at most one phase of each is open and its
    // parity says which.
    auto product_done = [&](uint32_t h) {   // the last product on barrier h, and all before it
      const bool done = wait_all(BAR_OD(t, h), ((h & 1u ? held1 : held0) - 1) & 1u, status, abort_flag);
      tc_fence_after();
      return done;
    };
#pragma unroll 1
    for (uint32_t seg = 0; ok; ++seg) {
      const uint32_t e = seg % kSegments;
      ok = wait_all(BAR_GF(e), (seg / kSegments) & 1u, status, abort_flag);
      if (!ok) break;
      const Segment sg = ring[e];
      mbar_arrive(BAR_GE(e));
      if (sg.tiles == 0) break;
      // this row tile's steps j, j + stride, ...; `half`: which of the unit's two partials they make
      const int stride = sg.wide ? 1 : 2, half = sg.wide ? t : (t ^ sg.tile_first) & 1;
      const bool own = sg.slot < 0;
      const int rows = sg.wide ? min(kTile, sg.rows - t * kTile) : sg.rows;   // of this tile
      const int row = lane_row;
      const bool live = row < rows, warp_live = quarter * 32 < rows;
      int j = sg.wide ? 0 : half;
      if (j >= sg.tiles) continue;
      // V rows that are no key get weight 0, and whatever is there must not turn
      // that into NaN: they are zeroed before the products read them (wide steps: by
      // both row tiles' warps, each before its own product).
      auto zero_values = [&](int j, int lo, int lim) {
        const uint32_t gj = sg.g0 + static_cast<uint32_t>(j), sv = gj % VS;
        if (!wait_all(BAR_VF(gj), (gj / VB) & 1u, status, abort_flag)) return false;
        if (lane_row >= lim || lane_row < lo) {
          const int pr = lane_row & (a.page_size - 1);
          uint8_t* base = smem + L::kV + sv * L::kTileBytes + (lane_row - pr) * D * 2 + pr * 128;
#pragma unroll 1
          for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
            for (int z = 0; z < 8; ++z)   // eight rows' pieces of eight different banks at a time
              reinterpret_cast<uint4*>(base + c * a.page_size * 128)[(z + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);
        }
        return true;
      };
      if (own) {
        // ---- own keys: this thread has key `lane_row` of the tile and one score per query row
        const int G = a.G;
        float m[kG], l[kG];
#pragma unroll
        for (int i = 0; i < kG; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.f;
        }
        // eight values of each of the row tile's four warps, joined through shared memory
        float* red = reinterpret_cast<float*>(smem + L::kRed) + t * 2 * 4 * 8;
        auto exchange = [&](float (&v)[kG], auto join) {
          float* buf = red + (exchanges & 1u) * 4 * kG;   // two in turn: one barrier an exchange
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kG; i += 4)
              *reinterpret_cast<float4*>(buf + quarter * kG + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            mbar_arrive(BAR_X(t));
          }
          if (!wait_all(BAR_X(t), exchanges++ & 1u, status, abort_flag)) return false;
#pragma unroll
          for (int i = 0; i < kG; i += 4) {
            float4 x = *reinterpret_cast<const float4*>(buf + i);
#pragma unroll
            for (int w = 1; w < 4; ++w) {
              const float4 y = *reinterpret_cast<const float4*>(buf + w * kG + i);
              x = make_float4(join(x.x, y.x), join(x.y, y.y), join(x.z, y.z), join(x.w, y.w));
            }
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
          }
          return true;
        };
        uint8_t* const prow = smem + L::kQ + t * L::kTileBytes + kOwnP + (lane_row >> 6) * (kOwnCols * 128);
        const uint32_t pcol = static_cast<uint32_t>(((lane_row & 63) >> 3) * 16), pbyte = static_cast<uint32_t>((lane_row & 7) * 2);
#pragma unroll 1
        for (bool first = true; j < sg.tiles; j += stride, first = false, ++own_k) {
          ok = wait_all(BAR_SO(t, own_k), (own_k >> 1) & 1u, status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          uint32_t sr[kG];
          tmem_ld(tS + (own_k & 1u) * kOwnCols, sr);
          const int lo = j == 0 ? sg.lo : 0, lim = min(kTile, sg.hi - j * kTile);
          const bool is_key = lane_row >= lo && lane_row < lim;
          if ((lim < kTile || lo > 0) && !(ok = zero_values(j, lo, lim))) break;
          tmem_wait_ld();
          float s[kG], mx[kG];
          bool raise = false;   // some row's max moves (by more than the margin)
#pragma unroll
          for (int i = 0; i < kG; ++i) {
            s[i] = is_key ? __uint_as_float(sr[i]) : -INFINITY;
            mx[i] = warp_max(s[i]);
          }
          if (!(ok = exchange(mx, [](float x, float y) { return fmaxf(x, y); }))) break;
#pragma unroll
          for (int i = 0; i < kG; ++i) raise = raise || (i < G && (mx[i] - m[i]) * c2 > kRescaleLog2);
          if (raise) {   // all 128 threads alike
            float alpha[kG];
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              const float m_new = fmaxf(m[i], mx[i]);
              alpha[i] = m[i] == m_new ? 1.f : ex2((m[i] - m_new) * c2);   // 0 from -inf
              m[i] = m_new;
              l[i] *= alpha[i];
            }
            if (!first) {   // O holds the products of the steps before, once the last of them is done
              if (!(ok = product_done(own_k + 1))) break;   // the step before
              uint32_t orr[kG];
              tmem_ld(tO, orr);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < kG; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha[i]);
              tmem_st(tO, orr);
              tmem_wait_st();
            }
          }
          // weights into P^T [query][key], 128-byte rows of 64 keys, 16-byte pieces swizzled by the row; rounded to bf16,
          // the type of V, as the prefix's are (below); the sum is of the unrounded ones
          uint8_t* const pk = prow + (own_k & 1u) * kOwnPBytes + pbyte;
          auto weigh = [&](int i) {
            const float negm = (m[i] == -INFINITY) ? 0.f : -m[i] * c2;
            const float p = ex2(fmaf(s[i], c2, negm));
            l[i] += p;
            *reinterpret_cast<__nv_bfloat16*>(pk + i * 128 + (pcol ^ (i * 16))) = __float2bfloat16(p);
          };
          weigh(0);
          if (G > 1) weigh(1);
          if (G > 2) {
#pragma unroll
            for (int i = 2; i < kG; ++i) weigh(i);
          }
          fence_proxy_async_smem();   // P (and zeroed V) before the products read them
          ++(own_k & 1u ? held1 : held0);
          tc_fence_before();
          mbar_arrive(BAR_PR(t, own_k & 1u));
        }
        if (!ok) break;
        // ---- the partial: this thread has column `lane_row` of d
#pragma unroll
        for (int i = 0; i < kG; ++i)
          if (i < G) {
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
          }
        if (!(ok = exchange(l, [](float x, float y) { return x + y; }) && product_done(own_k + 1))) break;
        uint32_t orr[kG];
        tmem_ld(tO, orr);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(BAR_OF(t));
        const size_t at = (static_cast<size_t>(~sg.slot) * 2 + half) * G;
#pragma unroll
        for (int i = 0; i < kG; ++i)
          if (i < G) {
            // no weight at all (every score -inf): an empty partial; a NaN sum (a score NaN or +inf) goes on to the join
            const float inv = l[i] == 0.f ? 0.f : __fdividef(1.f, l[i]);
            if (lane_row < D) a.own_o[(at + i) * D + lane_row] = __uint_as_float(orr[i]) * inv;
            if (lane_row == i && sg.tiles == 1) a.own_lse[(at ^ G) + i] = -INFINITY;   // the unit's other partial is none
            if (lane_row == i)
              a.own_lse[at + i] = l[i] == 0.f ? -INFINITY : fmaf(m[i], a.scale, __log2f(l[i]) * 0.69314718055994531f);
          }
        continue;
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (bool first = true; j < sg.tiles && ok; j += stride, ++steps_t) {
        // keys of this tile: columns [lo, lim); the rest of its shared memory holds none that count
        const int lo = j == 0 ? sg.lo : 0, lim = min(kTile, sg.hi - j * kTile);
        const bool need_mask = lim < kTile || lo > 0;
#pragma unroll 1
        for (int h = 0; h < 2; ++h, first = false) {   // 64 keys
          ok = wait_all(BAR_SF(t, h), steps_t & 1u, status, abort_flag);
          if (!ok) break;
          // Two row tiles in step form their exponentials at the same time (985 cycles for 64 of them, twice one warp's
          // time) and leave the unit idle at the same time.  Nothing moves them apart, so tile 1 starts a segment a
          // quarter of a step (of d = 128) late: figures at kApart.
          if (t == 1 && first && sg.wide)
            for (const long long t0 = clock64(); clock64() - t0 < kApart;) {
            }
          tc_fence_after();
          ++(h ? held1 : held0);   // this half's product is a phase of its barrier
          if (need_mask && h == 0) {
            if (!(ok = zero_values(j, lo, lim))) break;
            fence_proxy_async_smem();
          }
          if (!warp_live) {   // no row of this warp counts: its P may hold anything
            mbar_arrive(BAR_PR(t, h));
            continue;
          }
          uint32_t sr[2][32];
          tmem_ld32(tS + h * 64, sr[0]);
          tmem_ld32(tS + h * 64 + 32, sr[1]);
          tmem_wait_ld();
          if (need_mask) {
            const unsigned c0 = static_cast<unsigned>(h * 64 - lo), span = static_cast<unsigned>(lim - lo);
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c0 + c >= span) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
          }
          const float* s = reinterpret_cast<const float*>(&sr[0][0]);
          float mx;
          {
            float r0 = -INFINITY, r1 = -INFINITY, r2 = -INFINITY, r3 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; c += 8) {
              r0 = fmax3(r0, s[c + 0], s[c + 1]);
              r1 = fmax3(r1, s[c + 2], s[c + 3]);
              r2 = fmax3(r2, s[c + 4], s[c + 5]);
              r3 = fmax3(r3, s[c + 6], s[c + 7]);
            }
            mx = fmaxf(fmax3(r0, r1, r2), r3);
          }
          // rows that do not count hold anything: they ask for no rescale
          if (__any_sync(0xffffffffu, live && (mx - m) * c2 > kRescaleLog2)) {
            const float m_new = fmaxf(m, mx);
            const float alpha = m == m_new ? 1.f : ex2((m - m_new) * c2);   // 0 from -inf
            m = m_new;
            l *= alpha;
            if (!first) {   // O holds the products of the halves before, once the last of them is done
              if (!(ok = product_done(h ^ 1))) break;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t orr[32];
                tmem_ld32(tO + c * 32, orr);
                tmem_wait_ld();
#pragma unroll
                for (int z = 0; z < 32; ++z) orr[z] = __float_as_uint(__uint_as_float(orr[z]) * alpha);
                tmem_st32(tO + c * 32, orr);
              }
            }
          }
          // Weights 2^((s - m) c2), packed to bf16 for the tensor product (the rounding
          // of the prefill kernels: the operands of one product have one type, and V is
          // bf16.  An output is 0.0023 off, relative, where its own rounding alone makes
          // 0.0017; the sum is of the unrounded values).  c2 > 0 (see
          // the host side), so masked columns are exactly 0.  The weights take the
          // columns of their scores.
          const float negm = (m == -INFINITY) ? 0.f : -m * c2;
          const float2 c2v = make_float2(c2, c2), negv = make_float2(negm, negm);
          float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = ffma2(make_float2(s[2 * i], s[2 * i + 1]), c2v, negv);
            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
            if (i & 1) sb = fadd2(sb, pp);
            else sa = fadd2(sa, pp);
            pk[i] = pack_bf16x2(pp.x, pp.y);
          }
          l += (sa.x + sb.x) + (sa.y + sb.y);
          tmem_st32(tS + h * 64, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(BAR_PR(t, h));
        }
      }
      if (!ok) break;
      // ---- the partial: O / l and m scale + ln l, in fp32; NaN where l is (own keys do the same)
      if (!(ok = product_done(1))) break;
      if (warp_live) {
        const size_t slot = static_cast<size_t>(sg.slot);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        // [slot][4 columns][256 rows]: a warp's rows side by side
        float4* dst = reinterpret_cast<float4*>(a.pre_o) + slot * (D / 4) * kUnitRows + half * kTile + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orr[32];
          tmem_ld32(tO + c * 32, orr);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int z = 0; z < 8; ++z)
              dst[(c * 8 + z) * kUnitRows] =
                  make_float4(__uint_as_float(orr[4 * z]) * inv, __uint_as_float(orr[4 * z + 1]) * inv,
                              __uint_as_float(orr[4 * z + 2]) * inv, __uint_as_float(orr[4 * z + 3]) * inv);
          }
        }
        if (live) {
          if (!sg.wide && sg.tiles == 1)   // the unit's other partial is none
            a.pre_lse[slot * kUnitRows + (half ^ 1) * kTile + row] = -INFINITY;
          a.pre_lse[slot * kUnitRows + half * kTile + row] =
              l == 0.f ? -INFINITY : fmaf(m, a.scale, __log2f(l) * 0.69314718055994531f);
        }
      }
      tc_fence_before();
      mbar_arrive(BAR_OF(t));
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) a.cta_status[blockIdx.x] = *status;
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Combine: one CTA per (KV head, sequence), thread (c4, g) joins the partials of
// columns [4 c4, 4 c4 + 4) of query head g, with kLanes = 2 two threads half of
// them each.  Weights e^(lse_i - max) over all partials of a row.  Bound by
// latency: the release of the first grid, two dependent loads of the plan and one
// round of partials from L2, 7 us after the last attend CTA for 64 sequences of 32
// heads.  (16 partials in flight a thread instead of 8 were as good at small
// batches and 2% slower at 256 sequences.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ long long divide(long long x, long long y) {   // both >= 0; in 32 bits where it fits
  return ((x | y) >> 32) == 0 ? static_cast<unsigned>(x) / static_cast<unsigned>(y) : x / y;
}
// The CTAs [c0, c0 + n) that hold partials of a unit at place x0 on the line.
__device__ __forceinline__ void unit_ctas(long long x0, int tiles, int cost, long long per, int& c0, int& n) {
  x0 += start_of(cost);
  c0 = static_cast<int>(divide(x0, per));
  n = static_cast<int>(divide(x0 + static_cast<long long>(tiles - 1) * cost, per)) - c0 + 1;
}

template <int D, int G, int kLanes>
__global__ void __launch_bounds__(G * D / 4 * kLanes) shared_combine_kernel(const SharedArgs a, __nv_bfloat16* o, float* lse) {
  const int hkv = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x / kLanes, lane0 = threadIdx.x % kLanes;
  const int c4 = tid / G, gq = tid % G;
  grid_wait();   // the partials are complete
  const SeqPlan sp = a.seqs[seq];
  const long long per = *a.per_cta;
  // partials of the prefix (n_pre of them, `pre_step` floats apart; narrow rows have two a slot) and of the own keys
  int n_pre = 0, n_own = 0;
  size_t pre0 = 0, own0 = 0;
  bool wide = true;
  if (sp.group >= 0) {
    const GroupPlan g = a.groups[sp.group];
    const int blocks = blocks_of(g.n, G), cost = cost_of(g.n, G);
    const int r = (seq - g.first) * G, block = r / kUnitRows, unit = hkv * blocks + block;
    wide = min(kUnitRows, g.n * G - block * kUnitRows) > kTile;
    int c0;
    unit_ctas(g.x0 + unit * unit_cost(g.tiles, cost), g.tiles, cost, per, c0, n_pre);
    pre0 = static_cast<size_t>(c0 + g.unit0 + unit) * kUnitRows + r % kUnitRows + gq;
    if (!wide) n_pre *= 2;
  }
  if (sp.tiles > 0) {
    int c0;
    unit_ctas(sp.x0 + static_cast<long long>(hkv) * sp.tiles * kNarrowCost, sp.tiles, kNarrowCost, per, c0, n_own);
    own0 = static_cast<size_t>(c0 + seq * a.Hkv + hkv) * 2 * G + gq;
    n_own *= 2;
  }
  const int n = n_pre + n_own;
  auto place = [&](int i, const float*& w, const float4*& v) {
    if (i < n_pre) {
      const size_t row = pre0 + static_cast<size_t>(wide ? i * kUnitRows : i * kTile);   // two halves of 128 rows a slot
      w = a.pre_lse + row;
      v = reinterpret_cast<const float4*>(a.pre_o) + (row / kUnitRows * (D / 4) + c4) * kUnitRows + row % kUnitRows;
    } else {
      const size_t row = own0 + static_cast<size_t>(i - n_pre) * G;
      w = a.own_lse + row;
      v = reinterpret_cast<const float4*>(a.own_o) + row * (D / 4) + c4;
    }
  };
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 8;   // partials loaded before the first is joined
  for (int i0 = lane0; i0 < n; i0 += kAhead * kLanes) {
    float w[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      w[k] = -INFINITY;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + k * kLanes < n) {
        const float* pw;
        const float4* pv;
        place(i0 + k * kLanes, pw, pv);
        w[k] = *pw;
        v[k] = *pv;
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) mn = fmaxf(mn, w[k]);
    const float top = mn == -INFINITY ? 0.f : mn;   // the max passes over a NaN, whose weight must not be lost
    const float s0 = __expf(m - top);
    m = mn;
    l *= s0;
    acc = make_float4(acc.x * s0, acc.y * s0, acc.z * s0, acc.w * s0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (w[k] != -INFINITY) {   // an empty partial's values may be anything
        const float s1 = __expf(w[k] - top);
        l += s1;
        acc.x = fmaf(s1, v[k].x, acc.x);
        acc.y = fmaf(s1, v[k].y, acc.y);
        acc.z = fmaf(s1, v[k].z, acc.z);
        acc.w = fmaf(s1, v[k].w, acc.w);
      }
  }
  if constexpr (kLanes == 2) {   // the other lane's partials (the block is whole warps)
    const float m1 = __shfl_xor_sync(0xffffffffu, m, 1), l1 = __shfl_xor_sync(0xffffffffu, l, 1), mn = fmaxf(m, m1);
    const float s0 = m == -INFINITY ? 0.f : __expf(m - mn), s1 = m1 == -INFINITY ? 0.f : __expf(m1 - mn);
    // both lanes the same sums, term for term
    const float t0 = l * s0, t1 = l1 * s1;
    l = t0 + t1;
    acc.x = acc.x * s0 + __shfl_xor_sync(0xffffffffu, acc.x * s0, 1);
    acc.y = acc.y * s0 + __shfl_xor_sync(0xffffffffu, acc.y * s0, 1);
    acc.z = acc.z * s0 + __shfl_xor_sync(0xffffffffu, acc.z * s0, 1);
    acc.w = acc.w * s0 + __shfl_xor_sync(0xffffffffu, acc.w * s0, 1);
    m = mn;
  }
  constexpr int kThreadsHere = G * D / 4 * kLanes, kGather = kThreadsHere < 32 ? kThreadsHere : 32;
  if (hkv == 0 && seq == 0 && threadIdx.x < kGather) {   // the call's status: any CTA's
    unsigned bits = 0;
    for (int c = threadIdx.x; c < a.n_ctas; c += kGather) bits |= a.cta_status[c];
    bits = __reduce_or_sync(kGather == 32 ? 0xffffffffu : (1u << kGather) - 1u, bits);
    if (threadIdx.x == 0) *a.status = bits;
  }
  if (lane0 != 0) return;
  const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);   // NaN stays
  const size_t orow = static_cast<size_t>(seq) * a.Hq + hkv * G + gq;
  uint2 w2;
  w2.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  w2.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(o + orow * D)[c4] = w2;
  if (c4 == 0 && lse) lse[orow] = l == 0.f ? -INFINITY : m + __logf(l);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// pdl: programmatic dependent of the kernel before
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, bool pdl, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int kG>
ta_status launch_attend(const void* q, const void* k_cache, const void* v_cache, const SharedArgs& a,
                        cudaStream_t stream) {
  using L = AttendLayout<D>;
  CUtensorMap tq, tq1, tk, tv;
  ta_status st;
  // queries [S, Hq, d] as {64, Hq, S, d / 64}: a box of G heads of 128 / G sequences is one tile of 128 rows, a box
  // of G heads of one sequence one chunk of the rows that meet its own keys
  const uint64_t dims[4] = {64, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.num_seqs), D / 64};
  const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.Hq) * D * 2, 128};
  const uint32_t box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(kTile / a.G), D / 64};
  const uint32_t box1[4] = {64, static_cast<uint32_t>(a.G), 1, 1};
  if ((st = encode_bf16_tiled(&tq, q, 4, dims, strides, box)) != TA_OK) return st;
  if ((st = encode_bf16_tiled(&tq1, q, 4, dims, strides, box1)) != TA_OK) return st;
  {  // one page of one KV head a copy
    const uint64_t row = static_cast<uint64_t>(D) * 2, ps = static_cast<uint64_t>(a.page_size);
    const uint64_t heads = static_cast<uint64_t>(a.Hkv), pages = static_cast<uint64_t>(a.num_pages_total);
    const uint32_t rows = static_cast<uint32_t>(a.page_size), chunks = D / 64;
    // K as {64 columns, 8 rows, chunk, 8-row group, page and head}: lands [8-row group][chunk][8 rows][128 B], so all
    // 128 keys of a tile are 8-row groups at one stride, whichever page they came from
    const uint64_t dk[5] = {64, 8, chunks, ps / 8, pages * heads}, sk[4] = {row, 128, 8 * row, ps * row};
    const uint32_t bk[5] = {64, 8, chunks, rows / 8, 1};
    if ((st = encode_bf16_tiled(&tk, k_cache, 5, dk, sk, bk)) != TA_OK) return st;
    // V as {64 columns, page rows, chunk, head, page}: lands [chunk][page rows][128 B]
    const uint64_t dv[5] = {64, ps, chunks, heads, pages}, sv[4] = {row, 128, ps * row, heads * ps * row};
    const uint32_t bv[5] = {64, rows, chunks, 1, 1};
    if ((st = encode_bf16_tiled(&tv, v_cache, 5, dv, sv, bv)) != TA_OK) return st;
  }
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_limit(shared_attend_kernel<D, kG>, L::kAlloc, attr_done);
  if (e != cudaSuccess) return fail(TA_ERR_CUDA, "shared decode: shared-memory limit", e);
  e = launch(shared_attend_kernel<D, kG>, dim3(static_cast<unsigned>(a.n_ctas)), kThreads, L::kAlloc, false, stream, tq, tq1,
             tk, tv, a);
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "shared decode: attend kernel launch", e);
}

template <int D, int G>
cudaError_t launch_combine_of(const SharedArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.Hkv), static_cast<unsigned>(a.num_seqs));
  constexpr int kBlock = G * D / 4;
  // Two lanes an output, each with half of the partials, as long as all of them run at once (2048 threads an SM):
  // 64 sequences of 32 heads 43.9 -> 42.2 us for the whole call, 96 of 32 heads 47.1 -> 45.4.  Beyond that a second
  // wave costs more than the shorter loop gives (256 of 32 heads: 163.6 with one lane, 167.3 with two).
  if (static_cast<long long>(a.Hkv) * a.num_seqs * (2 * kBlock) <= a.n_ctas * 2048ll)
    return launch(shared_combine_kernel<D, G, 2>, grid, 2 * kBlock, 0, true, stream, a, o, lse);
  return launch(shared_combine_kernel<D, G, 1>, grid, kBlock, 0, true, stream, a, o, lse);
}
template <int D>
cudaError_t launch_combine(const SharedArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  switch (a.G) {
    case 1: return launch_combine_of<D, 1>(a, o, lse, stream);
    case 2: return launch_combine_of<D, 2>(a, o, lse, stream);
    case 4: return launch_combine_of<D, 4>(a, o, lse, stream);
    default: return launch_combine_of<D, 8>(a, o, lse, stream);
  }
}

}  // namespace

bool make_shared_plan(int num_seqs, int num_groups, int Hq, int Hkv, int d, SharedPlan* p) {
  if (num_seqs < 0 || num_groups < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || (d != 64 && d != 128)) return false;
  const int G = Hq / Hkv;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || num_seqs > 65535 || Hkv > 65535 || num_groups > 65535) return false;
  p->n_ctas = current_sm_count();
  // prefix units: every group has at most one block of rows that is not full, per KV head
  const long long units =
      num_groups == 0 ? 0 : static_cast<long long>(Hkv) * (num_groups + static_cast<long long>(num_seqs) * G / kUnitRows);
  const long long slots = units == 0 ? 0 : units + p->n_ctas;
  const long long own_slots = static_cast<long long>(num_seqs) * Hkv + p->n_ctas;
  if (slots > INT32_MAX || own_slots > INT32_MAX) return false;
  if (p->n_ctas < (kMaxWindows + 31) / 32 && (num_groups + num_seqs + 31) / 32 > 32 * p->n_ctas) return false;
  size_t at = 256;   // status word, a CTA's share
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  p->cta_status = take(static_cast<size_t>(p->n_ctas) * 4);
  p->groups = take(static_cast<size_t>(num_groups) * sizeof(GroupPlan));
  p->seqs = take(static_cast<size_t>(num_seqs) * sizeof(SeqPlan));
  p->pre_o = take(static_cast<size_t>(slots) * kUnitRows * d * 4);
  p->pre_lse = take(static_cast<size_t>(slots) * kUnitRows * 4);
  p->own_o = take(static_cast<size_t>(own_slots) * 2 * G * d * 4);
  p->own_lse = take(static_cast<size_t>(own_slots) * 2 * G * 4);
  p->bytes = at;
  return true;
}

ta_status launch_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* group_offsets, const int32_t* prefix_lens,
                               int page_size, int num_seqs, int num_groups, int max_own_len, int Hq, int Hkv, int d,
                               int max_pages, int num_pages_total, float scale, void* o, float* lse, void* workspace,
                               const SharedPlan& plan, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedArgs a = {};
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.group_offsets = group_offsets;
  a.prefix_lens = prefix_lens;
  a.page_size = page_size;
  while (1 << a.page_shift < page_size) ++a.page_shift;
  a.num_seqs = num_seqs;
  a.num_groups = num_groups;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  while (1 << a.g_shift < a.G) ++a.g_shift;
  a.max_pages = max_pages;
  a.num_pages_total = num_pages_total;
  a.n_ctas = plan.n_ctas;
  a.max_own = max_own_len;
  a.scale = scale;
  // a scale of 0 (equal weights) becomes the smallest number there is, 2^-149: masked scores are -inf, and 0 times
  // that would be NaN; finite ones come to less than 2^-21 and weigh 1
  a.scale_log2 = fmaxf(scale * 1.4426950408889634f, 1.4e-45f);
  a.status = reinterpret_cast<unsigned*>(ws);
  a.per_cta = reinterpret_cast<long long*>(ws + 128);
  a.cta_status = reinterpret_cast<unsigned*>(ws + plan.cta_status);
  a.groups = reinterpret_cast<GroupPlan*>(ws + plan.groups);
  a.seqs = reinterpret_cast<SeqPlan*>(ws + plan.seqs);
  a.pre_o = reinterpret_cast<float*>(ws + plan.pre_o);
  a.pre_lse = reinterpret_cast<float*>(ws + plan.pre_lse);
  a.own_o = reinterpret_cast<float*>(ws + plan.own_o);
  a.own_lse = reinterpret_cast<float*>(ws + plan.own_lse);

  const bool four = a.G <= 4;
  const ta_status st = d == 128 ? (four ? launch_attend<128, 4> : launch_attend<128, 8>)(q, k_cache, v_cache, a, stream)
                                : (four ? launch_attend<64, 4> : launch_attend<64, 8>)(q, k_cache, v_cache, a, stream);
  if (st != TA_OK) return st;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(o);
  const cudaError_t e = d == 128 ? launch_combine<128>(a, out, lse, stream) : launch_combine<64>(a, out, lse, stream);
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "shared decode: combine kernel launch", e);
}

}  // namespace ta
