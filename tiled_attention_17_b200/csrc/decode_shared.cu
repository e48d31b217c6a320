// Paged decode of a batch whose sequences share long prefixes: the prefix of a
// group of sequences is read and multiplied once for all of them.
//
// Softmax over a sequence's keys splits exactly into softmax over the group's
// prefix and softmax over the keys the sequence has of its own, joined by their
// log-sum-exp (FlashAttention optimisation article, section 3.2.2).  Decode
// alone reads every key once per sequence and is bound by those bytes.  Over a
// shared prefix the queries of the whole group meet each key, so the prefix is
// a matrix product: rows are (sequence, query head of one KV head) pairs, 128
// to a tile, and K/V tiles of 128 keys are read once for up to 256 rows.
//
// Four kernels, each a programmatic dependent of the one before where it can be:
//   shared_plan_kernel     one CTA: the group of each sequence, where its own
//                          keys start, and a running count of the prefix work
//   prefix_kernel          tcgen05: all prefix work, cut evenly over the SMs
//   decode_split_* <kOwn>  the paged decode's split kernels over own keys; they
//                          fill SMs as prefix CTAs leave
//   shared_combine_kernel  joins a row's partials by their log-sum-exp
//
// Work of the prefix kernel.  A unit is (group, KV head, 256 query rows); its
// steps are the prefix's 128-key tiles.  All units' steps are laid end to end
// and CTA c of n takes steps [c L, (c + 1) L), L = ceil(steps / n): equal shares
// whatever the groups' sizes and lengths, at the price of one partial result
// per CTA and unit it touches.  The (c, unit) pairs met along the line are
// monotone in both, so slot c + unit holds a pair's partial without a table.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"
#include "tiledattn_internal.h"

namespace ta {
namespace {

constexpr int kTile = 128;           // query rows and keys of a tile
constexpr int kUnitRows = 2 * kTile;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;
constexpr int kLaunchRegs = 168, kRegsControl = 56, kRegsSoftmax = 224;   // register split of the prefill kernel
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * kLaunchRegs, "register split");
constexpr float kRescaleLog2 = 8.0f;   // the stale-max margin of the prefill kernel
// Fewest steps a CTA takes.
constexpr int kMinSteps = 1;

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One group as the plan kernel found it: ranges checked, work counted.
struct __align__(16) Group {
  long long step0;   // steps of all groups before it
  int unit0;         // units of all groups before it
  int first, n;      // its sequences
  int len;           // prefix length
  int pad[2];
};
static_assert(sizeof(Group) == 32, "two 16-byte loads");

struct PlanHeader {
  long long steps;     // of all groups
  long long per_cta;   // L
};

__host__ __device__ __forceinline__ int prefix_tiles(int len) { return (len + kTile - 1) / kTile; }
__host__ __device__ __forceinline__ int row_blocks(int n, int G) {
  return static_cast<int>((static_cast<long long>(n) * G + kUnitRows - 1) / kUnitRows);
}

struct SharedArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* group_offsets;
  const int32_t* prefix_lens;
  int page_size, num_seqs, num_groups, Hq, Hkv, G, max_pages, num_pages_total, n_ctas;
  int own_splits, own_split_pages, max_own;
  float scale, scale_log2;
  // workspace
  unsigned* status;
  PlanHeader* header;
  Group* groups;        // [num_groups + 1]; the last only ends the counts
  int32_t* own_start;   // [num_seqs] first key a sequence reads itself
  int32_t* group_of;    // [num_seqs] group whose prefix it uses, or -1
  float* pre_o;         // [slots][D / 4][256][4] normalised prefix partials
  float* pre_lse;       // [slots][256]
  float* own_o;         // [num_seqs][Hq][own_splits][D]
  float* own_lse;       // [num_seqs][Hq][own_splits]
};

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

// bad_offsets: the offsets decrease or leave the batch, so groups might overlap.
__device__ __forceinline__ Group read_group(const SharedArgs& a, int g, bool& bad_offsets, bool& bad_len) {
  const int cap = a.max_pages * a.page_size;
  const int lo = __ldg(a.group_offsets + g), hi = __ldg(a.group_offsets + g + 1), len = __ldg(a.prefix_lens + g);
  Group r = {};
  r.first = min(max(lo, 0), a.num_seqs);
  const int end = min(max(hi, r.first), a.num_seqs);
  r.n = end - r.first;
  r.len = r.n > 0 ? min(max(len, 0), cap) : 0;   // a group without sequences shares nothing, whatever its length
  bad_offsets = bad_offsets || lo != r.first || hi != end;
  bad_len = bad_len || (r.n > 0 && len != r.len);
  return r;
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs a) {
  __shared__ long long s_steps[kPlanThreads / 32];
  __shared__ int s_units[kPlanThreads / 32];
  grid_launch_dependents();   // the prefix kernel sets up meanwhile; it waits before it reads the plan
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) *a.status = 0;
  __syncthreads();
  bool bad_offsets = false, bad_len = false, seen = false;

  // running counts over the groups: each thread a contiguous run of them
  const int run = (a.num_groups + kPlanThreads - 1) / kPlanThreads;
  const int g0 = min(tid * run, a.num_groups), g1 = min(g0 + run, a.num_groups);
  long long steps = 0;
  int units = 0;
  auto group_units = [&](const Group& r) { return r.len > 0 ? row_blocks(r.n, a.G) * a.Hkv : 0; };
  for (int g = g0; g < g1; ++g) {
    const Group r = read_group(a, g, bad_offsets, bad_len);
    const int u = group_units(r);
    units += u;
    steps += static_cast<long long>(u) * prefix_tiles(r.len);
  }
  long long st = steps;
  int un = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, st, o);
    const int y = __shfl_up_sync(0xffffffffu, un, o);
    if (lane >= o) {
      st += x;
      un += y;
    }
  }
  if (lane == 31) {
    s_steps[warp] = st;
    s_units[warp] = un;
  }
  // groups that might overlap are all left out (flagged): every sequence then reads its own keys only
  const bool ignore = __syncthreads_or(bad_offsets);
  long long before = st - steps, total = 0;
  int before_u = un - units;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      before += s_steps[w];
      before_u += s_units[w];
    }
    total += s_steps[w];
  }
  for (int g = g0; g < g1; ++g) {
    Group r = read_group(a, g, seen, seen);
    r.step0 = before;
    r.unit0 = before_u;
    a.groups[g] = r;
    const int u = group_units(r);
    before_u += u;
    before += static_cast<long long>(u) * prefix_tiles(r.len);
  }
  if (ignore) total = 0;
  if (tid == 0) {
    Group end = {};
    end.step0 = total;
    a.groups[a.num_groups] = end;
    a.header->steps = total;
    const long long per = (total + a.n_ctas - 1) / a.n_ctas;
    a.header->per_cta = per < kMinSteps ? kMinSteps : per;
  }

  // The group of each sequence: the first whose end lies behind it.  A
  // sequence shorter than its group's prefix does not use it (its keys are
  // all its own).
  for (int s = tid; s < a.num_seqs; s += kPlanThreads) {
    int lo = 0, hi = a.num_groups;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.group_offsets + mid + 1) <= s) lo = mid + 1;
      else hi = mid;
    }
    int start = 0, of = -1;
    if (lo < a.num_groups && !ignore) {
      const Group r = read_group(a, lo, seen, seen);
      if (s >= r.first && s < r.first + r.n && r.len > 0 && __ldg(a.seq_lens + s) >= r.len) {
        start = r.len;
        of = lo;
      }
    }
    a.own_start[s] = start;
    a.group_of[s] = of;
  }
  if (bad_offsets || bad_len) atomicOr(a.status, kDevBadSeqLen);
}

// ---------------------------------------------------------------------------
// Prefix
// ---------------------------------------------------------------------------
template <int D>
struct PrefixLayout {
  static constexpr int kChunks = D / 64;               // 128-byte swizzle rows along d
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kChunkBytes = kTile * 128;
  static constexpr int kStages = D == 128 ? 2 : 4;     // K ring and V ring depth
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBar = kV + kStages * kTileBytes;
  // q, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full[2], p_ready[2], o_done[2], p_half[2],
  // q_free, o_free[2], mma_done
  static constexpr int kNumBars = 1 + 4 * kStages + 12;
  static constexpr int kMisc = kBar + kNumBars * 8;     // tmem base, abort flag
  static constexpr int kAlloc = kMisc + 16 + 1024;      // slack to align the base to 1024 B
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kTmS0 = 0, kTmS1 = 128, kTmO0 = 256, kTmO1 = 256 + D;
};

// The CTA's place on the line of steps.  All roles walk it alike.
struct Segment {
  int row0;          // first row of the unit among the group's (sequence, head) rows
  int rows;          // rows of the unit (1..256)
  int first;         // first sequence of the group
  int hkv, len;      // KV head, prefix length
  int tile0, tiles;  // key tiles [tile0, tile0 + tiles)
  int slot;          // of its partial result
};
struct Walk {   // groups are read again for each segment: registers are scarcer than cached loads
  long long x, end;
  int g;

  __device__ __forceinline__ void start(const SharedArgs& a, long long steps, long long per) {
    x = per * blockIdx.x;
    end = min(steps, x + per);
    int lo = 0, hi = a.num_groups;   // the last group that starts at or before x: it owns step x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.groups[mid].step0 <= x) lo = mid;
      else hi = mid;
    }
    g = lo;
  }
  __device__ __forceinline__ bool more() const { return x < end; }
  __device__ __forceinline__ Segment next(const SharedArgs& a) {
    while (a.groups[g + 1].step0 <= x) ++g;   // the entry behind the last group holds the total
    const Group grp = a.groups[g];
    const int tiles = prefix_tiles(grp.len), blocks = row_blocks(grp.n, a.G);
    const long long in_group = x - grp.step0, unit = in_group / tiles;
    Segment s;
    s.tile0 = static_cast<int>(in_group - unit * tiles);
    s.tiles = static_cast<int>(min(static_cast<long long>(tiles - s.tile0), end - x));
    s.hkv = static_cast<int>(unit) / blocks;
    s.row0 = static_cast<int>(unit) % blocks * kUnitRows;
    s.rows = min(kUnitRows, grp.n * a.G - s.row0);
    s.first = grp.first;
    s.len = grp.len;
    s.slot = static_cast<int>(blockIdx.x) + grp.unit0 + static_cast<int>(unit);
    x += s.tiles;
    return s;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const SharedArgs a) {
  using L = PrefixLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::kQ, sK = sbase + L::kK, sV = sbase + L::kV;
  const uint32_t bar0 = sbase + L::kBar;
  constexpr int S4 = 4 * L::kStages;
  const uint32_t BAR_Q = bar0, BAR_QE = bar0 + 8u * (9 + S4), BAR_FIN = bar0 + 8u * (12 + S4);
  auto BAR_KF = [&](int s) { return bar0 + 8u * (1 + s); };
  auto BAR_KE = [&](int s) { return bar0 + 8u * (1 + L::kStages + s); };
  auto BAR_VF = [&](int s) { return bar0 + 8u * (1 + 2 * L::kStages + s); };
  auto BAR_VE = [&](int s) { return bar0 + 8u * (1 + 3 * L::kStages + s); };
  auto BAR_SF = [&](int t) { return bar0 + 8u * (1 + S4 + t); };
  auto BAR_PR = [&](int t) { return bar0 + 8u * (3 + S4 + t); };
  auto BAR_OD = [&](int t) { return bar0 + 8u * (5 + S4 + t); };
  auto BAR_PH = [&](int t) { return bar0 + 8u * (7 + S4 + t); };
  auto BAR_OF = [&](int t) { return bar0 + 8u * (10 + S4 + t); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- setup, before the plan is needed
  if (threadIdx.x == 0) {
    mbar_init(BAR_Q, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(BAR_KF(s), 1);
      mbar_init(BAR_KE(s), 1);
      mbar_init(BAR_VF(s), 1);
      mbar_init(BAR_VE(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR_SF(t), 1);
      mbar_init(BAR_PR(t), 128);
      mbar_init(BAR_OD(t), 1);
      mbar_init(BAR_PH(t), 128);
      mbar_init(BAR_OF(t), 128);
    }
    mbar_init(BAR_QE, 1);
    mbar_init(BAR_FIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_wait();                // the plan is complete
  grid_launch_dependents();   // the own-keys kernel may take the SMs this grid leaves
  const long long steps = a.header->steps, per = a.header->per_cta;
  Walk walk;
  walk.start(a, steps, per);

  if (warp < kSoftmaxWarp0) {
    setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
      // ======================= TMA producer (lane p: page p of a tile) =======================
      const int per_tile = kTile / a.page_size;
      const uint32_t page_bytes = static_cast<uint32_t>(a.page_size) * D * 2;
      bool ok = true;
      uint32_t g = 0, gv = 0;    // K and V tiles whose copies were issued
      int qi = 0;
      while (walk.more() && ok) {
        const Segment sg = walk.next(a);
        const int32_t* row = a.block_table + static_cast<size_t>(sg.first) * a.max_pages;
        // this lane's page of key tile j, -1 past the prefix; an entry outside the pool reads page 0 and is flagged
        auto page_of = [&](int j) {
          const int p = j * per_tile + lane;
          if (lane >= per_tile || static_cast<long long>(p) * a.page_size >= sg.len) return -1;
          int pg = __ldg(row + p);
          if (pg < 0 || pg >= a.num_pages_total) {
            atomicOr(a.status, kDevBadBlockTable);
            pg = 0;
          }
          return pg;
        };
        int pg = page_of(sg.tile0);
        if (qi > 0 && !(ok = mbar_wait_warp(BAR_QE, static_cast<uint32_t>(qi - 1) & 1u, a.status, abort_flag))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(BAR_Q, (sg.rows > kTile ? 2u : 1u) * L::kTileBytes);
          const int seq0 = sg.first + sg.row0 / a.G, seqs = kTile / a.G;
          tma_load_4d(sQ, &tmQ, BAR_Q, 0, sg.hkv * a.G, seq0, 0);
          if (sg.rows > kTile) tma_load_4d(sQ + L::kTileBytes, &tmQ, BAR_Q, 0, sg.hkv * a.G, seq0 + seqs, 0);
        }
        ++qi;
        // A page arrives in one copy, in the layouts of the paged prefill: with two
        // 64-column chunks K in the 32-byte swizzle ([8-row group][K step][8 rows]
        // [32 B]) and V page-major ([page][chunk][page rows][128 B]).
        auto copy = [&](const CUtensorMap* tm, uint32_t dst, uint32_t bar, bool is_v) {
          const uint32_t live = __ballot_sync(0xffffffffu, pg >= 0);
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(live)) * page_bytes);
          __syncwarp();
          if (pg >= 0) {
            const uint32_t at = dst + static_cast<uint32_t>(lane) * page_bytes;
            if (L::kChunks == 1) tma_load_4d(at, tm, bar, 0, 0, sg.hkv, pg);
            else if (is_v) tma_load_5d(at, tm, bar, 0, 0, 0, sg.hkv, pg);
            else tma_load_5d(at, tm, bar, 0, 0, 0, 0, pg * a.Hkv + sg.hkv);
          }
        };
        for (int j = 0; j < sg.tiles; ++j) {
          const int s = static_cast<int>(g % L::kStages);
          const uint32_t ph = (g / L::kStages) & 1u;
          if (!(ok = mbar_wait_warp(BAR_KE(s), ph ^ 1u, a.status, abort_flag))) break;
          copy(&tmK, sK + s * L::kTileBytes, BAR_KF(s), false);
          ++g;
          if (!(ok = mbar_wait_warp(BAR_VE(s), ph ^ 1u, a.status, abort_flag))) break;
          copy(&tmV, sV + s * L::kTileBytes, BAR_VF(s), true);
          ++gv;
          if (j + 1 < sg.tiles) pg = page_of(sg.tile0 + j + 1);
        }
      }
      // drain: no copy into this CTA's shared memory may still be in flight at exit
      if (lane == 0) {
        if (qi > 0) mbar_wait(BAR_Q, static_cast<uint32_t>(qi - 1) & 1u, nullptr, nullptr, kWaitLimitNs);
        constexpr uint32_t kS = L::kStages;
        for (uint32_t gg = (g > kS ? g - kS : 0u); gg < g; ++gg)
          mbar_wait(BAR_KF(static_cast<int>(gg % kS)), (gg / kS) & 1u, nullptr, nullptr, kWaitLimitNs);
        for (uint32_t gg = (gv > kS ? gv - kS : 0u); gg < gv; ++gg)
          mbar_wait(BAR_VF(static_cast<int>(gg % kS)), (gg / kS) & 1u, nullptr, nullptr, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ======================= MMA issuer (whole warp; the elected lane issues) =======================
      const bool leader = elect_one_sync();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kTile, kTile, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kTile, D, true);
      auto commit = [&](uint32_t bar) {
        if (leader) mma_commit(bar);
        __syncwarp();
      };
      auto tS = [&](int t) { return tmem + (t ? L::kTmS1 : L::kTmS0); };
      auto tO = [&](int t) { return tmem + (t ? L::kTmO1 : L::kTmO0); };
      constexpr bool kTwo = L::kChunks == 2;
      const uint64_t dQ = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dK = kTwo ? smem_desc_sw32(sK, 2048) : smem_desc_sw128(sK, 16, 1024);
      constexpr uint64_t kKStep = kTwo ? 16 : 2;
      const int ps = a.page_size;
      const uint64_t dV = kTwo ? smem_desc_sw128(sV, static_cast<uint32_t>(ps) * 128u, ps >= 16 ? 1024u : 2048u)
                               : smem_desc_sw128(sV, L::kChunkBytes, 1024);
      constexpr uint64_t kTileStep = L::kTileBytes >> 4;
      // page-major V: 16-key step kk starts at byte 2048 (kk + (kk & vmask))
      const int vmask = ~(max(ps / 16, 1) - 1);

      auto issue_qk = [&](int t, int s) {   // S_t = Q_t K^T
        uint64_t a0 = dQ + static_cast<uint64_t>(t) * kTileStep, b0 = dK + static_cast<uint64_t>(s) * kTileStep;
        if (leader) {
#pragma unroll 1
          for (int c = 0; c < L::kChunks; ++c) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
              mma_ss(tS(t), a0 + 2 * k4, b0 + kKStep * k4, idesc_qk, (c | k4) != 0 ? 1u : 0u);
            a0 += L::kChunkBytes >> 4;
            b0 += 4 * kKStep;
          }
        }
        __syncwarp();
      };
      auto issue_pv_half = [&](int t, int s, int half, bool acc) {   // O_t += P_t V over 64 keys
        const uint64_t b0 = dV + static_cast<uint64_t>(s) * kTileStep;
        if (leader) {
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int kk = half * 4 + k4;
            const uint32_t off = kTwo ? static_cast<uint32_t>((kk + (kk & vmask)) << 11) : kk * 2048u;
            mma_ts(tO(t), tS(t) + kk * 8, b0 + static_cast<uint64_t>(off >> 4), idesc_pv, (acc || kk > 0) ? 1u : 0u);
          }
        }
        __syncwarp();
      };

      bool ok = true;
      uint32_t g = 0;              // key tiles consumed
      uint32_t steps_t[2] = {0, 0};   // S/P/O barrier phases of each row tile
      int used[2] = {0, 0};        // segments whose O each row tile held
      int qi = 0;
      while (walk.more() && ok) {
        const Segment sg = walk.next(a);
        const int nt = sg.rows > kTile ? 2 : 1;
        if (!(ok = mbar_wait_warp(BAR_Q, static_cast<uint32_t>(qi) & 1u, a.status, abort_flag))) break;
        const int s0 = static_cast<int>(g % L::kStages);
        if (!(ok = mbar_wait_warp(BAR_KF(s0), (g / L::kStages) & 1u, a.status, abort_flag))) break;
        tc_fence_after();
        for (int t = 0; t < nt; ++t) {
          issue_qk(t, s0);
          commit(BAR_SF(t));
        }
        commit(BAR_KE(s0));
        if (sg.tiles == 1) commit(BAR_QE);
        for (int j = 0; j < sg.tiles && ok; ++j) {
          const uint32_t gj = g + static_cast<uint32_t>(j);
          const int s = static_cast<int>(gj % L::kStages), s1 = static_cast<int>((gj + 1) % L::kStages);
          if (!(ok = mbar_wait_warp(BAR_VF(s), (gj / L::kStages) & 1u, a.status, abort_flag))) break;
          for (int t = 0; t < nt; ++t) {
            const uint32_t c = steps_t[t];
            // the first P.V of a segment overwrites O_t: the last segment's epilogue must have read it
            if (j == 0 && used[t] > 0 &&
                !(ok = mbar_wait_warp(BAR_OF(t), static_cast<uint32_t>(used[t] - 1) & 1u, a.status, abort_flag)))
              break;
            if (!(ok = mbar_wait_warp(BAR_PH(t), c & 1u, a.status, abort_flag))) break;
            tc_fence_after();
            issue_pv_half(t, s, 0, j > 0);
            if (!(ok = mbar_wait_warp(BAR_PR(t), c & 1u, a.status, abort_flag))) break;
            tc_fence_after();
            issue_pv_half(t, s, 1, true);
            commit(BAR_OD(t));
            if (j + 1 < sg.tiles) {
              if (!(ok = mbar_wait_warp(BAR_KF(s1), ((gj + 1) / L::kStages) & 1u, a.status, abort_flag))) break;
              issue_qk(t, s1);
              commit(BAR_SF(t));
            }
            steps_t[t] = c + 1;
          }
          if (!ok) break;
          if (j + 2 == sg.tiles) commit(BAR_QE);   // the segment's last Q.K^T has been issued
          commit(BAR_VE(s));
          if (j + 1 < sg.tiles) commit(BAR_KE(s1));
        }
        if (!ok) break;
        for (int t = 0; t < nt; ++t) ++used[t];
        g += static_cast<uint32_t>(sg.tiles);
        ++qi;
      }
      // no commit may still be pending when the CTA exits
      commit(BAR_FIN);
      mbar_wait_warp(BAR_FIN, 0, nullptr, nullptr);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ======================= softmax warpgroups (one thread per query row) =======================
    const int t = (warp - kSoftmaxWarp0) / 4;
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + (t == 0 ? L::kTmS0 : L::kTmS1) + lane_off;
    const uint32_t tO = tmem + (t == 0 ? L::kTmO0 : L::kTmO1) + lane_off;
    const float c2 = a.scale_log2;
    bool ok = true;
    uint32_t steps_t = 0, g = 0;
    while (walk.more() && ok) {
      const Segment sg = walk.next(a);
      if (t * kTile >= sg.rows) {   // this row tile has no rows
        g += static_cast<uint32_t>(sg.tiles);
        continue;
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < sg.tiles; ++j, ++g) {
        ok = __all_sync(0xffffffffu, mbar_wait(BAR_SF(t), (steps_t + j) & 1u, a.status, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
        tmem_wait_ld();
        float* s = reinterpret_cast<float*>(&sr[0][0]);
        // keys of this tile: [0, lim); the rest of its shared memory holds no key
        const int lim = min(kTile, sg.len - (sg.tile0 + j) * kTile);
        const bool need_mask = lim < kTile;
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = c < lim ? s[c] : -INFINITY;
          // V rows past the keys get weight 0, and whatever is there must not
          // turn that into NaN: the first row tile's warps zero them (its P.V is
          // issued first).
          if (t == 0) {
            const int sv = static_cast<int>(g % L::kStages);
            ok = __all_sync(0xffffffffu, mbar_wait(BAR_VF(sv), (g / L::kStages) & 1u, a.status, abort_flag));
            if (!ok) break;
            if (row >= lim) {
              const int pr = row % a.page_size;
              uint8_t* base = smem + L::kV + sv * L::kTileBytes + (row - pr) * D * 2 + pr * 128;
#pragma unroll
              for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  reinterpret_cast<uint4*>(base + c * a.page_size * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();   // before the products read them
          }
        }
        // 64 columns: weights 2^((s - m) c2), packed to bf16; the sum of the
        // unrounded values.  Masked columns are exactly 0.
        auto exp_half = [&](auto masked, int h, float negm, uint32_t (&pk)[32]) -> float {
          constexpr bool kMasked = decltype(masked)::value;
          const float2 c2v = make_float2(c2, c2), negv = make_float2(negm, negm);
          float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = h * 64 + 2 * i;
            const float2 x = ffma2(make_float2(s[c], s[c + 1]), c2v, negv);
            float2 pp = make_float2(ex2(x.x), ex2(x.y));
            if constexpr (kMasked) {
              pp.x = c < lim ? pp.x : 0.f;
              pp.y = c + 1 < lim ? pp.y : 0.f;
            }
            if (i & 1) sb = fadd2(sb, pp);
            else sa = fadd2(sa, pp);
            pk[i] = pack_bf16x2(pp.x, pp.y);
          }
          return (sa.x + sb.x) + (sa.y + sb.y);
        };
        auto exp_half_any = [&](int h, float negm, uint32_t (&pk)[32]) -> float {
          return need_mask ? exp_half(std::true_type{}, h, negm, pk) : exp_half(std::false_type{}, h, negm, pk);
        };
        float mx;
        {
          float r0 = -INFINITY, r1 = -INFINITY, r2 = -INFINITY, r3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            r0 = fmax3(r0, s[c + 0], s[c + 1]);
            r1 = fmax3(r1, s[c + 2], s[c + 3]);
            r2 = fmax3(r2, s[c + 4], s[c + 5]);
            r3 = fmax3(r3, s[c + 6], s[c + 7]);
          }
          mx = fmaxf(fmax3(r0, r1, r2), r3);
        }
        const float m_new = fmaxf(m, mx);
        const bool upd = (m == -INFINITY) || ((m_new - m) * c2 > kRescaleLog2);
        const float m_use = upd ? m_new : m;
        const float alpha = (upd && m != -INFINITY) ? ex2((m - m_use) * c2) : (m == -INFINITY ? 0.f : 1.f);
        const float negm = (m_use == -INFINITY) ? 0.f : -m_use * c2;
        m = m_use;
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t orr[32];
            tmem_ld32(tO + c * 32, orr);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
            tmem_st32(tO + c * 32, orr);
          }
        }
        float psum;
        {
          uint32_t pk[32];
          psum = exp_half_any(0, negm, pk);
          tmem_st32(tS, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR_PH(t));
        {
          uint32_t pk[32];
          psum += exp_half_any(1, negm, pk);
          tmem_st32(tS + 32, pk);
        }
        l = alpha * l + psum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR_PR(t));
      }
      if (!ok) break;
      // ---- the segment's partial: O / l and m scale + ln l, in fp32
      ok = __all_sync(0xffffffffu, mbar_wait(BAR_OD(t), (steps_t + sg.tiles - 1) & 1u, a.status, abort_flag));
      tc_fence_after();
      if (!ok) break;
      steps_t += static_cast<uint32_t>(sg.tiles);
      const int urow = t * kTile + row;
      const bool store = urow < sg.rows;
      const float inv = (l > 0.f) ? 1.f / l : 0.f;
      float4* dst = reinterpret_cast<float4*>(a.pre_o) + static_cast<size_t>(sg.slot) * (D / 4) * kUnitRows + urow;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        tmem_ld32(tO + c * 32, orr);
        tmem_wait_ld();
        if (store) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[(c * 8 + e) * kUnitRows] =
                make_float4(__uint_as_float(orr[4 * e]) * inv, __uint_as_float(orr[4 * e + 1]) * inv,
                            __uint_as_float(orr[4 * e + 2]) * inv, __uint_as_float(orr[4 * e + 3]) * inv);
        }
      }
      tc_fence_before();
      mbar_arrive(BAR_OF(t));
      if (store)
        a.pre_lse[static_cast<size_t>(sg.slot) * kUnitRows + urow] =
            (l > 0.f) ? fmaf(m, a.scale, __log2f(l) * 0.69314718055994531f) : -INFINITY;
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Combine: one CTA per (KV head, sequence).  Thread (p, c4, g) joins every NP-th
// partial of columns [4 c4, 4 c4 + 4) of query head g, the NP runs meet in
// shared memory.  Weights e^(lse_i - max) over all partials of a row.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

template <int D, int G>
__global__ void __launch_bounds__(kCombineThreads) shared_combine_kernel(const SharedArgs a, __nv_bfloat16* o,
                                                                       float* lse) {
  constexpr int kPer = G * D / 4, NP = kCombineThreads / kPer;
  static_assert(kPer <= kCombineThreads && kCombineThreads % kPer == 0, "threads per partial");
  __shared__ float s_m[kCombineThreads], s_l[kCombineThreads];
  __shared__ float4 s_o[kCombineThreads];
  const int hkv = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
  const int p0 = tid / kPer, c4 = (tid % kPer) / G, gq = tid % G;
  grid_wait();   // both kernels that write partials are complete
  const int cap = a.max_pages * a.page_size;
  const int start = a.own_start[seq], of = a.group_of[seq];
  int len = min(max(__ldg(a.seq_lens + seq), 0), cap);
  len = min(len, start + a.max_own);
  const int split_tokens = a.own_split_pages * a.page_size;
  const int base = start / a.page_size * a.page_size;
  const int n_own = len > start ? (len - base + split_tokens - 1) / split_tokens : 0;
  int n_pre = 0, urow = 0;
  long long slot0 = 0;
  if (of >= 0) {
    const Group r = a.groups[of];
    const int tiles = prefix_tiles(r.len), blocks = row_blocks(r.n, G), rr = (seq - r.first) * G + gq;
    const long long unit = static_cast<long long>(hkv) * blocks + rr / kUnitRows;
    const long long x0 = r.step0 + unit * tiles, per = a.header->per_cta;
    const long long c0 = x0 / per, c1 = (x0 + tiles - 1) / per;
    n_pre = static_cast<int>(c1 - c0 + 1);
    slot0 = c0 + r.unit0 + unit;
    urow = rr % kUnitRows;
  }
  const int hq = hkv * G + gq;
  const size_t own0 = (static_cast<size_t>(seq) * a.Hq + hq) * a.own_splits;

  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = p0; i < n_pre + n_own; i += NP) {
    float w;
    float4 v;
    if (i < n_pre) {
      w = a.pre_lse[(slot0 + i) * kUnitRows + urow];
      v = reinterpret_cast<const float4*>(a.pre_o)[((slot0 + i) * (D / 4) + c4) * kUnitRows + urow];
    } else {
      w = a.own_lse[own0 + i - n_pre];
      v = reinterpret_cast<const float4*>(a.own_o + (own0 + i - n_pre) * D)[c4];
    }
    if (w == -INFINITY) continue;
    const float mn = fmaxf(m, w), s0 = __expf(m - mn), s1 = __expf(w - mn);
    l = fmaf(l, s0, s1);
    acc.x = fmaf(acc.x, s0, s1 * v.x);
    acc.y = fmaf(acc.y, s0, s1 * v.y);
    acc.z = fmaf(acc.z, s0, s1 * v.z);
    acc.w = fmaf(acc.w, s0, s1 * v.w);
    m = mn;
  }
  s_m[tid] = m;
  s_l[tid] = l;
  s_o[tid] = acc;
  __syncthreads();
  if (p0 != 0) return;
  float M = m;
  for (int p = 1; p < NP; ++p) M = fmaxf(M, s_m[p * kPer + tid]);
  float tot = 0.f;
  float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < NP; ++p) {
    const int e = p * kPer + tid;
    if (s_m[e] == -INFINITY) continue;
    const float w = __expf(s_m[e] - M);
    const float4 v = s_o[e];
    tot = fmaf(w, s_l[e], tot);
    out.x = fmaf(w, v.x, out.x);
    out.y = fmaf(w, v.y, out.y);
    out.z = fmaf(w, v.z, out.z);
    out.w = fmaf(w, v.w, out.w);
  }
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  const size_t orow = static_cast<size_t>(seq) * a.Hq + hq;
  uint2 w2;
  w2.x = pack_bf16x2(out.x * inv, out.y * inv);
  w2.y = pack_bf16x2(out.z * inv, out.w * inv);
  reinterpret_cast<uint2*>(o + orow * D)[c4] = w2;
  if (c4 == 0 && lse) lse[orow] = tot > 0.f ? M + __logf(tot) : -INFINITY;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
ta_status launch_prefix(const void* q, const void* k_cache, const void* v_cache, const SharedArgs& a,
                        cudaStream_t stream) {
  using L = PrefixLayout<D>;
  CUtensorMap tq, tk, tv;
  ta_status st;
  {  // queries [S, Hq, d] as {64, Hq, S, d / 64}: a box of G heads of 128 / G sequences is one tile of 128 rows
    const uint64_t dims[4] = {64, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.num_seqs), D / 64};
    const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(a.Hq) * D * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(kTile / a.G), D / 64};
    if ((st = encode_bf16_tiled(&tq, q, 4, dims, strides, box)) != TA_OK) return st;
  }
  if ((st = encode_pool_maps(&tk, &tv, k_cache, v_cache, D, a.page_size, a.Hkv, a.num_pages_total)) != TA_OK) return st;
  static int attr_done[64] = {0};
  cudaError_t e = ensure_smem_limit(prefix_kernel<D>, L::kAlloc, attr_done);
  if (e != cudaSuccess) return fail(TA_ERR_CUDA, "shared decode: shared-memory limit", e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefix_kernel<D>, tq, tk, tv, a);
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "shared decode: prefix kernel launch", e);
}

template <int D, int G>
cudaError_t launch_combine(const SharedArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.Hkv), static_cast<unsigned>(a.num_seqs));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_combine_kernel<D, G>, a, o, lse);
}

template <int D>
cudaError_t launch_combine_g(const SharedArgs& a, __nv_bfloat16* o, float* lse, cudaStream_t stream) {
  switch (a.G) {
    case 1: return launch_combine<D, 1>(a, o, lse, stream);
    case 2: return launch_combine<D, 2>(a, o, lse, stream);
    case 4: return launch_combine<D, 4>(a, o, lse, stream);
    default: return launch_combine<D, 8>(a, o, lse, stream);
  }
}

}  // namespace

bool make_shared_plan(int num_seqs, int num_groups, int Hq, int Hkv, int d, int max_own_len, int page_size,
                      SharedPlan* p) {
  if (num_seqs < 0 || num_groups < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || max_own_len < 0 || page_size <= 0) return false;
  const int G = Hq / Hkv;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || num_seqs > 65535 || Hkv > 65535 || num_groups > 65535) return false;
  // own keys start inside a page at worst: one page more than their own
  const int own_pages = max_own_len == 0 ? 0 : (max_own_len + page_size - 1) / page_size + 1;
  if (!make_decode_plan(num_seqs, Hq, Hkv, d, own_pages > 0 ? own_pages : 1, page_size, &p->own)) return false;
  if (own_pages == 0) p->own.max_splits = 0;
  p->n_ctas = current_sm_count();
  // units: every group has at most one block of rows that is not full, per KV head
  const long long units = num_groups == 0 ? 0 : static_cast<long long>(Hkv) * (num_groups + static_cast<long long>(num_seqs) * G / kUnitRows);
  const long long slots = units == 0 ? 0 : units + p->n_ctas;
  if (slots > INT32_MAX) return false;
  size_t at = 512;   // status word, plan header
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  p->groups = take((static_cast<size_t>(num_groups) + 1) * sizeof(Group));
  p->own_start = take(static_cast<size_t>(num_seqs) * 4);
  p->group_of = take(static_cast<size_t>(num_seqs) * 4);
  p->pre_o = take(static_cast<size_t>(slots) * kUnitRows * d * 4);
  p->pre_lse = take(static_cast<size_t>(slots) * kUnitRows * 4);
  const size_t rows = static_cast<size_t>(num_seqs) * Hq * p->own.max_splits;
  p->own_o = take(rows * d * 4);
  p->own_lse = take(rows * 4);
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
  a.num_seqs = num_seqs;
  a.num_groups = num_groups;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.max_pages = max_pages;
  a.num_pages_total = num_pages_total;
  a.n_ctas = plan.n_ctas;
  a.own_splits = plan.own.max_splits;
  a.own_split_pages = plan.own.split_pages;
  a.max_own = max_own_len;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = reinterpret_cast<unsigned*>(ws);
  a.header = reinterpret_cast<PlanHeader*>(ws + 256);
  a.groups = reinterpret_cast<Group*>(ws + plan.groups);
  a.own_start = reinterpret_cast<int32_t*>(ws + plan.own_start);
  a.group_of = reinterpret_cast<int32_t*>(ws + plan.group_of);
  a.pre_o = reinterpret_cast<float*>(ws + plan.pre_o);
  a.pre_lse = reinterpret_cast<float*>(ws + plan.pre_lse);
  a.own_o = reinterpret_cast<float*>(ws + plan.own_o);
  a.own_lse = reinterpret_cast<float*>(ws + plan.own_lse);

  shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TA_ERR_CUDA, "shared decode: plan kernel launch", e);
  if (num_groups > 0) {
    const ta_status st = d == 128 ? launch_prefix<128>(q, k_cache, v_cache, a, stream)
                                  : launch_prefix<64>(q, k_cache, v_cache, a, stream);
    if (st != TA_OK) return st;
  }
  if (plan.own.max_splits > 0) {
    // without a prefix kernel in between it has to wait for the plan kernel: an ordinary launch
    e = launch_decode_own(q, k_cache, v_cache, block_table, seq_lens, a.own_start, max_own_len, page_size, num_seqs,
                          Hq, Hkv, d, max_pages, num_pages_total, scale, plan.own, a.own_o, a.own_lse, a.status,
                          num_groups > 0, stream);
    if (e != cudaSuccess) return fail(TA_ERR_CUDA, "shared decode: own-keys kernel launch", e);
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(o);
  e = d == 128 ? launch_combine_g<128>(a, out, lse, stream) : launch_combine_g<64>(a, out, lse, stream);
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "shared decode: combine kernel launch", e);
}

}  // namespace ta
