// Rotary positions, and the write of new tokens into the paged cache with the
// rotation applied on the way.
//
// A row (one head of one token) holds rotary_dim / 2 pairs (a, b): neighbours
// (interleaved) or element i with element i + rotary_dim / 2 (half layout).
// Pair i of a token at position p turns by t = p * inv_freq[i]:
//   a' = amp (a cos t - b sin t),   b' = amp (a sin t + b cos t);
// the elements from rotary_dim on are copied.  The turn is linear, so the
// gradient is its transpose: the same with -t.
//
// The angle of a far position needs more than 32 bits (p = 10^6 at one radian
// a token leaves 0.06 rad of error in fp32): p * inv_freq / (2 pi) is formed in
// fp64, whole turns are dropped there, and only the fraction of a turn goes to
// fp32.  Sine and cosine of at most half a turn then come from the hardware's
// approximation: within 2^-21 of 1, next to the 2^-8 a bf16 result is rounded by.
//
// Bound: HBM bytes, each element read once and written once.  One thread owns
// 16 elements (8 pairs) of a row, in up to four heads of its token: the eight
// cosines and sines are formed once for them, while their loads (two of 16 bytes a
// head) are all in flight.  How many heads a thread takes is chosen in
// heads_per_thread (below).  Measured (B200): 4 x 4096 tokens, 16 heads of 128 in
// 24 us (5.6 TB/s), 16686 tokens of 48 rows of 128 appended in 69 us (5.9 TB/s), one
// token in 3.4 us.  With 2 or 8 heads in flight, blocks of 256, or loads marked as
// streaming the appends take 2 to 20% longer.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "tiledattn_internal.h"

namespace ta {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxHeads = 4;   // heads one thread takes at most, all loaded before the first is used

// Eight cosines and sines of pairs [8 u, 8 u + 8) at one position.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void make_turn(Turn& t, int position, const double* __restrict__ inv_freq, int u,
                                          float amp, float sign) {
  constexpr double kPerTurn = 0.15915494309189533577;   // 1 / (2 pi)
  constexpr double kRound = 6755399441055744.0;         // 1.5 * 2^52: adding and taking it off rounds to an integer
  constexpr float kTwoPi = 6.28318530717958647693f;
  const double p = static_cast<double>(position) * kPerTurn;   // |p f| < 2^51 for every int32 position and f < 2^20
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double turns = p * __ldg(inv_freq + 8 * u + e);
    const float angle = static_cast<float>(turns - ((turns + kRound) - kRound)) * kTwoPi;
    float s, c;
    __sincosf(angle, &s, &c);
    t.c[e] = c * amp;
    t.s[e] = s * (amp * sign);
  }
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = fmaf(x, c, -(y * s));
  b = fmaf(x, s, y * c);
}

// The 8 pairs of one row.  Half layout: va holds the pairs' first elements, vb
// the second ones.  Interleaved: va and vb are 16 consecutive elements.  fp32
// arithmetic, one rounding to bf16 (the cache's and the attention's type).
template <bool kPairs>
__device__ __forceinline__ void turn_row(uint4& va, uint4& vb, const Turn& t) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float2 x = bf16x2_to_f2(a[w]), y = bf16x2_to_f2(b[w]);
    if constexpr (kPairs) {
      turn_pair(x.x, x.y, t.c[w], t.s[w]);
      turn_pair(y.x, y.y, t.c[4 + w], t.s[4 + w]);
    } else {
      turn_pair(x.x, y.x, t.c[2 * w], t.s[2 * w]);
      turn_pair(x.y, y.y, t.c[2 * w + 1], t.s[2 * w + 1]);
    }
    a[w] = pack_bf16x2(x.x, x.y);
    b[w] = pack_bf16x2(y.x, y.y);
  }
}

// Where a thread's two 8-element vectors sit in a row.  Units below
// rotary_dim / 16 turn 8 pairs; the others copy 16 consecutive elements.
template <bool kPairs>
__device__ __forceinline__ void unit_vectors(int u, int rotary_dim, bool& turns, int& va, int& vb) {
  const int ru = rotary_dim >> 4;
  turns = u < ru;
  va = (!kPairs && turns) ? u : 2 * u;
  vb = (!kPairs && turns) ? u + ru : 2 * u + 1;
}

struct RopeArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  const int32_t* positions;   // null: the index in the sequence
  const double* inv_freq;
  int64_t xb, xh, xn, yb, yh, yn, pb;   // strides in elements
  int64_t tokens;                       // B * N
  int N, H, rotary_dim, heads;          // heads: heads one thread takes
  float amp, sign;
};

template <int D, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr int kUnits = D / 16;
  const int u = threadIdx.x % kUnits;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / kUnits) + threadIdx.x / kUnits;
  if (tok >= a.tokens) return;
  const int64_t b = tok / a.N, n = tok - b * a.N;
  bool turns;
  int va, vb;
  unit_vectors<kPairs>(u, a.rotary_dim, turns, va, vb);
  const int h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  const __nv_bfloat16* src = a.x + b * a.xb + n * a.xn;
  __nv_bfloat16* dst = a.y + b * a.yb + n * a.yn;

  uint4 ra[kMaxHeads], rb[kMaxHeads];   // in flight while the angles are formed
#pragma unroll
  for (int j = 0; j < kMaxHeads; ++j)
    if (h0 + j < h1) {
      const uint4* row = reinterpret_cast<const uint4*>(src + (h0 + j) * a.xh);
      ra[j] = row[va];
      rb[j] = row[vb];
    }
  Turn t;
  if (turns) make_turn(t, a.positions ? __ldg(a.positions + b * a.pb + n) : static_cast<int>(n), a.inv_freq, u, a.amp, a.sign);
#pragma unroll
  for (int j = 0; j < kMaxHeads; ++j)
    if (h0 + j < h1) {
      if (turns) turn_row<kPairs>(ra[j], rb[j], t);
      uint4* row = reinterpret_cast<uint4*>(dst + (h0 + j) * a.yh);
      row[va] = ra[j];
      row[vb] = rb[j];
    }
}

// ---------------------------------------------------------------------------
// Append to the paged cache
// ---------------------------------------------------------------------------
constexpr int kMaxStaged = 1024;   // sequence offsets (or samples of them) held in shared memory

struct AppendArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const int32_t* block_table;
  const int32_t* cu_seqlens;   // null: token s is sequence s's one new token
  const int32_t* seq_lens;
  const int32_t* positions;    // null: the slot in the sequence
  const double* inv_freq;
  int64_t qt, qh, kt, kh, vt, vh;   // strides in elements
  int page_size, num_seqs, total, Hq, Hkv, max_pages, num_pages_total, rotary_dim;
  int heads;                        // rows one thread takes
  int token_blocks;                 // blocks (in x) of tokens; those behind look at the sequences
  float amp;
  unsigned* status;
};

// Where one token goes: its slot in its sequence, and the first row of its
// page (-1: no page, nothing is written to the cache).
struct Place {
  int pos;          // rotation position; meaningful when `live`
  int live;         // 0: not a token of any sequence (or flagged): nothing is written
  int page, row;    // page -1: bad table entry
};

template <int D, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) paged_append_kernel(const AppendArgs a) {
  constexpr int kUnits = D / 16, kTokens = kRopeThreads / kUnits;
  __shared__ int s_cu[kMaxStaged];
  __shared__ Place s_place[kTokens];
  const int u = threadIdx.x % kUnits, in_block = threadIdx.x / kUnits;
  const int t0 = blockIdx.x * kTokens, tok = t0 + in_block;
  if (static_cast<int>(blockIdx.x) >= a.token_blocks) {
    // The blocks behind the tokens' look at every sequence's offsets and length: no token need lead to a bad one.  (In
    // the tokens' blocks the same loop took registers from their loads: 4 long prompts 131 -> 140 us.)
    unsigned bad = 0;
    for (int64_t s = static_cast<int64_t>(blockIdx.x - a.token_blocks) * kRopeThreads + threadIdx.x;
         s < a.num_seqs && blockIdx.y == 0; s += static_cast<int64_t>(gridDim.x - a.token_blocks) * kRopeThreads) {
      const int first = __ldg(a.cu_seqlens + s), end = __ldg(a.cu_seqlens + s + 1), len = __ldg(a.seq_lens + s);
      if (first < 0 || end < first || end > a.total || len < end - first || len > a.max_pages * a.page_size)
        bad = kDevBadSeqLen;
    }
    if (bad) atomicOr(a.status, bad);
    return;
  }
  bool turns;
  int va, vb;
  unit_vectors<kPairs>(u, a.rotary_dim, turns, va, vb);
  // rows of a token: query heads, then key heads, then value heads
  const int hq = a.q ? a.Hq : 0, rows = hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * a.heads, h1 = min(rows, h0 + a.heads);
  const bool in = tok < a.total;

  uint4 ra[kMaxHeads], rb[kMaxHeads];   // in flight while the tokens' places are found
#pragma unroll
  for (int j = 0; j < kMaxHeads; ++j)
    if (in && h0 + j < h1) {
      const int r = h0 + j;
      const __nv_bfloat16* p = r < hq            ? a.q + tok * a.qt + r * a.qh
                               : r < hq + a.Hkv ? a.k + tok * a.kt + (r - hq) * a.kh
                                                : a.v + tok * a.vt + (r - hq - a.Hkv) * a.vh;
      const uint4* row = reinterpret_cast<const uint4*>(p);
      ra[j] = row[va];
      rb[j] = row[vb];
    }

  // The sequence of a token: the number of sequence ends at or before it,
  // found by bisection among the ends staged in shared memory (every end up to
  // 1024 sequences, every stride-th beyond, the rest of the search in global
  // memory).  One pass of loads costs one memory latency; a bisection in
  // global memory would cost one for each step.
  int stride = 1, staged = 0;
  if (a.cu_seqlens) {
    stride = (a.num_seqs + kMaxStaged - 1) / kMaxStaged;
    staged = a.num_seqs / stride;   // samples: the ends of sequences stride - 1, 2 stride - 1, ...
    for (int i = threadIdx.x; i < staged; i += kRopeThreads) s_cu[i] = __ldg(a.cu_seqlens + (i + 1) * stride);
    __syncthreads();
  }
  if (threadIdx.x < kTokens) {
    const int t = t0 + threadIdx.x;
    Place pl = {0, 0, -1, 0};
    unsigned bad = 0;
    if (t < a.total) {
      int s = t, back = 1, brought = 1;   // the token sits `back` slots before the end of a sequence that brings `brought`
      bool found = true;
      if (a.cu_seqlens) {
        int lo = 0, hi = staged;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_cu[mid] <= t) lo = mid + 1;
          else hi = mid;
        }
        lo *= stride;
        hi = min(lo + stride - 1, a.num_seqs);
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(a.cu_seqlens + mid + 1) <= t) lo = mid + 1;
          else hi = mid;
        }
        s = lo;
        const int first = s < a.num_seqs ? __ldg(a.cu_seqlens + s) : INT32_MAX;
        found = first <= t;   // else a row outside every sequence
        if (found) {
          const int end = __ldg(a.cu_seqlens + s + 1);
          back = end - t;
          brought = end - first;
          if (first < 0 || end > a.total || back <= 0) {   // offsets that decrease, or run past the rows given
            bad |= kDevBadSeqLen;
            found = false;
          }
        }
      }
      if (found) {
        const int len = __ldg(a.seq_lens + s);
        if (!a.cu_seqlens && len == 0) {
          // an empty place of a fixed-size decode batch: no token
        } else if (len < brought || len > a.max_pages * a.page_size) {
          bad |= kDevBadSeqLen;
        } else {
          const int slot = len - back;
          pl.live = 1;
          pl.pos = a.positions ? __ldg(a.positions + t) : slot;
          pl.page = __ldg(a.block_table + static_cast<int64_t>(s) * a.max_pages + slot / a.page_size);
          pl.row = slot % a.page_size;
          if (pl.page < 0 || pl.page >= a.num_pages_total) {
            bad |= kDevBadBlockTable;
            pl.page = -1;
          }
        }
      }
    }
    if (bad && blockIdx.y == 0) atomicOr(a.status, bad);
    s_place[threadIdx.x] = pl;
  }
  __syncthreads();
  const Place pl = s_place[in_block];
  if (!pl.live) return;

  Turn t;
  if (turns && h0 < hq + a.Hkv) make_turn(t, pl.pos, a.inv_freq, u, a.amp, 1.f);
  const int64_t page_row = (static_cast<int64_t>(pl.page) * a.Hkv * a.page_size + pl.row) * D;
#pragma unroll
  for (int j = 0; j < kMaxHeads; ++j)
    if (h0 + j < h1) {
      const int r = h0 + j;
      const bool is_q = r < hq, is_v = r >= hq + a.Hkv;
      if (turns && !is_v) turn_row<kPairs>(ra[j], rb[j], t);
      if (is_q || pl.page >= 0) {
        const int64_t head = static_cast<int64_t>(is_v ? r - hq - a.Hkv : r - hq) * a.page_size * D;
        __nv_bfloat16* p = is_q   ? a.q_out + (static_cast<int64_t>(tok) * a.Hq + r) * D
                           : is_v ? a.v_cache + page_row + head
                                  : a.k_cache + page_row + head;
        uint4* row = reinterpret_cast<uint4*>(p);
        row[va] = ra[j];
        row[vb] = rb[j];
      }
    }
}

// Heads one thread takes.  More heads share one token's angles (about as much
// work as three heads), fewer give more threads.  Measured on a B200 (us, 1 / 2 /
// 4 / 8 heads): forward of 4 x 4096 tokens, 16 + 16 heads of 128: 97 / 61 / 48 / 49;
// ragged append of 16686 tokens, 48 rows: 167 / 98 / 72 / 76; 3 x 1021 tokens, 6 + 2
// heads: 10.1 / 8.6 / 8.5 / 9.8; 64 tokens, 48 rows: 4.4 / 4.3 / 4.6 / 7.9.  So one
// where threads are few enough to run at once with a block a scheduler, two up
// to a full machine, else four.
int heads_per_thread(int64_t threads_per_head, int heads) {
  const int64_t threads = threads_per_head * heads;
  const int per = threads <= 148 * 4 * 64 ? 1 : threads <= 148 * 1024 / 2 ? 2 : kMaxHeads;
  return per < heads ? per : heads;
}

}  // namespace

ta_status launch_rope(const void* x, void* y, const int32_t* positions, const double* inv_freq, int B, int H, int N,
                      int d, int rotary_dim, int interleaved, int inverse, float amplitude, const int64_t* x_strides,
                      const int64_t* y_strides, int64_t pos_stride, cudaStream_t stream) {
  RopeArgs a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.xb = x_strides[0];
  a.xh = x_strides[1];
  a.xn = x_strides[2];
  a.yb = y_strides[0];
  a.yh = y_strides[1];
  a.yn = y_strides[2];
  a.pb = pos_stride;
  a.tokens = static_cast<int64_t>(B) * N;
  a.N = N;
  a.H = H;
  a.rotary_dim = rotary_dim;
  a.amp = amplitude;
  a.sign = inverse ? -1.f : 1.f;
  const int units = d / 16, per_block = kRopeThreads / units;
  a.heads = heads_per_thread(a.tokens * units, H);
  const dim3 grid(static_cast<unsigned>((a.tokens + per_block - 1) / per_block),
                  static_cast<unsigned>((H + a.heads - 1) / a.heads));
  if (d == 128) {
    if (interleaved) rope_kernel<128, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else rope_kernel<128, false><<<grid, kRopeThreads, 0, stream>>>(a);
  } else {
    if (interleaved) rope_kernel<64, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else rope_kernel<64, false><<<grid, kRopeThreads, 0, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "attn_rope: launch", e);
}

ta_status launch_paged_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                              const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* seq_lens,
                              const int32_t* positions, const double* inv_freq, int page_size, int num_seqs,
                              int total, int Hq, int Hkv, int d, int max_pages, int num_pages_total, int rotary_dim,
                              int interleaved, float amplitude, const int64_t* strides, cudaStream_t stream) {
  AppendArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.block_table = block_table;
  a.cu_seqlens = cu_seqlens;
  a.seq_lens = seq_lens;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.qt = strides[0];
  a.qh = strides[1];
  a.kt = strides[2];
  a.kh = strides[3];
  a.vt = strides[4];
  a.vh = strides[5];
  a.page_size = page_size;
  a.num_seqs = num_seqs;
  a.total = total;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.max_pages = max_pages;
  a.num_pages_total = num_pages_total;
  a.rotary_dim = rotary_dim;
  a.amp = amplitude;
  a.status = device_status_ptr();
  if (!a.status) return fail(TA_ERR_CUDA, "attn_paged_append: device status word");
  const int units = d / 16, per_block = kRopeThreads / units;
  const int rows = (q ? Hq : 0) + 2 * Hkv;
  a.heads = heads_per_thread(static_cast<int64_t>(total) * units, rows);
  a.token_blocks = (total + per_block - 1) / per_block;
  int seq_blocks = 0;
  if (cu_seqlens) {   // with one token each the tokens are the sequences
    seq_blocks = (num_seqs - 1) / kRopeThreads + 1;
    if (seq_blocks > 148) seq_blocks = 148;
  }
  const dim3 grid(static_cast<unsigned>(a.token_blocks + seq_blocks), static_cast<unsigned>((rows + a.heads - 1) / a.heads));
  if (d == 128) {
    if (interleaved) paged_append_kernel<128, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else paged_append_kernel<128, false><<<grid, kRopeThreads, 0, stream>>>(a);
  } else {
    if (interleaved) paged_append_kernel<64, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else paged_append_kernel<64, false><<<grid, kRopeThreads, 0, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TA_OK : fail(TA_ERR_CUDA, "attn_paged_append: launch", e);
}

}  // namespace ta
