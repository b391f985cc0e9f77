// Attention of a chunk of new tokens over a paged cache, on the tensor cores
// (sm_100a): head sizes to 64 (D = 64) and to 128 (D = 128; columns behind d
// are zeros that the copy engine fills in), up to 128 query heads per KV head.
//
// For the new token i of sequence b and query head h of KV head g:
//     s_j = scale q_i . k_j for the visible keys j <= L - T + i (and, with a
//     window, j > L - T + i - window);  o = sum_j softmax_j(s) v_j;
//     lse = ln sum_j exp(s_j);  no visible key: o = 0, lse = -inf.
//
// Query rows of a KV head are (token, head of the group) pairs, token by
// token, so that the whole group shares each key tile read: a tile of 128 rows
// holds tt = 128 / G tokens. A work item is a pair of such tiles of one
// sequence and KV head; its steps are the tiles of 128 keys that any of its
// rows sees. Every CTA (one per SM) gets the same number w of steps, so that a
// chunk over a long cache fills the GPU however few rows it has and a mixed
// batch is balanced. The steps are dealt out in one of two ways:
//   - in order (sequence, KV head, tile pair, key tile), in contiguous ranges;
//   - when the batch's keys and values exceed what L2 can hold, an item of
//     n >= w steps first gives floor(n / w) chunks of w, a CTA each, and only
//     the rests go in contiguous ranges to the CTAs left. The pairs of a head
//     then run over the same keys at the same time, and all but the first find
//     them in L2. (1024 tokens over 64K, 32/8 heads: in contiguous ranges each
//     CTA was at another key, 3.9 GB came from DRAM where q, k and v have 0.28.)
// For the same reason a CTA that has done s steps begins a whole item of n at
// its key tile s mod n and wraps around: CTAs that work on one head stay
// together although they began their items at different times.
// A piece that is not a whole item leaves a normalised fp32 partial with its
// log-sum-exp, and the gather kernel folds the partials of an item together in
// the order of its keys.
//
// Two or three kernels per call:
//   attn_paged_plan_kernel    (batches above kInlineB sequences) one CTA: the
//                             steps, w, and where each CTA begins
//   attn_paged_kernel         the stream (below); for smaller batches each CTA
//                             works out the plan, and its own start, itself
//   attn_paged_gather_kernel  the cut items
//
// The stream has the warp roles of the prefill kernel: warps 0-3 and 4-7 are
// softmax groups 0 and 1 (one thread per row), warp 8 owns tensor memory and
// issues the products, warp 9 loads: Q by one copy per 64 columns (rows
// gathered over tokens and heads by the tensor map), K and V page by page, one
// lane per page and 64 columns, through a ring of tiles; a tile's pages land in
// the 128-byte-swizzled layout as if they were contiguous. Pages that the
// sequence does not have (behind its last, or an id outside the pool) are
// loaded at an out-of-range coordinate, which fills zeros and reads nothing.
//   Two tiles of rows (pair): both groups work on every key tile, S_t = Q_t K^T
// and O_t += P_t V, as in the prefill kernel.
//   With D = 64 tensor memory has room for P beside S: S_t is released as soon
// as it has been read, so the next scores run during the exponentials (s_free),
// and P_t waits for the previous product instead (pv_done). With D = 128 P
// overwrites S.
//   One tile of rows (a single token, or a short chunk): the groups share Q_0
// and take the key tiles in turns, each with its own running maximum, sum and
// O; group 0 folds O_1 into O_0 at the end of the piece. One group's
// exponentials then overlap the other's products and loads.
//
// Bound by the tensor cores and the exponential unit together, like the
// prefill kernel (a pair's step of 2 x 128 x 128 scores takes 3,500 cycles at d
// = 128 where either needs 2,048; 3,000 at d = 64), and at its ends by the
// chain of loads of a start (about 4 us) and the gather (4 us). Measured on
// B200: 1024 tokens over 64K, 32/8 heads, d = 128 0.88-0.89 ms once, 1.00-1.04
// ms in a row under the power limit (1.06 PFLOP/s, 0.76 of the measured
// sustained rate); 9 sequences of up to 301 tokens under a window of 4096, 16/2
// heads, d = 64 55 us.
//
// Scores, maxima, sums and outputs are held in 32 bits. Probabilities are rounded
// to the input's type for the value product, whose operands have 16 bits; the sum
// takes them unrounded. That puts o up to half a step times sum p |v| off, as much
// as the rounding of o itself (bf16, root mean square over all of o: 2.3e-3 of its
// size, where rounding o alone would give 1.7e-3).
//
// Rows of V behind the sequence's last key, and under a window those in front
// of the first key that any row of the item sees, are set to zero in shared
// memory before the product: their probabilities are zero, but what lies there
// in the pool may be infinite or NaN. Pages wholly in front of that key are not
// looked up (the cache may have given them up).
#pragma once

#include "paged_common.cuh"
#include "prefill_sm100.cuh"

namespace eta {
namespace paged {

constexpr int BM = 128;  // query rows per tile
constexpr int BN = 128;  // keys per tile
constexpr int NQT = 2;
constexpr int kThreads = 320;
constexpr int kMmaWarp = 8;
constexpr int kTmaWarp = 9;
constexpr int kPlanThreads = 1024;
constexpr int kSlotRows = NQT * BM;
constexpr int kInlineB = 2048;  // batches up to this many sequences plan in the stream kernel

// Wait sites reported in the status word.
enum : unsigned {
  kSiteQFull = 0x81,
  kSiteKvEmpty = 0x82,
  kSiteKvFull = 0x83,
  kSitePReady = 0x84,
  kSiteSReady = 0x85,
  kSiteODone = 0x86,
  kSiteDrain = 0x87,
  kSiteQEmpty = 0x88,
  kSiteXUp = 0x89,
  kSiteXDown = 0x8a,
  kSiteSFree = 0x8b,
  kSitePvDone = 0x8c,
};

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 128, "head size");
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = 128 * 128;  // 128 rows of 64 columns
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kKVOff = NQT * kTileBytes;
  // The inline plan's prefix sums (8 and 4 bytes a sequence), and once it is made
  // what the warps of group 1 hand over of their rows: (m, l), 256 bytes a warp.
  static constexpr int kScratchOff = kKVOff + kStages * kTileBytes;
  static constexpr int kScratchBytes = ((kInlineB + 1) * 12 + 15) / 16 * 16;
  static_assert(kScratchBytes >= 4 * 256, "exchange");
  static constexpr int kBarOff = kScratchOff + kScratchBytes;
  // kv_full[S], kv_empty[S], q_full[2], q_empty[2], s_ready[2], p_ready[2],
  // o_done[2], s_free[2], pv_done[2], x_up, x_down, drain
  static constexpr int kNumBars = 2 * kStages + 7 * NQT + 3;
  static constexpr int kCtlOff = kBarOff + kNumBars * 8;
  static constexpr int kWalkOff = kCtlOff + 64;  // each warp's way through the range
  static constexpr int kSmemBytes = kWalkOff + 10 * 104 + 1024;  // + runtime 1024-byte alignment
  static constexpr uint32_t kTmemCols = 512;
  static constexpr bool kOwnP = D == 64;  // P in columns of its own, else over S from column 64 on
  __host__ __device__ static constexpr uint32_t s_col(int t) { return kOwnP ? 256u * t : BN * t; }
  __host__ __device__ static constexpr uint32_t p_col(int t) {
    return kOwnP ? 256u * t + BN : BN * t + 64u;
  }
  __host__ __device__ static constexpr uint32_t o_col(int t) {
    return kOwnP ? 256u * t + BN + 64u : 2 * BN + D * t;
  }
  static_assert(kSmemBytes <= 232448, "shared memory");
};

// Where a CTA begins.
struct alignas(16) Start {
  int b, g, pair;
  int i;           // step of the item
  int chunk;       // the first chunk CTA of the item, or of the next that has one
  int pad;
  long long rest;  // positions of the rests before the item's
};

// The plan, in device memory.
struct Head {
  long long rest;   // positions of all rests
  int w;            // cost of a chunk, positions of a CTA that takes rests
  int chunks;       // CTAs that take a chunk: 0 .. chunks - 1; the rests follow
  int ctas;         // CTAs with work
};
struct Plan {
  Head* head;
  Start* starts;       // [nc]
  long long* rest_at;  // [B + 1] (plan kernel): rests before each sequence
  int* chunk_at;       // [B + 1] (plan kernel): chunks before each sequence
};

struct Params {
  const int* cu_q;
  const int* lens;
  const int* table;
  void* o;
  float* lse;
  float* part_o;    // [3 nc] slots of 256 rows: [row / 32][column / 4][row % 32][4]
  float* part_lse;  // [3 nc][256], log2 units
  Plan plan;
  int B, Hq, Hkv, G, tt;
  int total_q, max_q, d;
  int num_pages, page_log2, width;
  int window;
  int nc;
  int inline_plan;  // no plan kernel
  int warp_plan;    // up to 32 sequences, steps in 32 bits: a warp can make the plan
  int max_pairs;    // tile pairs that a sequence of max_q tokens has
  long long l2_bytes;
  float scale_log2;
  uint64_t wait_ns;

  __device__ __forceinline__ long long capacity() const {
    return static_cast<long long>(width) << page_log2;
  }
};

// The key tiles [lo, lo + n) that any row of tile pair `pair` sees; at least
// one, so that a pair of rows without keys goes the same way (all masked).
struct Span {
  int lo, n;
};
__device__ __forceinline__ Span span_of(const Params& p, const Seq& s, int pair) {
  const int t0 = pair * NQT * p.tt, t1 = min(s.T, t0 + NQT * p.tt);
  const int last = s.L - s.T + t1 - 1;
  Span r;
  r.lo = first_seen(s, t0, p.window) / BN;
  r.n = last < 0 ? 1 : max(1, last / BN + 1 - r.lo);
  if (last < 0) r.lo = 0;
  return r;
}
__device__ __forceinline__ int pairs_of(const Params& p, int T) {
  return (T + NQT * p.tt - 1) / (NQT * p.tt);
}

// n / d for 0 <= n, 0 < d, in 32 bits when both fit (the usual case).
__device__ __forceinline__ long long div_pos(long long n, long long d) {
  if (((n | d) >> 31) == 0)
    return static_cast<long long>(static_cast<unsigned>(n) / static_cast<unsigned>(d));
  return n / d;
}

// Costs are counted in thirds of a pair's step. A step with one tile of rows
// takes two of them (measured at d = 128: 3,550 cycles against 2,350, which is
// what its keys and values take to arrive; at d = 64, counted as two / as three:
// 48 mixed sequences of 1-64 tokens 122 / 136 us, tiles of 70-90 tokens of group 4
// 149 / 158, chunks of 128-512 168 / 172, prompts of 2K 89.3 / 88.6).
constexpr int kPairCost = 3, kSingleCost = 2;
__device__ __forceinline__ int step_cost(const Params& p, int T, int pair) {
  return pair * NQT * p.tt + p.tt < T ? kPairCost : kSingleCost;
}

// What beginning an item costs a CTA: loading its queries, and its end (the
// last product, the output). Measured with none / one / two / three / four
// steps on B200: 16 chunks of 128-512 tokens over 600-4000 275 / 251 / 242 /
// 237 / 224 us, 8K tokens 591 / 556 / 515 / 515 / 529, the mixed batch of 9
// 58.6 / 55.2 / 55.4 / 56.1 / 56.5.
#ifndef ETA_PAGED_ITEM_COST
#define ETA_PAGED_ITEM_COST 2
#endif
constexpr int kItemCost = ETA_PAGED_ITEM_COST * kPairCost;
// A range of less is not worth a CTA of its own. (It also holds a step's
// beginning wherever it lies.)
constexpr int kMinCost = 2 * kPairCost + kItemCost;

// Steps of a chunk, and chunks of an item of n steps (0: all of it goes to the rests).
__device__ __forceinline__ int chunk_steps(int w, int g) { return (w + g - 1) / g; }
__device__ __forceinline__ int chunks_of(int n, int wc, bool chunked) {
  return chunked && n >= wc ? static_cast<int>(static_cast<unsigned>(n) / static_cast<unsigned>(wc)) : 0;
}

// Positions of an item's rest of r steps: what its beginning costs, then the
// steps. A CTA takes the steps that begin in its range.
__device__ __forceinline__ int rest_cost(int r, int g) { return r > 0 ? r * g + kItemCost : 0; }

// Sums over a block of (a, b), which every thread gets; `red` holds 2 THREADS / 32 words.
template <int THREADS>
__device__ __forceinline__ void block_sum(long long& a, long long& b, long long* red) {
  constexpr int W = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();  // red's last use
  if (lane == 0) {
    red[2 * warp] = a;
    red[2 * warp + 1] = b;
  }
  __syncthreads();
  a = b = 0;
#pragma unroll 4
  for (int w = 0; w < W; ++w) {
    a += red[2 * w];
    b += red[2 * w + 1];
  }
}

// The plan, by a whole block of THREADS: its head, and the chunks and rests
// before each sequence (rest_at, chunk_at [B + 1]).
template <int THREADS>
__device__ __forceinline__ Head make_plan(const Params& p, long long* rest_at, int* chunk_at,
                                          long long* red, bool check) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // A thread per sequence; a warp per sequence where they have many tile pairs.
  const bool wide = p.max_pairs > 32;
  const int b_first = wide ? warp : tid, b_step = wide ? W : THREADS;
  const int i_first = wide ? lane : 0, i_step = wide ? 32 : 1;
  long long steps = 0, keys = 0;
  for (int b = b_first; b < p.B; b += b_step) {
    const Seq s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    const int n = pairs_of(p, s.T);
    for (int i = i_first; i < n; i += i_step)
      steps += rest_cost(span_of(p, s, i).n, step_cost(p, s.T, i));
    if (i_first == 0) {
      keys += s.T > 0 ? s.L : 0;
      if (check) check_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    }
  }
  block_sum<THREADS>(steps, keys, red);
  Head h;
  steps *= p.Hkv;
  const long long want = div_pos(steps, kMinCost);
  const int busy = static_cast<int>(want < p.nc ? (want > 0 ? want : 1) : p.nc);
  h.w = static_cast<int>(max(div_pos(steps + busy - 1, busy), 1LL));
  // Keys and values beyond half of L2 will not stay in it between two CTAs
  // that come by at different times (1024 tokens over 64K, 268 MB: 877 us with
  // chunks, 1020 us without; over 20K, 82 MB: 291 / 300 us; below, 49 MB, the
  // two differ by less than runs do. At d = 64, over 64K, 134 MB: 719 / 705 us;
  // over 40K, 82 MB, 453 / 453; over 24K, 49 MB, 273 / 276).
  const bool chunked = keys * p.Hkv * p.d * 4 > p.l2_bytes / 2;
  for (int b = b_first; b < p.B; b += b_step) {
    const Seq s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    const int n = pairs_of(p, s.T);
    long long rest = 0;
    int chunks = 0;
    for (int i = i_first; i < n; i += i_step) {
      const int k = span_of(p, s, i).n, g = step_cost(p, s.T, i), wc = chunk_steps(h.w, g);
      const int f = chunks_of(k, wc, chunked);
      chunks += f;
      rest += rest_cost(k - f * wc, g);
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        rest += __shfl_xor_sync(0xffffffffu, rest, o);
        chunks += __shfl_xor_sync(0xffffffffu, chunks, o);
      }
    }
    if (i_first == 0) {
      rest_at[b] = rest * p.Hkv;
      chunk_at[b] = chunks * p.Hkv;
    }
  }
  __syncthreads();
  // Exclusive prefix over the sequences, in place.
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long rest = 0, chunks = 0;
  for (int b = b0; b < b1; ++b) {
    rest += rest_at[b];
    chunks += chunk_at[b];
  }
  long long x = rest, y = chunks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x2 = __shfl_up_sync(0xffffffffu, x, o);
    const long long y2 = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += x2;
      y += y2;
    }
  }
  if (lane == 31) {
    red[2 * warp] = x;
    red[2 * warp + 1] = y;
  }
  __syncthreads();
  long long xb = 0, yb = 0, xa = 0, ya = 0;
#pragma unroll 4
  for (int w = 0; w < W; ++w) {
    const long long u = red[2 * w], v = red[2 * w + 1];
    if (w < warp) {
      xb += u;
      yb += v;
    }
    xa += u;
    ya += v;
  }
  x += xb - rest;
  y += yb - chunks;
  for (int b = b0; b < b1; ++b) {
    const long long r = rest_at[b];
    const int k = chunk_at[b];
    rest_at[b] = x;
    chunk_at[b] = static_cast<int>(y);
    x += r;
    y += k;
  }
  if (tid == 0) {
    rest_at[p.B] = xa;
    chunk_at[p.B] = static_cast<int>(ya);
  }
  h.rest = xa;
  h.chunks = static_cast<int>(ya);
  h.ctas = h.chunks + static_cast<int>(div_pos(xa + h.w - 1, h.w));
  __syncthreads();
  return h;
}

// Where CTA c (of those with work) begins, by a whole warp.
__device__ __forceinline__ Start plan_find(const Params& p, const Head& h, const long long* rest_at,
                                           const int* chunk_at, int c, int lane) {
  const bool chunked = h.chunks > 0, mine = c < h.chunks;
  const long long at = mine ? c : static_cast<long long>(c - h.chunks) * h.w;  // among the chunks, or the rests
  int lo = 0, hi = p.B - 1;  // the last sequence that begins at or before `at`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((mine ? chunk_at[mid] : rest_at[mid]) <= at)
      lo = mid;
    else
      hi = mid - 1;
  }
  const Seq s = load_seq(p.cu_q, p.lens, lo, p.total_q, p.max_q, p.capacity());
  const long long rest_head = div_pos(rest_at[lo + 1] - rest_at[lo], p.Hkv);
  const int chunk_head = (chunk_at[lo + 1] - chunk_at[lo]) / p.Hkv;
  long long r = mine ? c - chunk_at[lo] : at - rest_at[lo];
  const long long per_head = mine ? chunk_head : rest_head;
  Start st;
  st.b = lo;
  st.g = static_cast<int>(div_pos(r, per_head));
  st.pad = 0;
  r -= st.g * per_head;
  st.rest = rest_at[lo] + st.g * rest_head;
  st.chunk = chunk_at[lo] + st.g * chunk_head;
  st.pair = 0;
  st.i = 0;
  const int n = pairs_of(p, s.T);
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int k = i0 + lane < n ? span_of(p, s, i0 + lane).n : 0;
    const int g = step_cost(p, s.T, i0 + lane), wc = chunk_steps(h.w, g);
    const int f = chunks_of(k, wc, chunked);
    const int rr = rest_cost(k - f * wc, g);  // (32 spans stay below 2^31)
    int x = rr, y = f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x2 = __shfl_up_sync(0xffffffffu, x, o);
      const int y2 = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += x2;
        y += y2;
      }
    }
    const unsigned over = __ballot_sync(0xffffffffu, r < (mine ? y : x));
    if (over != 0) {
      const int l = __ffs(over) - 1;
      st.pair = i0 + l;
      st.rest += __shfl_sync(0xffffffffu, x - rr, l);
      st.chunk += __shfl_sync(0xffffffffu, y - f, l);
      const int before = __shfl_sync(0xffffffffu, mine ? y - f : x - rr, l);
      // (a rest: the walk finds the step from the range's position)
      st.i = mine ? static_cast<int>(r - before) * __shfl_sync(0xffffffffu, wc, l) : 0;
      break;
    }
    r -= __shfl_sync(0xffffffffu, mine ? y : x, 31);
    st.rest += __shfl_sync(0xffffffffu, x, 31);
    st.chunk += __shfl_sync(0xffffffffu, y, 31);
  }
  return st;
}

// The same for up to 32 sequences whose steps count in 32 bits and go in
// contiguous ranges, by one warp for itself: a lane per sequence, no barriers,
// little code (a kernel's start runs on cold instruction and data caches: with
// the block's plan a stream began its loads 10,000 cycles after its start, with
// this one 5,000). False: the block has to make the plan.
__device__ __forceinline__ bool plan_warp(const Params& p, int c, int lane, Head& h, Start& st) {
  Seq s{0, 0, 0};
  if (lane < p.B) s = load_seq(p.cu_q, p.lens, lane, p.total_q, p.max_q, p.capacity());
  const int n = pairs_of(p, s.T);
  int mine = 0, longest = 0;
  float keys = s.T > 0 ? static_cast<float>(s.L) : 0.f;
  if (p.max_pairs <= 32) {
    for (int i = 0; i < n; ++i) {
      const int k = span_of(p, s, i).n;
      mine += rest_cost(k, step_cost(p, s.T, i));
      longest = max(longest, k);
    }
  } else {
    for (int b = 0; b < p.B; ++b) {  // long chunks: the lanes share a sequence's pairs
      const Seq t{0, __shfl_sync(0xffffffffu, s.T, b), __shfl_sync(0xffffffffu, s.L, b)};
      const int m = pairs_of(p, t.T);
      int sum = 0;
      for (int i = lane; i < m; i += 32) {
        const int k = span_of(p, t, i).n;
        sum += rest_cost(k, step_cost(p, t.T, i));
        longest = max(longest, k);
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == b) mine = sum;
    }
  }
  mine *= p.Hkv;
  int x = mine;  // inclusive prefix
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    keys += __shfl_xor_sync(0xffffffffu, keys, o);
    if (lane >= o) x += y;
  }
  const unsigned steps = __shfl_sync(0xffffffffu, x, 31);
  const unsigned busy = min(max(steps / kMinCost, 1u), static_cast<unsigned>(p.nc));
  const unsigned w = max((steps + busy - 1) / busy, 1u);
  if (keys * p.Hkv * p.d * 4.f > static_cast<float>(p.l2_bytes / 2) &&
      __reduce_max_sync(0xffffffffu, longest) >= chunk_steps(w, kPairCost))
    return false;  // there are chunks
  h.rest = steps;
  h.w = static_cast<int>(w);
  h.chunks = 0;
  h.ctas = static_cast<int>((steps + w - 1) / w);
  if (c >= h.ctas) return true;
  const int at = c * static_cast<int>(w);
  const int b = __ffs(__ballot_sync(0xffffffffu, x > at)) - 1;
  const Seq t{0, __shfl_sync(0xffffffffu, s.T, b), __shfl_sync(0xffffffffu, s.L, b)};
  const unsigned per_head = static_cast<unsigned>(__shfl_sync(0xffffffffu, mine, b)) / p.Hkv;
  unsigned r = at - __shfl_sync(0xffffffffu, x - mine, b);
  st.b = b;
  st.g = static_cast<int>(r / per_head);
  r -= st.g * per_head;
  st.rest = at - static_cast<int>(r);
  st.chunk = 0;
  st.pad = 0;
  st.pair = st.i = 0;
  const int m = pairs_of(p, t.T);
  for (int i0 = 0; i0 < m; i0 += 32) {
    const int k = i0 + lane < m
                      ? rest_cost(span_of(p, t, i0 + lane).n, step_cost(p, t.T, i0 + lane)) : 0;
    int y = k;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    const unsigned over = __ballot_sync(0xffffffffu, static_cast<int>(r) < y);
    if (over != 0) {
      const int l = __ffs(over) - 1, before = __shfl_sync(0xffffffffu, y - k, l);
      st.pair = i0 + l;
      st.rest += before;
      break;
    }
    const int all = __shfl_sync(0xffffffffu, y, 31);
    r -= all;
    st.rest += all;
  }
  return true;
}

__global__ void __launch_bounds__(kPlanThreads) attn_paged_plan_kernel(const Params p) {
  __shared__ long long red[2 * kPlanThreads / 32];
  grid_launch_dependents();
  const Head h = make_plan<kPlanThreads>(p, p.plan.rest_at, p.plan.chunk_at, red, true);
  if (threadIdx.x == 0) *p.plan.head = h;
  for (int c = threadIdx.x >> 5; c < h.ctas; c += kPlanThreads / 32) {
    const Start st = plan_find(p, h, p.plan.rest_at, p.plan.chunk_at, c, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) p.plan.starts[c] = st;
  }
}

// A CTA's way through its range, piece by piece. Every warp keeps its own, in
// shared memory (in registers it would push the softmax's scores out): lane 0
// moves it on, the others read it.
struct Walk {
  int b, head, pair;
  int i0, i1, n;   // steps [i0, i1) of the item's n
  int first;       // the item's first step outside its chunks
  int lo;          // its first key tile
  int rot;         // the piece begins at its step rot and wraps around
  int chunk;       // the item's first chunk CTA (if it has chunks)
  int more;        // this is a piece (0: the range has ended)
  int w;           // cost of a chunk (0: no item has any)
  int wc;          // and its steps
  int g;           // cost of a step
  int left;        // positions of the range behind this piece
  int done;        // steps up to its end
  int chunks;      // CTAs that take a chunk
  // Softmax warps: phases of their piece-wise barriers used so far.
  uint32_t od0, od1, xp;
  Seq s;

  __device__ __forceinline__ void item(const Params& p) {
    const Span sp = span_of(p, s, pair);
    lo = sp.lo;
    n = sp.n;
    g = step_cost(p, s.T, pair);
    wc = chunk_steps(w, g);
    first = w > 0 ? chunks_of(n, wc, true) * wc : 0;
  }
  // The item's rest from its position r on: true if a step begins in the range.
  __device__ __forceinline__ bool piece(int r) {
    const int all = rest_cost(n - first, g), end = min(all, r + left);
    left -= all - r;
    i0 = first + (max(r - kItemCost, 0) + g - 1) / g;
    i1 = first + (max(end - kItemCost, 0) + g - 1) / g;
    if (i1 <= i0) return false;
    rot = i0 == first && i1 == n ? done % (n - first) : 0;
    done += i1 - i0;
    return true;
  }
  __device__ __forceinline__ void start(const Params& p, const Head& h, const Start& st, int c) {
    b = st.b, head = st.g, pair = st.pair, chunk = st.chunk;
    chunks = h.chunks;
    w = h.chunks > 0 ? h.w : 0;
    done = 0;
    od0 = od1 = xp = 0;
    more = 1;
    s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    item(p);
    if (c < h.chunks) {
      i0 = st.i;
      i1 = i0 + wc;
      rot = left = 0;
      return;
    }
    const long long at = static_cast<long long>(c - h.chunks) * h.w, behind = h.rest - at;
    left = behind < h.w ? static_cast<int>(behind) : h.w;
    if (!piece(static_cast<int>(at - st.rest))) next(p);
  }
  __device__ __forceinline__ void next(const Params& p) {
    do {
      more = 0;
      if (left <= 0) return;
      if (w > 0) chunk += first / wc;
      if (++pair >= pairs_of(p, s.T)) {
        pair = 0;
        if (++head >= p.Hkv) {
          head = 0;
          do {
            if (++b >= p.B) return;  // (the plan's range ends before this)
            s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
          } while (s.T == 0);
        }
      }
      item(p);
      more = 1;
    } while (!piece(0));
  }
  __device__ __forceinline__ int steps() const { return i1 - i0; }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == n; }
  // The slot of a piece that is not the whole item, in CTA c of nc: a chunk or
  // what goes on from the CTA before, what goes on in the next, all of a rest.
  __device__ __forceinline__ int slot(int c, int nc) const {
    return c < chunks || i0 != first ? c : i1 < n ? nc + c : 2 * nc + chunk;
  }
  // The first key that any row of the item sees.
  __device__ __forceinline__ int seen_from(const Params& p) const {
    return first_seen(s, pair * NQT * p.tt, p.window);
  }
  // Both tiles have rows?
  __device__ __forceinline__ bool two(const Params& p) const {
    return pair * NQT * p.tt + p.tt < s.T;
  }
};
static_assert(sizeof(Walk) <= 104, "shared memory of a warp's walk");

// The warp's walk to its next piece; false at the end of the range.
__device__ __forceinline__ bool walk_on(Walk& w, const Params& p, int lane) {
  __syncwarp();  // every lane is done with this piece
  if (lane == 0) w.next(p);
  __syncwarp();
  return w.more != 0;
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<D>;
  using prefill::warp_all;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::kKVOff;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* kv_empty = kv_full + S;
  uint64_t* q_full = kv_empty + S;
  uint64_t* q_empty = q_full + NQT;
  uint64_t* s_ready = q_empty + NQT;
  uint64_t* p_ready = s_ready + NQT;
  uint64_t* o_done = p_ready + NQT;
  uint64_t* s_free = o_done + NQT;   // S_t has been read (own P)
  uint64_t* pv_done = s_free + NQT;  // P_t V is complete (own P)
  uint64_t* x_up = pv_done + NQT;
  uint64_t* x_down = x_up + 1;
  uint64_t* drain = x_down + 1;
  CtaCtl* ctl = reinterpret_cast<CtaCtl*>(smem + C::kCtlOff);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kCtlOff + 32);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < NQT; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_ready[t], 1);
      mbar_init(&p_ready[t], BM);
      mbar_init(&o_done[t], 1);
      mbar_init(&s_free[t], BM);
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(x_up, BM);
    mbar_init(x_down, BM);
    mbar_init(drain, 1);
    ctl->abort = 0;
    ctl->wait_ns = p.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  grid_wait();  // the plan's writes (and the caller's before it) are visible
  grid_launch_dependents();
  Walk& w = *reinterpret_cast<Walk*>(smem + C::kWalkOff + warp * 104);
  bool work;
  Head h;
  Start st;
  if (p.warp_plan && plan_warp(p, c, lane, h, st)) {  // (the same answer in every warp)
    work = c < h.ctas;
    if (work) {
      if (lane == 0) w.start(p, h, st, c);
      __syncwarp();
      work = w.more != 0;  // (a short last range may hold no step's beginning)
      if (threadIdx.x == 0) p.plan.starts[c] = st;  // for the gather, as is the head
    }
    if (c == 0 && warp == 0) {
      if (lane == 0) *p.plan.head = h;
      if (lane < p.B) check_seq(p.cu_q, p.lens, lane, p.total_q, p.max_q, p.capacity());
    }
  } else if (p.inline_plan) {
    long long* rest_at = reinterpret_cast<long long*>(smem + C::kScratchOff);
    int* chunk_at = reinterpret_cast<int*>(rest_at + p.B + 1);
    h = make_plan<kThreads>(p, rest_at, chunk_at,
                                       reinterpret_cast<long long*>(smem + C::kWalkOff), c == 0);
    work = c < h.ctas;
    if (work) {
      st = plan_find(p, h, rest_at, chunk_at, c, lane);  // (every warp for itself)
      if (lane == 0) w.start(p, h, st, c);
      __syncwarp();
      work = w.more != 0;
      if (threadIdx.x == 0) p.plan.starts[c] = st;  // for the gather, as is the head
    }
    if (c == 0 && threadIdx.x == 0) *p.plan.head = h;
    __syncthreads();  // the scratch is free for the exchange of the softmax warps
  } else {
    h = *p.plan.head;
    work = c < h.ctas;
    if (work) {
      if (lane == 0) w.start(p, h, p.plan.starts[c], c);
      __syncwarp();
      work = w.more != 0;
    }
  }

  if (!work) {
    // nothing for this CTA (uniform over it)
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    // Lane l loads page l / kBoxes of a key tile, columns 64 (l % kBoxes) on.
    const int box_rows = min(1 << p.page_log2, BN);
    const int n_pages = BN / box_rows;  // pages (or parts of one) in a key tile
    const int pg = lane / C::kBoxes, bx = lane % C::kBoxes;
    const bool loads = lane < n_pages * C::kBoxes;
    const uint32_t dst_off = bx * C::kBoxBytes + pg * box_rows * 128;
    const uint32_t q_bytes = static_cast<uint32_t>(C::kBoxes * p.tt * p.G * 128);
    uint32_t L = 0;        // K/V tiles issued so far (K_j, V_j alternate)
    int qn[NQT] = {0, 0};  // Q loads issued so far, per tile
    bool ok = true;
    do {
      const int tiles = w.two(p) ? 2 : 1;
#pragma unroll
      for (int t = 0; t < NQT; ++t) {
        if (t >= tiles) break;
        if (qn[t] > 0 && !(ok = warp_all(wait_bar(&q_empty[t], (qn[t] - 1) & 1, ctl, kSiteQEmpty))))
          break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[t], q_bytes);
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(sQ + t * C::kTileBytes + x * C::kBoxBytes, &tm_q, &q_full[t], x * 64, 0,
                        w.head, w.s.q0 + (w.pair * NQT + t) * p.tt);
        }
        ++qn[t];
      }
      // The page that this lane loads of key tile j: its id, or num_pages
      // (out of range: zeros) where the sequence has none or no row sees any of it.
      const int* row = p.table + static_cast<size_t>(w.b) * p.width;
      const int keys = w.s.L, seen = w.seen_from(p), g = w.head, n = w.steps();
      const int j0 = w.lo + w.i0;
      int at = w.rot;  // step of the piece
      auto page_of = [&](int j) {
        const int key = j * BN + pg * box_rows;
        if (!loads || key >= keys || key + box_rows <= seen) return p.num_pages;
        const int id = row[key >> p.page_log2];
        if (id >= 0 && id < p.num_pages) return id;
        bad(kBadPage);
        return p.num_pages;
      };
      int page = page_of(j0 + at);
      for (int j = 0; ok && j < n; ++j) {
        const int y = ((j0 + at) * BN + pg * box_rows) & ((1 << p.page_log2) - 1);
        const int now = page;
        if (++at == n) at = 0;
        if (j + 1 < n) page = page_of(j0 + at);  // ahead of its use
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++L) {
          const uint32_t s = L % S, use = L / S;
          if (use > 0 &&
              !(ok = warp_all(wait_bar(&kv_empty[s], (use - 1) & 1, ctl, kSiteKvEmpty))))
            break;
          if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], C::kTileBytes);
          __syncwarp();
          if (loads)
            tma_load_4d(sKV + s * C::kTileBytes + dst_off, kv ? &tm_v : &tm_k, &kv_full[s], bx * 64,
                        y, g, now);
        }
      }
    } while (ok && walk_on(w, p, lane));
    // No copy may still be landing in shared memory when the CTA exits.
#pragma unroll
    for (int t = 0; t < NQT; ++t)
      if (qn[t] > 0) drain_bar(&q_full[t], (qn[t] - 1) & 1, ctl, kSiteDrain);
    for (uint32_t s = 0; s < static_cast<uint32_t>(S) && s < L; ++s) {
      const uint32_t cnt = (L - 1 - s) / S + 1;
      drain_bar(&kv_full[s], (cnt - 1) & 1, ctl, kSiteDrain);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t fmt = prefill::Fmt<T>::value;
    constexpr uint32_t idesc_s = umma_idesc_f16(fmt, BM, BN, 0, 0);
    constexpr uint32_t idesc_pv = umma_idesc_f16(fmt, BM, D, 0, 1);
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint32_t d_hi = static_cast<uint32_t>(dq >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(dq);
    const uint32_t k_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sKV), 16, 1024));
    const uint32_t v_lo =
        static_cast<uint32_t>(smem_desc_sw128(smem_u32(sKV), C::kBoxBytes, 1024));
    uint32_t L = 0;            // K/V tiles consumed before this piece
    int qi[NQT] = {0, 0};      // Q tiles used before this piece
    uint32_t pw[NQT] = {0, 0};  // P tiles used
    uint32_t sf[NQT] = {0, 0};  // score products issued (own P)
    bool ok = true;
    // With P in columns of its own, S_t is overwritten when it has been read.
    auto s_is_free = [&](int t) {
      if constexpr (C::kOwnP) {
        if (sf[t] > 0 && !warp_all(wait_bar(&s_free[t], (sf[t] - 1) & 1, ctl, kSiteSFree)))
          return false;
        tc_fence_after();
        ++sf[t];
      }
      return true;
    };
    auto score = [&](int t, int qt, uint32_t lk) {  // S_t = Q_qt K^T
      const uint32_t kd = k_lo + (((lk % S) * C::kTileBytes) >> 4);
      const uint32_t qd = q_lo + ((qt * C::kTileBytes) >> 4);
      const uint32_t tS = tmem + C::s_col(t);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t koff = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
        if (kk == 0)
          umma_ss_w<0>(tS, desc_words(qd + koff, d_hi), desc_words(kd + koff, d_hi), idesc_s);
        else
          umma_ss_w<1>(tS, desc_words(qd + koff, d_hi), desc_words(kd + koff, d_hi), idesc_s);
      }
      umma_commit_w(&s_ready[t]);
    };
    auto value = [&](int t, uint32_t lv, bool first) {  // O_t (+)= P_t V
      const uint32_t vd = v_lo + (((lv % S) * C::kTileBytes) >> 4);
      const uint32_t tP = tmem + C::p_col(t);
      const uint32_t tO = tmem + C::o_col(t);
      if (first)
        umma_ts_w<0>(tO, tP, desc_words(vd, d_hi), idesc_pv);
      else
        umma_ts_w<1>(tO, tP, desc_words(vd, d_hi), idesc_pv);
#pragma unroll
      for (int kk = 1; kk < BN / 16; ++kk)
        umma_ts_w<1>(tO, tP + kk * 8, desc_words(vd + kk * 128, d_hi), idesc_pv);
      if constexpr (C::kOwnP) umma_commit_w(&pv_done[t]);
    };
    // Rows of V behind the sequence's last key and in front of the first one seen:
    // zeros (the other pages there are zeros already; those of the last page, and
    // of the first one needed, may hold anything).
    int tail = 0, rot = 0, n = 0;  // keys of the sequence from the piece's first key tile on
    int front = 0;                 // those of them that no row sees
    const int box_rows = min(1 << p.page_log2, BN);
    auto clear_ends = [&](int j, uint32_t lv) {
      const int t0 = (j + rot < n ? j + rot : j + rot - n) * BN;  // (the piece's key tile)
      const int valid = tail - t0, unseen = front - t0;
      if (valid >= BN && unseen <= 0) return;
      uint8_t* base = sKV + (lv % S) * C::kTileBytes;
      auto clear = [&](int from, int to) {
        for (int i = lane; i < (to - from) * C::kBoxes * 8; i += 32) {
          const int u = i & 7, rb = i >> 3;
          const int r = from + rb / C::kBoxes, x = rb % C::kBoxes;
          *reinterpret_cast<uint4*>(base + x * C::kBoxBytes + r * 128 + u * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if (valid < BN) clear(max(valid, 0), BN);
      if (unseen > 0) clear(unseen & ~(box_rows - 1), unseen);
      fence_proxy_async_smem();
      __syncwarp();
    };
    do {
      n = w.steps();
      rot = w.rot;
      tail = w.s.L - (w.lo + w.i0) * BN;
      front = w.seen_from(p) - (w.lo + w.i0) * BN;
      if (w.two(p)) {
        for (int j = 0; ok && j <= n; ++j) {
          const uint32_t Lk = L + 2 * j, Lv = L + 2 * j - 1;
          auto scores = [&](int t) {
            if (j >= n || !ok) return;
            if (t == 0) {
              if (!(ok = warp_all(wait_bar(&kv_full[Lk % S], (Lk / S) & 1, ctl, kSiteKvFull)))) return;
              tc_fence_after();
            }
            if (j == 0) {
              if (!(ok = warp_all(wait_bar(&q_full[t], qi[t] & 1, ctl, kSiteQFull)))) return;
              tc_fence_after();
            }
            if (!(ok = s_is_free(t))) return;
            score(t, t, Lk);
            if (j == n - 1) umma_commit_w(&q_empty[t]);
            if (t == 1) umma_commit_w(&kv_empty[Lk % S]);
          };
          auto values = [&](int t) {
            if (j < 1 || !ok) return;
            if (t == 0) {
              if (!(ok = warp_all(wait_bar(&kv_full[Lv % S], (Lv / S) & 1, ctl, kSiteKvFull)))) return;
              clear_ends(j - 1, Lv);
            }
            if (!(ok = warp_all(wait_bar(&p_ready[t], pw[t] & 1, ctl, kSitePReady)))) return;
            ++pw[t];
            tc_fence_after();
            value(t, Lv, j == 1);
            if (j == n) umma_commit_w(&o_done[t]);
            if (t == 1) umma_commit_w(&kv_empty[Lv % S]);
          };
          if constexpr (C::kOwnP) {
            scores(0);
            scores(1);
            values(0);
            values(1);
          } else {  // S_t goes over P_t: after the product that reads it
            values(0);
            scores(0);
            values(1);
            scores(1);
          }
        }
        ++qi[0];
        ++qi[1];
      } else {
        // One tile of rows: S of key tile j into buffer j % 2, then P V of
        // tile j - 1. (S of tile j overwrites P of tile j - 2, whose product
        // was issued before it.)
        for (int j = 0; ok && j <= n; ++j) {
          if (j < n) {
            const uint32_t Lk = L + 2 * j;
            if (!(ok = warp_all(wait_bar(&kv_full[Lk % S], (Lk / S) & 1, ctl, kSiteKvFull)))) break;
            if (j == 0 && !(ok = warp_all(wait_bar(&q_full[0], qi[0] & 1, ctl, kSiteQFull)))) break;
            tc_fence_after();
            if (!(ok = s_is_free(j & 1))) break;
            score(j & 1, 0, Lk);
            if (j == n - 1) umma_commit_w(&q_empty[0]);
            umma_commit_w(&kv_empty[Lk % S]);
          }
          if (j >= 1) {
            const int t = (j - 1) & 1;
            const uint32_t Lv = L + 2 * j - 1;
            if (!(ok = warp_all(wait_bar(&kv_full[Lv % S], (Lv / S) & 1, ctl, kSiteKvFull)))) break;
            clear_ends(j - 1, Lv);
            if (!(ok = warp_all(wait_bar(&p_ready[t], pw[t] & 1, ctl, kSitePReady)))) break;
            ++pw[t];
            tc_fence_after();
            value(t, Lv, j - 1 == t);
            if (j + 1 >= n) umma_commit_w(&o_done[t]);  // this group's last step
            umma_commit_w(&kv_empty[Lv % S]);
          }
        }
        ++qi[0];
      }
      L += 2 * n;
    } while (ok && walk_on(w, p, lane));
    // Every MMA must be complete before tensor memory is released.
    umma_commit_w(drain);
    drain_bar(drain, 0, ctl, kSiteDrain);
  } else {
    // ------------------------------------------------------------ softmax
    // What a step needs stays in registers beside its 128 scores; everything
    // of a piece is worked out again from the walk at its end.
    const int t = warp >> 2;
    uint32_t sw = 0;                   // s_ready phases consumed
    [[maybe_unused]] uint32_t np = 0;  // P tiles written (own P)
    bool ok = true;
    do {
      float m = -INFINITY, l = 0.f;
      {
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + C::s_col(t);
        const uint32_t tP = tmem + lane_off + C::p_col(t);
        const uint32_t tO = tmem + lane_off + C::o_col(t);
        const float sl2 = p.scale_log2;
        const bool two = w.two(p);
        const int tok0 = (w.pair * NQT + (two ? t : 0)) * p.tt;  // first token of the group's tile
        const int base = w.s.L - w.s.T + tok0;                   // and its position
        int pos;  // this row's position (-1 where the row is none, or has no keys)
        bool live;
        {
          const int r = (warp & 3) * 32 + lane, tok = tok0 + r / p.G;
          const bool row_ok = r < p.tt * p.G && tok < w.s.T;
          pos = row_ok ? w.s.L - w.s.T + tok : -1;
          live = __any_sync(0xffffffffu, row_ok);
        }
        const int kend = (w.lo + w.i1) * BN, kwrap = w.steps() * BN;
        const int dk = two ? BN : 2 * BN;  // a shared tile's groups take its key tiles in turns
        int kv0 = (w.lo + w.i0 + w.rot) * BN + (two ? 0 : t * BN);
        if (kv0 >= kend) kv0 -= kwrap;
        int left = two ? w.steps() : (w.steps() + 1 - t) >> 1;
        bool first_step = true;
        for (; left > 0; --left, first_step = false) {
          if (!(ok = warp_all(wait_bar(&s_ready[t], sw & 1, ctl, kSiteSReady)))) break;
          ++sw;
          tc_fence_after();
          if (!live) {  // no rows in this warp: its P is never stored
            if constexpr (C::kOwnP) {
              mbar_arrive(&s_free[t]);
              // In step with the warps that have rows: the next scores come before
              // this step's product here, so an arrival for the next step could
              // otherwise stand in for one that this step's P still needs.
              if (np > 0 &&
                  !(ok = warp_all(wait_bar(&pv_done[t], (np - 1) & 1, ctl, kSitePvDone))))
                break;
              ++np;
            }
            mbar_arrive(&p_ready[t]);
            continue;
          }
          float s[BN];
          {
            uint32_t rr[BN / 32][32];
#pragma unroll
            for (int h = 0; h < BN / 32; ++h) tmem_ld_x32(tS + h * 32, rr[h]);
#pragma unroll
            for (int h = 0; h < BN / 32; ++h) tmem_wait_ld_x32(rr[h]);
#pragma unroll
            for (int h = 0; h < BN / 32; ++h)
#pragma unroll
              for (int k = 0; k < 32; ++k) s[h * 32 + k] = __uint_as_float(rr[h][k]);
          }
          if constexpr (C::kOwnP) {  // S_t read: its columns may take the next scores
            tc_fence_before();
            mbar_arrive(&s_free[t]);
          }
          if (kv0 + BN - 1 > base) {  // not every row sees the whole tile
            const int last = pos - kv0;
#pragma unroll
            for (int k = 0; k < BN; ++k) s[k] = (k > last) ? -INFINITY : s[k];
          }
          if (p.window > 0 && kv0 < base + p.tt - p.window) {
            const int first = pos - p.window + 1 - kv0;
#pragma unroll
            for (int k = 0; k < BN; ++k) s[k] = (k < first) ? -INFINITY : s[k];
          }
          kv0 += dk;
          if (kv0 >= kend) kv0 -= kwrap;
          constexpr int Q = BN / 4;
          float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[Q], s[Q + 1]);
          float mx2 = fmaxf(s[2 * Q], s[2 * Q + 1]), mx3 = fmaxf(s[3 * Q], s[3 * Q + 1]);
#pragma unroll
          for (int k = 2; k < Q; k += 2) {
            mx0 = fmax3(mx0, s[k], s[k + 1]);
            mx1 = fmax3(mx1, s[Q + k], s[Q + k + 1]);
            mx2 = fmax3(mx2, s[2 * Q + k], s[2 * Q + k + 1]);
            mx3 = fmax3(mx3, s[3 * Q + k], s[3 * Q + k + 1]);
          }
          const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
          // (Selects, no branch: tensor memory is written by the whole warp together.)
          const bool need = m_tile > m + prefill::kRescaleThreshold;
          const float alpha = ex2_approx(need ? m - m_tile : 0.f);  // m = -inf gives 0
          m = need ? m_tile : m;
          l *= alpha;
          const float m_use = (m == -INFINITY) ? 0.f : m;
          if constexpr (C::kOwnP) {
            // The first half of P in registers while the previous product may
            // still read P's columns (and write O).
            const uint64_t c2 = f2_make(sl2, sl2), nm2 = f2_make(-m_use, -m_use);
            uint64_t la = f2_make(0.f, 0.f), lb = la;
            uint32_t pa[32], pb[16];
            prefill::exp_cols_regs<T, 0, BN, 0, 64>(s, c2, nm2, pa, la, lb);
            if (np > 0) {
              if (!(ok = warp_all(wait_bar(&pv_done[t], (np - 1) & 1, ctl, kSitePvDone)))) break;
              tc_fence_after();
            }
            ++np;
            tmem_st_x16(tP, *reinterpret_cast<uint32_t(*)[16]>(pa));
            tmem_st_x16(tP + 16, *reinterpret_cast<uint32_t(*)[16]>(pa + 16));
            prefill::exp_cols_regs<T, 0, BN, 64, 96>(s, c2, nm2, pb, la, lb);
            tmem_st_x16(tP + 32, pb);
            prefill::exp_cols_regs<T, 0, BN, 96, 128>(s, c2, nm2, pb, la, lb);
            tmem_st_x16(tP + 48, pb);
            float a0, a1, b0, b1;
            f2_split(la, a0, a1);
            f2_split(lb, b0, b1);
            l += (a0 + a1) + (b0 + b1);
          } else {
            l += prefill::exp_tile<T, 0, BN>(s, sl2, m_use, tP);
          }
          if (!first_step && __any_sync(0xffffffffu, need)) {
            // O_t was last written by this group's previous product, complete
            // before S_t(j) was signalled (own P: waited for above).
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld_x32(tO + cc * 32, o);
              tmem_wait_ld_x32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_x32(tO + cc * 32, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_ready[t]);
        }
      }
      if (!ok) break;

      // ---- end of a piece
      const bool two = w.two(p);
      const bool shared = !two && w.steps() > 1;  // group 1 has a part of the same rows
      const int r = (warp & 3) * 32 + lane;       // row of the tile
      float2* xrow = reinterpret_cast<float2*>(smem + C::kScratchOff) + r;
      if (!two && t == 1) {
        if (shared) {
          // Hand (m, l) to group 0 and wait until it has read O_1.
          *xrow = make_float2(m, l);
          mbar_arrive(x_up);
          ok = warp_all(wait_bar(x_down, w.xp & 1, ctl, kSiteXDown));
          __syncwarp();
          if (lane == 0) {
            ++w.xp;
            ++w.od1;  // (group 0 waited for it)
          }
          if (!ok) break;
        }
        continue;
      }
      if (!(ok = warp_all(wait_bar(&o_done[t], (t ? w.od1 : w.od0) & 1, ctl, kSiteODone)))) break;
      float w0 = 1.f, w1 = 0.f;  // weights of O_0 and O_1
      if (shared) {
        if (!(ok = warp_all(wait_bar(&o_done[1], w.od1 & 1, ctl, kSiteODone)))) break;
        if (!(ok = warp_all(wait_bar(x_up, w.xp & 1, ctl, kSiteXUp)))) break;
        const float2 other = *xrow;
        const float mm = fmaxf(m, other.x);
        w0 = m == -INFINITY ? 0.f : ex2_approx(m - mm);
        w1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - mm);
        l = l * w0 + other.y * w1;
        m = mm;
      }
      __syncwarp();
      if (lane == 0) {  // (each group keeps count of the other's phases too)
        if (two || t == 0) ++w.od0;
        if (two || shared) ++w.od1;
        if (shared) ++w.xp;
      }
      tc_fence_after();
      const int tile = two ? t : 0, tok = (w.pair * NQT + tile) * p.tt + r / p.G;
      const bool row_ok = r < p.tt * p.G && tok < w.s.T;
      if (__any_sync(0xffffffffu, row_ok)) {
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        // (l = 0: no key, or every score -inf. A NaN score, or an infinite one, makes l
        // NaN, which goes on into o, lse and the gather.)
        const float inv = l == 0.f ? 0.f : 1.f / l;
        w0 *= inv;
        w1 *= inv;
        // 32 columns of the row's O, normalised; zeros for a row without keys
        // (O may hold anything). The whole warp reads tensor memory together, so
        // the lanes that have a row and those that have none meet here first.
        auto columns = [&](int col, float (&f)[32]) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld_x32(tmem + lane_off + C::o_col(t) + col, o);
          tmem_wait_ld_x32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * w0;
          if (shared) {
            tmem_ld_x32(tmem + lane_off + C::o_col(1) + col, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o[e]), w1, f[e]);
          }
          if (l == 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
          }
        };
        // (The loops over columns stay loops: this code runs once a piece, often on
        // a cold instruction cache; unrolled, 8K tokens took 497 us where they took
        // 479.)
        const float l2 = l == 0.f ? -INFINITY : m + lg2_approx(l);
        if (w.whole()) {
          // Each thread writes its own row, a 32-byte sector at a time. (Through
          // shared memory, in whole lines, it took twice as long.)
          const size_t orow = (static_cast<size_t>(w.s.q0) + tok) * p.Hq + w.head * p.G + r % p.G;
          T* dst = reinterpret_cast<T*>(p.o) + orow * p.d;
          const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            float f[32];
            columns(col, f);
            if (row_ok) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  v[e] = prefill::pack2<T>(f[16 * u + 2 * e], f[16 * u + 2 * e + 1]);
                const int at = col + 16 * u;
                if (sectors && at + 16 <= p.d) {
                  st_global_32(dst + at, v);
                } else {
                  if (at < p.d)
                    *reinterpret_cast<uint4*>(dst + at) = make_uint4(v[0], v[1], v[2], v[3]);
                  if (at + 8 < p.d)
                    *reinterpret_cast<uint4*>(dst + at + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                }
              }
            }
          }
          if (row_ok && p.lse != nullptr) p.lse[orow] = l2 * 0.69314718055994531f;
          __syncwarp();
        } else {
          // A partial, 32 rows of the slot per warp: columns 4u .. 4u + 3 of
          // all rows side by side, so that what a thread holds goes out in
          // whole lines as it is.
          const size_t rows32 = static_cast<size_t>(w.slot(c, p.nc)) * (kSlotRows / 32) +
                                (tile * BM + (warp & 3) * 32) / 32;
          float4* dst = reinterpret_cast<float4*>(p.part_o) + rows32 * (8 * D) + lane;
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            float f[32];
            columns(col, f);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[(col / 4 + u) * 32] =
                  make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
          }
          p.part_lse[rows32 * 32 + lane] = row_ok ? l2 : -INFINITY;
        }
      }
      tc_fence_before();
      if (shared) mbar_arrive(x_down);
    } while (walk_on(w, p, lane));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// The cut items: block (c, y) folds the one whose first chunk is CTA c's, or
// whose rest begins in CTA c's range and goes on in the next (if it has no
// chunks), rows 32 y .. 32 y + 31 of its 256: lane = row, warp w takes columns
// 4 (w + 8 k). All of a partial's columns are loaded before any is used, and
// the result goes out through shared memory in whole lines. (One row a warp at
// a time, partials in rows, this took 27 us for 148 cut items of 256 rows.)
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_paged_gather_kernel(const Params p) {
  constexpr int CW = D / 32;  // 4-column units of a thread
  __shared__ __align__(16) uint8_t stage[32 * (2 * D + 16)];
  grid_wait();
  const int c = blockIdx.x;
  const Head h = *p.plan.head;  // (loaded together; a start that no CTA wrote is not looked at)
  const Start at_c = p.plan.starts[c], at_next = p.plan.starts[min(c + 1, p.nc - 1)];
  if (c >= h.ctas) return;
  const bool has_chunks = c < h.chunks;
  if (!has_chunks && c + 1 >= h.ctas) return;
  const Start nx = has_chunks ? at_c : at_next;
  const Seq s = load_seq(p.cu_q, p.lens, nx.b, p.total_q, p.max_q, p.capacity());
  const int tile = blockIdx.y / 4, t0 = (nx.pair * NQT + tile) * p.tt;
  const int r0 = (blockIdx.y & 3) * 32;  // rows r0 .. r0 + 31 of the tile
  if (r0 >= p.tt * p.G || t0 + r0 / p.G >= s.T) return;  // none
  const int n = span_of(p, s, nx.pair).n, g = step_cost(p, s.T, nx.pair);
  const int wc = chunk_steps(h.w, g), f = chunks_of(n, wc, h.chunks > 0), rest = n - f * wc;
  if (has_chunks ? nx.i != 0 || (f == 1 && rest == 0) : f > 0)
    return;  // not the first chunk, or the whole item; the chunks' business
  // Its partials: chunks c .. c + f - 1, then the CTAs q0 .. q1 of the rest
  // (in whose ranges its first and its last step begin).
  const long long at = nx.rest + kItemCost;
  const int q0 = h.chunks + static_cast<int>(div_pos(at, h.w));
  const int q1 =
      rest > 0 ? h.chunks + static_cast<int>(div_pos(at + static_cast<long long>(rest - 1) * g, h.w))
               : q0 - 1;
  if (!has_chunks && (q0 != c || q1 == q0)) return;  // not begun in c's range, or not cut
  const int parts = f + q1 - q0 + 1;
  auto slot_of = [&](int k) {
    if (k < f) return c + k;
    if (q0 == q1) return 2 * p.nc + c;
    return k == f ? p.nc + q0 : q0 + k - f;
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float mx = -INFINITY, tot = 0.f;
  float4 acc[CW];
#pragma unroll
  for (int u = 0; u < CW; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const size_t rows32 = static_cast<size_t>(slot_of(k)) * (kSlotRows / 32) + blockIdx.y;
    const float lse = p.part_lse[rows32 * 32 + lane];
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + rows32 * (8 * D) + lane;
    float4 x[CW];
#pragma unroll
    for (int u = 0; u < CW; ++u) x[u] = src[(warp + 8 * u) * 32];
    if (lse == -INFINITY) continue;  // (saw no key; a NaN goes into the sums)
    const float nm = fmaxf(mx, lse);
    const float sc = ex2_approx(mx - nm), wt = ex2_approx(lse - nm);
    tot = tot * sc + wt;
#pragma unroll
    for (int u = 0; u < CW; ++u) {
      acc[u].x = fmaf(wt, x[u].x, acc[u].x * sc);
      acc[u].y = fmaf(wt, x[u].y, acc[u].y * sc);
      acc[u].z = fmaf(wt, x[u].z, acc[u].z * sc);
      acc[u].w = fmaf(wt, x[u].w, acc[u].w * sc);
    }
    mx = nm;
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
#pragma unroll
  for (int u = 0; u < CW; ++u) {
    uint2 v;
    v.x = prefill::pack2<T>(acc[u].x * inv, acc[u].y * inv);
    v.y = prefill::pack2<T>(acc[u].z * inv, acc[u].w * inv);
    *reinterpret_cast<uint2*>(stage + lane * (2 * D + 16) + (warp + 8 * u) * 8) = v;
  }
  auto out_row = [&](int q, long long& orow) {  // row q of the 32: is there one, and where
    const int r = r0 + q, tok = t0 + r / p.G;
    orow = (static_cast<long long>(s.q0) + tok) * p.Hq + nx.g * p.G + r % p.G;
    return r < p.tt * p.G && tok < s.T;
  };
  long long orow;
  if (warp == 0 && p.lse != nullptr && out_row(lane, orow))
    p.lse[orow] = tot == 0.f ? -INFINITY : (mx + lg2_approx(tot)) * 0.69314718055994531f;
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * D / 8; i += 256) {
    const int q = i / (D / 8), u = i % (D / 8);
    if (u * 8 < p.d && out_row(q, orow))
      *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.o) + orow * p.d + u * 8) =
          *reinterpret_cast<const uint4*>(stage + q * (2 * D + 16) + u * 16);
  }
}

}  // namespace paged
}  // namespace eta
