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
// rows sees. The steps of all items, in order (sequence, KV head, tile pair,
// key tile), are cut into equal contiguous ranges, one per CTA (one CTA per
// SM): a chunk over a long cache then fills the GPU however few rows it has,
// and a mixed batch is balanced. A piece that is not a whole item leaves a
// normalised fp32 partial with its log-sum-exp, and the gather kernel folds
// the partials of an item together in the order of its keys.
//
// Three kernels per call:
//   attn_paged_plan_kernel    one CTA: steps of each sequence, their prefix
//                             sums, each CTA's first (sequence, head, pair, step)
//   attn_paged_kernel         the stream (below)
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
//   One tile of rows (a single token, or a short chunk): the groups share Q_0
// and take the key tiles in turns, each with its own running maximum, sum and
// O; group 0 folds O_1 into O_0 at the end of the piece. One group's
// exponentials then overlap the other's products and loads.
//
// Rows of V behind the sequence's last key are set to zero in shared memory
// before the product: their probabilities are zero, but what lies there in the
// pool may be infinite or NaN.
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
};

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 128, "head size");
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = 128 * 128;  // 128 rows of 64 columns
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kKVOff = NQT * kTileBytes;
  static constexpr int kStgWarpBytes = 32 * 128;
  static constexpr int kStgOff = kKVOff + kStages * kTileBytes;
  static constexpr int kBarOff = kStgOff + 8 * kStgWarpBytes;
  // kv_full[S], kv_empty[S], q_full[2], q_empty[2], s_ready[2], p_ready[2],
  // o_done[2], x_up, x_down, drain
  static constexpr int kNumBars = 2 * kStages + 5 * NQT + 3;
  static constexpr int kCtlOff = kBarOff + kNumBars * 8;
  static constexpr int kXOff = kCtlOff + 64;  // (m, l) of group 1's rows
  static constexpr int kSmemBytes = kXOff + BM * 8 + 1024;  // + runtime 1024-byte alignment
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kPCol = 64;  // P_t overwrites S_t from this column on
  __host__ __device__ static constexpr uint32_t s_col(int t) { return BN * t; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 2 * BN + D * t; }
  static_assert(kSmemBytes <= 232448, "shared memory");
};

// The plan, in device memory.
struct Plan {
  long long* cost;  // [B + 1]: steps before sequence b (all its KV heads)
  int4* starts;     // [nc]: (b, g, pair, step) where CTA c begins
  int* busy;        // [1]: CTAs that have a range (min(nc, steps))
};

struct Params {
  const int* cu_q;
  const int* lens;
  const int* table;
  void* o;
  float* lse;
  float* part_o;    // [2 nc][256][d]
  float* part_lse;  // [2 nc][256], log2 units
  Plan plan;
  int B, Hq, Hkv, G, tt;
  int total_q, max_q, d;
  int num_pages, page_log2, width;
  int window;
  int nc;
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
  const int last = s.L - s.T + t1 - 1, first = s.L - s.T + t0;
  Span r;
  r.lo = p.window > 0 ? max(0, first - p.window + 1) / BN : 0;
  r.n = last < 0 ? 1 : max(1, last / BN + 1 - r.lo);
  if (last < 0) r.lo = 0;
  return r;
}
__device__ __forceinline__ int pairs_of(const Params& p, int T) {
  return (T + NQT * p.tt - 1) / (NQT * p.tt);
}

// Steps of one KV head of a sequence, by the whole warp.
__device__ __forceinline__ long long seq_steps(const Params& p, const Seq& s, int lane) {
  const int n = pairs_of(p, s.T);
  long long sum = 0;
  for (int i = lane; i < n; i += 32) sum += span_of(p, s, i).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__device__ __forceinline__ long long range_lo(int c, long long steps, int busy) {
  return c * steps / busy;
}

// A range of fewer steps than this is not worth a CTA of its own.
constexpr int kMinSteps = 2;

__global__ void __launch_bounds__(kPlanThreads) attn_paged_plan_kernel(const Params p) {
  __shared__ long long red[kPlanThreads / 32];
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = warp; b < p.B; b += kPlanThreads / 32) {
    const Seq s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    const long long c = seq_steps(p, s, lane) * p.Hkv;
    if (lane == 0) {
      p.plan.cost[b] = c;
      check_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    }
  }
  __syncthreads();
  // Exclusive prefix over the sequences, in place.
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += p.plan.cost[b];
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    red[lane] = w;
  }
  __syncthreads();
  const long long steps = red[kPlanThreads / 32 - 1];
  long long run = x - mine + (warp > 0 ? red[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) {
    const long long c = p.plan.cost[b];
    p.plan.cost[b] = run;
    run += c;
  }
  const long long want = (steps + kMinSteps - 1) / kMinSteps;
  const int busy = static_cast<int>(want < p.nc ? want : p.nc);
  if (tid == 0) {
    p.plan.cost[p.B] = steps;
    *p.plan.busy = busy;
  }
  __syncthreads();
  // Where each CTA begins: the sequence by bisection, the tile pair by a scan.
  for (int c = warp; c < busy; c += kPlanThreads / 32) {
    const long long at = range_lo(c, steps, busy);
    int lo = 0, hi = p.B - 1;  // largest b with cost[b] <= at
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.plan.cost[mid] <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    const long long per_head = (p.plan.cost[lo + 1] - p.plan.cost[lo]) / p.Hkv;
    long long r = at - p.plan.cost[lo];
    const int g = static_cast<int>(r / per_head);
    r -= g * per_head;
    const Seq s = load_seq(p.cu_q, p.lens, lo, p.total_q, p.max_q, p.capacity());
    const int n = pairs_of(p, s.T);
    int pair = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int k = i0 + lane < n ? span_of(p, s, i0 + lane).n : 0;
      int y = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      const unsigned over = __ballot_sync(0xffffffffu, r < y);  // (32 spans stay below 2^31)
      if (over != 0) {
        const int l = __ffs(over) - 1;
        r -= __shfl_sync(0xffffffffu, y - k, l);
        pair = i0 + l;
        break;
      }
      r -= __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) p.plan.starts[c] = make_int4(lo, g, pair, static_cast<int>(r));
  }
}

// A CTA's way through its range, piece by piece. Every role keeps its own.
struct Walk {
  int b, g, pair;
  int i0, i1, n;   // steps [i0, i1) of the item's n
  int lo;          // its first key tile
  long long left;  // steps of the range behind this piece
  Seq s;

  __device__ __forceinline__ void item(const Params& p, int from) {
    const Span sp = span_of(p, s, pair);
    lo = sp.lo;
    n = sp.n;
    i0 = from;
    i1 = static_cast<int>(min(static_cast<long long>(n), i0 + left));
    left -= i1 - i0;
  }
  __device__ __forceinline__ void start(const Params& p, int c, long long count) {
    const int4 st = p.plan.starts[c];
    b = st.x, g = st.y, pair = st.z;
    left = count;
    s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
    item(p, st.w);
  }
  // To the next piece; false at the end of the range.
  __device__ __forceinline__ bool next(const Params& p) {
    if (left <= 0) return false;
    if (++pair >= pairs_of(p, s.T)) {
      pair = 0;
      if (++g >= p.Hkv) {
        g = 0;
        do {
          if (++b >= p.B) return false;  // (the plan's range ends before this)
          s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, p.capacity());
        } while (s.T == 0);
      }
    }
    item(p, 0);
    return true;
  }
  __device__ __forceinline__ int token0() const { return pair; }
  __device__ __forceinline__ int steps() const { return i1 - i0; }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == n; }
  // Both tiles have rows?
  __device__ __forceinline__ bool two(const Params& p) const {
    return pair * NQT * p.tt + p.tt < s.T;
  }
};

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
  uint64_t* x_up = o_done + NQT;
  uint64_t* x_down = x_up + 1;
  uint64_t* drain = x_down + 1;
  CtaCtl* ctl = reinterpret_cast<CtaCtl*>(smem + C::kCtlOff);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kCtlOff + 32);
  float2* xrow = reinterpret_cast<float2*>(smem + C::kXOff);

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
  const long long steps = p.plan.cost[p.B];
  const int busy = *p.plan.busy;
  const long long r0 = c < busy ? range_lo(c, steps, busy) : 0;
  const long long r1 = c < busy ? range_lo(c + 1, steps, busy) : 0;

  if (r1 <= r0) {
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
    Walk w;
    w.start(p, c, r1 - r0);
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
                        w.g, w.s.q0 + (w.pair * NQT + t) * p.tt);
        }
        ++qn[t];
      }
      // The page that this lane loads of key tile j: its id, or num_pages
      // (out of range: zeros) where the sequence has none.
      const int* row = p.table + static_cast<size_t>(w.b) * p.width;
      auto page_of = [&](int j) {
        const int key = j * BN + pg * box_rows;
        if (!loads || key >= w.s.L) return p.num_pages;
        const int id = row[key >> p.page_log2];
        if (id >= 0 && id < p.num_pages) return id;
        bad(kBadPage);
        return p.num_pages;
      };
      int page = page_of(w.lo + w.i0);
      for (int j = w.lo + w.i0; ok && j < w.lo + w.i1; ++j) {
        const int y = (j * BN + pg * box_rows) & ((1 << p.page_log2) - 1);
        const int now = page;
        if (j + 1 < w.lo + w.i1) page = page_of(j + 1);  // ahead of its use
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
                        y, w.g, now);
        }
      }
    } while (ok && w.next(p));
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
    bool ok = true;
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
      const uint32_t tP = tmem + C::s_col(t) + C::kPCol;
      const uint32_t tO = tmem + C::o_col(t);
      if (first)
        umma_ts_w<0>(tO, tP, desc_words(vd, d_hi), idesc_pv);
      else
        umma_ts_w<1>(tO, tP, desc_words(vd, d_hi), idesc_pv);
#pragma unroll
      for (int kk = 1; kk < BN / 16; ++kk)
        umma_ts_w<1>(tO, tP + kk * 8, desc_words(vd + kk * 128, d_hi), idesc_pv);
    };
    Walk w;
    w.start(p, c, r1 - r0);
    // Rows of V behind the sequence's last key: zeros (the pages behind it are
    // zeros already; those of its last page may hold anything).
    auto clear_tail = [&](int j, uint32_t lv) {
      const int valid = w.s.L - (w.lo + w.i0 + j) * BN;
      if (valid >= BN) return;
      const int from = max(valid, 0);
      uint8_t* base = sKV + (lv % S) * C::kTileBytes;
      for (int i = lane; i < (BN - from) * C::kBoxes * 8; i += 32) {
        const int u = i & 7, rb = i >> 3;
        const int r = from + rb / C::kBoxes, x = rb % C::kBoxes;
        *reinterpret_cast<uint4*>(base + x * C::kBoxBytes + r * 128 + u * 16) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    do {
      const int n = w.steps();
      if (w.two(p)) {
        for (int j = 0; ok && j <= n; ++j) {
          const uint32_t Lk = L + 2 * j, Lv = L + 2 * j - 1;
          bool have_k = false, have_v = false;
#pragma unroll
          for (int t = 0; t < NQT; ++t) {
            if (!ok) break;
            if (j >= 1) {
              if (!have_v) {
                if (!(ok = warp_all(wait_bar(&kv_full[Lv % S], (Lv / S) & 1, ctl, kSiteKvFull))))
                  break;
                have_v = true;
                clear_tail(j - 1, Lv);
              }
              if (!(ok = warp_all(wait_bar(&p_ready[t], pw[t] & 1, ctl, kSitePReady)))) break;
              ++pw[t];
              tc_fence_after();
              value(t, Lv, j == 1);
              if (j == n) umma_commit_w(&o_done[t]);
            }
            if (j < n) {
              if (!have_k) {
                if (!(ok = warp_all(wait_bar(&kv_full[Lk % S], (Lk / S) & 1, ctl, kSiteKvFull))))
                  break;
                tc_fence_after();
                have_k = true;
              }
              if (j == 0) {
                if (!(ok = warp_all(wait_bar(&q_full[t], qi[t] & 1, ctl, kSiteQFull)))) break;
                tc_fence_after();
              }
              score(t, t, Lk);
              if (j == n - 1) umma_commit_w(&q_empty[t]);
            }
          }
          if (have_k) umma_commit_w(&kv_empty[Lk % S]);
          if (have_v) umma_commit_w(&kv_empty[Lv % S]);
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
            score(j & 1, 0, Lk);
            if (j == n - 1) umma_commit_w(&q_empty[0]);
            umma_commit_w(&kv_empty[Lk % S]);
          }
          if (j >= 1) {
            const int t = (j - 1) & 1;
            const uint32_t Lv = L + 2 * j - 1;
            if (!(ok = warp_all(wait_bar(&kv_full[Lv % S], (Lv / S) & 1, ctl, kSiteKvFull)))) break;
            clear_tail(j - 1, Lv);
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
    } while (ok && w.next(p));
    // Every MMA must be complete before tensor memory is released.
    umma_commit_w(drain);
    drain_bar(drain, 0, ctl, kSiteDrain);
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int q4 = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::s_col(t);
    const uint32_t tP = tS + C::kPCol;
    const uint32_t tO = tmem + lane_off + C::o_col(t);
    uint8_t* stg = smem + C::kStgOff + warp * C::kStgWarpBytes;
    const int r = q4 * 32 + lane;  // row of the tile
    const float sl2 = p.scale_log2;
    uint32_t sw = 0;  // s_ready phases consumed
    uint32_t od[NQT] = {0, 0};  // o_done phases (group 0 also follows group 1's in shared pieces)
    uint32_t xp = 0;  // exchanges
    bool ok = true;
    Walk w;
    w.start(p, c, r1 - r0);
    do {
      const int n = w.steps();
      const bool two = w.two(p);
      const int tile = two ? t : 0;                       // tile of rows this group works on
      const int j0 = two ? 0 : t, dj = two ? 1 : 2;       // its key tiles
      const int tok = (w.pair * NQT + tile) * p.tt + r / p.G;  // this row's token
      const bool row_ok = r < p.tt * p.G && tok < w.s.T;
      const bool live = __any_sync(0xffffffffu, row_ok);
      const int pos = row_ok ? w.s.L - w.s.T + tok : -1;
      const int kfirst = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      // Key tiles that every row of the tile sees whole need no mask.
      const int base = w.s.L - w.s.T + (w.pair * NQT + tile) * p.tt;
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < n; j += dj) {
        if (!(ok = warp_all(wait_bar(&s_ready[t], sw & 1, ctl, kSiteSReady)))) break;
        ++sw;
        tc_fence_after();
        if (!live) {  // no rows in this warp: its P is never stored
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
        const int kv0 = (w.lo + w.i0 + j) * BN;
        if (kv0 + BN - 1 > base) {
          const int last = pos - kv0;
#pragma unroll
          for (int k = 0; k < BN; ++k) s[k] = (k > last) ? -INFINITY : s[k];
        }
        if (p.window > 0 && kv0 < base + p.tt - p.window) {
          const int first = kfirst - kv0;
#pragma unroll
          for (int k = 0; k < BN; ++k) s[k] = (k < first) ? -INFINITY : s[k];
        }
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
        float alpha = 1.f;
        const bool need = m_tile > m + prefill::kRescaleThreshold;
        if (need) {
          alpha = ex2_approx(m - m_tile);  // m = -inf gives 0
          m = m_tile;
          l *= alpha;
        }
        const float m_use = (m == -INFINITY) ? 0.f : m;
        l += prefill::exp_tile<T, 0, BN>(s, sl2, m_use, tP);
        if (j > j0 && __any_sync(0xffffffffu, need)) {
          // O_t was last written by this group's previous product, which
          // completed before S_t(j) was signalled.
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
      if (!ok) break;

      // ---- end of a piece
      const bool shared = !two && n > 1;  // group 1 has a part of the same rows
      float w0 = 1.f, w1 = 0.f;           // weights of O_0 and O_1
      if (!two && t == 1) {
        if (shared) {
          // Hand (m, l) to group 0 and wait until it has read O_1.
          xrow[r] = make_float2(m, l);
          mbar_arrive(x_up);
          ok = warp_all(wait_bar(x_down, xp & 1, ctl, kSiteXDown));
          ++xp;
          ++od[1];  // (group 0 waited for it)
          if (!ok) break;
        }
        continue;
      }
      if (!(ok = warp_all(wait_bar(&o_done[t], od[t] & 1, ctl, kSiteODone)))) break;
      ++od[t];
      if (shared) {
        if (!(ok = warp_all(wait_bar(&o_done[1], od[1] & 1, ctl, kSiteODone)))) break;
        ++od[1];
        if (!(ok = warp_all(wait_bar(x_up, xp & 1, ctl, kSiteXUp)))) break;
        ++xp;
        const float2 other = xrow[r];
        const float mm = fmaxf(m, other.x);
        w0 = m == -INFINITY ? 0.f : ex2_approx(m - mm);
        w1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - mm);
        l = l * w0 + other.y * w1;
        m = mm;
      } else if (t == 0 && two) {
        ++od[1];  // group 1 waits for its own; keep count of its phases
      }
      tc_fence_after();
      if (live) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        w0 *= inv;
        w1 *= inv;
        const bool whole = w.whole();
        // The row's place: (token, head) in o, or its row in the piece's slot.
        const int slot = 2 * c + (w.i0 == 0 ? 1 : 0);
        const size_t prow = static_cast<size_t>(slot) * kSlotRows + tile * BM + r;
        const size_t orow = (static_cast<size_t>(w.s.q0) + tok) * p.Hq + w.g * p.G + r % p.G;
        // O, 32 columns at a time through the warp's staging rows, so that a
        // store instruction writes whole lines: 16-byte chunk u of row q sits
        // at chunk u ^ (q % 8).
        const long long my = row_ok ? static_cast<long long>(whole ? orow : prow) : -1;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          float f[64];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tmem_ld_x32(tO + half * 64 + h * 32, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[h * 32 + e] = __uint_as_float(o[e]) * w0;
            if (shared) {
              tmem_ld_x32(tmem + lane_off + C::o_col(1) + half * 64 + h * 32, o);
              tmem_wait_ld_x32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) f[h * 32 + e] = fmaf(__uint_as_float(o[e]), w1, f[h * 32 + e]);
            }
          }
          if (l <= 0.f) {  // no visible key: O may hold anything
#pragma unroll
            for (int e = 0; e < 64; ++e) f[e] = 0.f;
          }
          // whole: 64 columns of T are one staged line; partial: two of fp32.
          for (int h = 0; h < (whole ? 1 : 2); ++h) {
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint4 v;
              if (whole) {
                v.x = prefill::pack2<T>(f[8 * u], f[8 * u + 1]);
                v.y = prefill::pack2<T>(f[8 * u + 2], f[8 * u + 3]);
                v.z = prefill::pack2<T>(f[8 * u + 4], f[8 * u + 5]);
                v.w = prefill::pack2<T>(f[8 * u + 6], f[8 * u + 7]);
              } else {
                v.x = __float_as_uint(h ? f[32 + 4 * u] : f[4 * u]);
                v.y = __float_as_uint(h ? f[33 + 4 * u] : f[4 * u + 1]);
                v.z = __float_as_uint(h ? f[34 + 4 * u] : f[4 * u + 2]);
                v.w = __float_as_uint(h ? f[35 + 4 * u] : f[4 * u + 3]);
              }
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((u ^ (lane & 7)) << 4)) = v;
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int q = k * 4 + (lane >> 3), u = lane & 7;
              const long long to = __shfl_sync(0xffffffffu, my, q);
              const uint4 v = *reinterpret_cast<const uint4*>(stg + q * 128 + ((u ^ (q & 7)) << 4));
              const int col = whole ? half * 64 + u * 8 : half * 64 + h * 32 + u * 4;
              if (to >= 0 && col < p.d) {
                if (whole)
                  *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.o) + to * p.d + col) = v;
                else
                  *reinterpret_cast<uint4*>(p.part_o + to * p.d + col) = v;
              }
            }
          }
        }
        if (row_ok) {
          const float l2 = l > 0.f ? m + lg2_approx(l) : -INFINITY;
          if (!whole)
            p.part_lse[prow] = l2;
          else if (p.lse != nullptr)
            p.lse[orow] = l2 * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      if (shared) mbar_arrive(x_down);
    } while (w.next(p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// The items cut between CTAs: block (c, y) folds the one that begins in CTA
// c's range and goes on in the next ones, rows y, y + gridDim.y * 8, ... of it,
// one warp per row.
template <typename T>
__global__ void __launch_bounds__(256) attn_paged_gather_kernel(const Params p) {
  grid_wait();
  const long long steps = p.plan.cost[p.B];
  const int busy = *p.plan.busy;
  const int c = blockIdx.x;
  if (c + 1 >= busy) return;
  const int4 nx = p.plan.starts[c + 1];
  const long long r0 = range_lo(c, steps, busy), r1 = range_lo(c + 1, steps, busy);
  if (nx.w == 0 || nx.w > r1 - r0) return;  // a boundary between items, or begun before c
  const Seq s = load_seq(p.cu_q, p.lens, nx.x, p.total_q, p.max_q, p.capacity());
  const Span sp = span_of(p, s, nx.z);
  const long long end = r1 - nx.w + sp.n;  // one behind the item's last step
  const int t0 = nx.z * NQT * p.tt;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int rr = blockIdx.y * 8 + warp; rr < kSlotRows; rr += gridDim.y * 8) {
    const int tile = rr / BM, r = rr - tile * BM;
    const int tok = t0 + tile * p.tt + r / p.G;
    if (r >= p.tt * p.G || tok >= s.T) continue;
    // Partials: slot 2c + 1 of CTA c, then slot 2c' of the CTAs that go on.
    float mx = -INFINITY, tot = 0.f;
    float acc[8];  // two pieces of 4 columns: 4 lane, 128 + 4 lane (d <= 128: the first)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int cc = c; cc < busy && range_lo(cc, steps, busy) < end; ++cc) {
      const size_t row = static_cast<size_t>(2 * cc + (cc == c ? 1 : 0)) * kSlotRows + rr;
      const float lse = p.part_lse[row];
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lane * 4 < p.d) x = *reinterpret_cast<const float4*>(p.part_o + row * p.d + lane * 4);
      if (lse == -INFINITY) continue;
      const float nm = fmaxf(mx, lse);
      const float sc = ex2_approx(mx - nm), wt = ex2_approx(lse - nm);
      tot = tot * sc + wt;
      acc[0] = fmaf(wt, x.x, acc[0] * sc);
      acc[1] = fmaf(wt, x.y, acc[1] * sc);
      acc[2] = fmaf(wt, x.z, acc[2] * sc);
      acc[3] = fmaf(wt, x.w, acc[3] * sc);
      mx = nm;
    }
    const float inv = tot > 0.f ? 1.f / tot : 0.f;
    const size_t orow = (static_cast<size_t>(s.q0) + tok) * p.Hq + nx.y * p.G + r % p.G;
    if (lane * 4 < p.d) {
      uint2 v;
      v.x = prefill::pack2<T>(acc[0] * inv, acc[1] * inv);
      v.y = prefill::pack2<T>(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.o) + orow * p.d + lane * 4) = v;
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[orow] = tot > 0.f ? (mx + lg2_approx(tot)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace paged
}  // namespace eta
