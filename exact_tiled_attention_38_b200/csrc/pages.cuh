// Page operations of a paged cache: rows taking over other rows (forks, beam
// steps, ended and new sequences) and growing, and compaction of the live
// pages. Both first settle the whole numbers (block tables, reference counts,
// which page goes where), then copy page contents with the whole grid. When the
// counts fit shared memory and the tables are not large, one kernel does both:
// every CTA settles all of the whole numbers for itself, and writes and copies
// its share. Otherwise a cluster of CTAs settles them, its hardware barrier
// between the steps, and a second kernel copies.
//
// Free pages are those with a reference count <= 0, and are always taken
// lowest first in the order of the rows, so the result does not depend on
// timing: atomic additions and minima of whole numbers only.
//
// update: row b of the next state goes on from row source[b] of this one
// (-1: from nothing) and grows by add[b] tokens. Rows that share a source share
// its full pages. Its last, partly filled page stays with one of them -- the
// source row itself if it goes on, else the first that takes it over -- and the
// others get a copy in a page of their own.
// compact: with n live pages, those at n and above move, in order, into the
// free pages below n, in order: the fewest copies, and no page is both read
// and written, so the copies need no order among them.
//
// Bound: the whole numbers by latency (a few dependent passes over the tables
// and the counts), the contents by memory (each moved page is read once and
// written once). Measured on B200: a serving step of 64 rows, 9,934 pages 9.6
// us; a beam step of 96 rows with 66 copies in 16 layers, 277 MB 53 us (5.2
// TB/s); a compaction of 700 pages in 8 layers, 1.47 GB 245 us (6.0 TB/s, 0.91
// of the measured copy rate); a compaction of 20 small pages 6.4 us, the host's
// part of the call.
#pragma once

#include <climits>

#include "paged_common.cuh"

namespace eta {
namespace pages {

constexpr int kCtas = 8;
constexpr int kThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyBytes = 32 * 16 * kCopyUnroll;  // one warp's piece of a copy

__device__ __forceinline__ int cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// Barrier of the cluster's threads. Release / acquire at cluster scope: what
// any thread wrote to global memory before it, every thread sees after it.
__device__ __forceinline__ void cluster_barrier() {
  __threadfence();
  __syncthreads();  // (every warp converged, as the aligned form asks)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Reads and writes of data that other CTAs of the cluster write in the same
// launch go past L1.
__device__ __forceinline__ int ld(const int* p) { return __ldcg(p); }
__device__ __forceinline__ void st(int* p, int v) { __stcg(p, v); }

// The pools whose pages are copied. A page of a pool is `page_bytes` in one
// piece (a multiple of 16), in every layer of both pools.
struct CopyParams {
  uint8_t* pool[2];
  long long page_stride;   // bytes
  long long layer_stride;  // bytes
  long long page_bytes;
  int layers;
  const int* from;
  const int* to;
  const int* n_copies;
};

// Contents of the pages from[k] into to[k], k < n: pieces of 2 KB, one a warp
// at a time, `warps` warps in all.
__device__ __forceinline__ void copy_pages(const CopyParams& p, const int* from, const int* to,
                                           int n, long long me, long long warps) {
  const int lane = threadIdx.x & 31;
  const unsigned pieces = static_cast<unsigned>((p.page_bytes + kCopyBytes - 1) / kCopyBytes);
  const unsigned per_page = pieces * 2u * static_cast<unsigned>(p.layers);
  const long long units = static_cast<long long>(n) * per_page;
  for (long long w = me; w < units; w += warps) {
    unsigned k, r;
    if (units <= 0xffffffffLL) {
      k = static_cast<unsigned>(w) / per_page;
      r = static_cast<unsigned>(w) - k * per_page;
    } else {
      k = static_cast<unsigned>(w / per_page);
      r = static_cast<unsigned>(w - static_cast<long long>(k) * per_page);
    }
    const unsigned half = r / pieces, piece = r - half * pieces;  // (layer, pool)
    uint8_t* base = ((half & 1) ? p.pool[1] : p.pool[0]) + (half >> 1) * p.layer_stride;
    const long long at = static_cast<long long>(piece) * kCopyBytes + lane * 16;
    const uint8_t* src = base + from[k] * p.page_stride + at;
    uint8_t* dst = base + to[k] * p.page_stride + at;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 512 < p.page_bytes) v[i] = *reinterpret_cast<const uint4*>(src + i * 512);
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 512 < p.page_bytes) *reinterpret_cast<uint4*>(dst + i * 512) = v[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyParams p) {
  paged::grid_wait();
  paged::grid_launch_dependents();
  constexpr int W = kCopyThreads / 32;
  copy_pages(p, p.from, p.to, *p.n_copies, static_cast<long long>(blockIdx.x) * W + threadIdx.x / 32,
             static_cast<long long>(gridDim.x) * W);
}

// Exclusive prefix of v over the block's threads; *total gets the sum. `red`
// holds 33 words.
__device__ __forceinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // red's last use
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[31];
  return x - v + (warp > 0 ? red[warp - 1] : 0);
}

struct Params {
  const int* table;  // [B][width]
  const int* lens;
  const int* refs;   // [P]
  const int* source;
  const int* add;
  int* table_out;
  int* lens_out;
  int* refs_out;
  int* info;      // [2]
  int B, width, P, page_log2;
  // workspace
  int* keeper;    // [B]: update: the row (-1: the source itself) that keeps a source's last page
  int* need_off;  // [B + 1]: update: prefix of the fresh pages of each row
  int* counts;    // [kCtas]: free pages of each CTA's share
  int* list;      // [P]: free pages in order; compact: destination of move k
  int* from;      // [max(B, P)] sources, and
  int* to;        // destinations of the copies
  int* n_copies;  // [1]
};

__device__ __forceinline__ int ceil_pages(int len, int log2) {
  return static_cast<int>((static_cast<long long>(len) + (1 << log2) - 1) >> log2);
}

// Is there a page? An entry of -1 inside a row is one that the row has given up
// (a page in front of a sliding window); any other id outside the pool is
// reported. Neither is followed. (The kernel for small caches asks in place: with
// this function its loops over the tables took 10.1 us for 64 rows and 10,544
// pages, as nested conditions 9.5.)
__device__ __forceinline__ bool held_page(int page, const Params& p) {
  if (page >= 0 && page < p.P) return true;
  if (page != -1) paged::bad(paged::kBadPage);
  return false;
}

// One row of an update: what it goes on from and what it keeps.
struct Row {
  int s;      // source row, -1: none
  int L;      // its tokens
  int longer; // tokens after growing
  int held;   // pages of the source
  int kept;   // pages of them that this row keeps as they are
  int want;   // pages after growing
  bool copy;  // the source's last page is copied into this row's first fresh page
};

__device__ __forceinline__ int clamp_len(int l, const Params& p) {
  const long long cap = static_cast<long long>(p.width) << p.page_log2;
  return static_cast<int>(min(static_cast<long long>(max(l, 0)), cap));
}

__device__ __forceinline__ Row row_of(const Params& p, int b) {
  Row r;
  const int s = p.source[b];
  r.s = (s >= 0 && s < p.B) ? s : -1;
  r.L = r.s >= 0 ? clamp_len(p.lens[r.s], p) : 0;
  const long long longer = static_cast<long long>(r.L) + max(p.add[b], 0);
  r.longer = static_cast<int>(min(longer, static_cast<long long>(INT_MAX)));
  r.held = ceil_pages(r.L, p.page_log2);
  r.want = ceil_pages(r.longer, p.page_log2);
  const int full = r.L >> p.page_log2;
  const bool keeps = r.s >= 0 && ld(p.keeper + r.s) == (r.s == b ? -1 : b);
  r.kept = keeps ? r.held : full;
  r.copy = r.held > r.kept;
  return r;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_update_kernel(const Params p) {
  __shared__ int red[33];
  const int rank = cta_rank(), tid = threadIdx.x;
  const int all = kCtas * kThreads, me = rank * kThreads + tid;
  const int lane = tid & 31, wid = me >> 5, warps = all >> 5;
  paged::grid_wait();
  paged::grid_launch_dependents();

  // 1. The outputs start as the inputs; no row keeps a last page yet.
  for (int i = me; i < p.P; i += all) st(p.refs_out + i, p.refs[i]);
  for (int b = me; b < p.B; b += all) st(p.keeper + b, INT_MAX);
  if (me == 0) st(p.n_copies, 0);
  cluster_barrier();

  // 2. Every row lets go of its pages; the rows that take a source over find
  // out which of them keeps its last page.
  for (int b = wid; b < p.B; b += warps) {
    const int len = p.lens[b], L = clamp_len(len, p), n = ceil_pages(L, p.page_log2);
    if (lane == 0) {
      if (len > L) paged::bad(paged::kBadLength);
      const int s = p.source[b];
      if (s >= 0 && s < p.B)
        atomicMin(p.keeper + s, s == b ? -1 : b);
      else if (s != -1)
        paged::bad(paged::kBadSource);
    }
    for (int j = lane; j < n; j += 32) {
      const int page = p.table[static_cast<size_t>(b) * p.width + j];
      if (held_page(page, p)) atomicAdd(p.refs_out + page, -1);
    }
  }
  cluster_barrier();

  // 3. Every row holds the pages that it keeps. CTA 0 meanwhile sums up the
  // fresh pages that the rows need.
  for (int b = wid; b < p.B; b += warps) {
    const Row r = row_of(p, b);
    for (int j = lane; j < r.kept; j += 32) {
      const int page = p.table[static_cast<size_t>(r.s) * p.width + j];
      if (page >= 0 && page < p.P) atomicAdd(p.refs_out + page, 1);
    }
  }
  if (rank == 0) {
    int too_long = 0, sum = 0;
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    for (int b = b0; b < b1; ++b) {
      const Row r = row_of(p, b);
      if (r.want > p.width)
        ++too_long;  // the row's tokens do not fit its table
      else
        sum += r.want - r.kept;
    }
    int total, longs;
    block_scan(too_long, red, &longs);
    int run = block_scan(sum, red, &total);
    for (int b = b0; b < b1; ++b) {
      const Row r = row_of(p, b);
      st(p.need_off + b, run);
      if (r.want <= p.width) run += r.want - r.kept;
    }
    if (tid == 0) {
      st(p.need_off + p.B, total);
      st(p.info + 1, longs);
    }
  }
  cluster_barrier();

  // 4. Free pages, counted per thread's share of the pool.
  const int per = (p.P + all - 1) / all;
  const int p0 = static_cast<int>(min(static_cast<long long>(p.P), static_cast<long long>(me) * per));
  const int p1 = min(p.P, p0 + per);
  int mine = 0, cta_total;
  for (int i = p0; i < p1; ++i) mine += ld(p.refs_out + i) <= 0;
  int at = block_scan(mine, red, &cta_total);
  if (tid == 0) st(p.counts + rank, cta_total);
  cluster_barrier();
  int free_all = 0;
  for (int r = 0; r < kCtas; ++r) {
    const int c = ld(p.counts + r);
    if (r < rank) at += c;
    free_all += c;
  }
  const int need = ld(p.need_off + p.B);
  const bool refused = need > free_all || ld(p.info + 1) > 0;
  if (me == 0) st(p.info, max(need - free_all, 0));
  if (!refused)
    for (int i = p0; i < p1 && at < need; ++i)
      if (ld(p.refs_out + i) <= 0) st(p.list + at++, i);
  cluster_barrier();

  // 5. The new tables.
  for (int b = wid; b < p.B; b += warps) {
    const Row r = row_of(p, b);
    int* out = p.table_out + static_cast<size_t>(b) * p.width;
    if (refused) {  // everything stays as it was
      const int* in = p.table + static_cast<size_t>(b) * p.width;
      for (int j = lane; j < p.width; j += 32) out[j] = in[j];
      if (lane == 0) p.lens_out[b] = p.lens[b];
      continue;
    }
    const int first = ld(p.need_off + b);
    const int* in = p.table + static_cast<size_t>(max(r.s, 0)) * p.width;
    for (int j = lane; j < p.width; j += 32) {
      int page = -1;
      if (j < r.kept) {
        page = in[j];
      } else if (j < r.want) {
        page = ld(p.list + first + j - r.kept);
        st(p.refs_out + page, 1);
        if (r.copy && j == r.kept) {
          const int of = in[j];
          if (of >= 0 && of < p.P) {
            const int k = atomicAdd(p.n_copies, 1);
            p.from[k] = of;
            p.to[k] = page;
          }
        }
      }
      out[j] = page;
    }
    if (lane == 0) p.lens_out[b] = r.longer;
  }
  if (refused)
    for (int i = me; i < p.P; i += all) st(p.refs_out + i, p.refs[i]);
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_compact_kernel(const Params p) {
  __shared__ int red[33];
  const int rank = cta_rank(), tid = threadIdx.x;
  const int all = kCtas * kThreads, me = rank * kThreads + tid;
  const int lane = tid & 31, wid = me >> 5, warps = all >> 5;
  paged::grid_wait();
  paged::grid_launch_dependents();

  // 1. Live pages of each thread's share of the pool.
  const int per = (p.P + all - 1) / all;
  const int p0 = static_cast<int>(min(static_cast<long long>(p.P), static_cast<long long>(me) * per));
  const int p1 = min(p.P, p0 + per);
  int mine = 0, cta_total;
  for (int i = p0; i < p1; ++i) mine += p.refs[i] > 0;
  int at = block_scan(mine, red, &cta_total);
  if (tid == 0) st(p.counts + rank, cta_total);
  cluster_barrier();
  int n = 0;
  for (int r = 0; r < kCtas; ++r) {
    const int c = ld(p.counts + r);
    if (r < rank) at += c;
    n += c;
  }
  // 2. The live pages before n; the others move. `at` counts the live pages
  // before this share.
  if (n == p.P) {
    if (me == 0) st(p.n_copies, 0);
  } else if (p0 <= n && n < p1) {
    int before = at;
    for (int i = p0; i < n; ++i) before += p.refs[i] > 0;
    st(p.n_copies, n - before);
  }
  cluster_barrier();
  const int moves = ld(p.n_copies), below = n - moves;  // live pages that stay
  for (int i = p0; i < p1; ++i) {
    const bool live = p.refs[i] > 0;
    if (i < n && !live) st(p.to + (i - at), i);           // hole number i - (live before i)
    if (i >= n && live) {
      st(p.from + (at - below), i);
      st(p.list + i, at - below);  // which move takes page i
    }
    if (live && i < n) st(p.refs_out + i, p.refs[i]);
    if (i >= n) st(p.refs_out + i, 0);
    at += live;
  }
  cluster_barrier();
  // 3. Counts of the moved pages, and the tables.
  for (int k = me; k < moves; k += all) st(p.refs_out + ld(p.to + k), p.refs[ld(p.from + k)]);
  for (int b = wid; b < p.B; b += warps) {
    const int len = p.lens[b], L = clamp_len(len, p), held = ceil_pages(L, p.page_log2);
    if (lane == 0 && len > L) paged::bad(paged::kBadLength);
    for (int j = lane; j < p.width; j += 32) {
      const size_t e = static_cast<size_t>(b) * p.width + j;
      int page = -1;
      if (j < held) {
        page = p.table[e];
        if (held_page(page, p)) {
          if (p.refs[page] <= 0)
            paged::bad(paged::kBadPage);  // (left as it was)
          else if (page >= n)
            page = ld(p.to + ld(p.list + page));
        }
      }
      p.table_out[e] = page;
    }
  }
  if (me == 0) {
    p.info[0] = n;
    p.info[1] = moves;
  }
}

// ------------------------------------------------------------------ one kernel
// The same two operations with the counts in every CTA's shared memory.

// Words of dynamic shared memory.
inline size_t update_small_words(int B, int P) {
  return 2 * static_cast<size_t>(P) + 9 * static_cast<size_t>(B) + 1;
}
inline size_t compact_small_words(int P) { return 2 * static_cast<size_t>(P); }

// Calls f(i, rank) for the entries i of [0, n) where pick(i) holds, rank being
// their number in order, as long as it is below `most`; returns how many there
// are in all. A warp takes a contiguous share, 32 entries at a time. `red`
// holds 33 words.
template <typename Pick, typename F>
__device__ __forceinline__ int each_in_order(int n, int* red, int most, Pick pick, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = (n + kThreads - 1) / kThreads * 32;
  const int i0 = min(n, warp * share), i1 = min(n, i0 + share);
  int mine = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) mine += pick(i) ? 1 : 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();  // red's last use
  if (lane == 0) red[warp] = mine;
  __syncthreads();
  const int v = red[lane];
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  int at = __shfl_sync(0xffffffffu, x - v, warp);
  const int all = __shfl_sync(0xffffffffu, x, 31);
  for (int i = i0 + lane; i - lane < i1 && at < most; i += 32) {
    const bool p = i < i1 && pick(i);
    const unsigned m = __ballot_sync(0xffffffffu, p);
    const int k = at + __popc(m & ((1u << lane) - 1));
    if (p && k < most) f(i, k);
    at += __popc(m);
  }
  return all;
}

// Of a row that k rows go on from, the counts of the full pages change by k - 1,
// that of the last, partly filled page by -1 if k = 0. Rows that just go on
// (k = 1) need not be read for that.
__global__ void __launch_bounds__(kThreads, 1)
    pages_update_small_kernel(const Params p, const CopyParams cp) {
  extern __shared__ int sm[];
  __shared__ int red[33];
  __shared__ int s_long;
  int* refs = sm;               // [P]
  int* list = refs + p.P;       // [P] free pages in order
  int* len = list + p.P;        // [B]
  int* src = len + p.B;         // [B]
  int* longer = src + p.B;      // [B]
  int* keeper = longer + p.B;   // [B]
  int* takers = keeper + p.B;   // [B]
  int* kept = takers + p.B;     // [B]
  int* from = kept + p.B;       // [B] copies
  int* to = from + p.B;         // [B]
  int* first = to + p.B;        // [B + 1] fresh pages before each row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int me = blockIdx.x * (kThreads / 32) + warp, warps = gridDim.x * (kThreads / 32);
  paged::grid_wait();
  paged::grid_launch_dependents();

  for (int b = tid; b < p.B; b += kThreads) {
    const int l = p.lens[b], L = clamp_len(l, p), s = p.source[b];
    if (l > L) paged::bad(paged::kBadLength);
    if (s < -1 || s >= p.B) paged::bad(paged::kBadSource);
    len[b] = L;
    src[b] = s >= 0 && s < p.B ? s : -1;
    longer[b] = max(p.add[b], 0);  // (with the source's tokens below)
    keeper[b] = INT_MAX;
    takers[b] = 0;
  }
#pragma unroll 4
  for (int i = tid; i < p.P; i += kThreads) refs[i] = p.refs[i];
  if (tid == 0) s_long = 0;
  __syncthreads();

  for (int b = tid; b < p.B; b += kThreads) {
    const int s = src[b];
    if (s < 0) continue;
    atomicAdd(takers + s, 1);
    atomicMin(keeper + s, s == b ? -1 : b);
  }
  __syncthreads();

  for (int b = warp; b < p.B; b += kThreads / 32) {
    const int k = takers[b];
    if (k == 1) continue;
    const int full = len[b] >> p.page_log2, held = ceil_pages(len[b], p.page_log2);
    for (int j = lane; j < held; j += 32) {
      const int d = j < full ? k - 1 : k > 0 ? 0 : -1;
      const int page = p.table[static_cast<size_t>(b) * p.width + j];
      if (page < 0 || page >= p.P) {
        if (page != -1) paged::bad(paged::kBadPage);
      } else if (d != 0) {
        atomicAdd(refs + page, d);
      }
    }
  }
  // What each row keeps and needs, a few rows a thread.
  const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int sum = 0, need;
  for (int b = b0; b < b1; ++b) {
    const int s = src[b], L = s >= 0 ? len[s] : 0;
    const bool keeps = s >= 0 && keeper[s] == (s == b ? -1 : b);
    kept[b] = keeps ? ceil_pages(L, p.page_log2) : L >> p.page_log2;
    const long long n = static_cast<long long>(L) + longer[b];
    longer[b] = static_cast<int>(min(n, static_cast<long long>(INT_MAX)));
    const int want = ceil_pages(longer[b], p.page_log2);
    if (want > p.width)
      atomicAdd(&s_long, 1);
    else
      sum += want - kept[b];
  }
  int run = block_scan(sum, red, &need);
  for (int b = b0; b < b1; ++b) {
    first[b] = run;
    const int want = ceil_pages(longer[b], p.page_log2);
    if (want <= p.width) run += want - kept[b];
  }
  __syncthreads();
  const int n_free = each_in_order(
      p.P, red, need, [&](int i) { return refs[i] <= 0; }, [&](int i, int k) { list[k] = i; });
  const bool refused = need > n_free || s_long > 0;
  __syncthreads();

  // The tables, 32 entries of a row a warp at a time over the whole grid.
  const int blocks = (p.width + 31) / 32;
  for (int u = me; u < p.B * blocks; u += warps) {
    const int b = u / blocks, j = (u - b * blocks) * 32 + lane;
    const size_t row = static_cast<size_t>(b) * p.width;
    if (j == 0) p.lens_out[b] = refused ? p.lens[b] : longer[b];
    if (j >= p.width) continue;
    int page = -1;
    if (refused) {  // everything stays as it was
      page = p.table[row + j];
    } else if (j < kept[b]) {
      page = p.table[static_cast<size_t>(max(src[b], 0)) * p.width + j];
      if (page < 0 || page >= p.P)
        if (page != -1) paged::bad(paged::kBadPage);
    } else if (j < ceil_pages(longer[b], p.page_log2)) {
      page = list[first[b] + j - kept[b]];
    }
    p.table_out[row + j] = page;
  }
  if (refused) {
    for (int i = blockIdx.x * kThreads + tid; i < p.P; i += gridDim.x * kThreads)
      p.refs_out[i] = p.refs[i];
  } else {
    for (int k = tid; k < need; k += kThreads) refs[list[k]] = 1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.info[0] = max(need - n_free, 0);
    p.info[1] = s_long;
  }
  if (refused) return;
  // The copies, in the order of the rows.
  const int copies = each_in_order(
      p.B, red, p.B,
      [&](int b) { return src[b] >= 0 && ceil_pages(len[src[b]], p.page_log2) > kept[b]; },
      [&](int b, int k) {
        const int of = p.table[static_cast<size_t>(src[b]) * p.width + kept[b]], page = list[first[b]];
        from[k] = of >= 0 && of < p.P ? of : page;  // (no page there: nothing to copy)
        to[k] = page;
      });
  __syncthreads();
  for (int i = blockIdx.x * kThreads + tid; i < p.P; i += gridDim.x * kThreads)
    p.refs_out[i] = refs[i];
  copy_pages(cp, from, to, copies, me, warps);
}

__global__ void __launch_bounds__(kThreads, 1)
    pages_compact_small_kernel(const Params p, const CopyParams cp) {
  extern __shared__ int sm[];
  __shared__ int red[33];
  int* refs = sm;              // [P]
  int* to = refs + p.P;        // [P / 2] free pages below n in order
  int* from = to + p.P / 2;    // [P / 2] live pages from n on in order
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int me = blockIdx.x * (kThreads / 32) + warp, warps = gridDim.x * (kThreads / 32);
  paged::grid_wait();
  paged::grid_launch_dependents();
  int live = 0, n;
#pragma unroll 4
  for (int i = tid; i < p.P; i += kThreads) {
    const int r = max(p.refs[i], 0);  // (negative counts are free pages, too)
    refs[i] = r;
    live += r > 0;
  }
  block_scan(live, red, &n);
  __syncthreads();
  // The k-th live page from n on takes the k-th hole below n; there are as many
  // of both, so not more than P / 2.
  const int moves = each_in_order(
      n, red, p.P, [&](int i) { return refs[i] <= 0; }, [&](int i, int k) { to[k] = i; });
  __syncthreads();
  each_in_order(
      p.P - n, red, p.P, [&](int i) { return refs[n + i] > 0; },
      [&](int i, int k) {
        from[k] = n + i;
        refs[to[k]] = refs[n + i];
        refs[n + i] = ~to[k];  // negative: it moves to to[k]
      });
  __syncthreads();
  for (int i = blockIdx.x * kThreads + tid; i < p.P; i += gridDim.x * kThreads)
    p.refs_out[i] = i < n ? refs[i] : 0;
  const int blocks = (p.width + 31) / 32;
  for (int u = me; u < p.B * blocks; u += warps) {
    const int b = u / blocks, j = (u - b * blocks) * 32 + lane;
    const int l = p.lens[b], L = clamp_len(l, p);
    if (j == 0 && l > L) paged::bad(paged::kBadLength);
    if (j >= p.width) continue;
    const size_t e = static_cast<size_t>(b) * p.width + j;
    int page = -1;
    if (j < ceil_pages(L, p.page_log2)) {
      page = p.table[e];
      if (held_page(page, p)) {
        if (p.refs[page] <= 0)
          paged::bad(paged::kBadPage);  // (left as it was)
        else if (page >= n)
          page = ~refs[page];
      }
    }
    p.table_out[e] = page;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.info[0] = n;
    p.info[1] = moves;
  }
  copy_pages(cp, from, to, moves, me, warps);
}

}  // namespace pages
}  // namespace eta
