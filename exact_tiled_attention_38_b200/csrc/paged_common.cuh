// What the paged-cache kernels share: the cache's layout as a kernel sees it,
// a batch's sequences, and the status codes of bad tables and lengths.
//
// Sequence b has T_b new tokens (rows cu_q[b] .. cu_q[b + 1] of the packed
// tensors) and L_b cached tokens in all, the new ones included, so its new
// token i is at position L_b - T_b + i. Position t lies in page
// table[b][t / page_size], row t % page_size; element (page, head, row, c) of a
// pool is at page * page_stride + head * head_stride + row * token_stride + c.
//
// Nothing read from device memory is trusted as an index: lengths are clamped
// to what the table can hold, row ranges to the packed tensors, and a page id
// outside [0, num_pages) is never followed. Each such case records a status.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"

namespace eta {
namespace paged {

// Device status codes of bad cache descriptions (common.cuh holds the word).
constexpr unsigned kStatusPages = 0x2000u;
enum : unsigned {
  kBadPage = 1,    // a page id outside [0, num_pages) in the range a sequence needs
  kBadLength = 2,  // a cached length above the table's width * page_size
  kBadRows = 3,    // row offsets that decrease, leave [0, total_q] or exceed max_q
  kBadSource = 4,  // a source row outside [-1, B)
};

__device__ __forceinline__ void bad(unsigned what) { record_status(kStatusPages | what); }

// Programmatic dependent launch (see the decode kernels): wait for the kernel
// before this one on the stream, and let the one after it start its set-up.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct Cache {
  void* k;
  void* v;
  const int* table;       // [B][width]
  long long page_stride;  // elements
  long long head_stride;
  long long token_stride;
  int num_pages;
  int page_log2;  // page_size = 1 << page_log2
  int width;      // entries of a table row
  int Hkv;
  int d;

  __host__ __device__ __forceinline__ long long capacity() const {
    return static_cast<long long>(width) << page_log2;
  }
};

// One sequence of the batch: T new tokens at rows q0 .. q0 + T of the packed
// tensors, L cached tokens; token i is at position L - T + i.
struct Seq {
  int q0, T, L;
};

__device__ __forceinline__ Seq load_seq(const int* __restrict__ cu_q, const int* __restrict__ lens,
                                        int b, int total_q, int max_q, long long capacity) {
  Seq s;
  const int a = cu_q[b], e = cu_q[b + 1], l = lens[b];
  s.q0 = min(max(a, 0), total_q);
  s.T = min(min(max(e, s.q0), total_q) - s.q0, max_q);
  s.L = static_cast<int>(min(static_cast<long long>(max(l, 0)), capacity));
  return s;
}

// The first key that new token t of the sequence, and so any from t on, sees.
__device__ __forceinline__ int first_seen(const Seq& s, int t, int window) {
  return window > 0 ? max(0, s.L - s.T + t - window + 1) : 0;
}

// Records what load_seq() had to clamp (called once per sequence).
__device__ __forceinline__ void check_seq(const int* __restrict__ cu_q,
                                          const int* __restrict__ lens, int b, int total_q,
                                          int max_q, long long capacity) {
  const int a = cu_q[b], e = cu_q[b + 1];
  if (a < 0 || e < a || e > total_q || e - a > max_q) bad(kBadRows);
  if (lens[b] > capacity) bad(kBadLength);
}

// The sequence that holds packed row `row`: the last b with cu_q[b] <= row
// (rows of empty sequences are skipped), found by the whole warp, 32 pivots a
// round. Returns -1 for a row outside every sequence.
__device__ __forceinline__ int find_seq(const int* __restrict__ cu_q, int B, int row, int lane) {
  int lo = 0, n = B + 1;  // candidates cu_q[lo .. lo + n): the count of entries <= row
  int below = 0;          // entries known to be <= row
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + min((lane + 1) * step, n) - 1;  // last entry of this lane's share
    const bool le = lane * step < n && cu_q[at] <= row;
    const int full = __popc(__ballot_sync(0xffffffffu, le));  // shares wholly <= row (sorted)
    below = lo + min(full * step, n);
    if (step == 1 || full * step >= n) break;
    lo = below;
    n = min(step, n - full * step) - 1;  // the share's last entry is known to be > row
  }
  const int b = below - 1;
  return (b >= 0 && b < B) ? b : -1;
}

// 4-D tiled load of one box, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace paged
}  // namespace eta
