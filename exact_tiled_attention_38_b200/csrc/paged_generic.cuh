// Attention of new tokens over a paged cache on CUDA cores, in fp32: the head
// sizes above 128 and the groups above 128 query heads per KV head that the
// tensor-core kernel does not take (any d that is a multiple of 8, to 256).
//
// For the new token i of sequence b and query head h of KV head g:
//     s_j = scale q_i . k_j for the visible keys j <= L - T + i (and, with a
//     window, j > L - T + i - window);  o = sum_j softmax_j(s) v_j;
//     lse = ln sum_j exp(s_j);  no visible key: o = 0, lse = -inf.
//
// A CTA of 4 warps owns 16 query rows (4 a warp) of one sequence and KV head,
// the rows being (token, head of the group) pairs, so that the group shares
// each key it reads. Tiles of 32 keys of the pages go to shared memory, and
// each row keeps a running maximum and sum. Like the generic kernel over
// contiguous tensors it is far from the tensor-core kernel's speed.
#pragma once

#include "generic_fwd.cuh"
#include "paged_common.cuh"

namespace eta {
namespace paged {

struct GParams {
  const void* q;
  long long q_stride;  // elements between tokens
  Cache cache;
  const int* cu_q;
  const int* lens;
  void* o;
  float* lse;
  int B, Hq, G, total_q, max_q, window;
  float scale_log2;
};

template <typename T>
__global__ void __launch_bounds__(generic::kThreads) attn_paged_generic_kernel(const GParams p) {
  using generic::kRows;
  using generic::kRowsPerWarp;
  using generic::kThreads;
  using generic::kTK;
  extern __shared__ __align__(16) uint8_t smem[];
  const Cache& c = p.cache;
  const int d = c.d, stride = generic::row_stride(d), nchunk = d / 8;
  uint8_t* sK = smem;
  uint8_t* sV = smem + kTK * stride;
  T* sQ = reinterpret_cast<T*>(smem + 2 * kTK * stride);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long bg = static_cast<long long>(blockIdx.z) * generic::kGridY + blockIdx.y;
  if (bg >= static_cast<long long>(p.B) * c.Hkv) return;
  const int b = static_cast<int>(bg / c.Hkv), g = static_cast<int>(bg - static_cast<long long>(b) * c.Hkv);
  const Seq s = load_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, c.capacity());
  if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0)
    check_seq(p.cu_q, p.lens, b, p.total_q, p.max_q, c.capacity());
  const long long rows = static_cast<long long>(s.T) * p.G;
  const long long r0 = static_cast<long long>(blockIdx.x) * kRows;
  if (r0 >= rows) return;
  const int off = s.L - s.T;  // position of token 0

  auto row_ptr = [&](long long r) {  // element offset of row r's head in a [.., Hq, d] row
    return static_cast<size_t>(g * p.G + r % p.G) * d;
  };
  for (int i = threadIdx.x; i < kRows * nchunk; i += kThreads) {
    const int rr = i / nchunk, u = i - rr * nchunk;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + rr < rows)
      v = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.q) +
                                          (s.q0 + (r0 + rr) / p.G) * p.q_stride + row_ptr(r0 + rr) +
                                          u * 8);
    *reinterpret_cast<uint4*>(sQ + rr * d + u * 8) = v;
  }
  const long long rl = min(r0 + kRows, rows) - 1;
  const int khi = min(off + static_cast<int>(rl / p.G), s.L - 1);
  const int klo = first_seen(s, static_cast<int>(r0 / p.G), p.window);  // (for any row here)

  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][8];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[i][e] = 0.f;
  }
  const int* table = c.table + static_cast<size_t>(b) * c.width;
  for (int kv0 = klo / kTK * kTK; kv0 <= khi; kv0 += kTK) {
    __syncthreads();  // the previous tile is no longer read
    for (int i = threadIdx.x; i < kTK * nchunk; i += kThreads) {
      const int j = i / nchunk, u = i - j * nchunk;
      const int key = kv0 + j;
      uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
      if (key >= klo && key < s.L) {
        const int page = table[key >> c.page_log2];
        if (page >= 0 && page < c.num_pages) {
          const size_t at = page * c.page_stride + g * c.head_stride +
                            (key & ((1 << c.page_log2) - 1)) * c.token_stride + u * 8;
          kv = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(c.k) + at);
          vv = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(c.v) + at);
        } else if (u == 0) {
          bad(kBadPage);
        }
      }
      *reinterpret_cast<uint4*>(sK + j * stride + u * 16) = kv;
      *reinterpret_cast<uint4*>(sV + j * stride + u * 16) = vv;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const long long r = r0 + warp * kRowsPerWarp + i;
      if (r >= rows) continue;  // warp-uniform
      const int pos = off + static_cast<int>(r / p.G);
      const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float x = 0.f;
      const T* qrow = sQ + (warp * kRowsPerWarp + i) * d;
      for (int u = 0; u < nchunk; ++u) {
        float qf[8], kf[8];
        generic::to_f32x8<T>(*reinterpret_cast<const uint4*>(qrow + u * 8), qf);
        generic::to_f32x8<T>(*reinterpret_cast<const uint4*>(sK + lane * stride + u * 16), kf);
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaf(qf[e], kf[e], x);
      }
      const int key = kv0 + lane;
      x = (key >= lo && key <= pos) ? x * p.scale_log2 : -INFINITY;
      const float m_new = fmaxf(m[i], generic::warp_max(x));
      // No visible key for this row yet, or none whose score is above -inf. (The
      // maximum leaves NaN out; such scores go into the sum, which they make NaN.)
      if (m_new == -INFINITY && !__any_sync(0xffffffffu, isnan(x))) continue;
      const float alpha = exp2f(m[i] - m_new);  // m = -inf gives 0
      const float pj = exp2f(x - m_new);
      l[i] = l[i] * alpha + generic::warp_sum(pj);
      m[i] = m_new;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[i][e] *= alpha;
      for (int j = 0; j < kTK; ++j) {
        const float pb = __shfl_sync(0xffffffffu, pj, j);  // every lane takes part
        if (pb != 0.f && lane < nchunk) {  // a masked key's value is not touched (it may be NaN)
          float vf[8];
          generic::to_f32x8<T>(*reinterpret_cast<const uint4*>(sV + j * stride + lane * 16), vf);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[i][e] = fmaf(pb, vf[e], o[i][e]);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const long long r = r0 + warp * kRowsPerWarp + i;
    if (r >= rows) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const size_t token = static_cast<size_t>(s.q0 + r / p.G);
    if (lane < nchunk) {
      uint4 w;
      w.x = generic::pack_pair<T>(o[i][0] * inv, o[i][1] * inv);
      w.y = generic::pack_pair<T>(o[i][2] * inv, o[i][3] * inv);
      w.z = generic::pack_pair<T>(o[i][4] * inv, o[i][5] * inv);
      w.w = generic::pack_pair<T>(o[i][6] * inv, o[i][7] * inv);
      *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.o) + token * p.Hq * d + row_ptr(r) +
                                lane * 8) = w;
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[token * p.Hq + g * p.G + r % p.G] =
          l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994531f;
  }
}

}  // namespace paged
}  // namespace eta
