// Rotary positions, and their fusion with the append to a paged cache.
//
// Pair p of a head (of the first `rot` of its d values: values p and
// p + rot / 2, or 2p and 2p + 1 when interleaved) at position n is turned by
// the angle 2 pi n f_p and scaled by `amp`:
//     y_a = amp (x_a cos - x_b sin),   y_b = amp (x_b cos + x_a sin);
// the other d - rot values pass through. The gradient of that map is its
// transpose: the same with the angle negated.
//
// f_p comes as turns per position (angle / 2 pi) in 64 bits, and n f_p is
// formed and reduced to [-1/2, 1/2] turns in 64 bits: at position 10^6 a 32-bit
// product would be off by 0.03 rad. What is left is exact to 2^-25 turns in 32
// bits, and sincospif takes it from there. The rotation runs in 32 bits and
// rounds once, to the type of the output.
//
// Bound by memory: every value is read once and written once. A CTA takes a
// few tokens and some of their heads: the first heads' values are loaded, the
// tokens' cosines and sines go to shared memory, then each thread keeps the
// eight pairs of its place in the row in registers and goes through the heads
// with 16-byte loads. Measured on B200, of the 6554 GB/s of a copy: q and k of
// 4 x 16 + 16 heads x 2048 x 128 24.9 us (0.82; all launches of this length
// lose about 4 us at both ends), 32 + 8 heads x 32768 x 64 55.7 us (0.92), an
// append of 9 chunks of up to 1801 tokens 50.9 us (0.86).
#pragma once

#include "paged_common.cuh"

namespace eta {
namespace rope {

constexpr int kThreads = 256;
constexpr int kSlots = 64;                    // (token, unit) places of a CTA
constexpr int kGroups = kThreads / kSlots;    // threads that share a place, by heads
constexpr int kMaxTokens = 32;                // tokens of a CTA
constexpr int kHeadsAtOnce = 2;               // heads a thread loads before it stores any

struct Tensor {
  const void* x;
  void* y;
  long long xb, xh, xn;  // strides in elements: batch, head, token
  long long yb, yh, yn;
};

struct Params {
  Tensor t[2];  // q, k
  int H[2];
  int heads;    // H[0] + H[1] (and the value heads of an append)
  const int* pos;
  long long pos_b;      // stride of pos between batches (0: shared)
  const double* turns;  // [rot / 2]
  float amp;
  float sign;  // -1: the gradient
  int N;       // tokens of a batch
  long long tokens;  // B * N, or the packed rows of an append
  int d, rot;
  int units;        // places of a row: rot / 16 pair units, then 16 values each that pass
  int tokens_per_cta;
  int heads_per_cta;
  // append
  paged::Cache cache;
  const void* v;
  long long vh, vn;
  const int* cu_q;
  const int* lens;
  int B;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                    pack2<T>(f[6], f[7]));
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}

// Where one head of one token is read and written (y NULL: nowhere).
template <typename T>
struct Row {
  const T* x;
  T* y;
  bool turn;
};

// What a token needs besides its row of tensors, found once per CTA.
struct Place {
  long long page;  // element offset of its page row (append), -1: not stored
  int angle_pos;
};

template <typename T, bool APPEND>
__device__ __forceinline__ Row<T> row_of(const Params& p, long long token, int head, long long page) {
  Row<T> r;
  r.turn = true;
  if constexpr (APPEND) {
    if (head < p.H[0]) {
      r.x = reinterpret_cast<const T*>(p.t[0].x) + token * p.t[0].xn + head * p.t[0].xh;
      r.y = reinterpret_cast<T*>(p.t[0].y) + token * p.t[0].yn + head * p.t[0].yh;
      return r;
    }
    int g = head - p.H[0];
    const bool value = g >= p.H[1];
    if (value) g -= p.H[1];
    r.turn = !value;
    r.x = value ? reinterpret_cast<const T*>(p.v) + token * p.vn + g * p.vh
                : reinterpret_cast<const T*>(p.t[1].x) + token * p.t[1].xn + g * p.t[1].xh;
    T* pool = reinterpret_cast<T*>(value ? p.cache.v : p.cache.k);
    r.y = page < 0 ? nullptr : pool + page + g * p.cache.head_stride;
  } else {
    const int w = head < p.H[0] ? 0 : 1;
    const int h = w ? head - p.H[0] : head;
    const long long b = token / p.N, n = token - b * p.N;
    const Tensor& t = p.t[w];
    r.x = reinterpret_cast<const T*>(t.x) + b * t.xb + h * t.xh + n * t.xn;
    r.y = reinterpret_cast<T*>(t.y) + b * t.yb + h * t.yh + n * t.yn;
  }
  return r;
}

// VEC: rot is a multiple of 16 (units of eight pairs); otherwise the rotated
// part goes pair by pair.
template <typename T, bool APPEND, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* table = reinterpret_cast<float2*>(smem);  // [tokens][rot / 2] (cos, sin) times amp
  __shared__ Place place[kMaxTokens];
  const int half = p.rot / 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long first = static_cast<long long>(blockIdx.x) * p.tokens_per_cta;
  const int count = static_cast<int>(min(static_cast<long long>(p.tokens_per_cta), p.tokens - first));
  paged::grid_wait();  // (launched as a programmatic dependent: see launch_dependent)
  paged::grid_launch_dependents();
  const int h0 = blockIdx.y * p.heads_per_cta;
  const int h1 = min(h0 + p.heads_per_cta, p.heads);

  // This thread's place in a row: token t, the two 8-value pieces at c0 and c1.
  const int slot = tid % kSlots;
  const int t_mine = VEC ? slot / p.units : 0, u_mine = slot - t_mine * p.units;
  const int nrot = p.rot >> 4;
  const bool turned = u_mine < nrot;
  const int c0 = !turned ? p.rot + (u_mine - nrot) * 16 : INTERLEAVED ? u_mine * 16 : u_mine * 8;
  const int c1 = turned && !INTERLEAVED ? c0 + half : c0 + 8;
  const bool mine = VEC && t_mine < count, second = c1 < p.d;
  uint4 a[kHeadsAtOnce], b[kHeadsAtOnce];
  auto load = [&](int h) {  // the pieces of heads h, h + kGroups, ...
#pragma unroll
    for (int i = 0; i < kHeadsAtOnce; ++i) {
      if (h + i * kGroups >= h1) break;
      const Row<T> r = row_of<T, APPEND>(p, first + t_mine, h + i * kGroups, 0);
      a[i] = *reinterpret_cast<const uint4*>(r.x + c0);
      if (second) b[i] = *reinterpret_cast<const uint4*>(r.x + c1);
    }
  };
  // The first heads' values are on their way while the angles are worked out.
  if (mine) load(h0 + tid / kSlots);

  if constexpr (APPEND) {
    // The batch is checked while the values are on their way, by the first CTAs of
    // the last heads (64 tokens, device time: 3.68 us, as without the check; by those
    // of the first heads 3.86 us, at the kernel's end 4.07 us).
    const unsigned check_ctas = min(gridDim.x, 64u);
    if (blockIdx.y == gridDim.y - 1 && blockIdx.x < check_ctas) {
      const int total = static_cast<int>(p.tokens);
      for (unsigned b = blockIdx.x * kThreads + tid; b < static_cast<unsigned>(p.B); b += check_ctas * kThreads)
        paged::check_seq(p.cu_q, p.lens, static_cast<int>(b), total, total, p.cache.capacity());
    }
    // One warp per token: its sequence, its position, its page.
    for (int t = warp; t < count; t += kThreads / 32) {
      const int row = static_cast<int>(first) + t;
      const int b = paged::find_seq(p.cu_q, p.B, row, lane);
      if (lane == 0) {
        Place pl{-1, 0};
        if (b >= 0) {
          const int a = p.cu_q[b], e = p.cu_q[b + 1];
          const int at = p.lens[b] - (e - row);  // position: the last new token is at L - 1
          pl.angle_pos = at;
          if (at >= 0 && a <= row && row < e) {
            if (at < p.cache.capacity()) {
              const int page = p.cache.table[static_cast<size_t>(b) * p.cache.width +
                                             (at >> p.cache.page_log2)];
              if (page >= 0 && page < p.cache.num_pages)
                pl.page = page * p.cache.page_stride +
                          (at & ((1 << p.cache.page_log2) - 1)) * p.cache.token_stride;
              else
                paged::bad(paged::kBadPage);
            } else {
              paged::bad(paged::kBadLength);
            }
          }
        }
        if (p.pos != nullptr) pl.angle_pos = p.pos[row];
        place[t] = pl;
      }
    }
    __syncthreads();
  }

  for (int i = tid; i < count * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    int at;
    if constexpr (APPEND) {
      at = place[t].angle_pos;
    } else {
      const long long b = (first + t) / p.N;
      at = p.pos[b * p.pos_b + (first + t - b * p.N)];
    }
    double a = at * p.turns[pair];
    a -= rint(a);
    float s, c;
    sincospif(2.0f * static_cast<float>(a), &s, &c);
    c *= p.amp;
    s *= p.amp * p.sign;
    if constexpr (VEC) {
      // Pairs 2j, 2j + 1 of unit u at [t][j][u], as 16 bytes: threads of
      // neighbouring units read neighbouring words.
      const int u = pair >> 3, j = (pair >> 1) & 3;
      table[((t * 4 + j) * (half >> 3) + u) * 2 + (pair & 1)] = make_float2(c, s);
    } else {
      table[i] = make_float2(c, s);
    }
  }
  __syncthreads();

  if constexpr (VEC) {
    if (!mine) return;
    const long long page = APPEND ? place[t_mine].page : 0;
    float co[8], si[8];
    if (turned) {
      const float4* t4 = reinterpret_cast<const float4*>(table);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = t4[(t_mine * 4 + j) * nrot + u_mine];
        co[2 * j] = w.x, si[2 * j] = w.y, co[2 * j + 1] = w.z, si[2 * j + 1] = w.w;
      }
    }
    for (int h = h0 + tid / kSlots; h < h1;) {
#pragma unroll
      for (int i = 0; i < kHeadsAtOnce; ++i) {
        if (h + i * kGroups >= h1) break;
        const Row<T> r = row_of<T, APPEND>(p, first + t_mine, h + i * kGroups, page);
        if (r.y == nullptr) continue;
        if (turned && r.turn) {
          float x[8], y[8];
          unpack8<T>(a[i], x);
          unpack8<T>(b[i], y);
          float ox[8], oy[8];
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              ox[2 * j] = x[2 * j] * co[j] - x[2 * j + 1] * si[j];
              ox[2 * j + 1] = x[2 * j + 1] * co[j] + x[2 * j] * si[j];
              oy[2 * j] = y[2 * j] * co[4 + j] - y[2 * j + 1] * si[4 + j];
              oy[2 * j + 1] = y[2 * j + 1] * co[4 + j] + y[2 * j] * si[4 + j];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              ox[j] = x[j] * co[j] - y[j] * si[j];
              oy[j] = y[j] * co[j] + x[j] * si[j];
            }
          }
          a[i] = pack8<T>(ox);
          b[i] = pack8<T>(oy);
        }
        *reinterpret_cast<uint4*>(r.y + c0) = a[i];
        if (second) *reinterpret_cast<uint4*>(r.y + c1) = b[i];
      }
      h += kGroups * kHeadsAtOnce;
      if (h < h1) load(h);
    }
  } else {
    // Pair by pair, then value by value: any even rot.
    const int per = half + (p.d - p.rot);
    const long long all = static_cast<long long>(count) * (h1 - h0) * per;
    for (long long i = tid; i < all; i += kThreads) {
      const int e = static_cast<int>(i % per);
      const int th = static_cast<int>(i / per);
      const int t = th / (h1 - h0), h = h0 + th - t * (h1 - h0);
      const Row<T> r = row_of<T, APPEND>(p, first + t, h, APPEND ? place[t].page : 0);
      if (r.y == nullptr) continue;
      if (e >= half) {
        const int c = p.rot + e - half;
        r.y[c] = r.x[c];
        continue;
      }
      const int ca = INTERLEAVED ? 2 * e : e, cb = INTERLEAVED ? ca + 1 : e + half;
      const T xa = r.x[ca], xb = r.x[cb];
      if (!r.turn) {
        r.y[ca] = xa;
        r.y[cb] = xb;
        continue;
      }
      const float2 w = table[t * half + e];
      const float fa = to_float(xa), fb = to_float(xb);
      r.y[ca] = from_float<T>(fa * w.x - fb * w.y);
      r.y[cb] = from_float<T>(fb * w.x + fa * w.y);
    }
  }
}

}  // namespace rope
}  // namespace eta
