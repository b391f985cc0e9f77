// C-ABI boundary of the paged-cache operators: argument checks, tensor maps,
// workspaces and launches (included by attn_lib.cu, whose helpers it uses).
#pragma once

namespace eta {
namespace api {

// Limits that keep positions, rows and their differences inside 32 bits.
constexpr long long kMaxPositions = 1ll << 30;
constexpr int kMaxPackedRows = 1 << 29;

inline bool mult8(long long x) { return (x & 7) == 0; }

// ------------------------------------------------------------------ overlaps
// Outputs are written while inputs are still read by other CTAs, so an output
// that lies over an input (but for the in-place forms) or over another output
// is refused.

inline long long gap(const void* from, const void* to) {  // bytes
  return static_cast<long long>(reinterpret_cast<intptr_t>(to) - reinterpret_cast<intptr_t>(from));
}

// Blocks of na and nb bytes.
inline bool blocks_meet(const void* a, long long na, const void* b, long long nb) {
  const long long g = gap(a, b);
  return na > 0 && nb > 0 && g < na && g > -nb;
}

// Pieces of d elements (of 2 bytes) at base + i . s, 0 <= i < n.
struct Grid {
  const void* base;
  long long n[3], s[3];
  long long d;
  bool empty() const { return n[0] <= 0 || n[1] <= 0 || n[2] <= 0 || d <= 0; }
  // Elements from the first to behind the last; a dimension of one has no stride.
  double extent() const {
    double e = static_cast<double>(d);
    for (int k = 0; k < 3; ++k) e += static_cast<double>(n[k] - 1) * static_cast<double>(n[k] > 1 ? s[k] : 0);
    return e;
  }
  // No memory is that large (and within it the arithmetic below stays in 64 bits).
  bool too_large() const { return !empty() && extent() > 0x1p46; }
};

// Do two of a grid's own pieces overlap? (Also where its strides do not nest, so
// that it would take a search to tell.)
inline bool grid_meets_itself(const Grid& a) {
  if (a.empty()) return false;
  int by[3] = {0, 1, 2};  // ascending strides
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (a.s[by[j]] > a.s[by[j + 1]]) std::swap(by[j], by[j + 1]);
  long long extent = a.d;
  for (int k : by) {
    if (a.n[k] <= 1) continue;
    if (a.s[k] < extent) return true;
    extent += (a.n[k] - 1) * a.s[k];
  }
  return false;
}

// Are there whole numbers x[k] in [range[k][0], range[k][1]] with
// -below < at + x . s < above? Strides descend.
inline bool steps_reach(long long at, int dims, const long long (*range)[2], const long long* s,
                        long long below, long long above) {
  if (dims == 0) return at > -below && at < above;
  long long rest = 0;  // how far the other dimensions go
  for (int k = 1; k < dims; ++k) rest += s[k] * std::max(-range[k][0], range[k][1]);
  const auto floor_div = [](long long a, long long b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
  const long long lo = std::max(range[0][0], -floor_div(below - 1 + rest + at, s[0]));
  const long long hi = std::min(range[0][1], floor_div(above - 1 + rest - at, s[0]));
  if (hi - lo > 7) return true;  // (strides that do not nest: taken to meet)
  for (long long x = lo; x <= hi; ++x)
    if (steps_reach(at + x * s[0], dims - 1, range + 1, s + 1, below, above)) return true;
  return false;
}

// Do two grids overlap? Exact for parts of one tensor (equal strides, which
// nest); others are taken to if the memory between their ends does.
inline bool grids_meet(const Grid& a, const Grid& b) {
  if (a.empty() || b.empty() || !blocks_meet(a.base, 2 * static_cast<long long>(a.extent()), b.base,
                                             2 * static_cast<long long>(b.extent())))
    return false;
  long long s[3], range[3][2];
  int dims = 0;
  for (int k = 0; k < 3; ++k) {
    if (a.n[k] <= 1 && b.n[k] <= 1) continue;
    if (a.n[k] > 1 && b.n[k] > 1 && a.s[k] != b.s[k]) return true;
    const long long stride = a.n[k] > 1 ? a.s[k] : b.s[k];
    if (stride == 0) continue;  // (an input that is the same along this dimension)
    int at = dims++;
    for (; at > 0 && s[at - 1] < stride; --at) {
      s[at] = s[at - 1];
      range[at][0] = range[at - 1][0];
      range[at][1] = range[at - 1][1];
    }
    s[at] = stride;
    range[at][0] = -(a.n[k] - 1);
    range[at][1] = b.n[k] - 1;
  }
  return steps_reach(gap(a.base, b.base) / 2, dims, range, s, b.d, a.d);
}

// The same places, piece for piece (in place)?
inline bool grids_equal(const Grid& a, const Grid& b) {
  if (a.base != b.base) return false;
  for (int k = 0; k < 3; ++k)
    if (a.n[k] > 1 && a.s[k] != b.s[k]) return false;
  return true;
}

// The cache as the kernels see it; ATTN_OK or the error of a bad description
// (a batch of no sequences has no table).
inline int cache_of(const attn_pages* c, int B, paged::Cache* out) {
  if (c == nullptr) return ATTN_ERR_INVALID;
  if (c->d < 8 || c->d > generic::kMaxD || c->d % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return ATTN_ERR_UNSUPPORTED;
  if (c->Hkv < 1 || c->num_pages < 1 || c->table_width < 1 ||
      static_cast<long long>(c->table_width) * c->page_size > kMaxPositions)
    return ATTN_ERR_INVALID;
  if (c->k == nullptr || c->v == nullptr || (B > 0 && c->table == nullptr) ||
      !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4))
    return ATTN_ERR_INVALID;
  // Strides: whole 16-byte units, and no two elements of a page in one place.
  const long long ps = c->page_stride, hs = c->head_stride, ts = c->token_stride;
  if (!mult8(ps) || !mult8(hs) || !mult8(ts) || ts < c->d || hs < c->d || ps < c->d ||
      ps >= (1ll << 38) || hs >= (1ll << 38) || ts >= (1ll << 38))
    return ATTN_ERR_INVALID;
  out->k = c->k;
  out->v = c->v;
  out->table = c->table;
  out->page_stride = ps;
  out->head_stride = hs;
  out->token_stride = ts;
  out->num_pages = c->num_pages;
  out->page_log2 = 0;
  while ((1 << out->page_log2) < c->page_size) ++out->page_log2;
  out->width = c->table_width;
  out->Hkv = c->Hkv;
  out->d = c->d;
  return ATTN_OK;
}

// 4-D map of 16-bit elements with 128-byte-swizzled boxes of 64 columns.
inline int encode_4d(CUtensorMap* map, const void* base, bool bf16, const cuuint64_t (&dims)[4],
                     const cuuint64_t (&strides)[3], unsigned rows1, unsigned rows3) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return ATTN_ERR_CUDA;
  const cuuint32_t box[4] = {64, rows1, 1, rows3};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// A launch that may begin before the kernel in front of it ends (which it
// waits for on the device).
template <typename... A, typename... B>
int launch_dependent(void (*kern)(A...), dim3 grid, int threads, int smem, cudaStream_t st,
                     B&&... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<B>(args)...);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

// Stream-ordered workspace of one call.
struct Workspace {
  void* p = nullptr;
  cudaStream_t st;
  int take(size_t bytes, cudaStream_t stream) {
    cudaMemPool_t pool;
    st = stream;
    if (workspace_pool(&pool) != ATTN_OK) return ATTN_ERR_CUDA;
    const cudaError_t e = cudaMallocFromPoolAsync(&p, bytes, pool, st);
    if (e != cudaSuccess) {
      p = nullptr;
      cudaGetLastError();
      return cuda_fail(e);
    }
    return ATTN_OK;
  }
  int give_back(int rc) {
    const cudaError_t e = cudaFreeAsync(p, st);
    return rc != ATTN_OK ? rc : e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
};

// Maps of the pools, boxes of 64 columns and one page (or 128 rows of it).
inline int encode_pools(CUtensorMap* tk, CUtensorMap* tv, const paged::Cache& c, bool bf16) {
  const int page = 1 << c.page_log2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(page),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride) * 2,
                                 static_cast<cuuint64_t>(c.head_stride) * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const unsigned rows = static_cast<unsigned>(page < paged::BN ? page : paged::BN);
  const int rc = encode_4d(tk, c.k, bf16, dims, strides, rows, 1);
  return rc != ATTN_OK ? rc : encode_4d(tv, c.v, bf16, dims, strides, rows, 1);
}

// Map of the packed queries, boxes of 64 columns, a group's heads, `tokens` tokens.
inline int encode_queries(CUtensorMap* tq, const void* q, long long q_stride, const paged::Cache& c,
                          int G, int total_q, int tokens, bool bf16) {
  const cuuint64_t d = static_cast<cuuint64_t>(c.d);
  const cuuint64_t dims[4] = {d, static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(c.Hkv),
                              static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[3] = {d * 2, d * 2 * G, static_cast<cuuint64_t>(q_stride) * 2};
  return encode_4d(tq, q, bf16, dims, strides, static_cast<unsigned>(G),
                   static_cast<unsigned>(tokens));
}

template <int D, typename T>
int launch_paged(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 const paged::Params& p, cudaStream_t st) {
  auto kern = paged::attn_paged_kernel<D, T>;
  constexpr int smem = paged::Cfg<D>::kSmemBytes;
  static PerDeviceOnce attr;
  const cudaError_t attr_err = attr.run([&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr_err != cudaSuccess) return cuda_fail(attr_err);
  int rc = ATTN_OK;
  if (!p.inline_plan) {
    paged::attn_paged_plan_kernel<<<1, paged::kPlanThreads, 0, st>>>(p);
    rc = launch_status();
  }
  if (rc == ATTN_OK)
    rc = launch_dependent(kern, dim3(static_cast<unsigned>(p.nc)), paged::kThreads, smem, st, tq,
                          tk, tv, p);
  if (rc == ATTN_OK)
    rc = launch_dependent(paged::attn_paged_gather_kernel<D, T>,
                          dim3(static_cast<unsigned>(p.nc), paged::kSlotRows / 32), 256, 0, st, p);
  return rc;
}

// Cost of a segment's start, in tiles, when the CTAs of the paged decode pass
// share out the work. Measured on B200 with 0 / 1 / 2 / 3 / 4: the ragged batch
// of 64 x 1K-8K tokens 199 / 194 / 197 / 194 / 194 us, 256 sequences of 50-600
// tokens 116 / 91 / 87 / 88 / 90 us, 61 sequences under a window of 1006
// tokens 48 / 42 / 37 / 36 / 37 us, 1 to 4 new tokens over 500-4096 129 / 117 /
// 109 / 106 / 105 us; groups of 16 and 32 heads as before.
#ifndef ETA_PAGED_SEG_COST
#define ETA_PAGED_SEG_COST 3
#endif

// Few rows of a KV head (max_q G <= 32): the persistent decode pass, whose
// products have the keys on the tensor core's long side, over pages. Batches whose
// tiles could not be counted in 32 bits take the other kernel.
template <typename T>
int paged_decode_run(const void* q, long long q_stride, const paged::Cache& c, const int32_t* cu_q,
                     const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q,
                     int max_q, float scale, int window, int nc, cudaStream_t st) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int G = Hq / c.Hkv, D = c.d <= 64 ? 64 : 128;
  decode_ps::PParams p = {};
  p.q = q;
  p.kc = c.k;
  p.vc = c.v;
  p.seqlens = kv_lens;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = c.Hkv;
  p.G = G;
  p.window = window;
  p.inline_plan = B <= ETA_DECODE_INLINE_PLAN_MAX_B ? 1 : 0;
  p.R = max_q * G;
  p.wcost = p.inline_plan ? ETA_PAGED_SEG_COST : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_ns = kDefaultWaitNs;
  p.cu_q = cu_q;
  p.cache = c;
  p.total_q = total_q;
  p.max_q = max_q;
  CUtensorMap tq;
  decode_ps::KvMaps<true> kv;
  int rc = encode_queries(&tq, q, q_stride, c, G, total_q, max_q, bf16);
  if (rc == ATTN_OK) rc = encode_pools(&kv.k, &kv.v, c, bf16);
  if (rc != ATTN_OK) return rc;
  // Two slots of partial rows a CTA: what goes on from the CTA before, and what
  // goes on in the next.
  const PsLayout L = ps_layout(B, c.Hkv, p.R, D, nc, true, 2 * static_cast<size_t>(nc));
  Workspace ws;
  rc = ws.take(L.total, st);
  if (rc != ATTN_OK) return rc;
  rc = D == 128 ? launch_decode_ps_group<128, T, true>(tq, p, L, static_cast<char*>(ws.p), nc, st, kv)
                : launch_decode_ps_group<64, T, true>(tq, p, L, static_cast<char*>(ws.p), nc, st, kv);
  return ws.give_back(rc);
}

template <typename T>
int paged_run(const void* q, long long q_stride, const attn_pages* pages, const int32_t* cu_q,
              const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q, int max_q,
              float scale, int window, cudaStream_t st) {
  paged::Cache c;
  const int bad = cache_of(pages, B, &c);
  if (bad != ATTN_OK) return bad;
  if (B < 0 || total_q < 0 || total_q > kMaxPackedRows || max_q < 0 || Hq < 1 ||
      Hq % c.Hkv != 0 || !scale_ok(scale) || window < 0)
    return ATTN_ERR_INVALID;
  if (!mult8(q_stride) || q_stride < static_cast<long long>(Hq) * c.d || q_stride >= (1ll << 38))
    return ATTN_ERR_INVALID;
  if (static_cast<long long>(total_q) * Hq > 0x7fffffffLL ||
      static_cast<long long>(B) * c.Hkv > 0x7fffffffLL)
    return ATTN_ERR_INVALID;
  if (B == 0 || total_q == 0 || max_q == 0) return ATTN_OK;
  if (q == nullptr || o == nullptr || cu_q == nullptr || kv_lens == nullptr || !aligned(q, 16) ||
      !aligned(o, 16) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) ||
      (lse != nullptr && !aligned(lse, 4)))
    return ATTN_ERR_INVALID;
  const long long heads = static_cast<long long>(total_q) * Hq;
  const Grid q_rows{q, {total_q, 1, 1}, {q_stride, 0, 0}, static_cast<long long>(Hq) * c.d};
  const auto block = [](const void* at, long long bytes) { return Grid{at, {1, 1, 1}, {0, 0, 0}, bytes / 2}; };
  const Grid o_all = block(o, heads * c.d * 2), lse_all = block(lse, lse != nullptr ? heads * 4 : 0);
  if (q_rows.too_large() || grids_meet(o_all, q_rows) || grids_meet(lse_all, q_rows) ||
      grids_meet(o_all, lse_all))
    return ATTN_ERR_INVALID;
  DeviceInfo info;
  if (device_info(&info) != ATTN_OK) return ATTN_ERR_CUDA;
  if (!info.sm100) return ATTN_ERR_UNSUPPORTED;
  if (max_q > total_q) max_q = total_q;
  if (window >= kMaxPositions) window = 0;  // longer than any cache: none
  const int G = Hq / c.Hkv;

  if (c.d > 128 || G > paged::BM) {
    paged::GParams g;
    g.q = q;
    g.q_stride = q_stride;
    g.cache = c;
    g.cu_q = cu_q;
    g.lens = kv_lens;
    g.o = o;
    g.lse = lse;
    g.B = B;
    g.Hq = Hq;
    g.G = G;
    g.total_q = total_q;
    g.max_q = max_q;
    g.window = window;
    g.scale_log2 = scale * 1.4426950408889634f;
    const long long rows = static_cast<long long>(max_q) * G, bg = static_cast<long long>(B) * c.Hkv;
    const unsigned ny = static_cast<unsigned>(bg < generic::kGridY ? bg : generic::kGridY);
    const dim3 grid(static_cast<unsigned>((rows + generic::kRows - 1) / generic::kRows), ny,
                    static_cast<unsigned>((bg + generic::kGridY - 1) / generic::kGridY));
    paged::attn_paged_generic_kernel<T><<<grid, generic::kThreads, generic::smem_bytes(c.d), st>>>(g);
    return launch_status();
  }

  // Few rows of a KV head go to the decode pass, more to the pass of whole row
  // tiles. Measured on B200, decode pass / row tiles: one token at group 4 over
  // 64 x 1K-8K 196 / 213 us, at group 16 57 / 67 us, at group 32 39 / 47 us, at
  // group 32 of 4 x 50-700 13 / 18 us; 4 tokens at group 4 over 500-4096 108 /
  // 123 us, 8 tokens 126 / 124 us. With d <= 64 several tokens of more than 16
  // rows are better off in row tiles (8 tokens at group 4 120 / 94 us, 3 at
  // group 8 98 / 83 us; a single token at group 32 37 / 37 us).
  // (The global tile order and the gather's rows are counted in 32 bits.)
  const long long tiles = static_cast<long long>(B) * c.Hkv * ((c.capacity() >> 7) + 4);
  const int most_rows = c.d <= 64 && max_q > 1 ? 16 : 32;
  if (static_cast<long long>(max_q) * G <= most_rows && tiles < 0x7fffffffLL &&
      static_cast<long long>(B) * c.Hkv * max_q * G < (1ll << 32))
    return paged_decode_run<T>(q, q_stride, c, cu_q, kv_lens, o, lse, B, Hq, total_q, max_q, scale,
                               window, info.sm_count, st);

  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int tt = paged::BM / G;
  // (a CTA's steps are counted in 32 bits, each as up to 9 positions: with the
  // longest cache that the table allows for every token, this is weeks of work)
  const double most_steps = (static_cast<double>(total_q) / (paged::NQT * tt) + B) * c.Hkv *
                            (static_cast<double>(c.capacity()) / paged::BN + 1);
  if (most_steps / info.sm_count > 2e8) return ATTN_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv;
  int rc = encode_queries(&tq, q, q_stride, c, G, total_q, tt, bf16);
  if (rc == ATTN_OK) rc = encode_pools(&tk, &tv, c, bf16);
  if (rc != ATTN_OK) return rc;

  paged::Params p;
  p.cu_q = cu_q;
  p.lens = kv_lens;
  p.table = c.table;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = c.Hkv;
  p.G = G;
  p.tt = tt;
  p.total_q = total_q;
  p.max_q = max_q;
  p.d = c.d;
  p.num_pages = c.num_pages;
  p.page_log2 = c.page_log2;
  p.width = c.width;
  p.window = window;
  p.nc = info.sm_count;
  p.inline_plan = B <= paged::kInlineB ? 1 : 0;
  p.warp_plan = B <= 32 && most_steps < 2e8 ? 1 : 0;
  p.max_pairs = (max_q + paged::NQT * tt - 1) / (paged::NQT * tt);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_ns = kDefaultWaitNs;
  p.l2_bytes = info.l2_bytes;
  // Workspace: the plan, then three slots of partial rows per CTA.
  size_t end = 0;
  const auto part = [&end](size_t bytes) {
    const size_t at = end;
    end = align_up(end + bytes, 256);
    return at;
  };
  const size_t slots = static_cast<size_t>(3) * p.nc * paged::kSlotRows;
  const size_t head = part(sizeof(paged::Head)), starts = part(p.nc * sizeof(paged::Start)),
               rest_at = part(p.inline_plan ? 0 : (static_cast<size_t>(B) + 1) * 8),
               chunk_at = part(p.inline_plan ? 0 : (static_cast<size_t>(B) + 1) * 4),
               part_lse = part(slots * 4), part_o = part(slots * (c.d <= 64 ? 64 : 128) * 4);
  Workspace ws;
  rc = ws.take(end, st);
  if (rc != ATTN_OK) return rc;
  char* base = static_cast<char*>(ws.p);
  p.plan.head = reinterpret_cast<paged::Head*>(base + head);
  p.plan.starts = reinterpret_cast<paged::Start*>(base + starts);
  p.plan.rest_at = reinterpret_cast<long long*>(base + rest_at);
  p.plan.chunk_at = reinterpret_cast<int*>(base + chunk_at);
  p.part_lse = reinterpret_cast<float*>(base + part_lse);
  p.part_o = reinterpret_cast<float*>(base + part_o);
  rc = c.d <= 64 ? launch_paged<64, T>(tq, tk, tv, p, st) : launch_paged<128, T>(tq, tk, tv, p, st);
  return ws.give_back(rc);
}

// ------------------------------------------------------------------ rotary positions

inline int rope_sizes(int d, int rot) {
  if (d < 8 || d > generic::kMaxD || d % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  return rot >= 0 && rot <= d && rot % 2 == 0 ? ATTN_OK : ATTN_ERR_INVALID;
}

template <typename T, bool APPEND>
int launch_rope(rope::Params p, int interleaved, cudaStream_t st) {
  DeviceInfo info;
  if (device_info(&info) != ATTN_OK) return ATTN_ERR_CUDA;
  if (!info.sm100) return ATTN_ERR_UNSUPPORTED;
  const bool vec = p.rot % 16 == 0;
  p.units = p.rot / 16 + (p.d - p.rot + 15) / 16;
  int tokens = vec ? rope::kSlots / p.units : 8;
  if (tokens > rope::kMaxTokens) tokens = rope::kMaxTokens;
  if (tokens > p.tokens) tokens = static_cast<int>(p.tokens);
  // Heads of a CTA: as many as a thread loads at once, doubled up to 32 while
  // the grid still covers the GPU, since every CTA of a token works out the
  // same angles (8 / 16 / 32 / 64 heads: 30.3 / 26.3 / 24.9 / 24.9 us on the
  // 2K case of rope.cuh, 63.3 / 54.1 / 51.7 / 53.9 us on its append).
  int heads = rope::kGroups * rope::kHeadsAtOnce;
  const long long blocks_x = (p.tokens + tokens - 1) / tokens;
  if (blocks_x > 0x7fffffffLL) return ATTN_ERR_INVALID;
  while (heads < 32 && heads < p.heads &&
         blocks_x * ((p.heads + 2 * heads - 1) / (2 * heads)) >= 4LL * info.sm_count)
    heads *= 2;
  p.tokens_per_cta = tokens;
  p.heads_per_cta = heads;
  const int ny = (p.heads + heads - 1) / heads;
  if (ny > 65535) return ATTN_ERR_INVALID;
  const dim3 grid(static_cast<unsigned>(blocks_x), static_cast<unsigned>(ny));
  const int smem = tokens * (p.rot / 2) * 8;
  const auto kern = vec ? (interleaved ? rope::rope_kernel<T, APPEND, true, true>
                                       : rope::rope_kernel<T, APPEND, false, true>)
                        : (interleaved ? rope::rope_kernel<T, APPEND, true, false>
                                       : rope::rope_kernel<T, APPEND, false, false>);
  return launch_dependent(kern, grid, rope::kThreads, smem, st, p);
}

template <typename T>
int rope_run(const void* q, void* q_out, const void* k, void* k_out, const long long* strides,
             const int32_t* pos, long long pos_stride, const double* turns, int B, int Hq, int Hkv,
             int N, int d, int rot, float amp, int interleaved, int backward, cudaStream_t st) {
  const int rc = rope_sizes(d, rot);
  if (rc != ATTN_OK) return rc;
  if (B < 0 || N < 0 || Hq < 0 || Hkv < 0 || strides == nullptr || !std::isfinite(amp) ||
      static_cast<long long>(B) * N > 0x7fffffffLL || static_cast<long long>(Hq) + Hkv > 65535)
    return ATTN_ERR_INVALID;
  for (int i = 0; i < 12; ++i)
    if (!mult8(strides[i]) || strides[i] < 0) return ATTN_ERR_INVALID;
  if (B == 0 || N == 0 || Hq + Hkv == 0) return ATTN_OK;
  if (pos == nullptr || !aligned(pos, 4) || pos_stride < 0 ||
      (rot > 0 && (turns == nullptr || !aligned(turns, 8))))
    return ATTN_ERR_INVALID;
  if (Hq > 0 && (q == nullptr || q_out == nullptr || !aligned(q, 16) || !aligned(q_out, 16)))
    return ATTN_ERR_INVALID;
  if (Hkv > 0 && (k == nullptr || k_out == nullptr || !aligned(k, 16) || !aligned(k_out, 16)))
    return ATTN_ERR_INVALID;
  rope::Params p = {};
  const long long* s = strides;
  p.t[0] = {q, q_out, s[0], s[1], s[2], s[3], s[4], s[5]};
  p.t[1] = {k, k_out, s[6], s[7], s[8], s[9], s[10], s[11]};
  p.H[0] = Hq;
  p.H[1] = Hkv;
  p.heads = Hq + Hkv;
  p.pos = pos;
  p.pos_b = pos_stride;
  p.turns = turns;
  p.amp = amp;
  p.sign = backward ? -1.f : 1.f;
  p.N = N;
  p.tokens = static_cast<long long>(B) * N;
  const auto grid = [&](const void* base, int H, const long long* st) {
    return Grid{base, {B, H, N}, {st[0], st[1], st[2]}, d};
  };
  const Grid qi = grid(q, Hq, s), qo = grid(q_out, Hq, s + 3), ki = grid(k, Hkv, s + 6),
             ko = grid(k_out, Hkv, s + 9);
  const bool q_in_place = Hq == 0 || grids_equal(qi, qo), k_in_place = Hkv == 0 || grids_equal(ki, ko);
  // In place, the values that pass through are there already.
  const bool same = q_in_place && k_in_place;
  p.d = same ? rot : d;
  p.rot = rot;
  if (p.d == 0) return ATTN_OK;
  if (qi.too_large() || qo.too_large() || ki.too_large() || ko.too_large() || grid_meets_itself(qo) ||
      grid_meets_itself(ko) || (!q_in_place && grids_meet(qo, qi)) ||
      (!k_in_place && grids_meet(ko, ki)) || grids_meet(qo, ki) || grids_meet(ko, qi) ||
      grids_meet(qo, ko))
    return ATTN_ERR_INVALID;
  return launch_rope<T, false>(p, interleaved, st);
}

template <typename T>
int rope_append_run(const void* q, long long q_stride, void* q_out, long long q_out_stride,
                    const void* k, long long k_stride, const void* v, long long v_stride,
                    const attn_pages* pages, const int32_t* cu_q, const int32_t* kv_lens,
                    const int32_t* pos, const double* turns, int B, int Hq, int total_q, int rot,
                    float amp, int interleaved, cudaStream_t st) {
  rope::Params p = {};
  int rc = cache_of(pages, B, &p.cache);
  if (rc != ATTN_OK) return rc;
  const int d = p.cache.d, Hkv = p.cache.Hkv;
  rc = rope_sizes(d, rot);
  if (rc != ATTN_OK) return rc;
  if (B < 0 || Hq < 0 || total_q < 0 || total_q > kMaxPackedRows || !std::isfinite(amp) ||
      static_cast<long long>(Hq) + 2LL * Hkv > 65535)
    return ATTN_ERR_INVALID;
  const long long row_q = static_cast<long long>(Hq) * d, row_kv = static_cast<long long>(Hkv) * d;
  if (!mult8(q_stride) || !mult8(q_out_stride) || !mult8(k_stride) || !mult8(v_stride) ||
      q_stride < row_q || q_out_stride < row_q || k_stride < row_kv || v_stride < row_kv)
    return ATTN_ERR_INVALID;
  if (B == 0 || total_q == 0) return ATTN_OK;
  if (k == nullptr || v == nullptr || cu_q == nullptr || kv_lens == nullptr || !aligned(k, 16) ||
      !aligned(v, 16) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) ||
      (pos != nullptr && !aligned(pos, 4)) ||
      (rot > 0 && (turns == nullptr || !aligned(turns, 8))) ||
      (Hq > 0 && (q == nullptr || q_out == nullptr || !aligned(q, 16) || !aligned(q_out, 16))))
    return ATTN_ERR_INVALID;
  const auto rows = [&](const void* x, long long stride, long long row) {
    return Grid{x, {total_q, 1, 1}, {stride, 0, 0}, row};
  };
  const Grid qi = rows(q, q_stride, row_q), qo = rows(q_out, q_out_stride, row_q),
             ki = rows(k, k_stride, row_kv), vi = rows(v, v_stride, row_kv);
  if (qi.too_large() || qo.too_large() || ki.too_large() || vi.too_large() ||
      (!grids_equal(qi, qo) && grids_meet(qo, qi)) || grids_meet(qo, ki) || grids_meet(qo, vi))
    return ATTN_ERR_INVALID;
  p.t[0] = {q, q_out, 0, d, q_stride, 0, d, q_out_stride};
  p.t[1] = {k, nullptr, 0, d, k_stride, 0, 0, 0};
  p.v = v;
  p.vh = d;
  p.vn = v_stride;
  p.H[0] = Hq;
  p.H[1] = Hkv;
  p.heads = Hq + 2 * Hkv;
  p.pos = pos;
  p.turns = turns;
  p.amp = amp;
  p.sign = 1.f;
  p.N = total_q;
  p.tokens = total_q;
  p.d = d;
  p.rot = rot;
  p.cu_q = cu_q;
  p.lens = kv_lens;
  p.B = B;
  return launch_rope<T, true>(p, interleaved, st);
}

// ------------------------------------------------------------------ page operations

struct Block {
  const void* at;  // (NULL: none)
  long long bytes;
};
// Does an output lie over an input, or over another output?
inline bool overlap(std::initializer_list<Block> in, std::initializer_list<Block> out) {
  const auto meet = [](const Block& a, const Block& b) {
    return a.at != nullptr && b.at != nullptr && blocks_meet(a.at, a.bytes, b.at, b.bytes);
  };
  for (const Block* o = out.begin(); o != out.end(); ++o) {
    for (const Block& i : in)
      if (meet(*o, i)) return true;
    for (const Block* other = out.begin(); other != o; ++other)
      if (meet(*o, *other)) return true;
  }
  return false;
}

// Checks shared by update and compact (which has no source, add and lens_out);
// fills what both need.
inline int pages_setup(const attn_pages* c, int layers, long long layer_stride, int B,
                       const int32_t* lens, const int32_t* refs, const int32_t* source,
                       const int32_t* add, int32_t* table_out, int32_t* lens_out,
                       int32_t* refs_out, int32_t* info, paged::Cache* cache, pages::Params* p,
                       pages::CopyParams* cp) {
  const int rc = cache_of(c, B, cache);
  if (rc != ATTN_OK) return rc;
  if (B < 0 || layers < 1 || !mult8(layer_stride) || layer_stride < 0 ||
      static_cast<long long>(B) * c->table_width > 0x7fffffffLL)
    return ATTN_ERR_INVALID;
  // A page's values in one piece, heads or tokens outermost.
  const long long hs = c->head_stride, ts = c->token_stride, d = c->d;
  const bool heads_out = ts == d && (c->Hkv == 1 || hs == c->page_size * d);
  const bool tokens_out = (c->Hkv == 1 || hs == d) && ts == c->Hkv * d;
  if (!heads_out && !tokens_out) return ATTN_ERR_INVALID;
  const long long page = static_cast<long long>(c->Hkv) * c->page_size * d;
  if (c->page_stride < page) return ATTN_ERR_INVALID;
  if ((B > 0 && (lens == nullptr || table_out == nullptr)) || refs == nullptr ||
      refs_out == nullptr || info == nullptr || !aligned(lens, 4) || !aligned(refs, 4) || !aligned(table_out, 4) ||
      !aligned(refs_out, 4) || !aligned(info, 4))
    return ATTN_ERR_INVALID;
  const long long entries = 4LL * B * c->table_width, rows = 4LL * B, counts = 4LL * c->num_pages;
  if (overlap({{c->table, entries}, {lens, rows}, {refs, counts}, {source, rows}, {add, rows}},
              {{table_out, entries}, {lens_out, rows}, {refs_out, counts}, {info, 8}}))
    return ATTN_ERR_INVALID;
  p->table = c->table;
  p->lens = lens;
  p->refs = refs;
  p->table_out = table_out;
  p->refs_out = refs_out;
  p->info = info;
  p->B = B;
  p->width = c->table_width;
  p->P = c->num_pages;
  p->page_log2 = cache->page_log2;
  cp->pool[0] = static_cast<uint8_t*>(c->k);
  cp->pool[1] = static_cast<uint8_t*>(c->v);
  cp->page_stride = c->page_stride * 2;
  cp->layer_stride = layer_stride * 2;
  cp->page_bytes = page * 2;
  cp->layers = layers;
  return ATTN_OK;
}

// One kernel does everything when the counts fit shared memory (some 25,000
// pages) and the tables have few entries (every CTA reads what its share of the
// rows needs, and the rows that end or fork whole). Measured on B200 against
// the cluster and its copy kernel: update of 64 rows, 10,544 pages 10.2 against
// 16.6 us; compaction of 64 rows, 4,536 pages 8.7 / 11.6 us, of 256 rows of 251
// entries, 22,173 pages 11.9 / 14.3 us.
#ifndef ETA_PAGES_SMALL_ENTRIES
#define ETA_PAGES_SMALL_ENTRIES 65536
#endif
constexpr size_t kPagesSmallBytes = 200 * 1024;

template <void (*kern)(pages::Params, pages::CopyParams)>
int pages_launch_small(const pages::Params& p, const pages::CopyParams& cp, size_t words, int ctas,
                       cudaStream_t st) {
  static PerDeviceOnce attr;  // (one for each kernel)
  const cudaError_t e = attr.run([&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kPagesSmallBytes));
  });
  if (e != cudaSuccess) return cuda_fail(e);
  return launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), pages::kThreads,
                          static_cast<int>(words * 4), st, p, cp);
}

template <bool UPDATE>
int pages_launch(pages::Params p, pages::CopyParams cp, cudaStream_t st) {
  DeviceInfo dev;
  if (device_info(&dev) != ATTN_OK) return ATTN_ERR_CUDA;
  if (!dev.sm100) return ATTN_ERR_UNSUPPORTED;
  const size_t words = UPDATE ? pages::update_small_words(p.B, p.P) : pages::compact_small_words(p.P);
  if (words * 4 <= kPagesSmallBytes &&
      static_cast<long long>(p.B) * p.width <= ETA_PAGES_SMALL_ENTRIES) {
    if constexpr (UPDATE)
      return pages_launch_small<pages::pages_update_small_kernel>(p, cp, words, dev.sm_count, st);
    else
      return pages_launch_small<pages::pages_compact_small_kernel>(p, cp, words, dev.sm_count, st);
  }
  size_t end = 0;
  const auto part = [&end](size_t n) {
    const size_t at = end;
    end = align_up(end + n * 4, 256);
    return at;
  };
  const size_t B = static_cast<size_t>(p.B), P = static_cast<size_t>(p.P);
  const size_t moves = B > P ? B : P;
  const size_t keeper = part(B), need = part(B + 1), counts = part(pages::kCtas), list = part(P),
               from = part(moves), to = part(moves), n = part(1);
  Workspace ws;
  int rc = ws.take(end, st);
  if (rc != ATTN_OK) return rc;
  char* base = static_cast<char*>(ws.p);
  p.keeper = reinterpret_cast<int*>(base + keeper);
  p.need_off = reinterpret_cast<int*>(base + need);
  p.counts = reinterpret_cast<int*>(base + counts);
  p.list = reinterpret_cast<int*>(base + list);
  p.from = reinterpret_cast<int*>(base + from);
  p.to = reinterpret_cast<int*>(base + to);
  p.n_copies = reinterpret_cast<int*>(base + n);
  cp.from = p.from;
  cp.to = p.to;
  cp.n_copies = p.n_copies;
  rc = launch_dependent(UPDATE ? pages::pages_update_kernel : pages::pages_compact_kernel,
                        dim3(pages::kCtas), pages::kThreads, 0, st, p);
  if (rc == ATTN_OK)
    rc = launch_dependent(pages::pages_copy_kernel, dim3(static_cast<unsigned>(6 * dev.sm_count)),
                          pages::kCopyThreads, 0, st, cp);
  return ws.give_back(rc);
}

int pages_update(const attn_pages* c, int layers, long long layer_stride, const int32_t* lens,
                 const int32_t* refs, const int32_t* source, const int32_t* add,
                 int32_t* table_out, int32_t* lens_out, int32_t* refs_out, int32_t* info, int B,
                 cudaStream_t st) {
  paged::Cache cache;
  pages::Params p = {};
  pages::CopyParams cp = {};
  const int rc = pages_setup(c, layers, layer_stride, B, lens, refs, source, add, table_out,
                             lens_out, refs_out, info, &cache, &p, &cp);
  if (rc != ATTN_OK) return rc;
  if ((B > 0 && (source == nullptr || add == nullptr || lens_out == nullptr)) ||
      !aligned(source, 4) || !aligned(add, 4) || !aligned(lens_out, 4))
    return ATTN_ERR_INVALID;
  p.source = source;
  p.add = add;
  p.lens_out = lens_out;
  return pages_launch<true>(p, cp, st);
}

int pages_compact(const attn_pages* c, int layers, long long layer_stride, const int32_t* lens,
                  const int32_t* refs, int32_t* table_out, int32_t* refs_out, int32_t* info, int B,
                  cudaStream_t st) {
  paged::Cache cache;
  pages::Params p = {};
  pages::CopyParams cp = {};
  const int rc = pages_setup(c, layers, layer_stride, B, lens, refs, nullptr, nullptr, table_out,
                             nullptr, refs_out, info, &cache, &p, &cp);
  if (rc != ATTN_OK) return rc;
  return pages_launch<false>(p, cp, st);
}

// Turns per position of each pair, in 64 bits, on the host.
int rope_turns(double* turns, float* amp, int rot, double base, int scaling, double factor,
               double low, double high, double original) {
  if (turns == nullptr || amp == nullptr || rot < 2 || rot % 2 != 0 || rot > generic::kMaxD ||
      !std::isfinite(base) || base <= 1.0)
    return ATTN_ERR_INVALID;
  if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_BANDS) return ATTN_ERR_INVALID;
  if (scaling != ATTN_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return ATTN_ERR_INVALID;
  if (scaling == ATTN_ROPE_BASE && rot < 4) return ATTN_ERR_INVALID;
  if (scaling >= ATTN_ROPE_PARTS &&
      (!std::isfinite(low) || !std::isfinite(high) || low <= 0.0 || high <= low ||
       !std::isfinite(original) || original <= 0.0))
    return ATTN_ERR_INVALID;
  const double two_pi = 6.283185307179586476925286766559;
  const int n = rot / 2;
  *amp = 1.f;
  if (scaling == ATTN_ROPE_BASE) base *= std::pow(factor, rot / (rot - 2.0));
  double first = 0.0, last = 0.0;
  if (scaling == ATTN_ROPE_PARTS) {
    // The pair that makes t turns over the original context: its (real) index.
    const auto pair = [&](double t) {
      return rot * std::log(original / (t * two_pi)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(pair(high)), 0.0);
    last = std::fmin(std::ceil(pair(low)), rot - 1.0);
    *amp = static_cast<float>(0.1 * std::log(factor) + 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == ATTN_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == ATTN_ROPE_PARTS) {
      const double ramp = std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    } else if (scaling == ATTN_ROPE_BANDS) {
      const double mix =
          std::fmin(std::fmax((original * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = (1.0 - mix) * f / factor + mix * f;
    }
    turns[i] = f / two_pi;
  }
  return ATTN_OK;
}

}  // namespace api
}  // namespace eta

extern "C" {

int attn_paged(const void* q, long long q_stride, const attn_pages* cache, const int32_t* cu_q,
               const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q, int max_q,
               float scale, int window, attn_stream_t stream) {
  return eta::api::paged_run<__nv_bfloat16>(q, q_stride, cache, cu_q, kv_lens, o, lse, B, Hq,
                                            total_q, max_q, scale, window,
                                            reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_f16(const void* q, long long q_stride, const attn_pages* cache, const int32_t* cu_q,
                   const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q,
                   int max_q, float scale, int window, attn_stream_t stream) {
  return eta::api::paged_run<__half>(q, q_stride, cache, cu_q, kv_lens, o, lse, B, Hq, total_q,
                                     max_q, scale, window, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope(const void* q, void* q_out, const void* k, void* k_out, const long long* strides,
              const int32_t* pos, long long pos_stride, const double* turns, int B, int Hq, int Hkv,
              int N, int d, int rot, float amp, int interleaved, int backward,
              attn_stream_t stream) {
  return eta::api::rope_run<__nv_bfloat16>(q, q_out, k, k_out, strides, pos, pos_stride, turns, B,
                                           Hq, Hkv, N, d, rot, amp, interleaved, backward,
                                           reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_f16(const void* q, void* q_out, const void* k, void* k_out, const long long* strides,
                  const int32_t* pos, long long pos_stride, const double* turns, int B, int Hq,
                  int Hkv, int N, int d, int rot, float amp, int interleaved, int backward,
                  attn_stream_t stream) {
  return eta::api::rope_run<__half>(q, q_out, k, k_out, strides, pos, pos_stride, turns, B, Hq,
                                    Hkv, N, d, rot, amp, interleaved, backward,
                                    reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_append(const void* q, long long q_stride, void* q_out, long long q_out_stride,
                     const void* k, long long k_stride, const void* v, long long v_stride,
                     const attn_pages* cache, const int32_t* cu_q, const int32_t* kv_lens,
                     const int32_t* pos, const double* turns, int B, int Hq, int total_q, int rot,
                     float amp, int interleaved, attn_stream_t stream) {
  return eta::api::rope_append_run<__nv_bfloat16>(
      q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, cache, cu_q, kv_lens, pos, turns,
      B, Hq, total_q, rot, amp, interleaved, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_append_f16(const void* q, long long q_stride, void* q_out, long long q_out_stride,
                         const void* k, long long k_stride, const void* v, long long v_stride,
                         const attn_pages* cache, const int32_t* cu_q, const int32_t* kv_lens,
                         const int32_t* pos, const double* turns, int B, int Hq, int total_q,
                         int rot, float amp, int interleaved, attn_stream_t stream) {
  return eta::api::rope_append_run<__half>(
      q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, cache, cu_q, kv_lens, pos, turns,
      B, Hq, total_q, rot, amp, interleaved, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_turns(double* turns, float* amp, int rot, double base, int scaling, double factor,
                    double low, double high, double original) {
  return eta::api::rope_turns(turns, amp, rot, base, scaling, factor, low, high, original);
}

int attn_pages_update(const attn_pages* cache, int layers, long long layer_stride,
                      const int32_t* lens, const int32_t* refs, const int32_t* source,
                      const int32_t* add, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                      int32_t* info, int B, attn_stream_t stream) {
  return eta::api::pages_update(cache, layers, layer_stride, lens, refs, source, add, table_out,
                                lens_out, refs_out, info, B,
                                reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_compact(const attn_pages* cache, int layers, long long layer_stride,
                       const int32_t* lens, const int32_t* refs, int32_t* table_out,
                       int32_t* refs_out, int32_t* info, int B, attn_stream_t stream) {
  return eta::api::pages_compact(cache, layers, layer_stride, lens, refs, table_out, refs_out, info,
                                 B, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
