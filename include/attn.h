/*
 * exact_tiled_attention_38_b200: exact scaled-dot-product attention for B200
 * (sm_100a), as a C ABI.
 *
 * What is computed (every entry point): for each batch b, query head h and
 * query row i,
 *     s_ij  = scale * sum_c q[b,h,i,c] * k[b,g,j,c],   g = h / (Hq / Hkv)
 *     s_ij  = -inf where key j is masked (causal: j > i + Nk - Nq)
 *     o[b,h,i,:] = sum_j softmax_j(s_i.) * v[b,g,j,:]
 *     lse[b,h,i] = ln sum_j exp(s_ij)
 * This is exact attention (not an approximation): the aikaboom page
 * "11.4d FlashAttention" lists the tiled method's result as the same
 * mathematical result as standard attention (comparison table), and the
 * zimaspace page "How Does Flash Attention Reduce Memory Traffic During Local
 * Inference?" says the tiled algorithm still produces exact attention. It is
 * computed tile by tile with a running (online) softmax, so the score matrix
 * never reaches device memory (aikaboom page, sections "Tiling" and "Online
 * Softmax"; zimaspace page, "Online Softmax Avoids Storing the Full Score
 * Matrix" and "Kernel Fusion Keeps More of the Attention Chain in One
 * Execution Path"). GQA grouping follows the sicorps page's last paragraph
 * (n < n_head key/value heads, each shared by a group of query heads; MQA is
 * Hkv = 1).
 *
 * Conventions shared by all entry points:
 *   - All pointers are DEVICE pointers owned by the caller. The library never
 *     frees or retains them. q, k, v, o, kcache, vcache must be 16-byte
 *     aligned; lse and seqlens 4-byte aligned. Tensors are contiguous.
 *   - Element type: attn_fwd / attn_decode take bfloat16 q, k, v and write
 *     bfloat16 o; the _f16 twins take and write IEEE fp16. lse is float32.
 *     Products accumulate in fp32; softmax statistics are fp32.
 *   - scale must be finite and > 0 (the usual value is 1/sqrt(d)).
 *   - lse may be NULL: the log-sum-exp is then not written.
 *   - Work is enqueued on `stream` (NULL = legacy default stream); calls return
 *     without synchronising. Errors detected on the host return a negative
 *     code before anything is enqueued.
 *   - A row with no visible key (causal with Nq > Nk, or an empty decode
 *     sequence) gets o = 0 and lse = -inf.
 *   - Head size d: d = 64 and d = 128 run on the tensor-core kernels
 *     (tcgen05 MMA, TMA-fed tiles). Any other d that is a multiple of 8 in
 *     [8, 256] runs on a generic CUDA-core kernel with the same results to
 *     rounding (16 query rows per block, 32-key tiles staged in shared
 *     memory, fp32 online softmax); it is correct but far from the tensor-core
 *     kernels' speed. Other d return ATTN_ERR_UNSUPPORTED.
 *   - Every wait inside a kernel is bounded (about 2 s). If one gives up, the
 *     kernel ends early, its outputs are undefined, and
 *     attn_get_device_status() reports ATTN_ERR_TIMEOUT. No kernel traps.
 */
#ifndef EXACT_TILED_ATTENTION_ATTN_H
#define EXACT_TILED_ATTENTION_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; declared here so that callers need no
   CUDA header. */
typedef struct CUstream_st* attn_stream_t;

enum attn_status {
  ATTN_OK = 0,
  ATTN_ERR_INVALID = -1,     /* null pointer, bad size, misaligned, Hq % Hkv != 0, bad scale */
  ATTN_ERR_UNSUPPORTED = -2, /* d not a multiple of 8 in [8, 256]; decode with d = 64 / 128 and
                                B > 65,535; or the device is not sm_100 */
  ATTN_ERR_CUDA = -3,        /* a CUDA runtime call or launch failed */
  ATTN_ERR_TIMEOUT = -4,     /* a device-side wait gave up (see attn_get_device_status) */
  ATTN_ERR_SCRATCH = -5,     /* attn_decode_noalloc: sizes exceed its fixed scratch */
  ATTN_ERR_PAGES = -6        /* bad page ids, lengths or rows in device memory (paged cache; see
                                attn_get_device_status) */
};

/*
 * Prefill: many query tokens against keys/values of the same sequence
 * (aikaboom page, "The Core Problem" and "Tiling"; first page: prefill
 * processes n tokens, so the cost is quadratic).
 *   q   [B, Hq,  Nq, d]  bf16      k, v [B, Hkv, Nk, d] bf16
 *   o   [B, Hq,  Nq, d]  bf16      lse  [B, Hq, Nq] float32 (or NULL)
 *   causal != 0: bottom-right aligned mask, query i sees keys j <= i + Nk - Nq
 *                (equal to the usual lower-triangular mask when Nq == Nk).
 * Sizes: B >= 0, Nq >= 0, Nk >= 0 (B == 0 or Nq == 0: nothing to do;
 * Nk == 0: every row is empty), Hq >= 1, Hkv >= 1, Hq % Hkv == 0,
 * d a multiple of 8 in [8, 256], Nq <= 16,776,960, B * Hq < 2^31.
 * Allocates no device memory.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
             int Hkv, int Nq, int Nk, int d, float scale, int causal, attn_stream_t stream);

/* attn_fwd with IEEE fp16 q, k, v and o. */
int attn_fwd_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                 int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                 attn_stream_t stream);

/*
 * Decode: one new query token per sequence over a ragged KV cache (first
 * page: generating a token re-reads the whole KV cache plus the new entry, a
 * cost linear in the cache length; zimaspace page, "Reduced IO Is Not the Same
 * as Eliminating KV Cache").
 *   q       [B, Hq, d]  bf16
 *   kcache, vcache: packed per sequence. Sequence b starts at token offset
 *           off_b = sum_{j<b} seqlens[j] and is laid out [Hkv][seqlens[b]][d],
 *           i.e. element (b, g, t, c) is at ((off_b * Hkv + g * L_b + t) * d + c).
 *           The new token's key/value must already be appended.
 *           kcache and vcache must be non-NULL even if every sequence is empty.
 *   seqlens [B] int32, DEVICE memory, read only on the device (negative
 *           values count as 0; 0 gives o = 0, lse = -inf).
 *   o       [B, Hq, d]  bf16       lse [B, Hq] float32 (or NULL)
 * Sizes: B >= 0 (0: nothing to do), Hq >= 1, Hkv >= 1, Hq % Hkv == 0,
 * d a multiple of 8 in [8, 256], B * Hq < 2^29; for d = 64 and 128 also
 * B <= 65,535 (larger B returns ATTN_ERR_UNSUPPORTED).
 * Device memory: the call takes one workspace block from cudaMallocFromPoolAsync
 * on `stream` and returns it with cudaFreeAsync on the same stream
 * (stream-ordered; no block outlives the call's work). Its size:
 *   - d = 128 with 2 to 32 query heads per KV head (G = Hq / Hkv), the
 *     persistent tensor-core pass: B * 8 + (B + 1) * 4 bytes of per-sequence
 *     offsets, 16 bytes per SM, and (B * Hkv + SMs - 1) * G * (d + 1) * 4 bytes
 *     of partial results, each part rounded up to 256 bytes;
 *   - other d = 64 and 128 cases, the CUDA-core split pass: nsplit * B * Hq *
 *     (d + 1) * 4 bytes of split partials (nsplit = attn_decode_num_splits),
 *     plus B * 8 bytes of token offsets when B > 1024;
 *   - other d: B * 8 bytes of token offsets when B > 1024, else nothing.
 * The pool is the library's own, one per device, created on first use; it
 * keeps up to 256 MiB of freed blocks cached, so callers that synchronise
 * between calls do not pay for re-mapping device memory each time. The
 * caller's pools are not touched.
 */
int attn_decode(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens,
                void* o, float* lse, int B, int Hq, int Hkv, int d, float scale,
                attn_stream_t stream);

/* attn_decode with IEEE fp16 q, kcache, vcache and o. */
int attn_decode_f16(const void* q, const void* kcache, const void* vcache,
                    const int32_t* seqlens, void* o, float* lse, int B, int Hq, int Hkv, int d,
                    float scale, attn_stream_t stream);

/*
 * attn_decode that allocates nothing. The pages have no counterpart for this
 * entry point; it exists for callers that cannot allocate device memory where
 * they run decode: an engine that gives nearly all of HBM to its own KV-cache
 * pool at start-up, a latency-critical path where an allocator call may lock
 * or synchronise, or a runtime whose memory plan is fixed before serving.
 * Same arguments, layout and results as attn_decode (bf16), except:
 *   - The workspace is a fixed array of 2,097,152 floats (8 MiB) in this
 *     library's device memory, held by every GPU that loads the library
 *     until the process exits. It calls no cudaMalloc/cudaFree and no
 *     allocating library routine.
 *   - Persistent tensor-core pass (d = 128, 2 to 32 query heads per KV head):
 *     when its partial results (sizes as in attn_decode) do not fit, each SM
 *     takes whole (sequence, KV head) segments and writes o and lse itself;
 *     only the per-sequence offsets (under 1 MB for B <= 65,535) are kept in
 *     the array, so these calls are never refused. Results agree with
 *     attn_decode to rounding.
 *   - CUDA-core split pass (other d = 64 and 128 cases): one split needs
 *     B * Hq * (d + 1) floats besides the token offsets of a batch above 1024
 *     sequences. When the usual split count does not fit, fewer splits are
 *     used (results then agree with attn_decode to rounding); when not one
 *     split fits the call returns ATTN_ERR_SCRATCH and enqueues nothing.
 *   - Other d keep only the token offsets of a batch above 1024 sequences in
 *     the array (beyond a million sequences each block sums them itself).
 *   - The first call on a device looks up the array's device address (a
 *     runtime call); make that first call before any stream capture. The
 *     address is remembered with the id of the device's context; after
 *     cudaDeviceReset (a new context) the next call looks it up again, so
 *     make the first call after a reset before any capture too.
 *   - Every call on a device uses the same array, which keeps the previous
 *     call's contents (nothing in it needs to start at zero). Calls that can
 *     overlap on the GPU (different streams without ordering between them)
 *     race on it and give wrong results; order them on one stream or by events.
 */
int attn_decode_noalloc(const void* q, const void* kcache, const void* vcache,
                        const int32_t* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                        int d, float scale, attn_stream_t stream);

/*
 * Sliding-window variants (the "windowing" scheme the zimaspace page names in
 * "Reduced IO Is Not the Same as Eliminating KV Cache", applied as a mask).
 * attn_fwd_window: causal prefill where query i keeps only keys j with
 *   i + (Nk - Nq) - window < j <= i + (Nk - Nq), i.e. its `window` most recent
 *   positions including its own (bottom-right alignment as in attn_fwd).
 *   Key tiles wholly outside every row's window are never loaded.
 * attn_decode_window: the new token of sequence b reads only the last
 *   min(window, L_b) cached tokens (cache layout as in attn_decode).
 * window must be >= 1 (a window at least as long as the keys gives the plain
 * causal / full result). Other arguments, layouts, ownership and errors are
 * those of attn_fwd / attn_decode; the _f16 twins take and write fp16.
 */
int attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                    int Hq, int Hkv, int Nq, int Nk, int d, float scale, int window,
                    attn_stream_t stream);
int attn_fwd_window_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int Hq, int Hkv, int Nq, int Nk, int d, float scale, int window,
                        attn_stream_t stream);
int attn_decode_window(const void* q, const void* kcache, const void* vcache,
                       const int32_t* seqlens, void* o, float* lse, int B, int Hq, int Hkv, int d,
                       float scale, int window, attn_stream_t stream);
int attn_decode_window_f16(const void* q, const void* kcache, const void* vcache,
                           const int32_t* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                           int d, float scale, int window, attn_stream_t stream);

/*
 * Merge of partial results over disjoint key sets (context-parallel prefill:
 * each step computes a query block's attention over one key block with
 * attn_fwd, and the steps' results are folded together). The log-sum-exp
 * identity follows from the running softmax statistics (aikaboom page
 * "11.4d FlashAttention", "Online Softmax"): for one query row,
 *     LSE = ln(e^lse_acc + e^lse_part)
 *     O   = e^(lse_acc - LSE) * o_acc + e^(lse_part - LSE) * o_part.
 *   o_acc    [rows, d] float32, in/out: the running merged O (unrounded)
 *   lse_acc  [rows]    float32, in/out: the running LSE (natural log). A row
 *            whose lse_acc is -inf is empty and its o_acc is NOT read, so an
 *            accumulator starts as lse_acc = -inf with o_acc uninitialised.
 *   o_part   [rows, d] bf16 (attn_merge) or fp16 (attn_merge_f16), and
 *   lse_part [rows]    float32: one partial result, e.g. attn_fwd's o and lse
 *            over a key block (rows = B * Hq * Nq in attn_fwd's layout). A
 *            partial row with lse_part = -inf (no visible key) changes nothing.
 *   o_out    [rows, d] bf16 / fp16, or NULL: if not NULL, also receives the
 *            merged O rounded to nearest (the final merge of a sequence of
 *            merges writes the output this way); rows that stay empty get 0.
 * Sizes: rows >= 0 (0: nothing to do), d a multiple of 8 in [8, 256].
 * Pointers are device pointers owned by the caller; o_acc, o_part and o_out
 * 16-byte aligned, lse_acc and lse_part 4-byte aligned. o_out must not
 * overlap the other arrays. Allocates nothing.
 */
int attn_merge(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part,
               void* o_out, long long rows, int d, attn_stream_t stream);
int attn_merge_f16(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part,
                   void* o_out, long long rows, int d, attn_stream_t stream);

/*
 * Partial results kept in fp32, for a sequence of merges (context-parallel
 * prefill folds one query block's attention over every key block; rounding
 * each partial O to bf16 / fp16 before it is merged would add one rounding per
 * fold). The running-statistics merge is the aikaboom page's "Online Softmax"
 * applied to whole key blocks.
 * attn_fwd_partial / attn_fwd_partial_f16: attn_fwd / attn_fwd_f16 (bf16 /
 *   fp16 q, k, v; same layouts, masks, sizes and errors) except that o is
 *   float32 [B, Hq, Nq, d] holding O = sum_j softmax_j * v_j unrounded
 *   (16-byte aligned). No sliding window. Allocates nothing.
 * attn_merge_partial / attn_merge_partial_f16: attn_merge / attn_merge_f16
 *   with o_part float32 [rows, d] (such a partial O); o_out, if not NULL,
 *   receives the merged O rounded to bf16 / fp16.
 */
int attn_fwd_partial(const void* q, const void* k, const void* v, float* o, float* lse, int B,
                     int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                     attn_stream_t stream);
int attn_fwd_partial_f16(const void* q, const void* k, const void* v, float* o, float* lse, int B,
                         int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                         attn_stream_t stream);
int attn_merge_partial(float* o_acc, float* lse_acc, const float* o_part, const float* lse_part,
                       void* o_out, long long rows, int d, attn_stream_t stream);
int attn_merge_partial_f16(float* o_acc, float* lse_acc, const float* o_part,
                           const float* lse_part, void* o_out, long long rows, int d,
                           attn_stream_t stream);

/*
 * Paged key/value cache.
 *
 * A pool holds num_pages pages of page_size tokens for Hkv KV heads; element
 * (page, head, row, c) is at page * page_stride + head * head_stride +
 * row * token_stride + c, in elements of the pool's type, the same in k and v.
 * Both orders inside a page ([Hkv][page_size][d] and [page_size][Hkv][d]) and
 * pools interleaved with others are described by the strides.
 * Position t of sequence b lies in page table[b * table_width + t / page_size],
 * row t % page_size.
 *
 * New tokens are packed: sequence b has T_b = cu_q[b + 1] - cu_q[b] of them,
 * rows cu_q[b] .. cu_q[b + 1] of the packed tensors (cu_q: B + 1 entries, not
 * decreasing), and kv_lens[b] = L_b cached tokens in all, the new ones
 * included, so that its new token i is at position L_b - T_b + i. cu_q, kv_lens
 * and the table are DEVICE memory, read only on the device.
 *
 * Sizes: d a multiple of 8 in [8, 256], page_size a power of two in [8, 1024]
 * (others: ATTN_ERR_UNSUPPORTED), strides multiples of 8 elements and at least
 * d, k and v 16-byte aligned, num_pages >= 1, table_width >= 1,
 * table_width * page_size <= 2^30, at most 2^29 packed rows.
 *
 * Errors in device data cannot be refused on the host. They are never followed
 * out of bounds: a page id outside [0, num_pages) where a sequence needs a
 * page, lengths beyond the table, decreasing or overlong cu_q, a source row
 * outside [-1, B) make attn_get_device_status() return ATTN_ERR_PAGES (raw code
 * 0x2000 | what), and what the operators give for such a sequence is undefined.
 */
typedef struct attn_pages {
  void* k;
  void* v;
  const int32_t* table;  /* [B][table_width], DEVICE memory */
  long long page_stride; /* strides in elements */
  long long head_stride;
  long long token_stride;
  int num_pages;
  int page_size;
  int table_width;
  int Hkv;
  int d;
} attn_pages;

/*
 * Attention of new tokens over the paged cache: chunked prefill, decode (one
 * new token per sequence) and any mix of the two in one batch. For new token i
 * of sequence b, query head h and KV head g = h / (Hq / Hkv):
 *     s_j = scale * q_i . k_j  for the keys j <= L_b - T_b + i, and, with
 *           window >= 1, j > L_b - T_b + i - window
 *     o_i = sum_j softmax_j(s) v_j,   lse_i = ln sum_j exp(s_j).
 *   q    [total_q][Hq][d], rows of tokens q_stride elements apart (a multiple
 *        of 8, >= Hq * d: q may be a part of a wider projection)
 *   o    [total_q][Hq][d] contiguous     lse [total_q][Hq] float32, or NULL
 *        (neither over q nor over the other: ATTN_ERR_INVALID)
 *   max_q: no sequence has more new tokens than this. It decides which kernel
 *        runs, so a loose bound costs time: with 1 for 64 sequences of a token
 *        each, 1K-8K cached, 32/8 heads, the decode pass takes 190 us where whole
 *        row tiles, which 64 would choose, take 207.
 *   window: 0 for none.
 * The keys and values of the new tokens must be in the cache already
 * (attn_rope_append puts them there). A token that sees no key gets o = 0,
 * lse = -inf; rows of o and lse outside every sequence are left as they were.
 * The probabilities are rounded to q's type before the value product (d <= 128),
 * as in attn_fwd and attn_decode: besides the rounding of o itself, o is off by
 * at most half a step of that type times sum_j softmax_j |v_j| (fp16, whose steps
 * below 2^-14 no longer shrink: and by 2^-25 max_j softmax_j sum_j |v_j|).
 * A NaN or +infinite score at a key that a token sees makes its o and lse NaN;
 * keys with a score of -infinity do not count, and a token that sees no other
 * key is one that sees none.
 * What pages hold behind L_b, and in front of the first position that any new
 * token of the sequence sees under a window, is not looked at, NaN and
 * infinities included; pages wholly in front of it are not needed, and their
 * table entries may hold anything (-1, say, once the page serves another row).
 * Between the two they count as values: the value product runs over whole tiles
 * of 128 keys, so an infinite or NaN v at a position that a token does not see
 * may still reach it where other tokens see it (d <= 128).
 * d <= 128 with at most 128 query heads per KV head runs on the tensor cores
 * (any d below 64 or 128 at the cost of that size), other sizes on a CUDA-core
 * kernel, far from the former's speed.
 * Device memory: one workspace block from the library's pool, as attn_decode.
 * With D = 64 or 128, the least that holds d: max_q * Hq / Hkv <= 32 rows (16
 * for several tokens at d <= 64) take 12 bytes per sequence and per SM
 * 2 * max_q * (Hq / Hkv) * (D + 1) * 4 bytes of partial results; more rows take
 * 3 * 256 * (D + 1) * 4 bytes per SM, and 12 bytes per sequence above 2048 of
 * them; a few hundred bytes come on top. The CUDA-core kernel takes none.
 */
int attn_paged(const void* q, long long q_stride, const attn_pages* cache, const int32_t* cu_q,
               const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q, int max_q,
               float scale, int window, attn_stream_t stream);
int attn_paged_f16(const void* q, long long q_stride, const attn_pages* cache, const int32_t* cu_q,
                   const int32_t* kv_lens, void* o, float* lse, int B, int Hq, int total_q,
                   int max_q, float scale, int window, attn_stream_t stream);

/*
 * Rotary positions. Pair p of a head's first rot values -- values p and
 * p + rot / 2, or 2p and 2p + 1 when interleaved != 0 -- at position n is
 * turned by a = 2 pi n turns[p]:
 *     y_a = amp (x_a cos a - x_b sin a),   y_b = amp (x_b cos a + x_a sin a),
 * and the other d - rot values pass through. backward != 0 gives the gradient
 * of that map: q and k are then the gradients of its outputs (the angle is
 * negated; values and gradients pass alike). The angle is formed in 64 bits,
 * so far positions lose nothing; the rotation runs in fp32 and rounds once.
 *   q, q_out [B, Hq, N, d] and k, k_out [B, Hkv, N, d], by strides in elements:
 *        strides[0..2] batch, head, token of q, [3..5] of q_out, [6..8] of k,
 *        [9..11] of k_out (HOST memory; multiples of 8; d contiguous). An
 *        output may be its input (same pointer, same strides); else it must not
 *        lie over an input or the other output, and its own strides must nest,
 *        so that no two of its values share a place (ATTN_ERR_INVALID; exact for
 *        parts of one tensor). Hq or Hkv may be 0.
 *   pos  int32, DEVICE: pos[b * pos_stride + n] (pos_stride 0: shared)
 *   turns [rot / 2] float64, DEVICE (attn_rope_turns computes them)
 * Sizes: d a multiple of 8 in [8, 256], rot even in [0, d], Hq + Hkv <= 65,535,
 * B * N < 2^31. rot a multiple of 16 runs with 16-byte accesses.
 * Allocates nothing.
 */
int attn_rope(const void* q, void* q_out, const void* k, void* k_out, const long long* strides,
              const int32_t* pos, long long pos_stride, const double* turns, int B, int Hq, int Hkv,
              int N, int d, int rot, float amp, int interleaved, int backward,
              attn_stream_t stream);
int attn_rope_f16(const void* q, void* q_out, const void* k, void* k_out, const long long* strides,
                  const int32_t* pos, long long pos_stride, const double* turns, int B, int Hq,
                  int Hkv, int N, int d, int rot, float amp, int interleaved, int backward,
                  attn_stream_t stream);

/*
 * Rotary positions of a serving step, fused with the append to the cache: the
 * new tokens' q is rotated into q_out, k is rotated into the cache, v is copied
 * into it.
 *   q, q_out [total_q][Hq][d], k, v [total_q][Hkv][d], rows of tokens *_stride
 *        elements apart (multiples of 8, at least a row); q_out may be q (with
 *        its stride), and must not lie over q, k or v otherwise.
 *   pos  [total_q] int32, DEVICE, or NULL: the tokens' positions in the cache.
 * A token at a negative position (T_b > L_b) is not stored. rot = 0 appends
 * without rotating. Pages that several sequences share must not be written:
 * attn_pages_update gives each sequence that grows a last page of its own.
 * Other arguments as in attn_paged and attn_rope. Allocates nothing.
 */
int attn_rope_append(const void* q, long long q_stride, void* q_out, long long q_out_stride,
                     const void* k, long long k_stride, const void* v, long long v_stride,
                     const attn_pages* cache, const int32_t* cu_q, const int32_t* kv_lens,
                     const int32_t* pos, const double* turns, int B, int Hq, int total_q, int rot,
                     float amp, int interleaved, attn_stream_t stream);
int attn_rope_append_f16(const void* q, long long q_stride, void* q_out, long long q_out_stride,
                         const void* k, long long k_stride, const void* v, long long v_stride,
                         const attn_pages* cache, const int32_t* cu_q, const int32_t* kv_lens,
                         const int32_t* pos, const double* turns, int B, int Hq, int total_q,
                         int rot, float amp, int interleaved, attn_stream_t stream);

/*
 * Turns per position of each pair, f_p / 2 pi with f_p = base^(-2p / rot), and
 * the amplitude (1 but for ATTN_ROPE_PARTS). HOST function, HOST memory:
 * turns [rot / 2], amp [1]. rot even in [2, 256], base > 1. Scaling for contexts
 * longer than the original one (factor >= 1):
 *   ATTN_ROPE_LINEAR  f_p / factor
 *   ATTN_ROPE_BASE    base * factor^(rot / (rot - 2)) in place of base (rot >= 4)
 *   ATTN_ROPE_PARTS   pairs with more than `high` turns over `original`
 *                     positions keep f_p, those with fewer than `low` get
 *                     f_p / factor, with a ramp over the pairs between;
 *                     amp = 0.1 ln(factor) + 1
 *   ATTN_ROPE_BANDS   the same with the ramp over the number of turns:
 *                     (original f_p / 2 pi - low) / (high - low); amp = 1
 */
enum attn_rope_scaling {
  ATTN_ROPE_PLAIN = 0,
  ATTN_ROPE_LINEAR = 1,
  ATTN_ROPE_BASE = 2,
  ATTN_ROPE_PARTS = 3,
  ATTN_ROPE_BANDS = 4
};
int attn_rope_turns(double* turns, float* amp, int rot, double base, int scaling, double factor,
                    double low, double high, double original);

/*
 * One step of the cache's bookkeeping: forks, beam steps, ended, new and
 * growing sequences in one call. Row b of the next state goes on from row
 * source[b] of this one (-1: from nothing) and grows by add[b] >= 0 tokens:
 *   - rows that share a source share its full pages. Its last, partly filled
 *     page stays with one of them, the source row itself if it goes on
 *     (source[s] == s), else the first that takes it over; the others get a
 *     copy of it, in all layers of both pools, in a page of their own;
 *   - rows no longer taken over let go of their pages;
 *   - a row gets fresh pages for the tokens that it grows by (their contents
 *     are undefined). Free pages (refs <= 0 after the above) are taken lowest
 *     first, in the order of the rows.
 *   lens, refs, source, add: [B], [num_pages], [B], [B] int32; refs[p] counts
 *        the rows that hold page p (and whoever else pins it). A row of L
 *        tokens holds its first ceil(L / page_size) table entries. An entry of
 *        -1 among them is a page that the row has given up and stays -1: the
 *        caller gives up a full page (in front of a sliding window, say) by
 *        setting the entry to -1 and taking 1 off the page's count.
 *   table_out, lens_out, refs_out: the next state (entries behind a row's pages
 *        are -1). No output may lie over an input or another output.
 *   info [2] int32: pages that were missing, and rows longer than the table
 *        allows. If either is not 0 nothing has changed: the outputs are the
 *        inputs, and no page was copied.
 * All DEVICE memory. Values have 2 bytes; a page's Hkv * page_size * d values
 * must lie in one piece (either order); layer l of the pools begins
 * l * layer_stride elements behind k and v. Whole-number results do not depend
 * on timing. Caches of more than some 25,000 pages, or tables of more than
 * 65,536 entries in all, take one workspace block of (2 B + 3 max(B, num_pages))
 * * 4 bytes and a little more, as in attn_decode; smaller ones none.
 */
int attn_pages_update(const attn_pages* cache, int layers, long long layer_stride,
                      const int32_t* lens, const int32_t* refs, const int32_t* source,
                      const int32_t* add, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                      int32_t* info, int B, attn_stream_t stream);

/*
 * Compaction: with n live pages (refs > 0), the live pages at n and above move,
 * in order, into the free pages below n, in order -- the fewest copies -- in
 * all layers of both pools; the tables and counts follow. info [2]: n, and the
 * pages moved. Other arguments as in attn_pages_update.
 * A page that no row holds but someone else pins (refs counts it) moves like the
 * others. Its holder finds it by the rule above, from the counts before: the
 * k-th page with refs > 0 at n and above is now the k-th page that had refs <= 0
 * below n. Or it keeps the page in a row of the table, which follows by itself.
 */
int attn_pages_compact(const attn_pages* cache, int layers, long long layer_stride,
                       const int32_t* lens, const int32_t* refs, int32_t* table_out,
                       int32_t* refs_out, int32_t* info, int B, attn_stream_t stream);

/* Number of KV splits attn_decode uses for these sizes on the current device
   (>= 1; always 1 for d other than 64 and 128 and for the persistent pass of
   d = 128 with 2 to 32 query heads per KV head, which has no fixed split
   count), or a negative error code. */
int attn_decode_num_splits(int B, int Hq, int Hkv, int d);

/* The cudaError_t value (as an int) behind the calling thread's most recent
   ATTN_ERR_CUDA from this library, or 0 if there was none. */
int attn_last_cuda_error(void);

/* Human-readable text for a return code. Never NULL. */
const char* attn_strerror(int code);

/*
 * Synchronises `stream`, then reads and clears the library's device status
 * word on the current device. Returns ATTN_OK, ATTN_ERR_TIMEOUT (a device
 * wait gave up), ATTN_ERR_PAGES (a paged-cache operator met bad device data) or
 * ATTN_ERR_CUDA. *raw_code, if not NULL, receives the word: 0x1000 | site of
 * the wait, or 0x2000 | what was bad (1 page id, 2 length, 3 rows, 4 source).
 * The word holds the first error since it was last read.
 */
int attn_get_device_status(attn_stream_t stream, unsigned int* raw_code);

/*
 * Test hook for the bounded waits (not part of the attention computation).
 * Enqueues the attn_fwd prefill kernel with the same arguments and checks,
 * but with its TMA producers issuing no copies, so the kernel's first waits
 * for data can never complete; every wait gives up after wait_us
 * microseconds (1..1000000). The kernel then ends early with no copy or
 * tensor-core operation in flight, o and lse are left undefined, and the next
 * attn_get_device_status() returns ATTN_ERR_TIMEOUT with raw code
 * 0x1000 | site (site: which wait gave up first). The CUDA context stays
 * usable. Returns the enqueue status like attn_fwd, or ATTN_ERR_INVALID for
 * wait_us out of range, or ATTN_ERR_UNSUPPORTED for d other than 64 and 128
 * (the generic kernel has no waits).
 */
int attn_fwd_stall_test(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                        unsigned int wait_us, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_TILED_ATTENTION_ATTN_H */
