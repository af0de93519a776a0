/*
 * qgemm_attention.h -- C ABI of the attention operators that stand between two weight-only
 * quantized GEMMs (qgemm.h) on MI355X (gfx950): per-head norm and rotation of queries and keys,
 * a paged key/value cache held in 4 bits, and attention over that cache.
 *
 * Conventions are those of qgemm.h: status codes, qgemm_last_error, caller-owned buffers, calls
 * that validate on the host, enqueue on `stream` and return, no allocation, no exception.
 * 16-bit types are QGEMM_DT_F16 and QGEMM_DT_BF16; one call uses one of them throughout.
 * Every fp32 step below is rounded to 16 bits once, at the stored result.
 *
 * Values that live in device memory (positions, slots, page tables, lengths) cannot be checked on
 * the host.  The kernels bound every one of them before it becomes an address, so a wrong value
 * gives the stated result and never an access outside the buffers.
 */
#ifndef QGEMM_ATTENTION_H
#define QGEMM_ATTENTION_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * qgemm_norm_rope_t -- heads of `tokens` tokens: q [tokens][q_heads][head_dim] and
 * k [tokens][kv_heads][head_dim].
 *   tokens in [0, 2^24]; q_heads in [0, 1024], kv_heads in [0, 1024], not both 0 (more than about 2^36
 *   elements are beyond one launch: UNSUPPORTED);
 *   head_dim 64, 128 or 256; rot_dim a multiple of 8 in [0, head_dim]; max_pos in [1, 2^24]
 *   (rows of the table; ignored for rot_dim 0); dtype F16 or BF16.
 *   norm: 1 = RMS norm of every head first, 0 = rotation only.  eps >= 0 (finite), used with norm.
 *   interleaved: 0 = dim i is paired with i + rot_dim / 2, 1 = dim 2 i with 2 i + 1.
 */
typedef struct qgemm_norm_rope {
  int64_t tokens;
  int32_t q_heads, kv_heads, head_dim, rot_dim, max_pos, dtype, interleaved, norm;
  float eps;
  int32_t reserved;                 /* 0 */
} qgemm_norm_rope_t;

/*
 * qgemm_qk_norm_rope -- enqueue, for every head row x of q (and of k),
 *   y[d] = x[d] / sqrt(mean(x^2) + eps) * w[d]                  (norm = 1; w NULL means ones)
 *   (y[a], y[b]) <- (y[a] c_i - y[b] s_i, y[b] c_i + y[a] s_i)  for the rot_dim / 2 pairs (a, b)
 * in fp32, with c_i = cos_sin[pos][i], s_i = cos_sin[pos][rot_dim / 2 + i], pos = positions[token]
 * (a position outside [0, max_pos) takes the nearest row).
 *   q, k          16-bit; a token's heads are contiguous, tokens are q_stride / k_stride elements
 *                 apart (at least heads * head_dim, a multiple of 8), so both may be slices of one
 *                 projection's output.  q may be NULL when q_heads is 0, k when kv_heads is 0.
 *   q_weight, k_weight  head_dim 16-bit values each, or NULL; ignored for norm = 0.
 *   positions     int32 [tokens]; cos_sin fp32 [max_pos][rot_dim]; both ignored for rot_dim 0.
 *   q_out, k_out  as q, k with their own strides; may be the inputs themselves (same pointer and
 *                 stride), otherwise must not overlap them.
 * Pointers are 16-byte aligned (positions: 4).
 */
qgemm_status_t qgemm_qk_norm_rope(const qgemm_norm_rope_t* problem, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* q_weight, const void* k_weight,
                                  const int32_t* positions, const float* cos_sin, void* q_out, int64_t q_out_stride,
                                  void* k_out, int64_t k_out_stride, void* stream);

/*
 * qgemm_cache_t -- a paged key/value cache in 4 bits.  It holds num_pages pages of page_size token
 * slots; slot s is place s % page_size of page s / page_size.
 *   num_pages in [1, 2^31 - 1]; page_size a multiple of 16 in [16, 4096]; kv_heads in [1, 1024];
 *   head_dim 64, 128 or 256; group_size = head_dim / NG with NG = 1, 2 or 4 (NG 4 needs
 *   head_dim >= 128); dtype F16 or BF16, the type of keys, values and parameters.
 * Values: a group of group_size consecutive dims of one token, head and side (K or V) is held as
 * codes 0..15 and two 16-bit parameters, value = code * scale + zero, with
 *   zero = min, scale = RNE_16((max - min) / 15), code = clamp(rint((x - zero) / scale), 0, 15)
 * in fp32 (code 0 where scale is 0).  A group whose max - min is not finite gets NaN parameters and
 * codes 0: it reads back as NaN.
 * Layout: one block of bytes per (page, kv head), pages outermost:
 *   [K codes][V codes][K parameters][V parameters], with P = page_size, D = head_dim, u = D / 32
 *   K codes: a row of D / 2 bytes per token; dword u g + i of the row (g = 0..3, i < u) holds dims
 *     8 (4 i + g) .. + 7, the first in the low nibble: 16 tokens' rows are one MFMA A operand of
 *     S^T = K Q^T in lane order (lane l: token l & 15, g = l >> 4, i = the 32-wide step), whatever
 *     NG is, since a step never leaves its group.
 *   V codes: byte ((t / 4) * 16 + r) * 4 u + (t % 4) u + i / 2, nibble i % 2, holds dim 16 i + r of
 *     token t (r = 0..15): lane r of an MFMA A operand of O^T = V^T P^T finds four tokens of its
 *     dims 16 i + r side by side.
 *   parameters: [NG][P][scale, zero].
 */
typedef struct qgemm_cache {
  int64_t num_pages;
  int32_t page_size, kv_heads, head_dim, group_size, dtype;
  int32_t reserved;                 /* 0 */
} qgemm_cache_t;

/* qgemm_cache_bytes -- bytes of the cache buffer: num_pages * kv_heads * page_size * (D + 8 NG). */
qgemm_status_t qgemm_cache_bytes(const qgemm_cache_t* cache, size_t* bytes);

/*
 * qgemm_cache_write -- enqueue the quantization of `tokens` tokens into their slots.
 *   data    the cache buffer, 16-byte aligned; every other slot keeps its bytes.
 *   k, v    16-bit [tokens][kv_heads][head_dim] with token strides k_stride / v_stride (elements, a
 *           multiple of 8, at least kv_heads * head_dim); 16-byte aligned.
 *   slots   int64 [tokens]; a slot outside the cache (e.g. -1, padding) is skipped.  Slots of one
 *           call are distinct.
 * tokens in [0, 2^24]; more than about 2^35 elements of k are beyond one launch: UNSUPPORTED.
 */
qgemm_status_t qgemm_cache_write(const qgemm_cache_t* cache, void* data, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, const int64_t* slots, int64_t tokens, void* stream);

/*
 * qgemm_cache_read -- enqueue k_out, v_out [tokens][kv_heads][head_dim] (contiguous) = the values of
 * the slots, code * scale + zero in fp32, rounded to dtype; zeros for a slot outside the cache.
 */
qgemm_status_t qgemm_cache_read(const qgemm_cache_t* cache, const void* data, const int64_t* slots, int64_t tokens,
                                void* k_out, void* v_out, void* stream);

#define QGEMM_ATTENTION_AUTO 0
#define QGEMM_ATTENTION_ROWS 1      /* tokens of the cache over the wavefronts: few query rows per kv head */
#define QGEMM_ATTENTION_TILES 2     /* query rows over the wavefronts: many query rows per kv head         */

/*
 * qgemm_attention_t -- attention of `batch` sequences over the cache.
 *   total_q in [0, 2^24] query tokens in all; batch in [1, 65535]; q_heads a multiple of
 *   cache.kv_heads, at most 4096 (query head h reads kv head h / (q_heads / kv_heads));
 *   max_q_len in [1, total_q]: an upper bound of a sequence's query tokens; max_pages: the columns
 *   of the page table, max_pages * page_size <= 2^30;
 *   causal 0 or 1; window 0, or with causal the number of latest positions a query sees (>= 1);
 *   scale finite, the factor on q . k.  Queries, keys, values, scale and scale * q . k of up to 2^100 in magnitude
 *   are covered; beyond that fp32 steps may overflow.
 *   kernel_hint QGEMM_ATTENTION_* (testing and tuning; 0 is the right choice for applications).
 * The launch depends on the descriptor only, never on lengths in device memory.
 */
typedef struct qgemm_attention {
  qgemm_cache_t cache;
  int64_t total_q;
  int32_t batch, q_heads, max_q_len, max_pages, causal, window;
  float scale;
  int32_t kernel_hint;
  int32_t reserved[2];              /* 0 */
} qgemm_attention_t;

/* qgemm_attention_workspace_bytes -- device workspace of qgemm_attention: zero-filled once by the
 * caller, then reusable by later calls in stream order.  One workspace of the largest size asked for
 * serves any descriptors; calls that overlap in time need different ones. */
qgemm_status_t qgemm_attention_workspace_bytes(const qgemm_attention_t* problem, size_t* bytes);

/*
 * qgemm_attention -- enqueue out = softmax(scale * q . k^T) v over the cache's values.
 *   q, out      16-bit [total_q][q_heads][head_dim], token strides q_stride / out_stride (elements, a
 *               multiple of 8, at least q_heads * head_dim); 16-byte aligned; no overlap.
 *   data        the cache buffer.
 *   page_table  int32 [batch][max_pages]: the pages of each sequence in order (an entry outside
 *               [0, num_pages) reads page 0; entries past the length are not read).
 *   seq_lens    int32 [batch]: tokens of the sequence in the cache, this call's included (bounded to
 *               [0, max_pages * page_size]).
 *   q_start     int32 [batch + 1]: sequence b owns query rows q_start[b] .. q_start[b + 1] - 1, at most
 *               max_q_len, none is fine (also where it decreases); rows of no sequence keep their output.  Where
 *               the sequences claim more than total_q rows in all, the call writes nothing.
 * Query i of n of a sequence of length L stands at position L - n + i.  It sees positions t < L, with
 * causal t <= its own, with window t > its own - window.  A query that sees nothing gets zeros.  Bits
 * in slots that no query sees (unwritten pages, the rest of the last page) never reach the output.
 * Scores, the softmax's maximum and sum and the output are accumulated in fp32.  The weights that multiply
 * the codes, each times its value scale, are rounded to fp16: 11 bits, and no less than 2^-31 of the largest such
 * product, in the rows kernel of the row and group, in the tiles kernel of the row, where the groups' scales
 * count relative to their means over the first 64 tokens (32 for head_dim 256) of a workgroup's part.  The tiles
 * kernel over a BF16 cache also rounds the values to fp16, in units of a power of two per token, groups likewise relative to
 * their means: to 11 bits, three more than BF16 holds, down to 2^-14 of the token's largest, and to 2^-25 of it
 * below; and it holds keys in several groups exactly while a group's scale is at least 2^-25 of the token's
 * largest.  Results are bitwise deterministic.
 */
qgemm_status_t qgemm_attention(const qgemm_attention_t* problem, const void* q, int64_t q_stride, const void* data,
                               const int32_t* page_table, const int32_t* seq_lens, const int32_t* q_start, void* out,
                               int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream);

/* qgemm_attention_describe -- as qgemm_plan_describe: one line naming the launch. */
qgemm_status_t qgemm_attention_describe(const qgemm_attention_t* problem, char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_ATTENTION_H */
