/*
 * mx_attention.h -- C ABI of the gfx950 microscaling library, attention part: per-head norm of
 * queries and keys with the position rotation in the same pass (and its gradients), appending
 * keys and values to a paged MXFP4 cache with the rotation applied on the way, and attention
 * over that cache.  The entry points live in the same library as those of mx.h, return the same
 * status codes, and keep its conventions:
 *   - every buffer is device memory owned by the caller; nothing is allocated, freed or
 *     synchronized; work is enqueued on `stream` (a hipStream_t; NULL = the null stream);
 *   - argument errors are returned before any HIP call; calls with no tokens return MX_OK and
 *     enqueue nothing (except mx_qk_norm_rope_backward's weight gradients, which are zero then);
 *   - strides are counted in elements of each buffer (bf16 elements for bf16 buffers, bytes for
 *     code and scale buffers).
 *
 * The cache.  Keys and values of a token are MXFP4 rows of head_dim values, as mx_act_quant_fp4
 * writes them: packed E2M1 [head_dim / 2] (low nibble first) with one E8M0 byte per 32 values
 * [head_dim / 32].  `page_size` tokens of one head form a block with its tokens contiguous:
 * codes [pages, kv_heads, page_size, head_dim / 2], scales [pages, kv_heads, page_size,
 * head_dim / 32], with any page and head strides (multiples of 16 bytes, the same for keys and
 * values).  Slot s of the cache is token s % page_size of page s / page_size.  Where tokens are
 * appended, blocks must not lie on each other.
 * head_dim is 64, 128 or 256; page_size is a positive multiple of 16; pages * page_size < 2^31.
 * Attention takes no page of 2^20 tokens or more (its limits on pages and tables are with it, below).
 *
 * Arguments travel in structs of 8-byte fields (pointers, int64_t, double): no padding, and a
 * caller in any language can pack them.
 */
#ifndef MX_ATTENTION_H_
#define MX_ATTENTION_H_

#include <stdint.h>

#include "mx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mx_kv_cache_fp4 {
  void* k;               /* packed E2M1, 16-byte aligned                                      */
  void* k_scale;         /* E8M0, 16-byte aligned                                             */
  void* v;
  void* v_scale;
  int64_t pages, kv_heads, page_size, head_dim;
  int64_t code_page_stride, code_head_stride;     /* bytes, multiples of 16                   */
  int64_t scale_page_stride, scale_head_stride;   /* bytes, multiples of 16                   */
} mx_kv_cache_fp4;

/* ---------------------------------------------------------------------------------------------
 * Position rotation, shared by the calls below.  `positions` is int32 [tokens]; `cos` and `sin`
 * are fp32 [table_rows, rot / 2], contiguous and 16-byte aligned.  The first `rot` values of a
 * head are rotated (rot a positive multiple of 16, at most head_dim); with (c, s) entry i of the
 * token's row, the pair (a, b) becomes (a c - b s, b c + a s), where (a, b) is values
 * (i, i + rot / 2), or (2 i, 2 i + 1) when `interleaved` is non-zero.  positions == NULL: no
 * rotation (cos, sin, table_rows and rot are ignored).  A token whose position lies outside the
 * table has no rotation: its rows become NaN.
 *
 * mx_qk_norm_rope -- for every token and head of q (and k), in fp32 with one rounding to bf16:
 *   x' = R(position) (x * rsqrt(mean(x^2) + eps) * weight)
 * weight: bf16 [head_dim], or NULL for no norm (rotation alone).  An output may be its input.
 * k == NULL: queries alone (k_heads is then ignored).
 * Row starts must be 8-byte aligned (bases 8-byte aligned, strides multiples of 4 elements);
 * weights 8-byte aligned. tokens * heads < 2^31.
 */
typedef struct mx_qk_norm_rope_args {
  const void* q;                                  /* bf16 [tokens, q_heads, head_dim]         */
  const void* k;                                  /* bf16 [tokens, k_heads, head_dim] or NULL */
  void* q_out;
  void* k_out;
  const void* q_weight;
  const void* k_weight;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
  int64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
  int64_t tokens, q_heads, k_heads, head_dim;
  int64_t table_rows, rot, interleaved;
  double eps;
} mx_qk_norm_rope_args;

int mx_qk_norm_rope(const mx_qk_norm_rope_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Gradients of mx_qk_norm_rope.  With dy the gradient of an output row, n = R^T dy, r =
 * rsqrt(mean(x^2) + eps) and g = n * weight:
 *   dx = r (g - x r^2 mean(g x)),  dweight = sum over tokens and heads of n x r  (fp32 [head_dim])
 * and without a weight dx = R^T dy.  dx may be dy.  dq_weight / dk_weight are written (not added
 * to), and may be NULL when not wanted (always when there is no weight).  The sums are taken in
 * one fixed order: the same call gives the same bits.
 * workspace: mx_qk_norm_rope_backward_workspace_size bytes, 256-byte aligned, zero before its
 * first use and left reusable by every call; needed only where a weight gradient is summed, so not
 * without tokens (the size is 0 then).
 * Calls that may overlap need workspaces of their own.  Not to be shared with mx_attn_fp4: this call
 * leaves partial results where that one expects zeros.
 */
typedef struct mx_qk_norm_rope_backward_args {
  const void* dq_out;                             /* bf16 [tokens, q_heads, head_dim]         */
  const void* dk_out;                             /* or NULL                                  */
  const void* q;
  const void* k;
  void* dq;
  void* dk;
  const void* q_weight;
  const void* k_weight;
  float* dq_weight;
  float* dk_weight;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  void* workspace;
  int64_t workspace_bytes;
  int64_t dq_out_token_stride, dq_out_head_stride, dk_out_token_stride, dk_out_head_stride;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
  int64_t dq_token_stride, dq_head_stride, dk_token_stride, dk_head_stride;
  int64_t tokens, q_heads, k_heads, head_dim;
  int64_t table_rows, rot, interleaved;
  double eps;
} mx_qk_norm_rope_backward_args;

int mx_qk_norm_rope_backward(const mx_qk_norm_rope_backward_args* args, void* stream);
int64_t mx_qk_norm_rope_backward_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                                int64_t head_dim);

/* ---------------------------------------------------------------------------------------------
 * mx_kv_append_fp4 -- writes the keys and values of `tokens` new tokens into slots[token] of the
 * cache: the key rotated in fp32 (each product rounded, then their sum; no fused multiply-add),
 * then both quantized per 32 values of the head by the rule of mx_act_quant_fp4, from the fp32
 * values, with no rounding to bf16 in between.  A slot outside [0, pages * page_size) skips its
 * token (-1 marks padding).  No two tokens of a call may share a slot.
 * k_out / v_out (or NULL): the values that were stored, bf16 [tokens, kv_heads, head_dim]
 * contiguous: exactly what the attention will read (rows of skipped tokens are not written).
 * A token and head whose key or value holds NaN, an infinity, or a magnitude above 6 * 2^125
 * (which no finite code stands for), or whose position lies outside the table, is stored with
 * key scale bytes 255 (NaN) and zero codes: every query that sees it gets NaN, every other
 * query is untouched; its k_out and v_out rows are NaN.
 * Row starts of k and v must be 16-byte aligned (bases 16-byte aligned, strides multiples of 8).
 */
typedef struct mx_kv_append_fp4_args {
  const mx_kv_cache_fp4* cache;
  const void* k;                                  /* bf16 [tokens, kv_heads, head_dim]        */
  const void* v;
  const int64_t* slots;                           /* [tokens]                                 */
  const int32_t* positions;
  const float* cos;
  const float* sin;
  void* k_out;
  void* v_out;
  int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  int64_t tokens, table_rows, rot, interleaved;
} mx_kv_append_fp4_args;

int mx_kv_append_fp4(const mx_kv_append_fp4_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * mx_attn_fp4 -- attention of new queries over the cache.  Sequence b holds seq_lens[b] cached
 * tokens (its new ones included), found through page_table[b]: token t is token t % page_size of
 * page page_table[b][t / page_size].  Its queries are rows q_starts[b] .. q_starts[b + 1] of q
 * (at most max_q of them), or rows b * max_q .. (b + 1) * max_q when q_starts is NULL; query i of
 * n stands at position seq_lens[b] - n + i.  Query head h reads key/value head
 * h / (q_heads / kv_heads).  Key t is seen by a query at position p when
 *   t < seq_lens[b], and, if causal, t <= p, and, if window > 0, t > p - window
 * (window > 0 needs causal).  In fp32:
 *   s_t = scale * q . k_t;  out = sum_t softmax(s)_t v_t, rounded once to bf16;
 *   lse (or NULL) = ln sum_t exp(s_t), fp32 [total_q, q_heads].
 * A query that sees no key gets zeros and lse -infinity.  What lies in the cache beyond a
 * sequence's length, or before the window of its first query, is never used, whatever its bytes
 * (pages that hold nothing else may be freed, and their table entries be anything).  Among the tokens
 * between, a query's mask hides keys of any bytes but only finite values: a value scale byte of 253
 * to 255, which mx_kv_append_fp4 never stores, can make queries NaN that do not see its token.
 * |scale| must be below 1e30.
 * Pages and tables that attention takes: table_width * page_size at most 2^31 - 1024, and
 * table_width * (page_size / 16)^2 < 2^32.  The second allows pages of up to 2^20 - 16 tokens, in
 * tables of 1 page then; pages of 65536 tokens in tables of 255; pages of 496 and less in any.
 * seq_lens, q_starts and page_table entries are read on the device: lengths are clamped to what
 * the table covers, and an entry outside [0, pages) reads page 0 instead of memory that is not
 * the cache's.
 * workspace: mx_attn_fp4_workspace_size bytes, 256-byte aligned, zero before its first use and left
 * reusable by every call; the size depends on the sizes alone, not on lengths, and suffices for every
 * smaller max_q and batch too.  One workspace serves calls of any sizes it is large enough for;
 * calls that may overlap need workspaces of their own.  The size covers mx_attn_tree_fp4 (mx_draft.h) as well,
 * which needs more of it with 33 to 64 rows of heads of 128 (43 MB, mx_attn_fp4 itself 26) and 17 to 32 of
 * heads of 256 (77 and 26): mx_attn_fp4 is content with what it needs itself.  q and out rows must be 16-byte aligned
 * (bases 16-byte aligned, strides multiples of 8 elements).
 * At most 64 rows (queries of a sequence times q_heads / kv_heads; 32 with heads of 256) take a path
 * bound by reading the cache, for at most 2^21 sequences times kv_heads; more rows one bound by the
 * matrix instructions.
 * Rounding: products of bf16 queries and exactly decoded keys are summed in fp32; weights
 * exp(s - m) are rounded to bf16 for their product with the exactly decoded values, summed in
 * fp32; the softmax's maximum and sum stay in fp32.  The sum over the values is divided by that of
 * the weights at the end, and a weight may reach 2^8: values times 2^8 times the number of tokens
 * that share the weight have to stay within fp32's range.
 */
typedef struct mx_attn_fp4_args {
  const mx_kv_cache_fp4* cache;
  const void* q;                                  /* bf16 [total_q, q_heads, head_dim]        */
  void* out;                                      /* bf16 [total_q, q_heads, head_dim]        */
  float* lse;
  const int32_t* page_table;                      /* [batch, table_width]                     */
  const int32_t* seq_lens;                        /* [batch]                                  */
  const int32_t* q_starts;                        /* [batch + 1] or NULL                      */
  void* workspace;
  int64_t workspace_bytes;
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int64_t table_stride, table_width;
  int64_t batch, total_q, max_q, q_heads;
  int64_t causal, window;
  double scale;
} mx_attn_fp4_args;

int mx_attn_fp4(const mx_attn_fp4_args* args, void* stream);
int64_t mx_attn_fp4_workspace_size(int64_t batch, int64_t max_q, int64_t q_heads,
                                   int64_t kv_heads, int64_t head_dim);

#ifdef __cplusplus
}
#endif

#endif  /* MX_ATTENTION_H_ */
