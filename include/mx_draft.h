/*
 * mx_draft.h -- C ABI of the gfx950 microscaling library, drafted tokens: what a decoding step with a
 * tree of drafted tokens needs around the paged MXFP4 cache of mx_attention.h.  Masks and positions of
 * trees given by their nodes' parents, attention of the nodes over the cache, verification of the
 * drafted tokens against the target's probabilities from given random numbers, and the move of the
 * accepted path's keys and values to their places.  Nothing has to come back to the host between
 * them: a captured graph of the whole step serves growing sequences.
 *
 * The entry points live in the same library, return the same status codes and keep the conventions of
 * mx_attention.h: caller-owned device buffers, nothing allocated or synchronized, argument errors
 * before any HIP call, structs of 8-byte fields.
 *
 * Trees.  The nodes of all sequences lie one after the other: sequence b's are rows q_starts[b] ..
 * q_starts[b + 1] of every [total_q] buffer (at most max_q of them), or rows b * max_q ..
 * (b + 1) * max_q when q_starts is NULL; rows behind the last sequence's are neither read nor written.
 * Node 0 is the root, the last token of the text (its key and value are not cached before the step);
 * the others are drafted.  parents[i] is the number of node i's parent in its sequence and is less than
 * i; a node whose parent is not in [0, i) has none.  seq_lens[b] counts the cached tokens of sequence b
 * with its nodes: node i is cached as token seq_lens[b] - n + i of n nodes, whatever its depth.
 * q_starts and seq_lens are read on the device and clamped to total_q, max_q and what a page table
 * covers.  Outputs must not lie on each other, nor on inputs: MX_ERR_STRIDE (mx_attn_tree_fp4 does not look
 * for the latter).
 */
#ifndef MX_DRAFT_H_
#define MX_DRAFT_H_

#include "mx_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * mx_tree_mask -- for every node, which nodes of its sequence are itself or its ancestors: bit
 * j % 32 of word j / 32 of the node's row of `mask` for node j (all mask_words words are written),
 * and positions[node] = seq_lens[b] - n + depth, depth the number of its ancestors: where the node's
 * token would stand if its path were the text, as rotations and windows count it.
 * positions and seq_lens: both, or both NULL.  max_q at most 1024, mask_words at least max_q / 32
 * rounded up.  Rows of `mask` must not lie on each other.
 * Every word of a mask follows the node's ancestors, so the time grows with depth times nodes times words: 2
 * us for trees as deep as drafts are, but chains take 6 us with 64 nodes, 18 with 129, 0.54 ms with 512 and 4.3 ms
 * with 1024.
 */
typedef struct mx_tree_mask_args {
  const int32_t* parents;                         /* [total_q]                                */
  const int32_t* seq_lens;                        /* [batch] or NULL                          */
  const int32_t* q_starts;                        /* [batch + 1] or NULL                      */
  int32_t* mask;                                  /* [total_q, mask_words]                    */
  int32_t* positions;                             /* [total_q] or NULL                        */
  int64_t mask_stride, mask_words;
  int64_t batch, total_q, max_q;
} mx_tree_mask_args;

int mx_tree_mask(const mx_tree_mask_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * mx_attn_tree_fp4 -- mx_attn_fp4 for queries that are a tree's nodes, or any whose view of each
 * other a mask says: of the tokens before the tree (first = seq_lens[b] - n of them) a query sees
 * all, or those t > position - window where window > 0, position being positions[row] clamped to
 * [first, seq_lens[b] - 1]; of the tree's tokens, first + j for node j, it sees those whose bit j of
 * its row of `mask` is set (as mx_tree_mask writes them; bits past the nodes are ignored, and the
 * window takes none of these).  mask rows may be the same one (mask_stride 0).  positions may be NULL
 * without a window.  max_q at most 65536, mask_words at least max_q / 32 rounded up.
 * Everything else (arguments, formulas, roundings, limits, what lies beyond lengths, rows that see
 * nothing, the workspace and its size) is as in mx_attn_fp4.  A chain's nodes are off from what mx_attn_fp4's
 * causal mask gives by the roundings at most: trees are summed in other runs.  Nodes that no query sees are hidden
 * like other masked keys, any key bytes but values that are finite: where seq_lens counts padding nodes that are
 * never appended, their places have to hold some (zeros will do).
 */
typedef struct mx_attn_tree_fp4_args {
  const mx_kv_cache_fp4* cache;
  const void* q;                                  /* bf16 [total_q, q_heads, head_dim]        */
  void* out;                                      /* bf16 [total_q, q_heads, head_dim]        */
  float* lse;                                     /* fp32 [total_q, q_heads] or NULL          */
  const int32_t* mask;                            /* [total_q, mask_words]                    */
  const int32_t* positions;                       /* [total_q] or NULL                        */
  const int32_t* page_table;                      /* [batch, table_width]                     */
  const int32_t* seq_lens;                        /* [batch]                                  */
  const int32_t* q_starts;                        /* [batch + 1] or NULL                      */
  void* workspace;
  int64_t workspace_bytes;
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int64_t mask_stride, mask_words;
  int64_t table_stride, table_width;
  int64_t batch, total_q, max_q, q_heads;
  int64_t window;
  double scale;
} mx_attn_tree_fp4_args;

int mx_attn_tree_fp4(const mx_attn_tree_fp4_args* args, void* stream);

/* ---------------------------------------------------------------------------------------------
 * mx_tree_verify -- which drafted tokens stand, and the token after them, so that what is emitted is
 * distributed as if drawn from the target alone.  Row i of `target` is the target's distribution of the
 * token after node i's path, row i of `draft` the one that node i's children were drawn from.  From
 * the root on, a node's children are tried in their order; with p and q the node's rows, c = 0, S = 1
 * and Q = 1 at first, a child of token x and random number u = accept_u[child] is accepted when
 *     r(x) > 0 and u q(x) S < r(x) Q,   r(v) = max(p(v) - c q(v), 0),
 * and the walk goes on from it.  Rejected, c grows by S / Q, then Q shrinks by q(x) if the children
 * were drawn without replacement, and S becomes the sum of r(v) over the vocabulary (that of the
 * target's distribution given the rejections, up to its size; where Q is not positive the node's
 * other children are rejected as they are).  Where no child is left, the next token is the first v
 * at which the sum of r up to v exceeds sample_u[b] times the sum of all (the last v with r(v) > 0 if
 * none does; if r is 0 everywhere, p takes its place; -1 if p is 0 too).
 * draft == NULL: the drafts were chosen, not drawn (the most probable tokens, say).  A child is accepted
 * when p(x) > 0 and u S < p(x); a rejected token leaves r, and S shrinks by p(x) (to 0 at least).
 *
 * Entries that are negative, infinite or NaN count as 0, tokens outside [0, vocab) have probability 0.
 * Random numbers are meant to lie in [0, 1).  Probabilities are read in their type and computed with
 * in 64 bits; the order of the sums does not depend on what else runs, so the same call gives the same
 * tokens.
 *
 * path[b]: the accepted nodes, the root first, then -1.  tokens_out[b]: their tokens without the
 * root's, then the next token, then -1.  count[b]: the number of either, 0 for a sequence of no nodes.
 * `width` is that of both outputs, batch * width below 2^31; nodes deeper than width - 1 are not tried.
 * type: 0 fp32, 1 bf16, 2 fp16, of both matrices; row strides at least vocab (draft's 0: one row for
 * all), at most 2^30; rows need no alignment past their type's.  max_q at most 1024, vocab in [1, 2^30].
 * workspace: mx_tree_verify_workspace_size bytes, 256-byte aligned, zero before its first use and left
 * reusable; it may be one of mx_attn_fp4 that is as large.  Calls that may overlap need workspaces of
 * their own.
 */
typedef struct mx_tree_verify_args {
  const void* target;                             /* [total_q, vocab]                         */
  const void* draft;                              /* [total_q, vocab] or NULL                 */
  const int32_t* tokens;                          /* [total_q]                                */
  const int32_t* parents;                         /* [total_q]                                */
  const float* accept_u;                          /* [total_q]                                */
  const float* sample_u;                          /* [batch]                                  */
  const int32_t* q_starts;                        /* [batch + 1] or NULL                      */
  int32_t* path;                                  /* [batch, width], contiguous               */
  int32_t* tokens_out;                            /* [batch, width], contiguous               */
  int32_t* count;                                 /* [batch]                                  */
  void* workspace;
  int64_t workspace_bytes;
  int64_t target_stride, draft_stride;
  int64_t batch, total_q, max_q, vocab, width;
  int64_t type, replacement;
} mx_tree_verify_args;

int mx_tree_verify(const mx_tree_verify_args* args, void* stream);
int64_t mx_tree_verify_workspace_size(int64_t batch);

/* ---------------------------------------------------------------------------------------------
 * mx_kv_accept_fp4 -- in each of `layers` caches of one geometry (sizes and strides) that share a page
 * table, the keys and values of token first + path[b][i] of sequence b become those of token first + i,
 * for i < count[b], where first = seq_lens[b] - n for n nodes: the accepted path becomes the text.  Bytes
 * are moved as they are (a key is rotated for its depth already).  path [batch, width], contiguous,
 * rises strictly from 0 on, as mx_tree_verify writes it: then the rows are as if all were read before any
 * is written.  Entries outside [0, n), and tokens before 0 or past what the page table covers,
 * move nothing; page table entries outside [0, pages) neither.
 * lens_out (or NULL): first + count[b], at least 0: the sequences' lengths without what was rejected.
 * It is written without layers too (layers 0, say on a stage that has no attention; `caches` not NULL but
 * not read): there is no page size then, so lengths are taken as they are, negative ones as 0.  With layers 0
 * and caches NULL the call does nothing, lens_out or not.
 * Blocks of a cache must not lie on each other, nor those of two layers (the same cache twice is
 * refused), nor keys on values; a page that holds nodes belongs to one sequence.  layers at most 1024.
 */
typedef struct mx_kv_accept_fp4_args {
  const mx_kv_cache_fp4* caches;                  /* host array of `layers`                   */
  const int32_t* page_table;                      /* [batch, table_width]                     */
  const int32_t* seq_lens;                        /* [batch]                                  */
  const int32_t* q_starts;                        /* [batch + 1] or NULL                      */
  const int32_t* path;
  const int32_t* count;                           /* [batch]                                  */
  int32_t* lens_out;                              /* [batch] or NULL                          */
  int64_t layers, table_stride, table_width;
  int64_t batch, total_q, max_q, width;
} mx_kv_accept_fp4_args;

int mx_kv_accept_fp4(const mx_kv_accept_fp4_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif  /* MX_DRAFT_H_ */
