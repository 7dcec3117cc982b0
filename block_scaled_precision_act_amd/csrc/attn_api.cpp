// C ABI of the attention operators (declared in include/mx_attention.h, and the attention of a tree of
// drafted tokens in include/mx_draft.h): argument checks on the host, then one launch on the caller's
// stream.
#include "../../include/mx_draft.h"
#include "attn_checks.h"

#include <cfloat>
#include <cmath>

namespace {

using namespace mx;

int rotation_status(const int32_t* positions, const float* cos, const float* sin, int64_t rows,
                    int64_t rot, int64_t head_dim) {
  if (!positions) return MX_OK;
  if (rows < 0 || rows > kMax31 || rot <= 0 || rot % 16 != 0 || rot > head_dim) return MX_ERR_SHAPE;
  if (!cos || !sin) return MX_ERR_NULL;
  if (!aligned(cos, 16) || !aligned(sin, 16)) return MX_ERR_ALIGN;
  return MX_OK;
}

mx::Rotation rotation(const int32_t* positions, const float* cos, const float* sin, int64_t rows,
                      int64_t rot, int64_t interleaved) {
  if (!positions) return mx::Rotation{nullptr, nullptr, nullptr, 0, 0, false};
  return mx::Rotation{positions, cos, sin, static_cast<uint32_t>(rows), static_cast<int>(rot),
                      interleaved != 0};
}

// tokens and heads of the norm calls; k_heads counts only when there are keys.
int norm_shape_status(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                      double eps) {
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || !head_dim_ok(head_dim) || tokens > kMax31 ||
      q_heads > 65535 || k_heads > 65535 || !fits31(tokens, q_heads + k_heads) || !(eps >= 0))
    return MX_ERR_SHAPE;
  return MX_OK;
}

int64_t norm_back_workspace(int64_t head_dim) {
  return mx::kNormBackCounterBytes + mx::kNormBackGroups * head_dim * 4;
}

// A tree's mask (mx_draft.h), in place of a causal one.
struct Tree {
  const int32_t* mask;
  const int32_t* positions;
  int64_t stride, words;
};
constexpr int64_t kMostMaskedQueries = 65536;

int tree_status(const Tree& t, int64_t max_q, int64_t window) {
  if (max_q > kMostMaskedQueries || t.words < (max_q + 31) / 32 || t.words > kMax31) return MX_ERR_SHAPE;
  if (t.stride < 0) return MX_ERR_STRIDE;
  if (!t.mask || (window > 0 && !t.positions)) return MX_ERR_NULL;
  return aligned(t.mask, 4) && aligned(t.positions, 4) ? MX_OK : MX_ERR_ALIGN;
}

int attend(const mx_attn_fp4_args& args, const Tree* tree, void* stream) {
  const mx_attn_fp4_args* const a = &args;
  int st = cache_status(a->cache);
  if (st != MX_OK) return st;
  const mx_kv_cache_fp4& c = *a->cache;
  if (a->batch < 0 || a->batch > 65535 || a->total_q < 0 || a->max_q < 0 || a->q_heads <= 0 ||
      a->q_heads % c.kv_heads != 0 || !fits31(a->total_q, a->q_heads) ||
      !fits31(a->max_q, a->q_heads) || !fits31(a->batch, c.kv_heads) || a->table_width < 0 ||
      a->window < 0 || a->window > kMax31 || (a->window > 0 && !a->causal && !tree) ||
      !(std::fabs(a->scale) < 1e30))
    return MX_ERR_SHAPE;
  if (!a->q_starts && a->total_q != a->batch * a->max_q) return MX_ERR_SHAPE;
  // Tokens a table row covers: the kernels count in 31 bits, and look up to kLookAhead tokens past a
  // length.  And the exactness of the page number as a high product.
  if (!fits31(a->table_width, c.page_size) || a->table_width * c.page_size > kMax31 + 1 - mx::kLookAhead)
    return MX_ERR_SHAPE;
  const int64_t d = c.page_size / 16;
  if (a->table_width * d * d >= (int64_t{1} << 32)) return MX_ERR_SHAPE;
  if (a->table_stride < 0 || (a->batch > 1 && a->table_stride < a->table_width))
    return MX_ERR_STRIDE;
  if (a->batch == 0 || a->total_q == 0 || a->max_q == 0) return MX_OK;
  if (!a->seq_lens || (a->table_width > 0 && !a->page_table)) return MX_ERR_NULL;
  if (tree && (st = tree_status(*tree, a->max_q, a->window)) != MX_OK) return st;
  if ((st = first_error({rows_status(a->q, a->q_token_stride, a->q_head_stride, 8),
                         output_status(a->out, a->out_token_stride, a->out_head_stride, a->total_q,
                                       a->q_heads, c.head_dim, 8)})) != MX_OK)
    return st;
  mx::AttnPlan plan = mx::plan_attn(a->batch, a->max_q, a->q_heads, c.kv_heads,
                                    static_cast<int>(c.head_dim), tree != nullptr);
  // The deal of tiles of 128 tokens (plus a few slots for each sequence and head) counts in 31 bits.
  const int64_t units = a->batch * c.kv_heads;
  if (plan.few && (units > mx::kMaxUnits || !fits31(units, a->table_width * c.page_size / 128 + 8)))
    return MX_ERR_SHAPE;
  // So does that of tiles of 64 tokens; past it there is none.  Nor is there one where the table's tokens
  // are too few for it to gain what looking costs (the longest part's tiles; looking takes about 5 us, a
  // tile 2).
  const int64_t tiles = a->table_width * c.page_size / 64;
  const int64_t slots = plan.split == mx::AttnPlan::kMixed ? mx::AttnPlan::kMixedSlots : 1;
  if (!plan.few && plan.groups > 0 &&
      (tiles / plan.splits <= mx::kLeastDealTiles || !fits31(units * plan.row_blocks * slots, tiles + 8)))
    plan.groups = 0;
  if (plan.part_bytes > 0 && (!a->workspace || a->workspace_bytes < mx::kCounterBytes + plan.part_bytes ||
                              !aligned(a->workspace, 256)))
    return MX_ERR_WORKSPACE;
  if ((st = device_status()) != MX_OK) return st;
  mx::AttnTreeProblem p;
  p.cache = cache_of(c);
  p.q = rows(a->q, a->q_token_stride, a->q_head_stride);
  p.out = rows(a->out, a->out_token_stride, a->out_head_stride);
  p.lse = a->lse;
  p.table = a->page_table;
  p.lens = a->seq_lens;
  p.starts = a->q_starts;
  p.table_stride = a->table_stride;
  // An empty cache holds nothing that a length could speak of.
  p.table_width = static_cast<int32_t>(c.pages > 0 ? a->table_width : 0);
  p.page_div = static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d);   // d == 1: wraps to 0
  p.batch = static_cast<int32_t>(a->batch);
  p.total_q = static_cast<int32_t>(a->total_q);
  p.max_q = static_cast<int32_t>(a->max_q);
  p.group = static_cast<int32_t>(a->q_heads / c.kv_heads);
  // A scale of zero becomes the smallest normal number: every finite score still counts as zero, and
  // the -infinity of a masked one stays what it is.
  p.scale_log2 = static_cast<float>(std::fabs(a->scale) * 1.4426950408889634);
  if (p.scale_log2 < FLT_MIN) p.scale_log2 = FLT_MIN;
  p.flip = a->scale < 0 ? 0x80008000u : 0u;
  p.causal = a->causal != 0;
  p.window = static_cast<int32_t>(a->window);
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.counter_stride = mx::counter_stride(units);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + mx::kCounterBytes);
  p.tree = tree ? reinterpret_cast<const uint32_t*>(tree->mask) : nullptr;
  p.tree_at = tree ? tree->positions : nullptr;
  p.tree_stride = tree ? tree->stride : 0;
  p.tree_words = tree ? static_cast<int32_t>(tree->words) : 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(plan.few ? mx::launch_attn_few(p, plan, s) : mx::launch_attn_many(p, plan, s));
}

}  // namespace

extern "C" {

int mx_qk_norm_rope(const mx_qk_norm_rope_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  const int64_t k_heads = a->k ? a->k_heads : 0;
  int st = norm_shape_status(a->tokens, a->q_heads, k_heads, a->head_dim, a->eps);
  if (st != MX_OK) return st;
  if ((st = rotation_status(a->positions, a->cos, a->sin, a->table_rows, a->rot, a->head_dim)) !=
      MX_OK)
    return st;
  if (a->tokens == 0 || a->q_heads + k_heads == 0) return MX_OK;
  if (a->q_heads > 0)
    st = first_error({rows_status(a->q, a->q_token_stride, a->q_head_stride, 4),
                      output_status(a->q_out, a->q_out_token_stride, a->q_out_head_stride,
                                    a->tokens, a->q_heads, a->head_dim, 4)});
  if (st == MX_OK && k_heads > 0)
    st = first_error({rows_status(a->k, a->k_token_stride, a->k_head_stride, 4),
                      output_status(a->k_out, a->k_out_token_stride, a->k_out_head_stride,
                                    a->tokens, k_heads, a->head_dim, 4)});
  if (st != MX_OK) return st;
  if (!aligned(a->q_weight, 8) || !aligned(a->k_weight, 8)) return MX_ERR_ALIGN;
  if ((st = device_status()) != MX_OK) return st;
  mx::NormRopeProblem p;
  p.x[0] = rows(a->q, a->q_token_stride, a->q_head_stride);
  p.x[1] = rows(a->k, a->k_token_stride, a->k_head_stride);
  p.out[0] = rows(a->q_out, a->q_out_token_stride, a->q_out_head_stride);
  p.out[1] = rows(a->k_out, a->k_out_token_stride, a->k_out_head_stride);
  p.weight[0] = static_cast<const uint16_t*>(a->q_weight);
  p.weight[1] = static_cast<const uint16_t*>(a->k_weight);
  p.rot = rotation(a->positions, a->cos, a->sin, a->table_rows, a->rot, a->interleaved);
  p.tokens = static_cast<uint32_t>(a->tokens);
  p.heads[0] = static_cast<uint32_t>(a->q_heads);
  p.heads[1] = static_cast<uint32_t>(k_heads);
  p.head_dim = static_cast<int>(a->head_dim);
  p.eps = static_cast<float>(a->eps);
  return status_of(mx::launch_qk_norm_rope(p, static_cast<hipStream_t>(stream)));
}

int64_t mx_qk_norm_rope_backward_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                                int64_t head_dim) {
  if (norm_shape_status(tokens, q_heads, k_heads, head_dim, 0.0) != MX_OK || tokens == 0) return 0;
  return norm_back_workspace(head_dim);
}

int mx_qk_norm_rope_backward(const mx_qk_norm_rope_backward_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  const int64_t k_heads = a->k ? a->k_heads : 0;
  int st = norm_shape_status(a->tokens, a->q_heads, k_heads, a->head_dim, a->eps);
  if (st != MX_OK) return st;
  if ((st = rotation_status(a->positions, a->cos, a->sin, a->table_rows, a->rot, a->head_dim)) !=
      MX_OK)
    return st;
  // A gradient of a weight that is not there is a caller's mistake.
  if ((a->dq_weight && !a->q_weight) || (a->dk_weight && !a->k_weight)) return MX_ERR_NULL;
  const bool none = a->tokens == 0 || a->q_heads + k_heads == 0;
  if (none && !a->dq_weight && !a->dk_weight) return MX_OK;
  // Without rows a weight's gradient is zero, and is written as such by the kernel; no workspace needed.
  if (a->tokens > 0 && a->q_heads > 0)
    st = first_error({rows_status(a->q, a->q_token_stride, a->q_head_stride, 4),
                      rows_status(a->dq_out, a->dq_out_token_stride, a->dq_out_head_stride, 4),
                      output_status(a->dq, a->dq_token_stride, a->dq_head_stride, a->tokens,
                                    a->q_heads, a->head_dim, 4)});
  if (st == MX_OK && a->tokens > 0 && k_heads > 0)
    st = first_error({rows_status(a->k, a->k_token_stride, a->k_head_stride, 4),
                      rows_status(a->dk_out, a->dk_out_token_stride, a->dk_out_head_stride, 4),
                      output_status(a->dk, a->dk_token_stride, a->dk_head_stride, a->tokens,
                                    k_heads, a->head_dim, 4)});
  if (st != MX_OK) return st;
  if (!aligned(a->q_weight, 8) || !aligned(a->k_weight, 8) || !aligned(a->dq_weight, 4) ||
      !aligned(a->dk_weight, 4))
    return MX_ERR_ALIGN;
  const bool sums = a->tokens > 0 && ((a->dq_weight && a->q_heads > 0) || (a->dk_weight && k_heads > 0));
  if (sums &&
      (!a->workspace || a->workspace_bytes < norm_back_workspace(a->head_dim) ||
       !aligned(a->workspace, 256)))
    return MX_ERR_WORKSPACE;
  if ((st = device_status()) != MX_OK) return st;
  mx::NormRopeBackProblem p;
  p.dy[0] = rows(a->dq_out, a->dq_out_token_stride, a->dq_out_head_stride);
  p.dy[1] = rows(a->dk_out, a->dk_out_token_stride, a->dk_out_head_stride);
  p.x[0] = rows(a->q, a->q_token_stride, a->q_head_stride);
  p.x[1] = rows(a->k, a->k_token_stride, a->k_head_stride);
  p.dx[0] = rows(a->dq, a->dq_token_stride, a->dq_head_stride);
  p.dx[1] = rows(a->dk, a->dk_token_stride, a->dk_head_stride);
  p.weight[0] = static_cast<const uint16_t*>(a->q_weight);
  p.weight[1] = static_cast<const uint16_t*>(a->k_weight);
  p.dweight[0] = a->dq_weight;
  p.dweight[1] = a->dk_weight;
  p.rot = rotation(a->positions, a->cos, a->sin, a->table_rows, a->rot, a->interleaved);
  p.tokens = static_cast<uint32_t>(a->tokens);
  p.heads[0] = static_cast<uint32_t>(a->q_heads);
  p.heads[1] = static_cast<uint32_t>(k_heads);
  p.head_dim = static_cast<int>(a->head_dim);
  p.eps = static_cast<float>(a->eps);
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) +
                                     mx::kNormBackCounterBytes);
  return status_of(mx::launch_qk_norm_rope_backward(p, static_cast<hipStream_t>(stream)));
}

int mx_kv_append_fp4(const mx_kv_append_fp4_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  int st = cache_status(a->cache);
  if (st != MX_OK) return st;
  const mx_kv_cache_fp4& c = *a->cache;
  if (a->tokens < 0 || !fits31(a->tokens, c.kv_heads)) return MX_ERR_SHAPE;
  if ((st = rotation_status(a->positions, a->cos, a->sin, a->table_rows, a->rot, c.head_dim)) !=
      MX_OK)
    return st;
  if (a->tokens == 0) return MX_OK;
  // Written blocks must not lie on each other (attention may read any).
  if (blocks_meet(c.pages, c.code_page_stride, c.kv_heads, c.code_head_stride, c.page_size * c.head_dim / 2) ||
      blocks_meet(c.pages, c.scale_page_stride, c.kv_heads, c.scale_head_stride, c.page_size * c.head_dim / 32))
    return MX_ERR_STRIDE;
  if (!a->slots) return MX_ERR_NULL;
  if ((st = first_error({rows_status(a->k, a->k_token_stride, a->k_head_stride, 8),
                         rows_status(a->v, a->v_token_stride, a->v_head_stride, 8)})) !=
      MX_OK)
    return st;
  if (!aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !aligned(a->slots, 8))
    return MX_ERR_ALIGN;
  if (c.pages == 0) return MX_OK;                     // every slot is outside the cache
  if ((st = device_status()) != MX_OK) return st;
  mx::KvAppendProblem p;
  p.cache = cache_of(c);
  p.k = rows(a->k, a->k_token_stride, a->k_head_stride);
  p.v = rows(a->v, a->v_token_stride, a->v_head_stride);
  p.slots = a->slots;
  p.rot = rotation(a->positions, a->cos, a->sin, a->table_rows, a->rot, a->interleaved);
  p.k_out = static_cast<uint16_t*>(a->k_out);
  p.v_out = static_cast<uint16_t*>(a->v_out);
  p.tokens = static_cast<uint32_t>(a->tokens);
  return status_of(mx::launch_kv_append_fp4(p, static_cast<hipStream_t>(stream)));
}

int64_t mx_attn_fp4_workspace_size(int64_t batch, int64_t max_q, int64_t q_heads,
                                   int64_t kv_heads, int64_t head_dim) {
  if (batch <= 0 || max_q <= 0 || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0 ||
      !head_dim_ok(head_dim) || batch > 65535 || kv_heads > 65535 || !fits31(max_q, q_heads) ||
      !fits31(batch, kv_heads))
    return 0;
  return mx::kCounterBytes +
         mx::most_part_bytes(max_q, q_heads / kv_heads, static_cast<int>(head_dim));
}

int mx_attn_fp4(const mx_attn_fp4_args* a, void* stream) {
  return a ? attend(*a, nullptr, stream) : MX_ERR_NULL;
}

int mx_attn_tree_fp4(const mx_attn_tree_fp4_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  const mx_attn_fp4_args call = {
      a->cache, a->q, a->out, a->lse, a->page_table, a->seq_lens, a->q_starts, a->workspace,
      a->workspace_bytes, a->q_token_stride, a->q_head_stride, a->out_token_stride, a->out_head_stride,
      a->table_stride, a->table_width, a->batch, a->total_q, a->max_q, a->q_heads, 0, a->window, a->scale};
  const Tree tree = {a->mask, a->positions, a->mask_stride, a->mask_words};
  return attend(call, &tree, stream);
}

}  // extern "C"
