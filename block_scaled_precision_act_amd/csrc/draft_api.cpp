// C ABI of the draft operators (declared in include/mx_draft.h; the attention of a tree is in
// attn_api.cpp): argument checks on the host, then launches on the caller's stream.
#include "../../include/mx_draft.h"
#include "attn_checks.h"
#include "draft_internal.h"

#include <algorithm>

namespace {

using namespace mx;

constexpr int64_t kMostVocab = int64_t{1} << 30;
constexpr int64_t kMostStride = int64_t{1} << 30;      // elements: rows' addresses fit 64 bits
constexpr int64_t kMostLayers = 1024;

int nodes_status(int64_t batch, int64_t total_q, int64_t max_q, const int32_t* starts) {
  if (batch < 0 || batch > 65535 || total_q < 0 || total_q > kMax31 || max_q < 0 || max_q > kMostNodes)
    return MX_ERR_SHAPE;
  if (!starts && total_q != batch * max_q) return MX_ERR_SHAPE;
  return aligned(starts, 4) ? MX_OK : MX_ERR_ALIGN;
}

Nodes nodes(int64_t batch, int64_t total_q, int64_t max_q, const int32_t* starts) {
  return Nodes{starts, static_cast<int32_t>(batch), static_cast<int32_t>(total_q), static_cast<int32_t>(max_q)};
}

// Behind the counters, 64 sums of each sequence whose rows are cut: at most every second workgroup's.
constexpr int64_t kVerifyWorkspace = kCounterBytes + kVerifyGroups / 2 * 64 * 8;

// A buffer's address (nullptr: none) and bytes.
struct Range {
  const void* p;
  int64_t bytes;
};

bool meet(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
         y < x + static_cast<uintptr_t>(a.bytes);
}

// Whether an output lies on an input or another output: workgroups read what others may have written.
bool outputs_meet(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
  for (const Range* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Range& i : inputs)
      if (meet(*o, i)) return true;
    for (const Range* q = outputs.begin(); q != o; ++q)
      if (meet(*o, *q)) return true;
  }
  return false;
}

// Bytes of `rows` rows, or what no memory holds where they are more.
int64_t row_bytes(int64_t rows, int64_t stride, int64_t width, int64_t unit) {
  const __int128 n = rows > 0 ? (static_cast<__int128>(rows - 1) * stride + width) * unit : 0;
  return static_cast<int64_t>(std::min<__int128>(n, int64_t{1} << 62));
}

}  // namespace

extern "C" {

int mx_tree_mask(const mx_tree_mask_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  int st = nodes_status(a->batch, a->total_q, a->max_q, a->q_starts);
  if (st != MX_OK) return st;
  if (a->mask_words < (a->max_q + 31) / 32 || a->mask_words > kMax31) return MX_ERR_SHAPE;
  if (a->mask_stride < 0 || (a->total_q > 1 && a->mask_stride < a->mask_words)) return MX_ERR_STRIDE;
  if (a->batch == 0 || a->total_q == 0 || a->max_q == 0) return MX_OK;
  if (!a->parents || !a->mask || !a->seq_lens != !a->positions) return MX_ERR_NULL;
  if (!aligned(a->parents, 4) || !aligned(a->mask, 4) || !aligned(a->seq_lens, 4) || !aligned(a->positions, 4))
    return MX_ERR_ALIGN;
  if (outputs_meet({{a->mask, row_bytes(a->total_q, a->mask_stride, a->mask_words, 4)}, {a->positions, 4 * a->total_q}},
                   {{a->parents, 4 * a->total_q}, {a->seq_lens, 4 * a->batch}, {a->q_starts, 4 * (a->batch + 1)}}))
    return MX_ERR_STRIDE;
  if ((st = device_status()) != MX_OK) return st;
  TreeMaskProblem p;
  p.nodes = nodes(a->batch, a->total_q, a->max_q, a->q_starts);
  p.parents = a->parents;
  p.lens = a->seq_lens;
  p.mask = reinterpret_cast<uint32_t*>(a->mask);
  p.positions = a->positions;
  p.mask_stride = a->mask_stride;
  p.words = static_cast<int32_t>(a->mask_words);
  return status_of(launch_tree_mask(p, static_cast<hipStream_t>(stream)));
}

int64_t mx_tree_verify_workspace_size(int64_t batch) {
  return batch <= 0 || batch > 65535 ? 0 : kVerifyWorkspace;
}

int mx_tree_verify(const mx_tree_verify_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  int st = nodes_status(a->batch, a->total_q, a->max_q, a->q_starts);
  if (st != MX_OK) return st;
  if (a->vocab < 1 || a->vocab > kMostVocab || a->width < 1 || !fits31(a->batch, a->width) || a->type < 0 || a->type > 2)
    return MX_ERR_SHAPE;
  if (a->target_stride < 0 || a->target_stride > kMostStride || a->draft_stride > kMostStride ||
      (a->total_q > 1 && a->target_stride < a->vocab) || a->draft_stride < 0 ||
      (a->draft && a->draft_stride > 0 && a->draft_stride < a->vocab))
    return MX_ERR_STRIDE;
  if (a->batch == 0) return MX_OK;
  if (!a->path || !a->tokens_out || !a->count) return MX_ERR_NULL;
  const bool none = a->total_q == 0 || a->max_q == 0;     // every sequence's outputs are still written
  if (!none && (!a->target || !a->tokens || !a->parents || !a->accept_u || !a->sample_u)) return MX_ERR_NULL;
  const uintptr_t unit = a->type == 0 ? 4 : 2;
  if (!aligned(a->target, unit) || !aligned(a->draft, unit) || !aligned(a->tokens, 4) || !aligned(a->parents, 4) ||
      !aligned(a->accept_u, 4) || !aligned(a->sample_u, 4) || !aligned(a->path, 4) || !aligned(a->tokens_out, 4) ||
      !aligned(a->count, 4))
    return MX_ERR_ALIGN;
  const int64_t out = 4 * a->batch * a->width, each = 4 * a->total_q, width = unit;
  if (outputs_meet({{a->path, out}, {a->tokens_out, out}, {a->count, 4 * a->batch}},
                   {{a->tokens, each}, {a->parents, each}, {a->accept_u, each}, {a->sample_u, 4 * a->batch},
                    {a->q_starts, 4 * (a->batch + 1)},
                    {a->target, row_bytes(a->total_q, a->target_stride, a->vocab, width)},
                    {a->draft, row_bytes(a->total_q, a->draft_stride, a->vocab, width)}}))
    return MX_ERR_STRIDE;
  if (!a->workspace || a->workspace_bytes < kVerifyWorkspace || !aligned(a->workspace, 256))
    return MX_ERR_WORKSPACE;
  if ((st = device_status()) != MX_OK) return st;
  TreeVerifyProblem p;
  p.nodes = nodes(a->batch, none ? 0 : a->total_q, none ? 0 : a->max_q, none ? nullptr : a->q_starts);
  p.target = a->target;
  p.draft = a->draft;
  p.target_stride = a->target_stride;
  p.draft_stride = a->draft_stride;
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.accept_u = a->accept_u;
  p.sample_u = a->sample_u;
  p.path = a->path;
  p.tokens_out = a->tokens_out;
  p.count = a->count;
  p.vocab = static_cast<int32_t>(a->vocab);
  p.width = static_cast<int32_t>(a->width);
  p.type = static_cast<int>(a->type);
  p.replacement = a->replacement != 0;
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.parts = reinterpret_cast<double*>(static_cast<uint8_t*>(a->workspace) + kCounterBytes);
  return status_of(launch_tree_verify(p, static_cast<hipStream_t>(stream)));
}

int mx_kv_accept_fp4(const mx_kv_accept_fp4_args* a, void* stream) {
  if (!a) return MX_ERR_NULL;
  int st = nodes_status(a->batch, a->total_q, a->max_q, a->q_starts);
  if (st != MX_OK) return st;
  if (a->layers < 0 || a->layers > kMostLayers || a->width < 0 || !fits31(a->batch, a->width) || a->table_width < 0)
    return MX_ERR_SHAPE;
  if (a->batch == 0 || (a->layers == 0 && (!a->caches || !a->lens_out))) return MX_OK;
  if (!a->caches) return MX_ERR_NULL;
  // Without layers the new lengths alone are written: one cache of no pages, and lengths that no table covers.
  const bool none = a->layers == 0;
  const mx_kv_cache_fp4 empty = {nullptr, nullptr, nullptr, nullptr, 0, 1, 1, 64, 0, 0, 0, 0};
  const mx_kv_cache_fp4& c = none ? empty : a->caches[0];
  for (int64_t i = 0; i < a->layers; ++i) {
    const mx_kv_cache_fp4& x = a->caches[i];
    if ((st = cache_status(&x)) != MX_OK) return st;
    if (x.pages != c.pages || x.kv_heads != c.kv_heads || x.page_size != c.page_size || x.head_dim != c.head_dim)
      return MX_ERR_SHAPE;
    if (x.code_page_stride != c.code_page_stride || x.code_head_stride != c.code_head_stride ||
        x.scale_page_stride != c.scale_page_stride || x.scale_head_stride != c.scale_head_stride)
      return MX_ERR_STRIDE;
    // One layer's moves must not meet another's, nor keys' those of values.
    for (int64_t j = 0; c.pages > 0 && j <= i; ++j) {
      const mx_kv_cache_fp4& y = a->caches[j];
      if (x.k == y.v || x.k_scale == y.v_scale) return MX_ERR_STRIDE;
      if (j < i && (x.k == y.k || x.v == y.v || x.k_scale == y.k_scale || x.v_scale == y.v_scale || x.v == y.k ||
                    x.v_scale == y.k_scale))
        return MX_ERR_STRIDE;
    }
  }
  if (!fits31(a->batch, c.kv_heads) || !fits31(a->table_width, c.page_size)) return MX_ERR_SHAPE;
  if (a->table_stride < 0 || (a->batch > 1 && a->table_stride < a->table_width)) return MX_ERR_STRIDE;
  if (blocks_meet(c.pages, c.code_page_stride, c.kv_heads, c.code_head_stride, c.page_size * c.head_dim / 2) ||
      blocks_meet(c.pages, c.scale_page_stride, c.kv_heads, c.scale_head_stride, c.page_size * c.head_dim / 32))
    return MX_ERR_STRIDE;
  if (!a->seq_lens || !a->count || (a->width > 0 && !a->path) || (a->table_width > 0 && !a->page_table))
    return MX_ERR_NULL;
  if (!aligned(a->seq_lens, 4) || !aligned(a->count, 4) || !aligned(a->path, 4) || !aligned(a->page_table, 4) ||
      !aligned(a->lens_out, 4))
    return MX_ERR_ALIGN;
  if (outputs_meet({{a->lens_out, 4 * a->batch}},
                   {{a->seq_lens, 4 * a->batch}, {a->count, 4 * a->batch}, {a->q_starts, 4 * (a->batch + 1)},
                    {a->path, 4 * a->batch * a->width},
                    {a->page_table, row_bytes(a->batch, a->table_stride, a->table_width, 4)}}))
    return MX_ERR_STRIDE;
  if ((st = device_status()) != MX_OK) return st;
  KvAcceptProblem p;
  p.nodes = nodes(a->batch, a->total_q, a->max_q, a->q_starts);
  p.shape = cache_of(c);
  p.table = a->page_table;
  p.table_stride = a->table_stride;
  p.table_width = static_cast<int32_t>(none ? kMax31 : a->table_width);
  p.lens = a->seq_lens;
  p.path = a->path;
  p.count = a->count;
  p.width = static_cast<int32_t>(a->width);
  if (none) {
    p.layers = 1;
    p.layer[0] = {};
    p.lens_out = a->lens_out;
    return status_of(launch_kv_accept_fp4(p, static_cast<hipStream_t>(stream)));
  }
  for (int64_t at = 0; at < a->layers; at += kLayersALaunch) {
    p.layers = static_cast<int32_t>(std::min<int64_t>(kLayersALaunch, a->layers - at));
    p.lens_out = at == 0 ? a->lens_out : nullptr;
    for (int i = 0; i < p.layers; ++i) {
      const mx_kv_cache_fp4& x = a->caches[at + i];
      p.layer[i] = {static_cast<uint8_t*>(x.k), static_cast<uint8_t*>(x.k_scale), static_cast<uint8_t*>(x.v),
                    static_cast<uint8_t*>(x.v_scale)};
    }
    if ((st = status_of(launch_kv_accept_fp4(p, static_cast<hipStream_t>(stream)))) != MX_OK) return st;
  }
  return MX_OK;
}

}  // extern "C"
