// Internal interface between the C-ABI layer of the attention operators (attn_api.cpp) and their
// gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace mx {

// Workgroups of `threads` that one dimension of a grid holds: it counts fewer than 2^32 threads.
constexpr int64_t most_groups(int threads) { return ((int64_t{1} << 32) - 1) / threads; }

// Position rotation (see mx_attention.h).  positions == nullptr: none.
struct Rotation {
  const int32_t* positions;
  const float* cos;          // [rows, rot / 2]
  const float* sin;
  uint32_t rows;
  int rot;
  bool interleaved;
};

// One tensor of bf16 heads [tokens, heads, head_dim] and where its rows lie (element strides).
struct HeadRows {
  uint16_t* p;
  int64_t token_stride, head_stride;
};

struct NormRopeProblem {
  HeadRows x[2], out[2];     // queries, keys (heads[1] == 0: no keys)
  const uint16_t* weight[2]; // bf16 [head_dim] or nullptr
  Rotation rot;
  uint32_t tokens, heads[2];
  int head_dim;
  float eps;
};
hipError_t launch_qk_norm_rope(const NormRopeProblem& p, hipStream_t stream);

struct NormRopeBackProblem {
  HeadRows dy[2], x[2], dx[2];
  const uint16_t* weight[2];
  float* dweight[2];         // fp32 [head_dim] or nullptr
  Rotation rot;
  uint32_t tokens, heads[2];
  int head_dim;
  float eps;
  uint32_t* counters;        // two, zero between calls
  float* parts;              // [groups][head_dim]
};
// Workgroups that the gradients' rows are dealt to; each leaves one partial weight gradient.
constexpr int kNormBackGroups = 512;
constexpr int64_t kNormBackCounterBytes = 256;
hipError_t launch_qk_norm_rope_backward(const NormRopeBackProblem& p, hipStream_t stream);

struct KvCache {
  uint8_t *k, *ks, *v, *vs;
  int64_t code_page, code_head, scale_page, scale_head;   // byte strides
  uint32_t pages, heads, page_size;
  int head_dim;
};

struct KvAppendProblem {
  KvCache cache;
  HeadRows k, v;
  const int64_t* slots;
  Rotation rot;
  uint16_t *k_out, *v_out;   // or nullptr
  uint32_t tokens;
};
hipError_t launch_kv_append_fp4(const KvAppendProblem& p, hipStream_t stream);

struct AttnProblem {
  KvCache cache;
  HeadRows q, out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;     // or nullptr: max_q rows each
  int64_t table_stride;
  int32_t table_width;
  uint32_t page_div;         // ceil(2^32 / (page_size / 16)): n / (page_size / 16) as a high product
  int32_t batch, total_q, max_q, group;
  float scale_log2;          // |scale| * log2(e), at least the smallest normal fp32
  uint32_t flip;             // 0x80008000 where scale < 0: the queries' signs are turned instead
  bool causal;
  int32_t window;
  uint32_t* counters;
  uint32_t counter_stride;
  float* parts;
};

// Tokens past a sequence's length that the kernels' token numbers may reach (the rounding to a tile, and
// the next tiles' places, looked up before it is known whether they are needed): 128 and 256 at most.
constexpr int64_t kLookAhead = 1024;

// A workspace begins with the arrival counters of few rows, one per (sequence, key/value head), zero
// between calls; partial results follow at a fixed place, whatever the sizes, so calls of any sizes
// can share a workspace.  Counters lie a cache line apart while that fits (arrivals on neighbouring
// ones would pass one line around the XCDs).
constexpr int64_t kCounterBytes = int64_t{8} << 20;
constexpr int64_t kMaxUnits = kCounterBytes / 4;
constexpr uint32_t counter_stride(int64_t units) {
  uint32_t stride = 32;
  while (stride > 1 && units * stride > kMaxUnits) stride /= 2;
  return stride;
}

// How a problem's rows are dealt out, by its sizes alone.  A sequence's rows for one key/value
// head are its (query, grouped head) pairs, max_q * group of them at most.
struct AttnPlan {
  bool few;                  // few rows: the cache is what costs (attn_few.hip), else attn_many.hip
  int row_tiles;             // of a workgroup: 16-row tiles (few), wavefronts of 32 rows (many)
  int groups;                // workgroups that the cached tokens are dealt to (many: 0: no deal)
  int row_blocks, splits;    // many: blocks of rows of each (sequence, head), parts of their keys at most
  int64_t part_bytes;        // of partial results
};
// Wavefronts of attn_few.hip that a SIMD holds (by their registers), and so workgroups a CU.
constexpr int few_waves(int head_dim, int row_tiles) {
  return head_dim * row_tiles <= 128 ? 3 : head_dim * row_tiles <= 256 ? 2 : 1;
}
// A deal among many rows (attn_many.hip) is looked at where a part of a unit may have more tiles of 64
// tokens.
constexpr int64_t kLeastDealTiles = 32;
AttnPlan plan_attn(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int head_dim);
// Partial results of any plan with at most max_q queries a sequence.
int64_t most_part_bytes(int64_t max_q, int64_t group, int head_dim);

hipError_t launch_attn_few(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream);
hipError_t launch_attn_many(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream);

}  // namespace mx
