// Internal interface between the C-ABI layer of the draft operators (draft_api.cpp) and their gfx950
// kernels.
#pragma once

#include "attn_internal.h"

namespace mx {

// Nodes that a sequence's tree may have where their parents are followed (they lie in LDS).
constexpr int64_t kMostNodes = 1024;

// Where the sequences' nodes lie (see mx_draft.h).
struct Nodes {
  const int32_t* starts;     // or nullptr: max_q rows each
  int32_t batch, total, max_q;
};

struct TreeMaskProblem {
  Nodes nodes;
  const int32_t* parents;
  const int32_t* lens;       // or nullptr: no positions
  uint32_t* mask;
  int32_t* positions;
  int64_t mask_stride;
  int32_t words;
};
hipError_t launch_tree_mask(const TreeMaskProblem& p, hipStream_t stream);

struct TreeVerifyProblem {
  Nodes nodes;
  const void* target;
  const void* draft;         // or nullptr: chosen drafts
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* parents;
  const float* accept_u;
  const float* sample_u;
  int32_t* path;
  int32_t* tokens_out;
  int32_t* count;
  int32_t vocab, width;
  int type;                  // 0 fp32, 1 bf16, 2 fp16
  bool replacement;
  uint32_t* counters;        // kTeamWords of each
  double* parts;             // 64 of each sequence whose rows are cut
};
// Workgroups that a row's slices are dealt to, over all sequences: one a CU.
constexpr int64_t kVerifyGroups = 256;
constexpr int64_t kTeamWords = 32;       // a cache line
static_assert(kTeamWords * 65535 <= kMaxUnits, "every batch's counters lie in the workspace's first part");
hipError_t launch_tree_verify(const TreeVerifyProblem& p, hipStream_t stream);

constexpr int kLayersALaunch = 64;       // four pointers each: 2 KB of arguments
struct KvAcceptProblem {
  Nodes nodes;
  KvCache shape;             // the caches' sizes and strides
  struct { uint8_t *k, *ks, *v, *vs; } layer[kLayersALaunch];
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t* lens;
  const int32_t* path;
  const int32_t* count;
  int32_t* lens_out;         // or nullptr
  int32_t layers, width;
};
hipError_t launch_kv_accept_fp4(const KvAcceptProblem& p, hipStream_t stream);

}  // namespace mx
