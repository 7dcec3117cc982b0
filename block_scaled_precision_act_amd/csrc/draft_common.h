// Device pieces shared by the draft operators' kernels.
#pragma once

#include "attn_common.h"
#include "draft_internal.h"

namespace mx {
namespace {

// A sequence's nodes: the first one's row and how many.
struct Span {
  int32_t q0, n;
};

__device__ __forceinline__ Span nodes_of(const Nodes& s, int32_t b) {
  int32_t q0 = b * s.max_q, q1 = q0 + s.max_q;
  if (s.starts) {
    q0 = min(max(read_uniform(s.starts, b), 0), s.total);
    q1 = min(max(read_uniform(s.starts, b + 1), q0), s.total);
  }
  return Span{q0, min(q1 - q0, s.max_q)};
}

}  // namespace
}  // namespace mx
