// Masks and positions of trees of drafted tokens for gfx950.
//
// For node i: the bits of anc(i) = {i} and anc(parent(i)), and the number of its ancestors.  A workgroup
// takes a sequence's tree; its parents lie in LDS, and a thread makes one word of one node's mask by
// following the parents down to it (they only fall, so a word's thread stops below its nodes).
//
// Bound by latency: the parents' load, the stores, and between them LDS reads one after the other, an ancestor each,
// for every word that a thread makes: nodes x words / 256 words of up to `depth` reads.  That is little for trees as
// deep as drafts are (26 nodes: 1.8 us, the launch; 128 trees of up to 129 nodes, 3.4 to 3.8 us; 1024 nodes, three
// children each: 85 us), but it grows with the cube of a chain's length: 26 nodes 3.2 us, 64 5.5, 129 18, 200 44, 512
// 541, 1024 4278 (128 chains of 1024 as long).
#include "draft_common.h"

namespace mx {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void tree_mask_kernel(const TreeMaskProblem p) {
  __shared__ int32_t up[kMostNodes];
  const int32_t b = blockIdx.x;
  const Span s = nodes_of(p.nodes, b);
  const int32_t first = p.lens ? read_uniform(p.lens, b) - s.n : 0;
  for (int32_t i = threadIdx.x; i < s.n; i += kThreads) {
    const int32_t x = p.parents[s.q0 + i];
    up[i] = x >= 0 && x < i ? x : -1;
  }
  __syncthreads();
  const int64_t items = static_cast<int64_t>(s.n) * p.words;
  for (int64_t item = threadIdx.x; item < items; item += kThreads) {
    const int32_t i = static_cast<int32_t>(item / p.words), w = static_cast<int32_t>(item - int64_t{i} * p.words);
    uint32_t bits = 0;
    int32_t seen = 0;                     // of word 0: all of them
    for (int32_t j = i; j >= 0 && j >> 5 >= w; j = up[j]) {
      if (j >> 5 == w) bits |= 1u << (j & 31);
      ++seen;
    }
    p.mask[(s.q0 + i) * p.mask_stride + w] = bits;
    if (w == 0 && p.positions) p.positions[s.q0 + i] = first + seen - 1;
  }
}

}  // namespace

hipError_t launch_tree_mask(const TreeMaskProblem& p, hipStream_t stream) {
  hipLaunchKernelGGL(tree_mask_kernel, dim3(static_cast<unsigned>(p.nodes.batch)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mx
