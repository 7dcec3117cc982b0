// Moving the accepted path's keys and values to their places in the paged MXFP4 cache for gfx950.
//
// Token first + path[i] of a sequence becomes token first + i, in every layer and head, byte for byte.
// A wavefront takes a layer, a sequence and up to kHeads heads: D / 16 lanes a token, 16 bytes of key or value
// codes each (the first two its scales too), so 4 to 16 tokens at once, of all its heads before any is stored.
// path rises strictly and path[i] >= i, so a token's place is no later token's source but those moved with it,
// whose loads come before: the wavefront goes over the path in order with no barrier.
//
// Bound by latency (path, table, codes, one after the other), whatever the layers: 64 go in one launch.  One
// layer, one sequence: 3.0 us; 32 layers, 41 sequences, 8 heads of 128: 5.1 us for 8 MB.
#include "draft_common.h"

#include <algorithm>

namespace mx {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kMostBlocks = 1 << 20;
constexpr int kHeads = 4;            // of a wavefront (32 layers x 41 sequences x 8 heads: 5.2 us; 1: 7.2, 8: 5.7)

template <int BYTES> struct ScaleWord;
template <> struct ScaleWord<2> { typedef uint16_t type; };
template <> struct ScaleWord<4> { typedef uint32_t type; };
template <> struct ScaleWord<8> { typedef uint64_t type; };

template <int D>
__global__ __launch_bounds__(kThreads) void kv_accept_kernel(const KvAcceptProblem p, uint32_t head_groups,
                                                             int64_t units) {
  constexpr int kLanes = D / 16, kTokens = 64 / kLanes;       // lanes a token: half for keys, half for values
  typedef typename ScaleWord<D / 32>::type Scales;
  const int lane = threadIdx.x & 63;
  const int token = lane / kLanes, part = lane % kLanes;
  const int32_t page_size = p.shape.page_size;
  const int64_t covered = static_cast<int64_t>(p.table_width) * page_size;
  for (int64_t unit = blockIdx.x * int64_t{kWaves} + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units;
       unit += int64_t{gridDim.x} * kWaves) {
    const uint32_t h0 = static_cast<uint32_t>(unit % head_groups) * kHeads;
    const int64_t rest = unit / head_groups;
    const int32_t b = static_cast<int32_t>(rest % p.nodes.batch), layer = static_cast<int32_t>(rest / p.nodes.batch);
    const Span s = nodes_of(p.nodes, b);
    const int32_t raw = read_uniform(p.lens, b);
    const int32_t len = raw < 0 ? 0 : (raw < covered ? raw : static_cast<int32_t>(covered));
    const int32_t first = len - s.n, count = min(max(read_uniform(p.count, b), 0), min(s.n, p.width));
    if (p.lens_out && layer == 0 && h0 == 0 && lane == 0) p.lens_out[b] = max(first + count, 0);
    if (p.shape.pages == 0) continue;      // nothing moves, and the table is not what `covered` says without layers
    const int32_t heads = min(static_cast<int32_t>(p.shape.heads - h0), kHeads);
    const int32_t* const path = p.path + static_cast<int64_t>(b) * p.width;
    const int32_t* const table = p.table + b * p.table_stride;
    uint8_t* const codes = (part >= kLanes / 2 ? p.layer[layer].v : p.layer[layer].k) + part % (kLanes / 2) * 16;
    uint8_t* const scales = (part & 1) ? p.layer[layer].vs : p.layer[layer].ks;
    // Where a token lies: its page and place, no page where it is none.
    auto place = [&](int32_t t, uint32_t* off) {
      if (t < 0 || t >= covered) return p.shape.pages;
      const uint32_t page = static_cast<uint32_t>(t) / page_size;
      *off = static_cast<uint32_t>(t) - page * page_size;
      return static_cast<uint32_t>(table[page]);
    };
    for (int32_t i0 = 0; i0 < count; i0 += kTokens) {
      const int32_t i = i0 + token;
      const int32_t j = i < count ? path[i] : i;
      uint32_t from = p.shape.pages, to = p.shape.pages, from_off = 0, to_off = 0;
      if (j != i && j >= 0 && j < s.n) {
        from = place(first + j, &from_off);
        to = place(first + i, &to_off);
      }
      const bool moves = from < p.shape.pages && to < p.shape.pages;
      if (!__any(moves)) continue;
      const int64_t at = from * p.shape.code_page + h0 * p.shape.code_head + int64_t{from_off} * (D / 2);
      const int64_t scale_at = from * p.shape.scale_page + h0 * p.shape.scale_head + int64_t{from_off} * (D / 32);
      v4u x[kHeads];
      Scales y[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (moves && h < heads) {
          x[h] = *reinterpret_cast<const v4u*>(codes + at + h * p.shape.code_head);
          if (part < 2) y[h] = *reinterpret_cast<const Scales*>(scales + scale_at + h * p.shape.scale_head);
        }
      }
      // Every lane's loads are complete before any lane's store: one lane's place may be another's source.
      __builtin_amdgcn_s_waitcnt(kVmcntZero);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int64_t put = to * p.shape.code_page + h0 * p.shape.code_head + int64_t{to_off} * (D / 2);
      const int64_t scale_put = to * p.shape.scale_page + h0 * p.shape.scale_head + int64_t{to_off} * (D / 32);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (moves && h < heads) {
          *reinterpret_cast<v4u*>(codes + put + h * p.shape.code_head) = x[h];
          if (part < 2) *reinterpret_cast<Scales*>(scales + scale_put + h * p.shape.scale_head) = y[h];
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_accept_fp4(const KvAcceptProblem& p, hipStream_t stream) {
  const uint32_t head_groups = (p.shape.heads + kHeads - 1) / kHeads;
  const int64_t units = int64_t{p.layers} * p.nodes.batch * head_groups;
  const dim3 grid(static_cast<unsigned>(std::min((units + kWaves - 1) / kWaves, kMostBlocks)));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, head_groups, units); };
  if (p.shape.head_dim == 64) go(kv_accept_kernel<64>);
  else if (p.shape.head_dim == 128) go(kv_accept_kernel<128>);
  else go(kv_accept_kernel<256>);
  return hipGetLastError();
}

}  // namespace mx
