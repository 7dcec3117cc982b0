// Verification of trees of drafted tokens against the target's probabilities for gfx950.
//
// The walk (see mx_draft.h): at a node with target row p and draft row q, a child of token x is accepted
// when u q(x) S < r(x) Q with r(v) = max(p(v) - c q(v), 0); each rejection needs S = sum r(v) over the
// vocabulary, and the last one's r is what the next token is drawn from.  (What is left of a target
// distribution r / S after a token of q / Q was rejected is max(r / S - q / Q, 0) = max(p - (c + S / Q) q,
// 0) / S: its shape is kept in the one number c, and no row is ever written.)
//
// Bound by latency and by one pass over a row of p and one of q.  All that the tests need of the rows is
// p(x) and q(x) of every child, loaded at once into LDS; then the walk costs no memory access until
// the first sum.  For that one the rows are cut into slices, a workgroup each, which all take the same
// walk to find out what to sum; the last to arrive has S and goes on alone: what remains for a chain is to
// find the token within one slice.  A tree may need more sums, which that workgroup takes by itself: a
// wait for other workgroups would need all of them resident.
//
// In 64 bits, each product and sum rounded by itself: a token is decided by where a random number falls
// between sums of up to 2^30 terms, and 32 bits would misplace it once in some hundred tokens.
#include "draft_common.h"

#include <type_traits>

namespace mx {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// What is no probability counts as none.
__device__ __forceinline__ float probability(float x) { return x > 0.f && x < kInf ? x : 0.f; }

template <int TYPE>
__device__ __forceinline__ float widened(uint32_t bits) {
  if constexpr (TYPE == 0) return __uint_as_float(bits);
  if constexpr (TYPE == 1) return __uint_as_float(bits << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

template <int TYPE>
__device__ __forceinline__ float load_one(const void* row, int64_t i) {
  if constexpr (TYPE == 0) return static_cast<const float*>(row)[i];
  else return widened<TYPE>(static_cast<const uint16_t*>(row)[i]);
}

// 16 bytes of neighbouring probabilities; rows are aligned to their elements only.
template <int TYPE>
struct Chunk {
  static constexpr int kSize = TYPE == 0 ? 4 : 8;
  typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t Words2 __attribute__((ext_vector_type(4), aligned(2)));
  typedef std::conditional_t<TYPE == 0, Words4, Words2> Words;
  uint32_t x[4];

  // Those from v on of the row's first `end`; past it 0.
  __device__ __forceinline__ void load(const uint8_t* row, int32_t v, int32_t end) {
    constexpr int kBytes = TYPE == 0 ? 4 : 2;
    const uint8_t* at = row + int64_t{v} * kBytes;
    if (v + kSize <= end) {
      const Words w = *reinterpret_cast<const Words*>(at);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 0;
#pragma unroll
    for (int e = 0; e < kSize; ++e) {
      if (v + e >= end) break;
      if constexpr (TYPE == 0) x[e] = reinterpret_cast<const uint32_t*>(at)[e];
      else x[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[e]) << (16 * (e & 1));
    }
  }
  __device__ __forceinline__ double get(int e) const {
    return probability(widened<TYPE>(TYPE == 0 ? x[e] : x[e / 2] >> (16 * (e & 1)) & 0xFFFFu));
  }
};

// max(p - c q, 0)
__device__ __forceinline__ double residual(double p, double c, double q) {
#pragma clang fp contract(off)
  const double t = c * q;
  const double r = p - t;
  return r > 0.0 ? r : 0.0;
}

__device__ __forceinline__ double shifted_up(double v, int d) { return __shfl_up(v, d, 64); }

// Sums over the lanes up to and with this one.
__device__ __forceinline__ double wave_prefix(double v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double o = shifted_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

// The walk through a sequence's tree; every wavefront takes it for itself, with the same result.
struct Walk {
  int32_t cur, next, count;    // the node, the first one that may still be its child, nodes accepted
  double c, s, q;              // what r is made of, its sum, what is left of the draft's distribution
  bool summed;                 // s is r's sum over the vocabulary
};

// What the tests need, in LDS.
struct Tests {
  int32_t up[kMostNodes], token[kMostNodes];
  float u[kMostNodes], p[kMostNodes], q[kMostNodes];      // of the token in its parent's rows
  int32_t path[kMostNodes];
};

// Goes on until r's sum is needed (true: a child was rejected, others may follow) or no child is left.
template <bool DRAFT>
__device__ __forceinline__ bool walk_on(Walk& w, Tests& t, int32_t n, int32_t width, bool replacement) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  while (w.count < width) {
    // The next child of cur.
    int32_t i = n;
    for (int32_t at = w.next; at < n; at += 64) {
      const uint64_t its = __ballot(at + lane < n && t.up[min(at + lane, n - 1)] == w.cur);
      if (its) {
        i = at + __builtin_ctzll(its);
        break;
      }
    }
    i = __builtin_amdgcn_readfirstlane(i);
    w.next = min(i + 1, n);
    if (i >= n) return false;
    const double u = t.u[i], p = t.p[i];
    bool accepted;
    if constexpr (DRAFT) {
      const double q = t.q[i], r = residual(p, w.c, q);
      const double a = u * q, left = a * w.s, right = r * w.q;
      accepted = w.q > 0.0 && r > 0.0 && left < right;
      if (!accepted) {
        if (!(w.q > 0.0)) continue;
        const double step = w.s / w.q;
        w.c = w.c + step;
        if (!replacement) w.q = w.q - q;
        w.summed = false;
        return true;
      }
    } else {
      // A token that was rejected here before is no longer there.
      bool again = false;
      for (int32_t at = w.cur + 1; at < i; at += 64) {
        const int32_t j = min(at + lane, i - 1);
        again = again || __any(t.up[j] == w.cur && t.token[j] == t.token[i]);
      }
      const double r = again ? 0.0 : p, left = u * w.s;
      accepted = r > 0.0 && left < r;
      if (!accepted) {
        const double rest = w.s - r;
        w.s = rest > 0.0 ? rest : 0.0;
        continue;
      }
    }
    w.cur = i;
    if (threadIdx.x == 0) t.path[w.count] = i;
    ++w.count;
    w.c = 0.0;
    w.s = 1.0;
    w.q = 1.0;
    w.summed = false;
  }
  return false;
}

// A node's residual over the vocabulary.
template <int TYPE, bool DRAFT>
struct Rest {
  static constexpr int kSize = Chunk<TYPE>::kSize;
  const uint8_t *p, *q;        // its rows
  double c;                    // 0: q is not read
  const int32_t* gone;         // tokens that have left it (chosen drafts)
  int32_t ngone;

  struct Loaded {
    Chunk<TYPE> p, q;
  };
  __device__ __forceinline__ void load(Loaded& w, int32_t v, int32_t end) const {
    w.p.load(p, v, end);
    if constexpr (DRAFT)
      if (c != 0.0) w.q.load(q, v, end);
  }
  __device__ __forceinline__ void values(const Loaded& w, int32_t v, double (&r)[kSize]) const {
#pragma unroll
    for (int e = 0; e < kSize; ++e) r[e] = w.p.get(e);
    if constexpr (DRAFT) {
      if (c != 0.0) {
#pragma unroll
        for (int e = 0; e < kSize; ++e) r[e] = residual(r[e], c, w.q.get(e));
      }
    } else {
      for (int32_t i = 0; i < ngone; ++i) {
        const int32_t x = gone[i] - v;
#pragma unroll
        for (int e = 0; e < kSize; ++e)
          if (x == e) r[e] = 0.0;
      }
    }
  }
  // The calling lanes' shares of [begin, end), chunk by chunk, `lanes` of them one after the other.
  __device__ __forceinline__ double share(int32_t begin, int32_t end, int32_t lanes, int32_t lane) const {
    constexpr int kAhead = 4;
    double sum = 0.0;
    for (int64_t v0 = begin + int64_t{lane} * kSize; v0 < end; v0 += int64_t{kAhead} * lanes * kSize) {
      Loaded w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t v = v0 + int64_t{i} * lanes * kSize;
        load(w[i], static_cast<int32_t>(v < end ? v : end), end);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t v = v0 + int64_t{i} * lanes * kSize;
        double r[kSize];
        values(w[i], static_cast<int32_t>(v < end ? v : end), r);
#pragma unroll
        for (int e = 0; e < kSize; ++e) sum += r[e];
      }
    }
    return sum;
  }
};

// Sums of up to 64 neighbouring segments of the vocabulary.
struct Segments {
  double sum;                  // the lane's
  int32_t length;
};

template <int TYPE, bool DRAFT>
__global__ __launch_bounds__(kThreads) void tree_verify_kernel(const TreeVerifyProblem p, int32_t slices,
                                                               int32_t slice) {
  typedef Rest<TYPE, DRAFT> R;
  constexpr int kBytes = TYPE == 0 ? 4 : 2, kSize = R::kSize;
  __shared__ Tests t;
  __shared__ int32_t gone[DRAFT ? 1 : kMostNodes];
  __shared__ int32_t ngone, hit, last;
  __shared__ double sums[kWaves];
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t b = blockIdx.x / slices, mine = blockIdx.x - b * slices;
  const Span s = nodes_of(p.nodes, b);
  const int32_t V = p.vocab;
  int32_t* const path = p.path + static_cast<int64_t>(b) * p.width;
  int32_t* const out = p.tokens_out + static_cast<int64_t>(b) * p.width;
  if (s.n == 0) {
    if (mine != 0) return;
    for (int32_t i = tid; i < p.width; i += kThreads) path[i] = out[i] = -1;
    if (tid == 0) p.count[b] = 0;
    return;
  }
  auto row = [&](const void* m, int64_t stride, int32_t i) {
    return static_cast<const uint8_t*>(m) + (s.q0 + i) * stride * kBytes;
  };
  for (int32_t i = tid; i < s.n; i += kThreads) {
    const int32_t up = p.parents[s.q0 + i], x = p.tokens[s.q0 + i];
    const bool child = up >= 0 && up < i, real = child && x >= 0 && x < V;
    t.up[i] = child ? up : -1;
    t.token[i] = x;
    t.u[i] = p.accept_u[s.q0 + i];
    t.p[i] = real ? probability(load_one<TYPE>(row(p.target, p.target_stride, up), x)) : 0.f;
    if constexpr (DRAFT) t.q[i] = real ? probability(load_one<TYPE>(row(p.draft, p.draft_stride, up), x)) : 0.f;
  }
  if (tid == 0) t.path[0] = 0;
  __syncthreads();
  Walk w = {0, 1, 1, 0.0, 1.0, 1.0, false};
  bool more = walk_on<DRAFT>(w, t, s.n, p.width, p.replacement);

  auto rest = [&](bool whole) {            // of the walk's node; whole: the target's row itself
    R r;
    r.p = row(p.target, p.target_stride, w.cur);
    r.q = DRAFT ? row(p.draft, p.draft_stride, w.cur) : nullptr;
    r.c = whole ? 0.0 : w.c;
    r.gone = gone;
    r.ngone = 0;
    if constexpr (!DRAFT) {
      if (!whole) {
        // The tokens of the children that were rejected.
        if (wave == 0) {
          int32_t n = 0;
          for (int32_t at = w.cur + 1; at < w.next; at += 64) {
            const int32_t i = min(at + lane, w.next - 1);
            const bool its = at + lane < w.next && t.up[i] == w.cur;
            const uint64_t all = __ballot(its);
            if (its) gone[n + __builtin_popcountll(all & ((uint64_t{1} << lane) - 1))] = t.token[i];
            n += __builtin_popcountll(all);
          }
          if (lane == 0) ngone = n;
        }
        __syncthreads();
        r.ngone = ngone;
      }
    }
    return r;
  };
  // A wavefront's sum of a run each, by this workgroup.
  auto sum_alone = [&](const R& r) {
    Segments g;
    g.length = ((V + kWaves - 1) / kWaves + kSize - 1) / kSize * kSize;
    const int64_t begin = int64_t{wave} * g.length;
    const double mine_of = begin < V ? wave_total(r.share(static_cast<int32_t>(begin),
                                                          static_cast<int32_t>(min(begin + g.length, int64_t{V})), 64, lane))
                                     : 0.0;
    __syncthreads();
    if (lane == 0) sums[wave] = mine_of;
    __syncthreads();
    g.sum = lane < kWaves ? sums[lane] : 0.0;
    return g;
  };

  R r = rest(false);
  Segments g;
  if (slices > 1) {
    const int64_t begin = int64_t{mine} * slice, end = min(begin + slice, int64_t{V});
    const double part = begin < end ? wave_total(r.share(static_cast<int32_t>(begin), static_cast<int32_t>(end), kThreads, tid))
                                    : 0.0;
    if (lane == 0) sums[wave] = part;
    __syncthreads();
    double* const parts = p.parts + static_cast<int64_t>(b) * slices;
    if (tid == 0) {
      double all = 0.0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) all += sums[i];
      __hip_atomic_store(reinterpret_cast<uint64_t*>(parts + mine), __builtin_bit_cast(uint64_t, all),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!arrive_last(p.counters + static_cast<int64_t>(b) * p.counter_stride, slices, &flag)) return;
    g.sum = lane < slices ? parts[lane] : 0.0;
    g.length = slice;
  } else {
    g = sum_alone(r);
  }
  // The last workgroup has the sum; a tree's walk may need others.
  double upto;
  for (;;) {
    upto = wave_prefix(g.sum);
    w.s = __shfl(upto, 63, 64);
    w.summed = true;
    if (!more) break;
    more = walk_on<DRAFT>(w, t, s.n, p.width, p.replacement);
    if (!more && w.summed) break;
    r = rest(false);
    g = sum_alone(r);
  }
  if (!(w.s > 0.0)) {                      // nothing is left: the target's row itself
    r = rest(true);
    g = sum_alone(r);
    upto = wave_prefix(g.sum);
    w.s = __shfl(upto, 63, 64);
  }
  int32_t token = -1;
  if (w.s > 0.0) {
    // The first v at which the sum exceeds `aim`: its segment, then chunks of neighbouring values.
    const double aim = static_cast<double>(p.sample_u[b]) * w.s;
    const uint64_t past = __ballot(upto > aim);
    const int seg = past ? __builtin_ctzll(past) : 0;
    double base = seg > 0 ? __shfl(upto, seg - 1, 64) : 0.0;
    const double target = past ? aim : static_cast<double>(kInf);
    for (int64_t v0 = int64_t{seg} * g.length;; v0 = 0, base = 0.0) {
      const bool from_start = v0 == 0;
      __syncthreads();
      if (tid == 0) {
        hit = V;
        last = -1;
      }
      for (; v0 < V; v0 += kThreads * kSize) {
        const int64_t at = v0 + int64_t{tid} * kSize;
        const int32_t v = static_cast<int32_t>(min(at, int64_t{V}));
        typename R::Loaded x;
        r.load(x, v, V);
        double y[kSize], sum = 0.0;
        r.values(x, v, y);
#pragma unroll
        for (int e = 0; e < kSize; ++e) sum += y[e];
        const double incl = wave_prefix(sum);
        __syncthreads();                   // before: sums and hit are read
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        double at_sum = base, all = base;
        for (int i = 0; i < kWaves; ++i) {
          if (i < wave) at_sum += sums[i];
          all += sums[i];
        }
        const double before = shifted_up(incl, 1);
        if (lane > 0) at_sum += before;
        int32_t found = V, positive = -1;
#pragma unroll
        for (int e = kSize - 1; e >= 0; --e)
          if (y[e] > 0.0 && positive < 0) positive = v + e;
#pragma unroll
        for (int e = 0; e < kSize; ++e) {
          at_sum += y[e];
          if (y[e] > 0.0 && at_sum > target && found == V) found = v + e;
        }
        if (found < V) atomicMin(&hit, found);
        if (positive >= 0) atomicMax(&last, positive);
        __syncthreads();
        if (hit < V) break;
        base = all;
      }
      __syncthreads();
      // Sums in two orders may differ in their last bit, past the last positive value too.
      token = hit < V ? hit : last;
      if (token >= 0 || from_start) break;
    }
  }
  for (int32_t i = tid; i < p.width; i += kThreads) {
    path[i] = i < w.count ? t.path[i] : -1;
    out[i] = i + 1 < w.count ? t.token[t.path[i + 1]] : i + 1 == w.count ? token : -1;
  }
  if (tid == 0) p.count[b] = w.count;
}

template <int TYPE, bool DRAFT>
hipError_t launch(const TreeVerifyProblem& p, hipStream_t stream) {
  constexpr int64_t kChunk = int64_t{kThreads} * Chunk<TYPE>::kSize;
  const int64_t chunks = (p.vocab + kChunk - 1) / kChunk;
  int64_t most = kVerifyGroups / p.nodes.batch;
  most = most < 1 ? 1 : most > 64 ? 64 : most;
  const int64_t each = (chunks + most - 1) / most, slices = (chunks + each - 1) / each;
  hipLaunchKernelGGL((tree_verify_kernel<TYPE, DRAFT>), dim3(static_cast<unsigned>(slices * p.nodes.batch)),
                     dim3(kThreads), 0, stream, p, static_cast<int32_t>(slices), static_cast<int32_t>(each * kChunk));
  return hipGetLastError();
}

template <int TYPE>
hipError_t launch_type(const TreeVerifyProblem& p, hipStream_t stream) {
  return p.draft ? launch<TYPE, true>(p, stream) : launch<TYPE, false>(p, stream);
}

}  // namespace

hipError_t launch_tree_verify(const TreeVerifyProblem& p, hipStream_t stream) {
  if (p.type == 0) return launch_type<0>(p, stream);
  return p.type == 1 ? launch_type<1>(p, stream) : launch_type<2>(p, stream);
}

}  // namespace mx
