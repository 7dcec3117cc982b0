// Verification of trees of drafted tokens against the target's probabilities for gfx950.
//
// The walk (see mx_draft.h): at a node with target row p and draft row q, a child of token x is accepted
// when u q(x) S < r(x) Q with r(v) = max(p(v) - c q(v), 0); each rejection needs S = sum r(v) over the
// vocabulary, and the last one's r is what the next token is drawn from.  (What is left of a target
// distribution r / S after a token of q / Q was rejected is max(r / S - q / Q, 0) = max(p - (c + S / Q) q,
// 0) / S: its shape is kept in the one number c, and no row is ever written.)
//
// Bound by latency, and by the sums: each is a pass over a row of p and one of q.  All that the tests need of
// the rows is p(x) and q(x) of every child, loaded at once into LDS; then the walk costs no memory access until
// the first sum.  For that one a row is cut into parts, a workgroup each, which all take the same walk to find
// out what to sum; the last to arrive has S.  A chain is done then but for finding the token within one
// 64th of its row.  A tree may need more sums: the same workgroups take parts of them (Team), as one CU reads
// no more than 67 GB/s (100003 fp32 of both rows: 12 us by itself, 6.8 us so).
//
// Measured, whole calls in a graph: a chain of 4 over 32000 fp32, 9.6 us: launch 2, the children's
// probabilities 1, walk 1.3, sum 2.5, arrival 1, the token 2.2.  16 trees of 26 nodes over 100003: 31 us, the
// slowest of them four sums.  41 trees of 64 chosen drafts over 131072 bf16: 13 us.  Most of the code runs
// once a call, and fetching it is much of that: loops stay rolled where unrolling would not feed more loads.
//
// In 64 bits: a token is decided by where a random number falls between sums of up to 2^30 terms, and 32 bits
// would misplace it once in some hundred tokens.
#include "draft_common.h"

#include <type_traits>

namespace mx {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// 16 bytes of neighbouring probabilities; rows are aligned to their elements only.
template <int TYPE>
struct Chunk {
  static constexpr int kBytes = TYPE == 0 ? 4 : 2, kSize = 16 / kBytes;
  typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t Words2 __attribute__((ext_vector_type(4), aligned(2)));
  typedef std::conditional_t<TYPE == 0, Words4, Words2> Words;
  // The bits of 0 and of all positive finite numbers are the smallest: these are the first past them.
  static constexpr uint32_t kPast = TYPE == 0 ? 0x7F800000u : TYPE == 1 ? 0x7F80u : 0x7C00u;
  uint32_t x[4];

  __device__ __forceinline__ void load(const uint8_t* row, int64_t v) {
    const Words w = *reinterpret_cast<const Words*>(row + v * kBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = w[i];
  }
  // The first `n` elements alone (rows shorter than a chunk).
  __device__ __forceinline__ void load_some(const uint8_t* row, int32_t n) {
    for (int i = 0; i < 4; ++i) x[i] = 0;
#pragma unroll
    for (int e = 0; e < kSize; ++e) {
      if (e >= n) break;
      if constexpr (TYPE == 0) x[e] = reinterpret_cast<const uint32_t*>(row)[e];
      else x[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[e]) << (16 * (e & 1));
    }
  }
  // Its first n elements become 0.
  __device__ __forceinline__ void drop(int32_t n) {
#pragma unroll
    for (int e = 0; e < kSize; ++e) {
      if (e >= n) break;
      if constexpr (TYPE == 0) x[e] = 0;
      else x[e / 2] &= e & 1 ? 0xFFFFu : 0xFFFF0000u;
    }
  }
  // Whether some element is none of the numbers that count, and what each is then.
  __device__ __forceinline__ bool odd() const {
    if constexpr (TYPE == 0) return max(max(x[0], x[1]), max(x[2], x[3])) >= kPast;
    typedef uint16_t Halves __attribute__((ext_vector_type(2)));
    const Halves m = __builtin_elementwise_max(
        __builtin_elementwise_max(__builtin_bit_cast(Halves, x[0]), __builtin_bit_cast(Halves, x[1])),
        __builtin_elementwise_max(__builtin_bit_cast(Halves, x[2]), __builtin_bit_cast(Halves, x[3])));
    return m[0] >= kPast || m[1] >= kPast;
  }
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == 0) {
        if (x[i] >= kPast) x[i] = 0;
      } else {
        if ((x[i] & 0xFFFFu) >= kPast) x[i] &= 0xFFFF0000u;
        if (x[i] >> 16 >= kPast) x[i] &= 0xFFFFu;
      }
    }
  }
  // Element e of a clean chunk.
  __device__ __forceinline__ double get(int e) const {
    if constexpr (TYPE == 0) return __uint_as_float(x[e]);
    const uint32_t w = x[e / 2];
    if constexpr (TYPE == 1) return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(e & 1 ? w >> 16 : w & 0xFFFFu)));
  }
};

// A row's element; what is no probability (negative, infinite, NaN) counts as 0.
template <int TYPE>
__device__ __forceinline__ float load_one(const uint8_t* row, int64_t i) {
  if constexpr (TYPE == 0) {
    const uint32_t x = reinterpret_cast<const uint32_t*>(row)[i];
    return __uint_as_float(x < Chunk<0>::kPast ? x : 0u);
  }
  uint16_t x = reinterpret_cast<const uint16_t*>(row)[i];
  if (x >= Chunk<TYPE>::kPast) x = 0;
  if constexpr (TYPE == 1) return __uint_as_float(uint32_t{x} << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, x));
}

// max(p - c q, 0)
__device__ __forceinline__ double residual(double p, double c, double q) {
  return __builtin_fmax(__builtin_fma(-c, q, p), 0.0);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(x >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, uint64_t{hi} << 32 | lo);
}

// Sums over the lanes up to and with this one (every lane active): within rows of 16, then the rows'.
__device__ __forceinline__ double wave_prefix(double v) {
  v += moved<0x111, 0xF>(v);
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);               // rows 1 and 3: the last lane's of the row before
  v += moved<0x143, 0xC>(v);               // rows 2 and 3: that of lane 31
  return v;
}

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(x), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(x >> 32), lane);
  return __builtin_bit_cast(double, uint64_t{hi} << 32 | lo);
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ double wave_total(double v) { return lane_value(wave_prefix(v), 63); }

// The walk through a sequence's tree: one wavefront takes it.
struct Walk {
  int32_t cur, next, count;    // the node, the first one that may still be its child, nodes accepted
  int32_t more, summed;        // children may be left to try; s is r's sum over the vocabulary
  double c, s, q;              // what r is made of, its sum, what is left of the draft's distribution
};

// What the tests need, in LDS.
struct Tests {
  int32_t up[kMostNodes], token[kMostNodes];
  float u[kMostNodes], p[kMostNodes], q[kMostNodes];      // of the token in its parent's rows
  int32_t path[kMostNodes];
};

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Goes on until a child was rejected and r's sum is needed for others that may follow (true), or none is
// left (false).
// 64 nodes at a time lie in the lanes' registers: a test reads no memory.
template <bool DRAFT>
__device__ __forceinline__ bool walk_on(Walk& w, Tests& t, int32_t n, int32_t width, bool replacement) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  while (w.next < n && w.count < width) {
    const int32_t at = w.next & ~63, mine = min(at + lane, n - 1);
    const int32_t up = at + lane < n ? t.up[mine] : -1, token = t.token[mine];
    const float us = t.u[mine], ps = t.p[mine], qs = DRAFT ? t.q[mine] : 0.f;
    for (;;) {                             // the children of cur among them from `next` on
      const uint64_t its = __ballot(up == w.cur) & (~uint64_t{0} << (w.next - at));
      if (its == 0) {
        w.next = min(at + 64, n);
        break;
      }
      const int x = __builtin_ctzll(its);
      const int32_t i = at + x;
      w.next = i + 1;
      const double u = lane_value(us, x), p = lane_value(ps, x);
      bool accepted;
      if constexpr (DRAFT) {
        const double q = lane_value(qs, x), r = residual(p, w.c, q);
        const double a = u * q, left = a * w.s, right = r * w.q;
        accepted = w.q > 0.0 && r > 0.0 && left < right;
        if (!accepted && w.q > 0.0) {
          const double step = w.s / w.q;
          w.c = w.c + step;
          if (!replacement) w.q = w.q - q;
          w.summed = 0;
          return (its & (its - 1)) != 0 || at + 64 < n;
        }
      } else {
        // A token that was rejected here before is no longer there.
        const int32_t tx = __builtin_amdgcn_readlane(token, x);
        bool again = __any(up == w.cur && token == tx && lane < x);
        for (int32_t k = w.cur + 1; k < at && !again; k += 64) {
          const int32_t j = min(k + lane, at - 1);
          again = __any(t.up[j] == w.cur && t.token[j] == tx);
        }
        const double r = again ? 0.0 : p, left = u * w.s;
        accepted = r > 0.0 && left < r;
        if (!accepted) {
          const double rest = w.s - r;
          w.s = rest > 0.0 ? rest : 0.0;
        }
      }
      if (accepted) {
        w.cur = i;
        if (lane == 0) t.path[w.count] = i;
        ++w.count;
        w.c = 0.0;
        w.s = 1.0;
        w.q = 1.0;
        w.summed = 0;
        if (w.count >= width) return false;
      }
      if (w.next - at >= 64) break;
    }
  }
  return false;
}

// A row is summed in 64 segments, which say where a token lies to within one chunk of a workgroup.  Of 2^k
// workgroups' wavefronts, 2^k / 4 have a segment between them, or one has 4 / 2^k of them.
constexpr int kSegments = 64;

// How a row is cut for `parts` workgroups (a power of two): into runs of `length` elements.
struct Cut {
  int32_t length;
  int a_wave, a_segment;       // runs
};

template <int TYPE>
__device__ __forceinline__ Cut cut_of(int32_t vocab, int32_t parts) {
  constexpr int kSize = Chunk<TYPE>::kSize;
  Cut c;
  c.a_wave = max(1, 4 / parts);
  c.a_segment = max(1, parts / 4);
  const int32_t runs = kSegments * c.a_segment;
  c.length = (((vocab + runs - 1) >> __builtin_ctz(runs)) + kSize - 1) & ~(kSize - 1);
  return c;
}

// A node's residual over the vocabulary.
template <int TYPE, bool DRAFT>
struct Rest {
  static constexpr int kSize = Chunk<TYPE>::kSize;
  const uint8_t *p, *q;        // its rows
  int32_t vocab;
  double c;                    // 0: q is not read
  const int32_t* gone;         // tokens that have left it (chosen drafts)
  int32_t ngone;

  // The chunk at v: loaded from where a whole one lies, `from`; its first v - from elements are not its.
  struct Loaded {
    Chunk<TYPE> p, q;
    int32_t v, from;
  };
  __device__ __forceinline__ void load(Loaded& w, int32_t v) const {
    w.v = v;
    w.from = max(min(v, vocab - kSize), 0);
    if (__builtin_expect(vocab >= kSize, 1)) {
      w.p.load(p, w.from);
      if (DRAFT && c != 0.0) w.q.load(q, w.from);
    } else {
      w.p.load_some(p, vocab);
      if (DRAFT && c != 0.0) w.q.load_some(q, vocab);
    }
  }
  // Its values, element by element from `from`.  A wavefront's chunks lie one after
  // the other.
  __device__ __forceinline__ void values(Loaded& w, double (&r)[kSize]) const {
    const bool has_q = DRAFT && c != 0.0;
    if (__builtin_expect(__any(w.p.odd() || (has_q && w.q.odd())), 0)) {
      w.p.clean();
      if (has_q) w.q.clean();
    }
    if (__builtin_expect(__any(w.v != w.from), 0)) w.p.drop(w.v - w.from);
#pragma unroll
    for (int e = 0; e < kSize; ++e) r[e] = w.p.get(e);
    if (has_q) {
#pragma unroll
      for (int e = 0; e < kSize; ++e) r[e] = residual(r[e], c, w.q.get(e));
    }
    if constexpr (!DRAFT) {
      const int lane = threadIdx.x & 63;
      const int32_t first = __builtin_amdgcn_readfirstlane(w.from);
      for (int32_t i = 0; i < ngone; i += 64) {
        // Few lie among the wavefront's: those are looked for in the lanes'.
        const int32_t mine = gone[min(i + lane, ngone - 1)];
        uint64_t all = __ballot(i + lane < ngone && mine >= first && mine - first < 64 * kSize);
        for (; all; all &= all - 1) {
          const int32_t x = __builtin_amdgcn_readlane(mine, __builtin_ctzll(all)) - w.from;
#pragma unroll
          for (int e = 0; e < kSize; ++e)
            if (x == e) r[e] = 0.0;
        }
      }
    }
  }
  // The wavefront's sum of [begin, end).  Code that runs once a call costs its fetching: two chunks a lane
  // at once, no more.
  __device__ __forceinline__ double sum_run(int32_t begin, int32_t end) const {
    const int32_t at = static_cast<int32_t>(threadIdx.x & 63) * kSize;
    double sum = 0.0;
#pragma unroll 1
    for (int32_t v0 = begin; v0 < end; v0 += 128 * kSize) {
      Loaded w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) load(w[i], min(v0 + i * 64 * kSize + at, vocab));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        double r[kSize], of = 0.0;
        values(w[i], r);
#pragma unroll
        for (int e = 0; e < kSize; ++e) of += r[e];
        sum += w[i].v < end ? of : 0.0;
      }
    }
    return wave_total(sum);
  }
};

// What a workgroup is to sum: a part of the residual r(v) = max(p(v) - c q(v), 0) at node cur; part < 0: nothing.
struct Job {
  int32_t part, cur;
  double c;
};

// The workgroups of a sequence that sum its rows together.  Parts are taken, not given: who leads asks for a
// sum and takes parts of it like the others, so it needs none of them.  A helper waits for kPatience at most
// and leaves then (it may be that workgroups which have to come before there is a leader wait for its place);
// the leader waits for parts that running workgroups have taken.  So every wait ends, whoever is resident.
//
// A sequence's line of counters, all zero between calls: arrivals; the ticket (sums asked for in the upper
// half, parts taken of the last one in the lower); parts done of all sums; workgroups that have left; the
// node; c.
struct Team {
  uint32_t* words;
  double* sums;                // the segments'
  Job* job;
  int32_t size;                // 1: alone
  uint32_t asked;              // sums so far

  static constexpr uint32_t kOne = 0x10000u, kDismissed = 0xFFFF0000u;
  static constexpr int64_t kPatience = 10000;        // of wall_clock64: 100 us

  __device__ __forceinline__ Team(const TreeVerifyProblem& p, int32_t b, int32_t slices, Job* j)
      : words(p.counters + static_cast<int64_t>(b) * kTeamWords), sums(p.parts + static_cast<int64_t>(b) * kSegments),
        job(j), size(slices), asked(0) {}

  __device__ __forceinline__ static uint32_t read(const uint32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ static void write(uint32_t* p, uint32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ static uint32_t add(uint32_t* p, uint32_t v) {
    return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // Every store of this workgroup that came before is where all see it.
  __device__ __forceinline__ static void stored() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(kVmcntZero);
    __syncthreads();
  }
  __device__ __forceinline__ void store(int32_t i, double v) const {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(sums + i), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ double load(int32_t i) const {
    return __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(sums + i), __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT));
  }

  // The leader's: a sum over all parts.  Every part of the one before is done.
  __device__ __forceinline__ void ask(int32_t cur, double c) {
    ++asked;
    if (threadIdx.x != 0) return;
    write(words + 4, static_cast<uint32_t>(cur));
    __hip_atomic_store(reinterpret_cast<uint64_t*>(words + 6), __builtin_bit_cast(uint64_t, c), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(kVmcntZero);
    write(words + 1, asked * kOne);
  }
  // A part of the sum asked for (-1: none is left, or a helper is not needed), and of what.
  __device__ __forceinline__ int32_t claim(bool leads, int32_t* cur, double* c) const {
    __syncthreads();
    if (threadIdx.x == 0) {
      int32_t part = -1;
      for (const int64_t since = wall_clock64();;) {
        uint32_t t = leads ? 0 : read(words + 1);
        if (t >= kDismissed) break;
        if (leads || (t >= kOne && (t & (kOne - 1)) < static_cast<uint32_t>(size))) {
          t = add(words + 1, 1u);
          if (t < kDismissed && (t & (kOne - 1)) < static_cast<uint32_t>(size)) part = t & (kOne - 1);
          if (leads || part >= 0 || t >= kDismissed) break;
        }
        if (wall_clock64() - since > kPatience) break;
        __builtin_amdgcn_s_sleep(1);
      }
      job->part = part;
      if (part >= 0 && !leads) {
        // What was asked stays until this part is done.
        job->cur = static_cast<int32_t>(read(words + 4));
        job->c = __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(words + 6),
                                                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      }
    }
    __syncthreads();
    const int32_t part = uniform(job->part);
    if (part >= 0 && !leads) {
      *cur = uniform(job->cur);
      *c = lane_value(job->c, 0);
    }
    return part;
  }
  __device__ __forceinline__ void done() const {
    stored();
    if (threadIdx.x == 0) add(words + 2, 1u);
  }
  // The leader's: until every part is done, by workgroups that run.
  __device__ __forceinline__ void wait() const {
    if (threadIdx.x == 0)
      while (read(words + 2) != asked * static_cast<uint32_t>(size)) __builtin_amdgcn_s_sleep(1);
    __syncthreads();
  }
  __device__ __forceinline__ void dismiss() const {
    if (threadIdx.x == 0) write(words + 1, kDismissed);
  }
  // The last to leave clears what it leaves behind (nobody reads it any more).
  __device__ __forceinline__ void leave() const {
    if (threadIdx.x != 0) return;
    __builtin_amdgcn_s_waitcnt(kVmcntZero);          // what it wrote lies before what the last one clears
    if (add(words + 3, 1u) + 1 != static_cast<uint32_t>(size)) return;
    for (int i = 1; i < 8; ++i) write(words + i, 0u);
  }
};

template <int TYPE, bool DRAFT>
__global__ __launch_bounds__(kThreads) void tree_verify_kernel(const TreeVerifyProblem p, int32_t slices) {
  typedef Rest<TYPE, DRAFT> R;
  constexpr int kBytes = Chunk<TYPE>::kBytes, kSize = R::kSize;
  __shared__ Tests t;
  __shared__ int32_t gone[DRAFT ? 1 : kMostNodes];
  __shared__ int32_t ngone, hit[kWaves], last[kWaves];
  __shared__ double sums[kWaves], runs[kSegments];
  __shared__ uint32_t flag;
  __shared__ Job job;
  __shared__ Walk walk;
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
    t.p[i] = real ? load_one<TYPE>(row(p.target, p.target_stride, up), x) : 0.f;
    if constexpr (DRAFT) t.q[i] = real ? load_one<TYPE>(row(p.draft, p.draft_stride, up), x) : 0.f;
  }
  if (tid == 0) t.path[0] = 0;
  __syncthreads();
  Walk w = {0, 1, 1, 1, 0, 0.0, 1.0, 1.0};
  Team team(p, b, slices, &job);
  bool whole = false;                      // r is the target's row itself
  R r;
  r.vocab = V;
  r.gone = gone;
  auto look_at_node = [&]() {
    r.p = row(p.target, p.target_stride, w.cur);
    r.q = DRAFT ? row(p.draft, p.draft_stride, w.cur) : nullptr;
    r.c = whole ? 0.0 : w.c;
    r.ngone = DRAFT || whole ? 0 : uniform(ngone);
  };
  // The first sum is every workgroup's, a part each.  The last to arrive has it, and leads: it takes the walk
  // on, and where another sum is needed the others, who have waited for it, help.
  bool first = true, leads = true;
  int32_t parts = slices;                  // what makes the segments
  double upto = 0.0;
  for (;;) {
    if (leads) {
      // One wavefront's walk, not each its own: 16 at once take 3 us for 1.
      if (w.more) {
        if (wave == 0) {
          w.more = walk_on<DRAFT>(w, t, s.n, p.width, p.replacement);
          if constexpr (!DRAFT) {
            // The tokens of the children that were rejected.
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
          if (lane == 0) walk = w;
        }
        __syncthreads();
        w = Walk{uniform(walk.cur), uniform(walk.next), uniform(walk.count), uniform(walk.more), uniform(walk.summed),
                 lane_value(walk.c, 0), lane_value(walk.s, 0), lane_value(walk.q, 0)};
      }
      if (!w.more && w.summed) {
        if (whole || w.s > 0.0) break;
        whole = true;                      // nothing is left: the target's row itself
      }
      if (!first) {
        parts = whole ? 1 : team.size;
        if (parts > 1) team.ask(w.cur, w.c);
      }
    }
    double seg_sum;
    for (int32_t part = first ? mine : 0;;) {
      if (!first && parts > 1) {
        part = team.claim(leads, &w.cur, &w.c);
        if (part < 0) break;
      }
      look_at_node();
      const Cut cut = cut_of<TYPE>(V, parts);
      __syncthreads();                     // what the last sums left is read
      for (int i = 0; i < cut.a_wave; ++i) {
        const int32_t run = (part * kWaves + wave) * cut.a_wave + i;
        const int64_t begin = int64_t{run} * cut.length;
        const double sum = begin < V ? r.sum_run(static_cast<int32_t>(begin), static_cast<int32_t>(min(begin + cut.length, int64_t{V})))
                                     : 0.0;
        if (lane == 0) runs[wave * cut.a_wave + i] = sum;
      }
      __syncthreads();
      seg_sum = lane < kWaves * cut.a_wave ? runs[lane] : 0.0;
      for (int d = 1; d < cut.a_segment; d *= 2) seg_sum += __shfl_xor(seg_sum, d, 64);
      if (parts == 1) break;
      if (wave == 0 && lane % cut.a_segment == 0 && lane < kWaves * cut.a_wave)
        team.store((part * kWaves * cut.a_wave + lane) / cut.a_segment, seg_sum);
      if (first) break;
      team.done();
    }
    if (parts > 1) {
      if (first) {
        leads = arrive_last(team.words, parts, &flag);
        if (!w.more) {                     // no other sum
          if (!leads) return;
          team.size = 1;
        }
      } else if (leads) {
        team.wait();
      } else {
        team.leave();
        return;
      }
    }
    first = false;
    if (!leads) continue;
    if (parts > 1) seg_sum = team.load(lane);
    upto = wave_prefix(seg_sum);
    w.s = lane_value(upto, 63);
    w.summed = 1;
  }
  if (team.size > 1) {
    team.dismiss();
    team.leave();
  }
  look_at_node();
  int32_t token = -1;
  if (w.s > 0.0) {
    // The first v at which the sum exceeds `aim`: its segment, then chunks of neighbouring values.
    const double aim = static_cast<double>(p.sample_u[b]) * lane_value(upto, 63);
    const uint64_t past = __ballot(upto > aim);
    const int seg = past ? __builtin_ctzll(past) : 0;
    double base = seg > 0 ? lane_value(upto, seg - 1) : 0.0;
    const Cut cut = cut_of<TYPE>(V, parts);
    const double target = past ? aim : static_cast<double>(kInf);
    for (int64_t v0 = int64_t{seg} * cut.length * cut.a_segment;; v0 = 0, base = 0.0) {
      const bool from_start = v0 == 0;
      int32_t final_one = -1;              // the last positive value so far
      for (; v0 < V && token < 0; v0 += kThreads * kSize) {
        typename R::Loaded x;
        r.load(x, static_cast<int32_t>(min(v0 + tid * kSize, int64_t{V})));
        double y[kSize], sum = 0.0;
        r.values(x, y);
#pragma unroll
        for (int e = 0; e < kSize; ++e) sum += y[e];
        const double incl = wave_prefix(sum), before = __shfl_up(incl, 1, 64);
        __syncthreads();                   // what the last chunk left is read
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        // Sums up to each wavefront's values: lane i those of wavefront i.
        const double of_waves = wave_prefix(lane < kWaves ? sums[lane] : 0.0);
        double at_sum = base + (wave > 0 ? lane_value(of_waves, wave - 1) : 0.0);
        base += lane_value(of_waves, 63);
        if (lane > 0) at_sum += before;
        int32_t found = -1, positive = -1;
#pragma unroll
        for (int e = 0; e < kSize; ++e) {
          at_sum += y[e];
          if (y[e] > 0.0) {
            positive = x.from + e;
            if (at_sum > target && found < 0) found = positive;
          }
        }
        const uint64_t have = __ballot(found >= 0), some = __ballot(positive >= 0);
        if (lane == 0) {
          hit[wave] = have ? __builtin_amdgcn_readlane(found, __builtin_ctzll(have)) : -1;
          last[wave] = some ? __builtin_amdgcn_readlane(positive, 63 - __builtin_clzll(some)) : -1;
        }
        __syncthreads();
        const int32_t h = lane < kWaves ? hit[lane] : -1, l = lane < kWaves ? last[lane] : -1;
        const uint64_t hits = __ballot(h >= 0), lasts = __ballot(l >= 0);
        if (hits) token = __builtin_amdgcn_readlane(h, __builtin_ctzll(hits));
        if (lasts) final_one = __builtin_amdgcn_readlane(l, 63 - __builtin_clzll(lasts));
      }
      // Sums in two orders may differ in their last bit, past the last positive value too.
      if (token < 0) token = final_one;
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
  // Parts of a row: no smaller than half a chunk of each lane, as many as the chip has CUs for.
  constexpr int64_t kLeast = int64_t{kThreads} * Chunk<TYPE>::kSize / 2;
  int64_t slices = 1;
  while (slices < kSegments && 2 * slices * p.nodes.batch <= kVerifyGroups && 2 * slices * kLeast <= p.vocab) slices *= 2;
  hipLaunchKernelGGL((tree_verify_kernel<TYPE, DRAFT>), dim3(static_cast<unsigned>(slices * p.nodes.batch)),
                     dim3(kThreads), 0, stream, p, static_cast<int32_t>(slices));
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
