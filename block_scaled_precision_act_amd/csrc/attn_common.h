// Device pieces shared by the attention operators' kernels.
#pragma once

#include "attn_internal.h"
#include "mx_quant.h"

#include <type_traits>

namespace mx {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// s_waitcnt operand that waits for every vector-memory access of the wavefront and nothing else.
constexpr int kVmcntZero = 0x0F70;

constexpr float kNaN = __builtin_nanf("");
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 rounded to nearest even into packed bf16 (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <int V>
struct IntC { static constexpr int value = V; };

// 8 E2M1 codes times the scale -> 8 bf16, exact.
__device__ __forceinline__ uint4 decode8(uint32_t d, float s) {
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3)));
}

// Byte `a` (0..3, constant after unrolling) of d: two codes times the scale -> two bf16.
__device__ __forceinline__ uint32_t decode2(uint32_t d, float s, int a) {
  return __builtin_bit_cast(uint32_t, a == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0)
                                      : a == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1)
                                      : a == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3));
}

// v_perm selectors: the low (high) halves of (second, first) operand, first in the low half.
constexpr uint32_t kLowHalves = 0x05040100u, kHighHalves = 0x07060302u;

// Reads an int32 that no kernel writes meanwhile (a scalar load where the index is uniform).
typedef const __attribute__((address_space(4))) int32_t* ConstInts;

__device__ __forceinline__ int32_t read_uniform(const int32_t* p, int64_t i) {
  return reinterpret_cast<ConstInts>(reinterpret_cast<uintptr_t>(p))[i];
}

// The scale in a byte of `word`, for the scaled conversions: they read a scale's exponent field alone
// (its sign and mantissa bits change nothing, checked for every byte and code), so rotating the word
// right by 9 + 8 * byte is enough.
__device__ __forceinline__ float scale_of_byte(uint32_t word, uint32_t turn) {
  return __uint_as_float(__builtin_amdgcn_alignbit(word, word, turn));
}

constexpr uint32_t kScalesOfOne = 0x7F7F7F7Fu;       // four E8M0 bytes

// The value of lane `i` (0..3, constant after unrolling) of each group of four.
__device__ __forceinline__ uint32_t quad_lane(uint32_t v, int i) {
  const int x = static_cast<int>(v);
  return static_cast<uint32_t>(i == 0   ? __builtin_amdgcn_mov_dpp(x, 0x00, 0xF, 0xF, false)
                               : i == 1 ? __builtin_amdgcn_mov_dpp(x, 0x55, 0xF, 0xF, false)
                               : i == 2 ? __builtin_amdgcn_mov_dpp(x, 0xAA, 0xF, 0xF, false)
                                        : __builtin_amdgcn_mov_dpp(x, 0xFF, 0xF, 0xF, false));
}

// The largest of the values of lanes that differ in bit 4 (every lane active).
__device__ __forceinline__ float max_rows(float v) {
  const v2u r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The larger of the lane's value and that of the lane 32 away (every lane active).
__device__ __forceinline__ float max_halves(float v) {
  const v2u r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The first key that a query at position `at` sees, or a number below 0.  A position is negative where a
// sequence is shorter than its queries; such a query sees no key, and counting it as -1 keeps the
// difference within 32 bits for windows of up to 2^31 - 1.
__device__ __forceinline__ int32_t window_start(int32_t at, int32_t window) {
  return max(at, -1) + 1 - window;
}

template <bool TREE>
using ProblemOf = std::conditional_t<TREE, AttnTreeProblem, AttnProblem>;

// Of a tree's query, which of the 32 tokens from `d` tokens behind the first node on it sees: its own
// bits from there on, ones for what lies before the tree.  A word is read where it exists.
__device__ __forceinline__ uint32_t tree_bits(const AttnTreeProblem& p, int32_t query, int32_t d) {
  const uint32_t* row = p.tree + query * p.tree_stride;
  const int32_t w = d >> 5;
  const uint32_t lo = w < 0 ? ~0u : w < p.tree_words ? row[w] : 0u;
  const uint32_t hi = w < -1 ? ~0u : w + 1 < p.tree_words ? row[w + 1] : 0u;
  return __builtin_amdgcn_alignbit(hi, lo, d & 31);
}

// The first key before the tree that its query sees: the query's position lies within the tree's
// [first, end), as its depth does (whatever the caller's says).
__device__ __forceinline__ int32_t tree_window_start(const AttnTreeProblem& p, int32_t query, int32_t first,
                                                     int32_t end) {
  return window_start(min(max(p.tree_at[query], first), end - 1), p.window);
}

// A row's weights are exp2(s scale - m), one fused multiply-add each, with m the rounded product of its
// largest score and the scale.  The maximum that is subtracted moves only when some row's rose by more
// than `kSlack`: until then weights stay below 2^8, and bf16 and fp32 hold them as well as those below
// one.  (Moved at every rise, a prompt of 8192 tokens takes 5% more.)
//
// At the largest score the fused form gives m's rounding error, the same for all of the row's weights, so
// it cancels in their mean; but from |m| = 2^28 on it may pass 2^8, and from 2^31 on the largest weight
// could overflow or vanish.  There the scores are multiplied first, and rounded as m is: the largest
// weight is then 1.  A slack of -infinity brings every later step to where that is done, so the others
// spend nothing on it.
constexpr float kSlack = 8.f, kLargeScore = 268435456.f;         // 2^28

// Whether some row of the wavefront has such a maximum (m = -infinity: has seen nothing).
__device__ __forceinline__ bool large_scores(float m) { return __any(fabsf(m) >= kLargeScore && m != -kInf); }

// A product rounded by itself, whatever it is added to.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// The same value, but not known to be: what was computed from it before is computed again.
__device__ __forceinline__ uint32_t again(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Workgroup barrier for data passed through LDS: waits for the wavefront's LDS accesses only, so
// loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Stores of partial results that other workgroups will read: device scope, so they are written
// through this XCD's L2 to where every XCD sees them.  (Plain stores would need the L2 written back
// before the handoff, and that L2 also holds whatever else the kernel writes: with the gradients of
// 16384 x 40 heads in it, 1024 workgroups' write-backs cost 44 us.)
__device__ __forceinline__ void store_shared(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_shared4(float* p, float a, float b, float c, float d) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(q, __builtin_bit_cast(uint64_t, v2u{__float_as_uint(a), __float_as_uint(b)}),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, __builtin_bit_cast(uint64_t, v2u{__float_as_uint(c), __float_as_uint(d)}),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Called by every thread of a workgroup once it has stored its partial results with the functions
// above: counts the workgroup in at `counter`.  Returns (to every thread) whether it is the last of
// `expected`; the last one then sees what all others stored, and has put the counter back to zero.
//   (1) Every wavefront waits until its own stores are complete (written through); (2) past the
//   barrier the whole workgroup's are, so they precede thread 0's arrival; (3) the last arrival's
//   acquire drops what this XCD's caches may hold stale, before the barrier lets any thread load.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, uint32_t expected, uint32_t* flag) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(kVmcntZero);
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
    const bool last = n + 1 == expected;
    if (last) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    *flag = last;
  }
  __syncthreads();
  return *flag != 0u;
}

}  // namespace
}  // namespace mx
