// Per-head norm of queries and keys with the position rotation in the same pass, and its
// gradients, for gfx950.
//
// Forward, for a head x of D values at position p, in fp32:
//   r = rsqrt(mean(x^2) + eps), n = x r w, y = R(p) n, rounded once to bf16.
// Backward (the rotation's transpose turns back): n' = R(p)^T dy, g = n' w,
//   dx = r (g - x r^2 mean(g x)),  dw = sum over rows of n' x r.
//
// Both are bound by HBM: every input read once, every output written once.  D / 8 lanes own a row,
// 8 values each, chosen so that a lane holds both members of its rotated pairs: values
// [4 j, 4 j + 4) and [rot/2 + 4 j, ...) for pairs half a rotation apart, 8 neighbours for
// interleaved pairs and for what lies past `rot`.  So the rotation needs no exchange, the row sums
// are log2(D / 8) lane exchanges, and loads are 8 bytes a lane in runs of at least 32 bytes.
#include "attn_common.h"

#include <algorithm>

namespace mx {
namespace {

constexpr int kThreads = 256;

// From this many values on a row's owners take four heads at once (more loads in flight); below, one,
// as the rows then do not fill the chip.  Four and one: forward, 3.1 M values 5.1 and 4.8 us, 6.1 M 6.2
// and 7.9 us; backward (its workgroups are 511 at most), 0.8 M 9.4 and 9.1 us, 1.5 M 10.1 and 12.8 us
// (heads of 128; 64 and 256 cross over within the same steps).
constexpr uint64_t kManyForward = uint64_t{1} << 22, kManyBackward = uint64_t{1} << 20;

// Sum over the LR lanes that own a row, by DPP: quads, then mirrors of 8 and 16 lanes (whose quads
// and halves already hold equal sums), then the two rows of 16.  All lanes are active.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(
                 static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, false)));
}

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<0xB1>(v);                       // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);                       // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);                      // row_half_mirror
  if constexpr (LR >= 16) v = dpp_add<0x140>(v);   // row_mirror
  if constexpr (LR >= 32) {
    const v2u r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Which 8 values of a row lane j owns: [c0, c0 + 4) and [c1, c1 + 4).
struct LaneChunks {
  int c0, c1;
  bool turned;     // the lane's values are rotated, by table entries [4 j, 4 j + 4)
};

template <bool INTER>
__device__ __forceinline__ LaneChunks lane_chunks(int j, int rot) {
  const int half = rot >> 1;
  const bool turned = 8 * j < rot;
  if (INTER || !turned) return {8 * j, 8 * j + 4, turned};
  return {4 * j, half + 4 * j, true};
}

// Turns the lane's pairs by (c, s): (a, b) -> (a c - b s, b c + a s).
template <bool INTER>
__device__ __forceinline__ void turn(float (&x)[8], const float4& c, const float4& s) {
  const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 4;
    const float a = x[ia], b = x[ib];
    x[ia] = a * cc[i] - b * ss[i];
    x[ib] = b * cc[i] + a * ss[i];
  }
}

__device__ __forceinline__ void widen(const uint2& lo, const uint2& hi, float (&x)[8]) {
  x[0] = bf16_lo(lo.x); x[1] = bf16_hi(lo.x); x[2] = bf16_lo(lo.y); x[3] = bf16_hi(lo.y);
  x[4] = bf16_lo(hi.x); x[5] = bf16_hi(hi.x); x[6] = bf16_lo(hi.y); x[7] = bf16_hi(hi.y);
}

__device__ __forceinline__ void load8(const uint16_t* row, const LaneChunks& lc, float (&x)[8]) {
  widen(*reinterpret_cast<const uint2*>(row + lc.c0), *reinterpret_cast<const uint2*>(row + lc.c1),
        x);
}

// Rows are loaded and stored past the caches, each being read or written once: 16384 x 40 heads of 128
// take 60 us so (68 us through the caches), their gradients 100 us (107 us): 5.6 and 5.0 TB/s.
__device__ __forceinline__ void load_stream(const uint16_t* row, const LaneChunks& lc, uint2* lo, uint2* hi) {
  const v2u a = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(row + lc.c0));
  const v2u b = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(row + lc.c1));
  *lo = make_uint2(a[0], a[1]);
  *hi = make_uint2(b[0], b[1]);
}

__device__ __forceinline__ void store8(uint16_t* row, const LaneChunks& lc, const float (&x)[8]) {
  __builtin_nontemporal_store(v2u{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])},
                              reinterpret_cast<v2u*>(row + lc.c0));
  __builtin_nontemporal_store(v2u{pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])},
                              reinterpret_cast<v2u*>(row + lc.c1));
}

// A token's table entries of lane j; a position outside the table sets `bad`.
__device__ __forceinline__ void load_turn(const Rotation& r, uint32_t t, int j, bool turned,
                                          float4* c, float4* s, bool* bad) {
  *c = make_float4(1.f, 1.f, 1.f, 1.f);
  *s = make_float4(0.f, 0.f, 0.f, 0.f);
  *bad = false;
  if (!r.positions) return;
  const uint32_t pos = static_cast<uint32_t>(r.positions[t]);
  *bad = pos >= r.rows;
  if (turned && !*bad) {
    const int64_t at = static_cast<int64_t>(pos) * (r.rot >> 1) + 4 * j;
    *c = *reinterpret_cast<const float4*>(r.cos + at);
    *s = *reinterpret_cast<const float4*>(r.sin + at);
  }
}

// A row's owners handle U heads of one token (one tensor's), all loaded before the first is used;
// the token's table entries are loaded once.  Units of a token: its queries' heads by U, then its
// keys'.
template <int LR, bool INTER, int U>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(const NormRopeProblem p,
                                                             uint32_t units_q, uint32_t units) {
  constexpr int D = 8 * LR, RG = kThreads / LR;
  const int j = threadIdx.x % LR;
  const LaneChunks lc = lane_chunks<INTER>(j, p.rot.rot);
  const uint32_t unit = blockIdx.x * RG + threadIdx.x / LR;
  // Owners past the last unit repeat it (the row sums need every lane) and write nothing.
  const uint32_t all = p.tokens * units, at = min(unit, all - 1);
  const uint32_t t = at / units, part = at - t * units;
  const int i = part >= units_q;
  const uint32_t h0 = (part - (i ? units_q : 0)) * U, heads = p.heads[i];
  const HeadRows& in = p.x[i];
  const uint16_t* src = in.p + t * in.token_stride + h0 * in.head_stride;
  uint2 lo[U], hi[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint16_t* row = src + (h0 + u < heads ? u : 0) * in.head_stride;
    load_stream(row, lc, &lo[u], &hi[u]);
  }
  float w[8];
  const bool norm = p.weight[i] != nullptr;
  if (norm) load8(p.weight[i], lc, w);
  float4 c, s;
  bool bad;
  load_turn(p.rot, t, j, lc.turned, &c, &s, &bad);
  const HeadRows& o = p.out[i];
  uint16_t* dst = o.p + t * o.token_stride + h0 * o.head_stride;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8];
    widen(lo[u], hi[u], x);
    if (norm) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq += x[e] * x[e];
      const float r = rsqrtf(row_sum<LR>(sq) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    }
    turn<INTER>(x, c, s);
    if (bad) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = kNaN;
    }
    if (h0 + u < heads && unit < all) store8(dst + u * o.head_stride, lc, x);
  }
}

// Rows after which a lane's sums are folded into its totals in LDS, with what each addition rounds off
// carried on: no chain of plain additions is longer, however many rows there are.  Calls of fewer rows a
// lane (of 16384 x 40 heads of 128, 81) do without: folding costs them 3%.
constexpr int kFoldRows = 256;

// total[0 .. 4) += v, the carry of the total's rounding errors beside it.
__device__ __forceinline__ void fold4(float4* total, float4* carry, const float* v) {
  const float4 s = *total, c = *carry;
  const float t[4] = {s.x, s.y, s.z, s.w}, k[4] = {c.x, c.y, c.z, c.w};
  float nt[4], nk[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = v[e] - k[e];
    nt[e] = t[e] + y;
    const float off = (nt[e] - t[e]) - y;
    nk[e] = fabsf(off) < kInf ? off : 0.f;   // an infinite total has no rounding error
  }
  *total = make_float4(nt[0], nt[1], nt[2], nt[3]);
  *carry = make_float4(nk[0], nk[1], nk[2], nk[3]);
}

// Workgroups [0, groups_q) take the queries' rows, the rest the keys'; rows are dealt round robin,
// RG at a time.  A lane sums its 8 weight gradients over its rows in fp32 (kFoldRows a chain), the
// workgroup's lanes are summed through LDS, and the last workgroup of a tensor to arrive sums all its
// workgroups' partials in their order, so the result does not depend on which one that is.
template <int LR, bool INTER, int U, bool FOLD>
__global__ __launch_bounds__(kThreads) void norm_rope_back_kernel(const NormRopeBackProblem p,
                                                                  uint32_t groups_q,
                                                                  uint32_t groups_k) {
  constexpr int D = 8 * LR, RG = kThreads / LR;
  __shared__ __align__(16) float sums[RG * D], carries[FOLD ? RG * D : 4];
  __shared__ uint32_t flag;
  const int i = blockIdx.x >= groups_q;
  const uint32_t group = blockIdx.x - (i ? groups_q : 0), groups = i ? groups_k : groups_q;
  const int j = threadIdx.x % LR, rg = threadIdx.x / LR;
  const LaneChunks lc = lane_chunks<INTER>(j, p.rot.rot);
  const uint32_t heads = p.heads[i], units = (heads + U - 1) / U, all = p.tokens * units;
  const bool norm = p.weight[i] != nullptr;
  float w[8], acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.f, acc[e] = 0.f;
  if (norm) load8(p.weight[i], lc, w);
  const HeadRows &gy = p.dy[i], &in = p.x[i], &gx = p.dx[i];
  int unfolded = 0;                          // units since the last fold
  auto fold = [&]() {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int at = rg * D + (c ? lc.c1 : lc.c0);
      fold4(reinterpret_cast<float4*>(sums + at), reinterpret_cast<float4*>(carries + at), acc + 4 * c);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  };
  if constexpr (FOLD) {
    for (int e = threadIdx.x; e < RG * D; e += kThreads) sums[e] = carries[e] = 0.f;
    __syncthreads();
  }
  // Every owner walks the same number of units (the row sums need every lane); past the last one it
  // repeats it, writes nothing and adds nothing.
  for (uint32_t base = group * RG; base < all; base += groups * RG) {
    const uint32_t at = min(base + rg, all - 1);
    const bool real = base + rg < all;
    const uint32_t t = at / units, h0 = (at - t * units) * U;
    uint2 ylo[U], yhi[U], xlo[U], xhi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t h = h0 + u < heads ? h0 + u : h0;
      const uint16_t* row = gy.p + t * gy.token_stride + h * gy.head_stride;
      load_stream(row, lc, &ylo[u], &yhi[u]);
      if (norm) {
        row = in.p + t * in.token_stride + h * in.head_stride;
        load_stream(row, lc, &xlo[u], &xhi[u]);
      }
    }
    float4 c, s;
    bool bad;
    load_turn(p.rot, t, j, lc.turned, &c, &s, &bad);
    s = make_float4(-s.x, -s.y, -s.z, -s.w);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = real && h0 + u < heads;
      float dy[8];
      widen(ylo[u], yhi[u], dy);
      turn<INTER>(dy, c, s);
      if (bad) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dy[e] = kNaN;
      }
      if (norm) {
        float x[8], sq = 0.f, dot = 0.f;
        widen(xlo[u], xhi[u], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sq += x[e] * x[e];
          dot += dy[e] * w[e] * x[e];
        }
        const float r = rsqrtf(row_sum<LR>(sq) * (1.f / D) + p.eps);
        const float m = row_sum<LR>(dot) * (1.f / D) * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (live) acc[e] += dy[e] * (x[e] * r);
          dy[e] = r * (dy[e] * w[e] - x[e] * m);
        }
      }
      if (live) store8(gx.p + t * gx.token_stride + (h0 + u) * gx.head_stride, lc, dy);
    }
    if (FOLD && ++unfolded == kFoldRows / U) {
      fold();
      unfolded = 0;
    }
  }
  if (!p.dweight[i]) return;
  if (all == 0) {                            // no rows: a workgroup of its own, and no workspace
    if (threadIdx.x < D) p.dweight[i][threadIdx.x] = 0.f;
    return;
  }
  if constexpr (FOLD) {
    fold();
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[rg * D + (e < 4 ? lc.c0 + e : lc.c1 + e - 4)] = acc[e];
  }
  __syncthreads();
  float* const parts = p.parts + static_cast<int64_t>(blockIdx.x) * D;
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll 8
    for (int g = 0; g < RG; ++g) v += sums[g * D + threadIdx.x];
    store_shared(parts + threadIdx.x, v);
  }
  if (!arrive_last(p.counters + i, groups, &flag)) return;
  // The last workgroup: D / 4 lanes by kThreads * 4 / D runs of partials, then the runs' sums.
  constexpr int L4 = D / 4, RUNS = kThreads / L4;
  const float* parts_i = p.parts + static_cast<int64_t>(i ? groups_q : 0) * D;
  const int d4 = threadIdx.x % L4, run = threadIdx.x / L4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  // Loads in flight; their latency is what the join costs (48000 rows of 256: 29.5 us, 32.2 with 8).
  constexpr int kBatch = 16;
  for (uint32_t g0 = run; g0 < groups; g0 += kBatch * RUNS) {
    float4 a[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      a[b] = *reinterpret_cast<const float4*>(
          parts_i + static_cast<int64_t>(min(g0 + b * RUNS, groups - 1)) * D + 4 * d4);
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (g0 + b * RUNS < groups) v.x += a[b].x, v.y += a[b].y, v.z += a[b].z, v.w += a[b].w;
  }
  *reinterpret_cast<float4*>(&sums[run * D + 4 * d4]) = v;
  __syncthreads();
  if (threadIdx.x < D) {
    float z = 0.f;
    for (int g = 0; g < RUNS; ++g) z += sums[g * D + threadIdx.x];
    p.dweight[i][threadIdx.x] = z;
  }
}

template <int LR, int U>
hipError_t launch_forward_u(NormRopeProblem p, hipStream_t stream) {
  constexpr int64_t RG = kThreads / LR;
  const uint32_t units_q = (p.heads[0] + U - 1) / U, units = units_q + (p.heads[1] + U - 1) / U;
  const uint32_t tokens = p.tokens;
  const uint32_t most = static_cast<uint32_t>(std::min<int64_t>(tokens, most_groups(kThreads) * RG / units));
  for (uint32_t t = 0; t < tokens; t += most) {      // all at once, unless a grid does not hold them
    p.tokens = std::min(most, tokens - t);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.tokens) * units + RG - 1) / RG));
    if (p.rot.interleaved)
      hipLaunchKernelGGL((norm_rope_kernel<LR, true, U>), grid, dim3(kThreads), 0, stream, p, units_q,
                         units);
    else
      hipLaunchKernelGGL((norm_rope_kernel<LR, false, U>), grid, dim3(kThreads), 0, stream, p, units_q,
                         units);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    for (int i = 0; i < 2; ++i) {
      if (p.heads[i] == 0) continue;
      p.x[i].p += p.tokens * p.x[i].token_stride;
      p.out[i].p += p.tokens * p.out[i].token_stride;
    }
    if (p.rot.positions) p.rot.positions += p.tokens;
  }
  return hipSuccess;
}

template <int LR>
hipError_t launch_forward(const NormRopeProblem& p, hipStream_t stream) {
  const uint64_t rows = static_cast<uint64_t>(p.tokens) * (p.heads[0] + p.heads[1]);
  return rows * (8 * LR) >= kManyForward ? launch_forward_u<LR, 4>(p, stream) : launch_forward_u<LR, 1>(p, stream);
}

template <int LR, int U>
hipError_t launch_backward_u(const NormRopeBackProblem& p, hipStream_t stream) {
  constexpr uint64_t RG = kThreads / LR;
  // Workgroups in proportion to the rows, each owner with two units at least; one for a
  // weight gradient without rows, which it writes as zero.
  uint32_t groups[2];
  const uint64_t heads = p.heads[0] + p.heads[1];
  for (int i = 0; i < 2; ++i) {
    const uint64_t units = static_cast<uint64_t>(p.tokens) * ((p.heads[i] + U - 1) / U);
    const uint64_t share = heads ? (kNormBackGroups - 1) * p.heads[i] / heads : 0;
    const uint64_t most = (units + 2 * RG - 1) / (2 * RG);
    groups[i] = static_cast<uint32_t>(most < share ? most : share);
    if (groups[i] == 0 && (units > 0 || p.dweight[i])) groups[i] = 1;
  }
  if (groups[0] + groups[1] == 0) return hipSuccess;
  bool fold = false;
  for (int i = 0; i < 2; ++i) {
    const uint64_t units = static_cast<uint64_t>(p.tokens) * ((p.heads[i] + U - 1) / U);
    if (p.dweight[i] && units * U > groups[i] * RG * kFoldRows) fold = true;
  }
  const dim3 grid(groups[0] + groups[1]);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, groups[0], groups[1]);
  };
  if (p.rot.interleaved)
    fold ? go(norm_rope_back_kernel<LR, true, U, true>) : go(norm_rope_back_kernel<LR, true, U, false>);
  else
    fold ? go(norm_rope_back_kernel<LR, false, U, true>) : go(norm_rope_back_kernel<LR, false, U, false>);
  return hipGetLastError();
}

template <int LR>
hipError_t launch_backward(const NormRopeBackProblem& p, hipStream_t stream) {
  const uint64_t rows = static_cast<uint64_t>(p.tokens) * (p.heads[0] + p.heads[1]);
  return rows * (8 * LR) >= kManyBackward ? launch_backward_u<LR, 4>(p, stream) : launch_backward_u<LR, 1>(p, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(const NormRopeProblem& p, hipStream_t stream) {
  if (p.head_dim == 64) return launch_forward<8>(p, stream);
  if (p.head_dim == 128) return launch_forward<16>(p, stream);
  return launch_forward<32>(p, stream);
}

hipError_t launch_qk_norm_rope_backward(const NormRopeBackProblem& p, hipStream_t stream) {
  if (p.head_dim == 64) return launch_backward<8>(p, stream);
  if (p.head_dim == 128) return launch_backward<16>(p, stream);
  return launch_backward<32>(p, stream);
}

}  // namespace mx
