// Attention over the paged MXFP4 cache for many query rows (prompts, chunks of them), for gfx950:
// bound by the bf16 matrix instructions and the softmax between them.
//
// A workgroup holds a block of query rows of one sequence and key/value head, rows r = (query,
// grouped head), 32 to a wavefront, and walks over its keys 64 tokens at a time (one pass, running
// maximum and sum).  The 64 tokens' codes are decoded to bf16 once for the workgroup, into LDS, in
// the order the matrix operands are read in: every LDS access of the loop is 16 bytes a lane, 1 KB
// in a row.  Scores are computed transposed, S^T = K Q^T on v_mfma_f32_32x32x16_bf16, so a lane
// holds one row's scores of 16 of 32 tokens, and those are its B operand of O^T = V^T P^T with the
// product's token order (4 h + i, 8 + 4 h + i), h the lane's half: the weights never leave the lane.
// V^T's operand is made by the thread that decodes 8 tokens' same codes.
#include "attn_common.h"

namespace mx {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 32 * kWaves, kTok = 64;
constexpr float kLn2 = 0.6931471805599453f;
typedef float v16f __attribute__((ext_vector_type(16)));

template <int D>
struct Tile {                 // one thread's undecoded share of 64 tokens
  static constexpr int KW = D / 32, EPI = D / 32, SW = D == 64 ? 2 : 4;
  uint32_t k[KW];             // a quarter of token tid % 64's key codes
  uint32_t ks;                // their scale byte(s)
  uint32_t v[8];              // D / 32 codes of 8 tokens
  uint32_t vs[2][SW];
};

template <int D>
__global__ __launch_bounds__(kThreads) void attn_many_kernel(const AttnProblem p, int row_blocks,
                                                             int splits) {
  constexpr int KS = D / 16, DT = D / 32, EPI = D / 32;
  __shared__ uint4 kl[2 * KS * 64];         // [32-token half][k step][lane]
  __shared__ uint4 vl[4 * DT * 64];         // [16-token step][head value % DT][lane]
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, hh = lane >> 5;
  const int heads = static_cast<int>(p.cache.heads);
  // Heads fastest: with 8 of them a head's keys stay on one XCD's L2.  Late rows (the longest under
  // a causal mask) first.
  uint32_t idx = blockIdx.x;
  const int h = idx % heads;
  idx /= heads;
  const int b = idx % p.batch;
  idx /= p.batch;
  const int part_id = idx % splits;
  const int blk = row_blocks - 1 - static_cast<int>(idx / splits);

  const int64_t most = static_cast<int64_t>(p.table_width) * p.cache.page_size;
  const int32_t raw_len = p.lens[b];
  const int32_t len = raw_len < 0 ? 0 : (raw_len < most ? raw_len : static_cast<int32_t>(most));
  int32_t q0 = b * p.max_q, q1 = q0 + p.max_q;
  if (p.starts) {
    q0 = min(max(p.starts[b], 0), p.total_q);
    q1 = min(max(p.starts[b + 1], q0), p.total_q);
  }
  const int32_t n = min(q1 - q0, p.max_q);
  const int32_t rows = n * p.group, r0 = blk * kRows;
  if (r0 >= rows) return;
  const int32_t first = len - n;
  const int32_t tok_lo = r0 / p.group, tok_hi = (min(r0 + kRows, rows) - 1) / p.group;
  const int32_t hi = p.causal ? min(max(first + tok_hi + 1, 0), len) : len;
  const int32_t lo = p.window > 0 ? max(first + tok_lo + 1 - p.window, 0) & ~(kTok - 1) : 0;
  const int32_t all = max(0, (hi - lo + kTok - 1) / kTok);
  const int32_t parts = max(1, min(splits, all / 4));
  if (part_id >= parts) return;
  const int32_t t_begin = lo + static_cast<int32_t>(static_cast<int64_t>(all) * part_id / parts) * kTok;
  const int32_t t_end = min(hi, lo + static_cast<int32_t>(static_cast<int64_t>(all) * (part_id + 1) / parts) * kTok);

  // The lane's query row.
  const int32_t r = r0 + wave * 32 + c;
  const bool live = r < rows;
  const int32_t tok = live ? r / p.group : 0, hg = live ? r - tok * p.group : 0;
  const int32_t row_hi = live && p.causal ? first + tok + 1 : len;
  const int32_t row_lo = live && p.window > 0 ? first + tok + 1 - p.window : 0;
  bf16x8 qf[KS];
  {
    const uint16_t* row = p.q.p + static_cast<int64_t>(q0 + tok) * p.q.token_stride +
                          static_cast<int64_t>(h * p.group + hg) * p.q.head_stride + 8 * hh;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      qf[s] = __builtin_bit_cast(bf16x8, live ? *reinterpret_cast<const uint4*>(row + 16 * s)
                                              : make_uint4(0, 0, 0, 0));
  }
  const int32_t full_hi = p.causal ? min(first + tok_lo + 1, len) : len;
  const int32_t full_lo = p.window > 0 ? first + tok_hi + 1 - p.window : 0;

  // The thread's share of decoding: key token kt, codes [kq D / 4, (kq + 1) D / 4); the values of 8
  // tokens of 16-token step vstep, head values [EPI vc, EPI (vc + 1)).
  const int kt = tid & 63, kq = tid >> 6;
  const int vc = tid & 31, vset = tid >> 5, vstep = vset >> 1, vh = vset & 1;
  const int32_t last16 = (hi - 1) >> 4;
  const int32_t* const trow = p.table + static_cast<int64_t>(b) * p.table_stride;
  const uint32_t page16 = p.cache.page_size >> 4;

  auto place = [&](int32_t t0, int sub, uint32_t* off) {     // a 16-token step's page and offset
    const uint32_t t16 = static_cast<uint32_t>(min((t0 >> 4) + sub, last16));
    const uint32_t page = p.page_div ? __umulhi(t16, p.page_div) : t16;
    *off = (t16 - page * page16) * 16u;
    const uint32_t id = static_cast<uint32_t>(trow[page]);
    return id < p.cache.pages ? id : 0u;
  };
  auto load = [&](Tile<D>& w, int32_t t0) {
    uint32_t off;
    uint32_t id = place(t0, kt >> 4, &off);
    off += kt & 15;
    const uint8_t* kp = p.cache.k + id * p.cache.code_page + h * p.cache.code_head + off * (D / 2) +
                        kq * (D / 8);
    const uint8_t* ksp = p.cache.ks + id * p.cache.scale_page + h * p.cache.scale_head +
                         off * (D / 32);
    if constexpr (D == 64) {
      const uint2 t = *reinterpret_cast<const uint2*>(kp);
      w.k[0] = t.x; w.k[1] = t.y;
      w.ks = ksp[kq >> 1];
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 t = *reinterpret_cast<const uint4*>(kp + 16 * i);
        w.k[4 * i] = t.x; w.k[4 * i + 1] = t.y; w.k[4 * i + 2] = t.z; w.k[4 * i + 3] = t.w;
      }
      if constexpr (D == 128) w.ks = ksp[kq];
      else w.ks = *reinterpret_cast<const uint16_t*>(ksp + 2 * kq);
    }
    id = place(t0, vstep, &off);
    const uint8_t* vp = p.cache.v + id * p.cache.code_page + h * p.cache.code_head + vc * (EPI / 2);
    const uint8_t* vsp = p.cache.vs + id * p.cache.scale_page + h * p.cache.scale_head;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t t = off + (i >> 2) * 8 + vh * 4 + (i & 3);
      const uint8_t* a = vp + t * (D / 2);
      if constexpr (D == 64) w.v[i] = *a;
      if constexpr (D == 128) w.v[i] = *reinterpret_cast<const uint16_t*>(a);
      if constexpr (D == 256) w.v[i] = *reinterpret_cast<const uint32_t*>(a);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t = off + i * 8 + vh * 4;
      if constexpr (D == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(vsp + t * 2);
        w.vs[i][0] = x.x; w.vs[i][1] = x.y;
      } else if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(vsp + t * 4);
        w.vs[i][0] = x.x; w.vs[i][1] = x.y; w.vs[i][2] = x.z; w.vs[i][3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w.vs[i][e] = *reinterpret_cast<const uint32_t*>(vsp + (t + e) * 8 + (vc >> 4) * 4);
      }
    }
  };
  auto decode = [&](const Tile<D>& w, int32_t t0) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t byte = D == 256 ? (w.ks >> (i < 4 ? 0 : 8)) & 0xFFu : w.ks;
      const float sc = __uint_as_float(byte << 23);
      const int word = kq * (D / 32) + i;               // 8 codes: k step word / 2, half word % 2
      const uint4 o = make_uint4(
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.k[i], sc, 0)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.k[i], sc, 1)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.k[i], sc, 2)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.k[i], sc, 3)));
      kl[((kt >> 5) * KS + (word >> 1)) * 64 + (word & 1) * 32 + (kt & 31)] = o;
    }
    float sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int sh = D == 64 ? 8 * (vc >> 4) + 16 * (i & 1) : D == 128 ? 8 * (vc >> 3) : 8 * ((vc >> 2) & 3);
      const uint32_t word = D == 64 ? w.vs[i >> 2][(i & 3) >> 1] : w.vs[i >> 2][i & 3];
      sc[i] = __uint_as_float(((word >> sh) & 0xFFu) << 23);
      // What lies past the keys is given scale 1: finite, and its weight is 0.
      if (t0 + vstep * 16 + (i >> 2) * 8 + vh * 4 + (i & 3) >= hi) sc[i] = 1.f;
    }
#pragma unroll
    for (int a = 0; a < EPI / 2; ++a) {
      uint32_t pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16x2 x = a == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], sc[i], 0)
                         : a == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], sc[i], 1)
                         : a == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], sc[i], 2)
                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], sc[i], 3);
        pr[i] = __builtin_bit_cast(uint32_t, x);
      }
      uint4 x, y;
      x.x = __builtin_amdgcn_perm(pr[1], pr[0], 0x05040100u);
      x.y = __builtin_amdgcn_perm(pr[3], pr[2], 0x05040100u);
      x.z = __builtin_amdgcn_perm(pr[5], pr[4], 0x05040100u);
      x.w = __builtin_amdgcn_perm(pr[7], pr[6], 0x05040100u);
      y.x = __builtin_amdgcn_perm(pr[1], pr[0], 0x07060302u);
      y.y = __builtin_amdgcn_perm(pr[3], pr[2], 0x07060302u);
      y.z = __builtin_amdgcn_perm(pr[5], pr[4], 0x07060302u);
      y.w = __builtin_amdgcn_perm(pr[7], pr[6], 0x07060302u);
      vl[(vstep * DT + 2 * a) * 64 + vh * 32 + vc] = x;
      vl[(vstep * DT + 2 * a + 1) * 64 + vh * 32 + vc] = y;
    }
  };

  v16f acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -kInf, l = 0.f;

  Tile<D> w;
  if (t_begin < t_end) load(w, t_begin);
  for (int32_t t0 = t_begin; t0 < t_end; t0 += kTok) {
    __syncthreads();                        // the previous tile's operands are read
    decode(w, t0);
    __syncthreads();
    if (t0 + kTok < t_end) load(w, t0 + kTok);
    const bool edge = t0 + kTok > full_hi || t0 < full_lo;
    v16f s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; ++j)
        s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, kl[(t * KS + j) * 64 + lane]), qf[j], s[t], 0, 0, 0);
    }
    float top = -kInf;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = s[t][i] * p.scale_log2;
        if (edge) {
          const int32_t key = t0 + t * 32 + (i & 3) + 8 * (i >> 2) + 4 * hh;
          x = key < row_hi && key >= row_lo ? x : -kInf;
        }
        s[t][i] = x;
        top = fmaxf(top, x);
      }
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    // The maximum that is subtracted moves only when some row's rose by more than 2^8 (weights below
    // that are held as exactly as those below one).
    if (__any(top > m + 8.f)) {
      const float now = fmaxf(m, top);
      const float f = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= f;
    }
    const float sub = m == -kInf ? 0.f : m;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(s[t][i] - sub);
        l += s[t][i];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 pf = __builtin_bit_cast(
            bf16x8, make_uint4(pack_bf16(s[t][8 * u], s[t][8 * u + 1]),
                               pack_bf16(s[t][8 * u + 2], s[t][8 * u + 3]),
                               pack_bf16(s[t][8 * u + 4], s[t][8 * u + 5]),
                               pack_bf16(s[t][8 * u + 6], s[t][8 * u + 7])));
#pragma unroll
        for (int d = 0; d < DT; ++d)
          acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, vl[((t * 2 + u) * DT + d) * 64 + lane]), pf, acc[d], 0, 0, 0);
      }
    }
  }
  l += __shfl_xor(l, 32, 64);

  // Lane (c, hh) holds row r's head values DT (i % 4 + 8 (i / 4) + 4 hh) + d.
  auto write_row = [&](float mm, float ll) {
    const int head = h * p.group + hg;
    const int64_t qrow = q0 + tok;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    uint16_t* dst = p.out.p + qrow * p.out.token_stride + head * p.out.head_stride;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t x[DT / 2];
#pragma unroll
      for (int d = 0; d < DT / 2; ++d) x[d] = pack_bf16(acc[2 * d][i] * inv, acc[2 * d + 1][i] * inv);
      uint16_t* at = dst + DT * ((i & 3) + 8 * (i >> 2) + 4 * hh);
      if constexpr (DT == 2) *reinterpret_cast<uint32_t*>(at) = x[0];
      if constexpr (DT == 4) *reinterpret_cast<uint2*>(at) = make_uint2(x[0], x[1]);
      if constexpr (DT == 8) *reinterpret_cast<uint4*>(at) = make_uint4(x[0], x[1], x[2], x[3]);
    }
    if (p.lse && hh == 0)
      p.lse[qrow * (static_cast<int64_t>(p.group) * heads) + head] =
          ll == 0.f ? -kInf : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
  };
  if (parts == 1) {
    if (live) write_row(m, l);
    return;
  }
  // Partial (m, l, O) of each part: values as the lanes hold them, 4 to a lane, lanes in a row.
  const int64_t unit = (static_cast<int64_t>(blk) * p.batch + b) * heads + h;
  constexpr int64_t kPart = static_cast<int64_t>(kRows) * (D + 2);
  float* const mine = p.parts + (unit * splits + part_id) * kPart;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store_shared4(mine + ((d * 4 + i / 4) * kThreads + tid) * 4, acc[d][i], acc[d][i + 1],
                    acc[d][i + 2], acc[d][i + 3]);
  if (hh == 0) {
    store_shared(mine + kRows * D + wave * 32 + c, m);
    store_shared(mine + kRows * D + kRows + wave * 32 + c, l);
  }
  if (!arrive_last(p.counters + unit, static_cast<uint32_t>(parts), &flag)) return;
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  for (int q = 0; q < parts; ++q) {
    const float* src = p.parts + (unit * splits + q) * kPart;
    const float pm = src[kRows * D + wave * 32 + c], pl = src[kRows * D + kRows + wave * 32 + c];
    const float now = fmaxf(m, pm);
    const float fo = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
    const float fn = pm == -kInf ? 0.f : __builtin_amdgcn_exp2f(pm - now);
    m = now;
    l = l * fo + pl * fn;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(src + ((d * 4 + i / 4) * kThreads + tid) * 4);
        acc[d][i] = acc[d][i] * fo + x.x * fn;
        acc[d][i + 1] = acc[d][i + 1] * fo + x.y * fn;
        acc[d][i + 2] = acc[d][i + 2] * fo + x.z * fn;
        acc[d][i + 3] = acc[d][i + 3] * fo + x.w * fn;
      }
  }
  if (live) write_row(m, l);
}

template <int D>
hipError_t launch(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  const int64_t grid = static_cast<int64_t>(plan.row_blocks) * plan.splits * p.batch * p.cache.heads;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((attn_many_kernel<D>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                     stream, p, plan.row_blocks, plan.splits);
  return hipGetLastError();
}

}  // namespace

AttnPlan plan_attn(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int head_dim) {
  AttnPlan a = {};
  const int64_t rows = max_q * (q_heads / kv_heads), units = batch * kv_heads;
  const int64_t most = head_dim == 256 ? 16 : 64;
  a.few = rows <= most;
  if (a.few) {
    a.row_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    a.groups = 512;
    a.counter_bytes = (units * 4 + 255) / 256 * 256;
    a.bytes = a.counter_bytes +
              2 * static_cast<int64_t>(a.groups) * 16 * a.row_tiles * (head_dim + 2) * 4;
    return a;
  }
  const int64_t blocks = (rows + kRows - 1) / kRows;
  a.row_blocks = static_cast<int>(blocks);
  const int64_t fit = 512 / (blocks * units);
  a.splits = static_cast<int>(fit < 1 ? 1 : fit > 64 ? 64 : fit);
  if (a.splits > 1) {
    a.counter_bytes = (blocks * units * 4 + 255) / 256 * 256;
    a.bytes = a.counter_bytes +
              blocks * units * a.splits * static_cast<int64_t>(kRows) * (head_dim + 2) * 4;
  }
  return a;
}

hipError_t launch_attn_many(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  if (p.cache.head_dim == 64) return launch<64>(p, plan, stream);
  if (p.cache.head_dim == 128) return launch<128>(p, plan, stream);
  return launch<256>(p, plan, stream);
}

}  // namespace mx
