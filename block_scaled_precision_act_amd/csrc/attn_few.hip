// Attention over the paged MXFP4 cache for few query rows (single tokens, a few drafted ones), for
// gfx950: every cached byte is read once, and that is what bounds it.
//
// For one sequence and key/value head, with rows r = (query, grouped head):
//   s = scale q k^T, p = exp(s - m), out = (p v) / sum p, m the running maximum (one pass).
//
// A wavefront takes 32 tokens at a time.  Scores are computed transposed, S^T = K Q^T on
// v_mfma_f32_16x16x32_bf16 (A: 16 tokens, B: 16 query rows), so that a lane ends with 8 tokens'
// scores of one row, and those 8 are exactly the B operand its lane has to hold for
// O^T = V^T P^T when the product's token order is taken to be (4 g + i, 16 + 4 g + i), g the lane's
// group of 16: the weights never cross lanes.  V^T's operand, 8 tokens of one head value, is made in
// the lane too: it loads the same D / 16 neighbouring codes of its group's 8 tokens, decodes them
// (value pairs) and regroups the halves by v_perm.  Nothing passes through LDS in the loop.
// Codes are decoded exactly (v_cvt_scalef32_pk_bf16_fp4 applies the E8M0 scale).
//
// The cached tokens of all sequences and heads are laid end to end in tiles of 128 and dealt in
// equal runs to a fixed number of workgroups, from the lengths on the device, so ragged batches are
// balanced and one long sequence fills the chip.  A sequence and head that a run's end cuts leaves
// partial (m, sum, O) in the workspace; the last of its workgroups to arrive joins them, in order.
#include "attn_common.h"

namespace mx {
namespace {

constexpr int kThreads = 256, kWaves = 4, kWaveTokens = 32, kTile = kWaves * kWaveTokens;

// One sequence's rows and keys.
struct Sequence {
  int32_t len, rows, q0, n;    // cached tokens; query rows (n queries x group); first query
  int32_t lo, hi;              // keys that any of its rows sees, lo down to a multiple of 32
  int32_t tiles;               // 0: no rows; at least 1 otherwise (a row that sees nothing is written)
};

__device__ __forceinline__ Sequence sequence(const AttnProblem& p, int32_t b) {
  Sequence s;
  const int64_t most = static_cast<int64_t>(p.table_width) * p.cache.page_size;
  const int32_t len = read_uniform(p.lens, b);
  s.len = len < 0 ? 0 : (len < most ? len : static_cast<int32_t>(most));
  int32_t q0 = b * p.max_q, q1 = q0 + p.max_q;
  if (p.starts) {
    q0 = read_uniform(p.starts, b);
    q1 = read_uniform(p.starts, b + 1);
    q0 = min(max(q0, 0), p.total_q);
    q1 = min(max(q1, q0), p.total_q);
  }
  s.q0 = q0;
  s.n = min(q1 - q0, p.max_q);
  s.rows = s.n * p.group;
  s.hi = s.len;
  const int32_t first = s.len - s.n;                     // the first query's position
  s.lo = p.window > 0 ? max(first + 1 - p.window, 0) & ~31 : 0;
  s.tiles = s.n == 0 ? 0 : max(1, (s.hi - s.lo + kTile - 1) / kTile);
  return s;
}

// What a wavefront loads for 32 tokens, undecoded.
template <int D>
struct Raw {
  static constexpr int KW = D / 32, VW = D <= 128 ? 1 : 2, SW = D == 64 ? 2 : 4;
  uint32_t k[2][KW];      // per 16 tokens: the lane's D / 4 codes of token lane % 16
  uint32_t ks[2];         // their scale byte(s)
  uint32_t v[8][VW];      // D / 16 codes of the lane's 8 tokens
  uint32_t vs[2][SW];     // words that hold their scale bytes
};

template <int D, int MT>
__global__ __launch_bounds__(kThreads) void attn_few_kernel(const AttnProblem p) {
  constexpr int KS = D / 32;               // k steps of a score product
  constexpr int EPL = D / 16;              // head values a lane decodes of a token's value row
  constexpr int PAD = D + 4;
  __shared__ float obuf[kWaves][16][PAD];
  __shared__ float mbuf[kWaves][16], lbuf[kWaves][16];
  __shared__ uint32_t scan[kThreads / 64 + 2];
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int heads = static_cast<int>(p.cache.heads);

  // This workgroup's run of tiles: a prefix sum of the sequences' tiles, each thread a run of
  // sequences.
  const int seg = (p.batch + kThreads - 1) / kThreads;
  uint32_t mine = 0;
  for (int i = 0; i < seg; ++i) {
    const int b = tid * seg + i;
    if (b < p.batch) mine += static_cast<uint32_t>(sequence(p, b).tiles * heads);
  }
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) scan[wave] = incl;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  const uint32_t share = max(1u, (total + gridDim.x - 1) / gridDim.x);
  const uint32_t start = blockIdx.x * share, end = min(start + share, total);
  if (start >= total) return;
  const uint32_t excl = before + incl - mine;
  if (start >= excl && start < excl + mine) {
    uint32_t at = excl;
    int b = tid * seg;
    for (;;) {
      const uint32_t n = static_cast<uint32_t>(sequence(p, b).tiles * heads);
      if (start < at + n) break;
      at += n;
      ++b;
    }
    scan[kWaves] = static_cast<uint32_t>(b);
    scan[kWaves + 1] = at;
  }
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(static_cast<int>(scan[kWaves]));
  uint32_t base = __builtin_amdgcn_readfirstlane(static_cast<int>(scan[kWaves + 1]));
  uint32_t at = start;

  while (at < end) {
    const Sequence sq = sequence(p, b);
    const uint32_t seq_tiles = static_cast<uint32_t>(sq.tiles) * heads;
    if (at - base >= seq_tiles) {            // also a sequence without rows
      base += seq_tiles;
      ++b;
      continue;
    }
    const int h = static_cast<int>((at - base) / sq.tiles);
    const uint32_t unit0 = base + static_cast<uint32_t>(h) * sq.tiles;
    const int tile0 = static_cast<int>(at - unit0);
    const int ntiles = min(sq.tiles - tile0, static_cast<int>(end - at));

    // Query rows, as B operands: lane (c, g) holds row c's values [g D/4, (g+1) D/4).
    bf16x8 qf[MT][KS];
    int32_t hi_row[MT], lo_row[MT];
    const int32_t first = sq.len - sq.n;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 16 + c;
      const int tok = r / p.group, hg = r - tok * p.group;
      const bool live = r < sq.rows;
      hi_row[mt] = live && p.causal ? first + tok + 1 : sq.len;
      lo_row[mt] = live && p.window > 0 ? first + tok + 1 - p.window : 0;
      const uint16_t* row = p.q.p + static_cast<int64_t>(sq.q0 + tok) * p.q.token_stride +
                            static_cast<int64_t>(h * p.group + hg) * p.q.head_stride + g * (D / 4);
#pragma unroll
      for (int s = 0; s < KS; ++s)
      {
        uint4 w = live ? *reinterpret_cast<const uint4*>(row + 8 * s) : make_uint4(0, 0, 0, 0);
        w.x ^= p.flip; w.y ^= p.flip; w.z ^= p.flip; w.w ^= p.flip;
        qf[mt][s] = __builtin_bit_cast(bf16x8, w);
      }
    }
    // Tokens below `full_hi` and from `full_lo` on are seen by every row.
    const int32_t full_hi = p.causal ? min(first + 1, sq.len) : sq.len;
    const int32_t full_lo = p.window > 0 ? sq.len - p.window : 0;

    v4f acc[MT][EPL];
    float m[MT], l[MT];       // row c's running maximum (base 2) and the lane's share of the sum
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = -kInf;
      l[mt] = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[mt][e] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t last16 = (sq.hi - 1) >> 4;
    const int64_t trow = static_cast<int64_t>(b) * p.table_stride;
    const uint8_t* const kh = p.cache.k + h * p.cache.code_head;
    const uint8_t* const vh = p.cache.v + h * p.cache.code_head;
    const uint8_t* const ksh = p.cache.ks + h * p.cache.scale_head;
    const uint8_t* const vsh = p.cache.vs + h * p.cache.scale_head;
    const uint32_t page16 = p.cache.page_size >> 4;

    auto load = [&](Raw<D>& w, int32_t tok0) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t t16 = static_cast<uint32_t>(min((tok0 >> 4) + s, last16));
        const uint32_t page = p.page_div ? __umulhi(t16, p.page_div) : t16;
        const uint32_t off = (t16 - page * page16) * 16u;
        uint32_t id = static_cast<uint32_t>(read_uniform(p.table, trow + page));
        id = id < p.cache.pages ? id : 0u;
        const int64_t cb = id * p.cache.code_page + off * (D / 2);
        const int64_t sb = id * p.cache.scale_page + off * (D / 32);
        const uint8_t* const kp = kh + cb;
        const uint8_t* const vp = vh + cb;
        const uint8_t* const ksp = ksh + sb;
        const uint8_t* const vsp = vsh + sb;
        const uint32_t ko = c * (D / 2) + g * (D / 8);
        if constexpr (D == 64) {
          const uint2 t = *reinterpret_cast<const uint2*>(kp + ko);
          w.k[s][0] = t.x; w.k[s][1] = t.y;
          w.ks[s] = ksp[c * 2 + (g >> 1)];
        } else {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {
            const uint4 t = *reinterpret_cast<const uint4*>(kp + ko + 16 * i);
            w.k[s][4 * i] = t.x; w.k[s][4 * i + 1] = t.y;
            w.k[s][4 * i + 2] = t.z; w.k[s][4 * i + 3] = t.w;
          }
          if constexpr (D == 128) w.ks[s] = ksp[c * 4 + g];
          else w.ks[s] = *reinterpret_cast<const uint16_t*>(ksp + c * 8 + g * 2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* a = vp + (g * 4 + i) * (D / 2) + c * (D / 32);
          if constexpr (D == 64) w.v[4 * s + i][0] = *reinterpret_cast<const uint16_t*>(a);
          if constexpr (D == 128) w.v[4 * s + i][0] = *reinterpret_cast<const uint32_t*>(a);
          if constexpr (D == 256) {
            const uint2 t = *reinterpret_cast<const uint2*>(a);
            w.v[4 * s + i][0] = t.x; w.v[4 * s + i][1] = t.y;
          }
        }
        if constexpr (D == 64) {
          const uint2 t = *reinterpret_cast<const uint2*>(vsp + g * 8);
          w.vs[s][0] = t.x; w.vs[s][1] = t.y;
        } else if constexpr (D == 128) {
          const uint4 t = *reinterpret_cast<const uint4*>(vsp + g * 16);
          w.vs[s][0] = t.x; w.vs[s][1] = t.y; w.vs[s][2] = t.z; w.vs[s][3] = t.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w.vs[s][i] = *reinterpret_cast<const uint32_t*>(vsp + (g * 4 + i) * 8 + (c >> 3) * 4);
        }
      }
    };

    auto compute = [&](const Raw<D>& w, int32_t tok0) {
      v4f s[MT][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt][t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const uint32_t byte = D == 256 ? (w.ks[t] >> (j < 4 ? 0 : 8)) & 0xFFu : w.ks[t];
          const float sc = __uint_as_float(byte << 23);
          const uint32_t d = w.k[t][j];
          const bf16x8 kf = __builtin_bit_cast(bf16x8, decode8(d, sc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            s[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[mt][j], s[mt][t], 0, 0, 0);
        }
      }
      const bool edge = tok0 + kWaveTokens > full_hi || tok0 < full_lo;
      bf16x8 pf[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = s[mt][i >> 2][i & 3] * p.scale_log2;
        if (edge) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int32_t t = tok0 + (i >> 2) * 16 + g * 4 + (i & 3);
            x[i] = t < hi_row[mt] && t >= lo_row[mt] ? x[i] : -kInf;
          }
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // The maximum that is subtracted moves only when some row's rose by more than 2^8: until
        // then weights stay below 2^8, and bf16 and fp32 hold them as well as those below one.
        if (__any(top > m[mt] + 8.f)) {
          const float now = fmaxf(m[mt], top);
          const float f = m[mt] == -kInf ? 0.f : __builtin_amdgcn_exp2f(m[mt] - now);
          m[mt] = now;
          l[mt] *= f;
#pragma unroll
          for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][e][i] *= f;
        }
        const float sub = m[mt] == -kInf ? 0.f : m[mt];
        float w8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w8[i] = __builtin_amdgcn_exp2f(x[i] - sub);
          l[mt] += w8[i];
        }
        pf[mt] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(w8[0], w8[1]), pack_bf16(w8[2], w8[3]),
                                                       pack_bf16(w8[4], w8[5]), pack_bf16(w8[6], w8[7])));
      }
      // The values' scales; what lies past the keys is given scale 1: finite, and its weight is 0.
      float vsc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int sh = D == 64 ? 8 * (c >> 3) + 16 * (i & 1) : D == 128 ? 8 * (c >> 2) : 8 * ((c >> 1) & 3);
        const uint32_t word = D == 64 ? w.vs[i >> 2][(i & 3) >> 1] : w.vs[i >> 2][i & 3];
        vsc[i] = __uint_as_float(((word >> sh) & 0xFFu) << 23);
      }
      if (tok0 + kWaveTokens > sq.hi) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (tok0 + (i >> 2) * 16 + g * 4 + (i & 3) >= sq.hi) vsc[i] = 1.f;
      }
      auto value_pair = [&](int a) {           // head values 2 a and 2 a + 1 of the lane's EPL
        uint32_t pr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pr[i] = decode2(w.v[i][a >> 2], vsc[i], a & 3);
        v4u lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __builtin_amdgcn_perm(pr[2 * i + 1], pr[2 * i], kLowHalves);
          hi[i] = __builtin_amdgcn_perm(pr[2 * i + 1], pr[2 * i], kHighHalves);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][2 * a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, lo), pf[mt], acc[mt][2 * a], 0, 0, 0);
          acc[mt][2 * a + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, hi), pf[mt], acc[mt][2 * a + 1], 0, 0, 0);
        }
      };
#pragma unroll
      for (int a = 0; a < EPL / 2; ++a) value_pair(a);
    };

    const int32_t tok_begin = sq.lo + tile0 * kTile + wave * kWaveTokens;
    const int32_t tok_end = min(sq.lo + (tile0 + ntiles) * kTile, sq.hi);
    if (tok_begin < tok_end) {
      Raw<D> ra, rb;
      load(ra, tok_begin);
      for (int32_t t = tok_begin;;) {
        int32_t nx = t + kTile;
        if (nx < tok_end) load(rb, nx);
        compute(ra, t);
        if (nx >= tok_end) break;
        t = nx;
        nx = t + kTile;
        if (nx < tok_end) load(ra, nx);
        compute(rb, t);
        if (nx >= tok_end) break;
        t = nx;
      }
    }

    // Join the four wavefronts through LDS, 16 rows at a time; thread t then holds EPL values of
    // row t / 16.
    const bool whole = ntiles == sq.tiles;
    const uint32_t wg0 = unit0 / share, wg1 = (unit0 + sq.tiles - 1) / share;
    constexpr int RB = MT * 16;
    constexpr int64_t kPart = static_cast<int64_t>(RB) * (D + 2);
    float* const part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (blockIdx.x == wg0)) * kPart;
    const int orow = tid >> 4, od = (tid & 15) * EPL;
    auto write_row = [&](int r, const float (&o)[EPL], float mm, float ll) {
      const int tok = r / p.group, hg = r - tok * p.group;
      const int64_t qrow = sq.q0 + tok;
      const int head = h * p.group + hg;
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      uint32_t w[EPL / 2];
#pragma unroll
      for (int e = 0; e < EPL / 2; ++e) w[e] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
      uint16_t* dst = p.out.p + qrow * p.out.token_stride + head * p.out.head_stride + od;
      if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else
#pragma unroll
        for (int e = 0; e < EPL / 8; ++e)
          reinterpret_cast<uint4*>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      if (p.lse && (tid & 15) == 0)
        p.lse[qrow * (static_cast<int64_t>(p.group) * heads) + head] =
            ll == 0.f ? -kInf : (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f;
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= sq.rows) break;
      float ls = l[mt];
      ls += __shfl_xor(ls, 16, 64);
      ls += __shfl_xor(ls, 32, 64);
      if (g == 0) {
        mbuf[wave][c] = m[mt];
        lbuf[wave][c] = ls;
      }
      __syncthreads();
      const float mall = fmaxf(fmaxf(mbuf[0][c], mbuf[1][c]), fmaxf(mbuf[2][c], mbuf[3][c]));
      const float f = m[mt] == -kInf ? 0.f : __builtin_amdgcn_exp2f(m[mt] - mall);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < EPL; e += 4)
          *reinterpret_cast<float4*>(&obuf[wave][c][(g * 4 + i) * EPL + e]) =
              make_float4(acc[mt][e][i] * f, acc[mt][e + 1][i] * f, acc[mt][e + 2][i] * f,
                          acc[mt][e + 3][i] * f);
      __syncthreads();
      const int r = mt * 16 + orow;
      float o[EPL], mm = -kInf, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, mbuf[w][orow]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        ll += lbuf[w][orow] * (mbuf[w][orow] == -kInf ? 0.f : __builtin_amdgcn_exp2f(mbuf[w][orow] - mm));
#pragma unroll
      for (int e = 0; e < EPL; ++e)
        o[e] = (obuf[0][orow][od + e] + obuf[1][orow][od + e]) +
               (obuf[2][orow][od + e] + obuf[3][orow][od + e]);
      if (r < sq.rows) {
        if (whole) {
          write_row(r, o, mm, ll);
        } else {
#pragma unroll
          for (int e = 0; e < EPL; e += 4)
            store_shared4(part + r * D + od + e, o[e], o[e + 1], o[e + 2], o[e + 3]);
          if ((tid & 15) == 0) {
            store_shared(part + RB * D + r, mm);
            store_shared(part + RB * D + RB + r, ll);
          }
        }
      }
      __syncthreads();
    }
    if (!whole) {
      const uint32_t count = wg1 - wg0 + 1;
      if (arrive_last(p.counters + static_cast<int64_t>(b) * heads + h, count, &flag)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int r = mt * 16 + orow;
          if (r >= sq.rows) break;
          float o[EPL], mm = -kInf, ll = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[e] = 0.f;
#pragma unroll 4
          for (uint32_t w = wg0; w <= wg1; ++w) {
            const float* src = p.parts + (2 * static_cast<int64_t>(w) + (w == wg0)) * kPart;
            const float pm = src[RB * D + r], pl = src[RB * D + RB + r];
            const float now = fmaxf(mm, pm);
            const float fo = mm == -kInf ? 0.f : __builtin_amdgcn_exp2f(mm - now);
            const float fn = pm == -kInf ? 0.f : __builtin_amdgcn_exp2f(pm - now);
            mm = now;
            ll = ll * fo + pl * fn;
#pragma unroll
            for (int e = 0; e < EPL; e += 4) {
              const float4 v = *reinterpret_cast<const float4*>(src + r * D + od + e);
              o[e] = o[e] * fo + v.x * fn;
              o[e + 1] = o[e + 1] * fo + v.y * fn;
              o[e + 2] = o[e + 2] * fo + v.z * fn;
              o[e + 3] = o[e + 3] * fo + v.w * fn;
            }
          }
          write_row(r, o, mm, ll);
        }
      }
      __syncthreads();
    }
    at += static_cast<uint32_t>(ntiles);
  }
}

template <int D, int MT>
hipError_t launch(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  hipLaunchKernelGGL((attn_few_kernel<D, MT>), dim3(static_cast<unsigned>(plan.groups)),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  if (plan.row_tiles == 1) return launch<D, 1>(p, plan, stream);
  if constexpr (D < 256) {
    if (plan.row_tiles == 2) return launch<D, 2>(p, plan, stream);
    return launch<D, 4>(p, plan, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attn_few(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  if (p.cache.head_dim == 64) return launch_d<64>(p, plan, stream);
  if (p.cache.head_dim == 128) return launch_d<128>(p, plan, stream);
  return launch_d<256>(p, plan, stream);
}

}  // namespace mx
