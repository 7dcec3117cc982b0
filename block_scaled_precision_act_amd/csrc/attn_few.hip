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
// The cached tokens of all sequences and heads are laid end to end in tiles of 128, with a few empty
// slots before each sequence and head for what it costs beside its tokens, and dealt in equal runs to
// a fixed number of workgroups, from the lengths on the device: ragged batches are balanced and one
// long sequence fills the chip.  A sequence and head that a run's end cuts leaves
// partial (m, sum, O) in the workspace; the last of its workgroups to arrive joins them, in order.
//
// Measured, 8 heads of 128: 4 sequences of up to 131073 tokens, 4 rows each: 93 us for 555 MB, 5.95
// TB/s (a large copy reaches 5.1); 41 sequences of 1 to 8192 tokens, 7 rows: 41 us, 4.5 TB/s, the ramp
// and the join being 6 of them; 1000 tokens: 8 us, nearly all latency.  Heads of 64 have half the bytes
// a token for the same instructions and nearly the same loads a step: 32 sequences, 12 heads, 4 rows, a
// window of 4096: 28 us, 3.2 TB/s (22 without the loads; without decoding or exponentials no less).
#include "attn_common.h"

namespace mx {
namespace {

constexpr int kThreads = 256, kWaves = 4, kWaveTokens = 32, kTile = kWaves * kWaveTokens;

// One sequence's rows and keys.
struct Sequence {
  int32_t len, rows, q0, n;    // cached tokens; query rows (n queries x group); first query
  int32_t low, lo, hi;         // keys that any of its rows sees: [low, hi); lo: low down to a multiple of 32
  int32_t tiles;               // 0: no rows; at least 1 otherwise (a row that sees nothing is written)
};

// From its cached tokens and its queries.
__device__ __forceinline__ Sequence sequence_of(const AttnProblem& p, int32_t len, int32_t q0,
                                                int32_t n) {
  Sequence s;
  s.len = len;
  s.q0 = q0;
  s.n = n;
  s.rows = s.n * p.group;
  s.hi = s.len;
  const int32_t first = s.len - s.n;                     // the first query's position
  s.low = p.window > 0 ? max(window_start(first, p.window), 0) : 0;
  s.lo = s.low & ~31;
  s.tiles = s.n == 0 ? 0 : max(1, (s.hi - s.lo + kTile - 1) / kTile);
  return s;
}

// The first of the D / 16 neighbouring head values that lane c of 16 decodes.
template <int D>
__device__ __forceinline__ int value_of(int c) {
  return D == 64 ? 8 * (c & 7) + 4 * (c >> 3) : c * (D / 16);
}

// What a lane holds of 32 tokens, undecoded.  Whole words: the widening of a loaded byte or half waits
// for the load at once, where these wait until the next step needs them.
template <int D>
struct RawKeys {
  uint32_t k[2][D / 32];  // per 16 tokens: D / 4 codes of token lane % 16
  uint32_t s;             // the word that holds their scale byte(s), of step g % 2
};
template <int D>
struct RawValues {
  // D / 16 codes of the lane's 8 tokens.  D == 64: the first four words, 8 codes each of every second
  // token, whose halves lanes c and c + 8 exchange (value_words).
  uint32_t v[8][D <= 128 ? 1 : 2];
  uint32_t s;         // the word that holds token 4 (lane % 4) + g's scale byte, of step lane / 4 % 2
};

struct Places {           // where the two 16-token steps of 32 tokens lie: pages and first tokens
  uint32_t id[2], off[2];
};

// Loads codes, which are read once: past the caches (4 x 131073 tokens: 94 us, 108 us without).
template <class T>
__device__ __forceinline__ T stream(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}

// exp2(m - now), and 0 where nothing was seen yet (m = -infinity).
__device__ __forceinline__ float weight_of(float m, float now) {
  return m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
}

__device__ __forceinline__ Sequence sequence(const AttnProblem& p, int32_t b) {
  const int64_t most = static_cast<int64_t>(p.table_width) * p.cache.page_size;
  const int32_t len = read_uniform(p.lens, b);
  int32_t q0 = b * p.max_q, q1 = q0 + p.max_q;
  if (p.starts) {
    q0 = min(max(read_uniform(p.starts, b), 0), p.total_q);
    q1 = min(max(read_uniform(p.starts, b + 1), q0), p.total_q);
  }
  return sequence_of(p, len < 0 ? 0 : (len < most ? len : static_cast<int32_t>(most)), q0,
                     min(q1 - q0, p.max_q));
}

// What a sequence and head costs beside its tiles (queries, joins, latencies), counted in tiles.
constexpr uint32_t kUnitSlots = 2;

// What joining one part costs, counted in tiles: a sequence and head of n tiles cut into runs of s
// takes about s + kJoinCost * n / s, least at s = sqrt(kJoinCost * n), so runs are no shorter.
constexpr float kJoinCost = 0.2f;

// The slots of a sequence: for each head, kUnitSlots and its tiles.
__device__ __forceinline__ uint32_t slots(const Sequence& s, int heads) {
  return s.tiles ? (static_cast<uint32_t>(s.tiles) + kUnitSlots) * heads : 0u;
}

// Inclusive prefix sum over the wavefront.
__device__ __forceinline__ uint32_t prefix_sum(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = max(v, static_cast<uint32_t>(__shfl_xor(v, d, 64)));
  return __builtin_amdgcn_readfirstlane(v);
}

template <int D, int MT>
__global__ __launch_bounds__(kThreads, (few_waves(D, MT))) void attn_few_kernel(const AttnProblem p) {
  constexpr int KS = D / 32;               // k steps of a score product
  constexpr int EPL = D / 16;              // head values a lane decodes of a token's value row
  constexpr int PAD = D + 4;
  __shared__ float obuf[kWaves][16][PAD];
  __shared__ float mbuf[kWaves][16], lbuf[kWaves][16];
  __shared__ uint32_t scan[2 * kWaves + 2];
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int heads = static_cast<int>(p.cache.heads);
  const int key_c = (c & 3) * 4 + (c >> 2);    // the token of 16 whose key the lane loads
  // Rotations that bring the bytes of the lane's head values to a scale's exponent field.
  const uint32_t turn_vs = 9 + 8 * (D == 64 ? 2 * (g & 1) + ((c & 7) >> 2) : D == 128 ? c >> 2 : (c >> 1) & 3);
  const uint32_t turn_ks =
      9 + 8 * (D == 64 ? 2 * (key_c & 1) + (g >> 1) : D == 128 ? g : 2 * (g & 1));

  // This workgroup's run of slots: a prefix sum over the sequences' slots finds the sequence that its
  // run begins in (b) and that sequence's first slot (base).
  uint32_t total, longest, base;           // all slots; the most of one sequence and head
  int b;
  Sequence mine_of = {};                   // up to 64 sequences: the lane's
  auto share_of = [&]() {
    const uint32_t even = (total + gridDim.x - 1) / gridDim.x;
    const float least = __builtin_sqrtf(kJoinCost * static_cast<float>(longest));
    return max(max(even, 1u), static_cast<uint32_t>(least));
  };
  if (p.batch <= 64) {                     // a lane each, every wavefront for itself
    mine_of = sequence(p, min(lane, p.batch - 1));
    const uint32_t mine = lane < p.batch ? slots(mine_of, heads) : 0u;
    const uint32_t incl = prefix_sum(mine);
    total = __builtin_amdgcn_readlane(incl, 63);
    longest = wave_max(static_cast<uint32_t>(mine_of.tiles));
    const uint32_t start = blockIdx.x * share_of();
    if (start >= total) return;
    b = __builtin_ctzll(__ballot(start < incl));
    base = __builtin_amdgcn_readlane(incl - mine, b);
  } else {                                 // a thread for each run of sequences
    const int seg = (p.batch + kThreads - 1) / kThreads;
    uint32_t mine = 0, most = 0;
    for (int i = 0; i < seg; ++i) {
      if (tid * seg + i >= p.batch) break;
      const Sequence s = sequence(p, tid * seg + i);
      mine += slots(s, heads);
      most = max(most, static_cast<uint32_t>(s.tiles));
    }
    const uint32_t incl = prefix_sum(mine);
    most = wave_max(most);
    if (lane == 63) {
      scan[wave] = incl;
      scan[kWaves + wave] = most;
    }
    __syncthreads();
    uint32_t excl = incl - mine;
    total = longest = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) excl += scan[w];
      total += scan[w];
      longest = max(longest, scan[kWaves + w]);
    }
    total = __builtin_amdgcn_readfirstlane(total);
    longest = __builtin_amdgcn_readfirstlane(longest);
    const uint32_t start = blockIdx.x * share_of();
    if (start >= total) return;
    if (start >= excl && start < excl + mine) {
      int i = tid * seg;
      for (;;) {
        const uint32_t n = slots(sequence(p, i), heads);
        if (start < excl + n) break;
        excl += n;
        ++i;
      }
      scan[2 * kWaves] = static_cast<uint32_t>(i);
      scan[2 * kWaves + 1] = excl;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(static_cast<int>(scan[2 * kWaves]));
    base = __builtin_amdgcn_readfirstlane(static_cast<int>(scan[2 * kWaves + 1]));
  }
  const uint32_t share = share_of();
  uint32_t at = blockIdx.x * share;
  const uint32_t end = min(at + share, total);

  while (at < end) {
    const Sequence sq = p.batch > 64 ? sequence(p, b)
                                     : sequence_of(p, __builtin_amdgcn_readlane(mine_of.len, b),
                                                   __builtin_amdgcn_readlane(mine_of.q0, b),
                                                   __builtin_amdgcn_readlane(mine_of.n, b));
    const uint32_t per = static_cast<uint32_t>(sq.tiles) + kUnitSlots, all = slots(sq, heads);
    if (at - base >= all) {                  // also a sequence without rows
      base += all;
      ++b;
      continue;
    }
    const int h = static_cast<int>((at - base) / per);
    const uint32_t unit0 = base + static_cast<uint32_t>(h) * per;
    const uint32_t s0 = at - unit0, s1 = min(per, end - unit0);
    const int tile0 = static_cast<int>(max(s0, kUnitSlots) - kUnitSlots);
    const int ntiles = static_cast<int>(max(s1, kUnitSlots) - kUnitSlots) - tile0;
    at = unit0 + s1;
    if (ntiles == 0) continue;

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
      lo_row[mt] = live && p.window > 0 ? window_start(first + tok, p.window) : 0;
      const uint16_t* row = p.q.p + static_cast<int64_t>(sq.q0 + tok) * p.q.token_stride +
                            static_cast<int64_t>(h * p.group + hg) * p.q.head_stride + g * (D / 4);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
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
    float slack[MT];          // what a row's maximum may rise by before it is moved
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = -kInf;
      l[mt] = 0.f;
      slack[mt] = kSlack;
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

    auto place = [&](int32_t tok0) {
      Places at;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t t16 = static_cast<uint32_t>(min((tok0 >> 4) + s, last16));
        const uint32_t page = p.page_div ? __umulhi(t16, p.page_div) : t16;
        const uint32_t id = static_cast<uint32_t>(read_uniform(p.table, trow + page));
        at.id[s] = id < p.cache.pages ? id : 0u;
        at.off[s] = (t16 - page * page16) * 16u;
      }
      return at;
    };
    // Both steps' scales come in one load, half of the lanes each, and are handed over in registers (4 x
    // 131073 tokens of 8 heads of 64: 64 us, 72 with a load for each step).  The codes are not: 16 bytes
    // a lane of all that lies together, exchanged among lanes, 67 us.
    auto scales_of = [&](const Places& at, int second) {
      const int64_t a = at.id[0] * p.cache.scale_page + at.off[0] * (D / 32);
      const int64_t b = at.id[1] * p.cache.scale_page + at.off[1] * (D / 32);
      return second ? b : a;
    };
    auto load_keys = [&](RawKeys<D>& w, const Places& at) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* const kp = kh + (at.id[s] * p.cache.code_page + at.off[s] * (D / 2)) +
                                  (key_c * (D / 2) + g * (D / 8));
        if constexpr (D == 64) {
          const v2u t = stream<v2u>(kp);
          w.k[s][0] = t[0]; w.k[s][1] = t[1];
        } else {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {
            const v4u t = stream<v4u>(kp + 16 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) w.k[s][4 * i + e] = t[e];
          }
        }
      }
      w.s = *reinterpret_cast<const uint32_t*>(
          ksh + scales_of(at, g & 1) +
          (D == 64 ? (key_c >> 1) * 4 : D == 128 ? key_c * 4 : key_c * 8 + (g >> 1) * 4));
    };
    auto load_values = [&](RawValues<D>& w, const Places& at) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* const vp = vh + (at.id[s] * p.cache.code_page + at.off[s] * (D / 2)) +
                                  (D == 64 ? ((c >> 3) * 4 + g) * 32 + (c & 7) * 4 : g * (D / 2) + c * (D / 32));
        if constexpr (D == 64) {
          w.v[2 * s][0] = stream<uint32_t>(vp);
          w.v[2 * s + 1][0] = stream<uint32_t>(vp + 8 * 32);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* a = vp + i * 4 * (D / 2);
            if constexpr (D == 128) {
              w.v[4 * s + i][0] = stream<uint32_t>(a);
            } else {
              const v2u t = stream<v2u>(a);
              w.v[4 * s + i][0] = t[0]; w.v[4 * s + i][1] = t[1];
            }
          }
        }
      }
      w.s = *reinterpret_cast<const uint32_t*>(
          vsh + scales_of(at, c & 4) +
          (D == 64 ? ((c & 3) * 2 + (g >> 1)) * 4 : ((c & 3) * 4 + g) * (D / 32) + (D == 256 ? (c >> 3) * 4 : 0)));
    };

    // 32 tokens from tok0; what was loaded for them is replaced by the loads of `next` as soon as it
    // is decoded.
    auto step = [&](RawKeys<D>& rk, RawValues<D>& rv, int32_t tok0, const Places& next, auto more) {
      v4f s[MT][2];
      const v2u ks = __builtin_amdgcn_permlane16_swap(rk.s, rk.s, false, false);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const float sc = scale_of_byte(ks[t], D == 256 && j >= 4 ? turn_ks + 8 : turn_ks);
          const bf16x8 kf = __builtin_bit_cast(bf16x8, decode8(rk.k[t][j], sc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            s[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[mt][j], j == 0 ? v4f(0.f) : s[mt][t],
                                                               0, 0, 0);
        }
      }
      if constexpr (decltype(more)::value) load_keys(rk, next);
      if (tok0 + kWaveTokens > full_hi || tok0 < full_lo) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int32_t t = tok0 + (i >> 2) * 16 + (i & 3) * 4 + g;
            if (t >= hi_row[mt] || t < lo_row[mt]) s[mt][i >> 2][i & 3] = -kInf;
          }
        __builtin_amdgcn_sched_barrier(0);        // keeps the masks a branch
      }
      bf16x8 pf[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top = s[mt][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, s[mt][i >> 2][i & 3]);
        top = max_halves(max_rows(top)) * p.scale_log2;
        float scale = p.scale_log2;
        if (__any(top > m[mt] + slack[mt])) {
          const float now = fmaxf(m[mt], top);
          const float f = weight_of(m[mt], now);
          m[mt] = now;
          l[mt] *= f;
#pragma unroll
          for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][e][i] *= f;
          slack[mt] = kSlack;
          if (large_scores(now)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              s[mt][i >> 2][i & 3] = rounded_product(s[mt][i >> 2][i & 3], scale);
            scale = 1.f;
            slack[mt] = -kInf;
          }
        }
        const float sub = m[mt] == -kInf ? 0.f : m[mt];
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[mt][i >> 2][i & 3], scale, -sub));
          l[mt] += w[i];
        }
        // In bf16, the product's type; summed unrounded (weights in attn_many.hip).
        pf[mt] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]),
                                                       pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])));
      }
      // The values' scales: the scaled conversions read a scale's exponent field alone, so the word is
      // rotated until the lane's byte lies there.  What lies past the keys, or before the oldest window,
      // is given scale 1: finite, and its weight is 0.
      const int vs = static_cast<int>(rv.s);
      const uint32_t vss[2] = {
          static_cast<uint32_t>(__builtin_amdgcn_update_dpp(vs, vs, 0x114, 0xF, 0xA, false)),   // from quads 0, 2
          static_cast<uint32_t>(__builtin_amdgcn_update_dpp(vs, vs, 0x104, 0xF, 0x5, false))};  // from quads 1, 3
      float vsc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        vsc[i] = scale_of_byte(quad_lane(vss[i >> 2], i & 3), turn_vs);
      if (tok0 + kWaveTokens > sq.hi || tok0 < sq.low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t t = tok0 + (i >> 2) * 16 + (i & 3) * 4 + g;
          if (t >= sq.hi || t < sq.low) vsc[i] = 1.f;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // D == 64: lane c loaded 8 codes of one token, lane c + 8 the same 8 of another; each keeps its
      // half of both, the first token's in the low half of the word.
      uint32_t vw[4];
      if constexpr (D == 64) {
        const uint32_t halves = c < 8 ? kLowHalves : 0x03020706u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vw[i] = __builtin_amdgcn_perm(
              static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(rv.v[i][0]), 0x128, 0xF, 0xF, false)),
              rv.v[i][0], halves);
      }
#pragma unroll
      for (int a = 0; a < EPL / 2; ++a) {        // head values 2 a and 2 a + 1 of the lane's EPL
        uint32_t pr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          pr[i] = D == 64 ? decode2(vw[i >> 1], vsc[i], 2 * (i & 1) + a) : decode2(rv.v[i][a >> 2], vsc[i], a & 3);
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
      }
      if constexpr (decltype(more)::value) load_values(rv, next);
    };

    const int32_t tok_begin = sq.lo + tile0 * kTile + wave * kWaveTokens;
    const int32_t tok_end = min(sq.lo + (tile0 + ntiles) * kTile, sq.hi);
    if (tok_begin < tok_end) {
      RawKeys<D> rk;
      RawValues<D> rv;
      Places at = place(tok_begin);
      load_keys(rk, at);
      load_values(rv, at);
      at = place(tok_begin + kTile);             // past the end: the last step's
      // The last step is apart: loads that depended on a condition would make every wait for keys one
      // for the values behind them too.
      int32_t t = tok_begin;
      for (; t + kTile < tok_end; t += kTile) {
        const Places next = place(t + 2 * kTile);
        step(rk, rv, t, at, IntC<1>{});
        at = next;
      }
      step(rk, rv, t, at, IntC<0>{});
    }

    // Join the four wavefronts through LDS, 16 rows at a time; thread t then holds EPL values of
    // row t / 16.
    const bool whole = ntiles == sq.tiles;
    const uint32_t wg0 = (unit0 + kUnitSlots) / share, wg1 = (unit0 + per - 1) / share;
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
      const float f = weight_of(m[mt], mall);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < EPL; e += 4)
          *reinterpret_cast<float4*>(&obuf[wave][c][value_of<D>(g * 4 + i) + e]) =
              make_float4(acc[mt][e][i] * f, acc[mt][e + 1][i] * f, acc[mt][e + 2][i] * f,
                          acc[mt][e + 3][i] * f);
      __syncthreads();
      const int r = mt * 16 + orow;
      float o[EPL], mm = -kInf, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, mbuf[w][orow]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        ll += lbuf[w][orow] * weight_of(mbuf[w][orow], mm);
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
    // The last workgroup to arrive joins the parts: its 16 lots of 16 threads take the tile's live
    // rows, and the parts by turns where rows leave lots over; the lots of a row are then joined.
    if (!whole && arrive_last(p.counters + (static_cast<int64_t>(b) * heads + h) * p.counter_stride, wg1 - wg0 + 1, &flag)) {
      const int lot = tid >> 4;
      for (int mt = 0; mt < MT && mt * 16 < sq.rows; ++mt) {
        const int live = min(16, sq.rows - mt * 16), turns = 16 / live;
        const int turn = lot / live, r = mt * 16 + lot - turn * live;
        float o[EPL], mm = -kInf, ll = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] = 0.f;
        if (turn < turns) {
          constexpr int kBatch = D == 256 ? 4 : 8;
          for (uint32_t w0 = wg0 + turn; w0 <= wg1; w0 += kBatch * turns) {
            float pm[kBatch], pl[kBatch];
            float4 v[kBatch][EPL / 4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {     // past the last part: that part, with no weight
              const uint32_t w = min(w0 + i * turns, wg1);
              const float* src = p.parts + (2 * static_cast<int64_t>(w) + (w == wg0)) * kPart;
              pm[i] = src[RB * D + r];
              pl[i] = src[RB * D + RB + r];
#pragma unroll
              for (int e = 0; e < EPL / 4; ++e) v[i][e] = *reinterpret_cast<const float4*>(src + r * D + od + 4 * e);
            }
            float now = mm;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (w0 + i * turns > wg1) pm[i] = -kInf;
              now = fmaxf(now, pm[i]);
            }
            const float fo = weight_of(mm, now);
            mm = now;
            ll *= fo;
#pragma unroll
            for (int e = 0; e < EPL; ++e) o[e] *= fo;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (w0 + i * turns > wg1) break;
              const float f = weight_of(pm[i], now);
              ll += pl[i] * f;
#pragma unroll
              for (int e = 0; e < EPL / 4; ++e) {
                o[4 * e] += v[i][e].x * f;
                o[4 * e + 1] += v[i][e].y * f;
                o[4 * e + 2] += v[i][e].z * f;
                o[4 * e + 3] += v[i][e].w * f;
              }
            }
          }
        }
        if (turns > 1) {
#pragma unroll
          for (int e = 0; e < EPL; ++e) obuf[0][lot][od + e] = o[e];
          if ((tid & 15) == 0) {
            mbuf[0][lot] = mm;
            lbuf[0][lot] = ll;
          }
          __syncthreads();
          if (turn == 0) {
            for (int i = 1; i < turns; ++i) {
              const int other = lot + i * live;
              const float pm = mbuf[0][other], now = fmaxf(mm, pm);
              const float fo = weight_of(mm, now), fn = weight_of(pm, now);
              mm = now;
              ll = ll * fo + lbuf[0][other] * fn;
#pragma unroll
              for (int e = 0; e < EPL; ++e) o[e] = o[e] * fo + obuf[0][other][od + e] * fn;
            }
          }
        }
        if (turn == 0) write_row(r, o, mm, ll);
        __syncthreads();
      }
    }
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
  if (plan.row_tiles == 2) return launch<D, 2>(p, plan, stream);
  if constexpr (D < 256) return launch<D, 4>(p, plan, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attn_few(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  if (p.cache.head_dim == 64) return launch_d<64>(p, plan, stream);
  if (p.cache.head_dim == 128) return launch_d<128>(p, plan, stream);
  return launch_d<256>(p, plan, stream);
}

}  // namespace mx
