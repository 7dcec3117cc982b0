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

constexpr int kTok = 64;
constexpr float kLn2 = 0.6931471805599453f;
typedef float v16f __attribute__((ext_vector_type(16)));

// A decoding thread's undecoded share of 64 tokens: a quarter of a token's key codes and the word that
// holds their scale byte(s); or the words of 8 tokens that hold its D / 32 value codes, and those that
// hold their scale bytes.  Whole words: the widening of a loaded byte or half waits for the load at
// once, where these wait until the next tile needs them.
template <int D>
struct RawKeys {
  uint32_t k[D / 32], s;
};
template <int D>
struct RawValues {
  uint32_t v[8], s[2][D == 64 ? 2 : 4];
};

struct Place {                // where a 16-token step lies: its page and the first token's offset
  uint32_t id, off;
};

// NW wavefronts of 32 query rows each.  Of 8, the first four decode keys and the others values (one
// of each to a SIMD); of 4, all decode both.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_many_kernel(const AttnProblem p,
                                                                              int row_blocks,
                                                                              int splits) {
  constexpr int KS = D / 16, DT = D / 32, EPI = D / 32, kRows = 32 * NW, kThreads = 64 * NW;
  constexpr bool kPipe = D < 256;
  __shared__ uint4 kl[2][2 * KS * 64];      // [32-token half][k step][lane]
  __shared__ uint4 vl[2][4 * DT * 64];      // [16-token step][head value % DT][lane]
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
  const int32_t tile0 = static_cast<int32_t>(static_cast<int64_t>(all) * part_id / parts);
  const int32_t tiles = static_cast<int32_t>(static_cast<int64_t>(all) * (part_id + 1) / parts) - tile0;
  const int32_t t_begin = lo + tile0 * kTok;

  // The lane's query row, as B operands.
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
    for (int s = 0; s < KS; ++s) {
      uint4 w = live ? *reinterpret_cast<const uint4*>(row + 16 * s) : make_uint4(0, 0, 0, 0);
      w.x ^= p.flip; w.y ^= p.flip; w.z ^= p.flip; w.w ^= p.flip;
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
  }
  const int32_t full_hi = p.causal ? min(first + tok_lo + 1, len) : len;
  const int32_t full_lo = p.window > 0 ? first + tok_hi + 1 - p.window : 0;

  // A wavefront decodes the keys or values of one 16-token step (its page is the same for all lanes):
  // of key lane % 16, codes [kq D / 4, (kq + 1) D / 4); of 8 tokens (half vh), head values
  // [EPI vc, EPI (vc + 1)).
  const bool keys = NW == 4 || wave < 4, values = NW == 4 || wave >= 4;
  const int sub = wave & 3;
  const int k16 = lane & 15, kq = lane >> 4, vc = lane & 31, vh = lane >> 5;
  const uint32_t turn_k = 9 + 8 * (D == 64 ? 2 * (k16 & 1) + (kq >> 1) : D == 128 ? kq : 2 * (kq & 1));
  const int32_t last16 = (hi - 1) >> 4;
  const int64_t trow = static_cast<int64_t>(b) * p.table_stride;
  const uint32_t page16 = p.cache.page_size >> 4;
  const uint8_t* const kbase = p.cache.k + h * p.cache.code_head;
  const uint8_t* const vbase = p.cache.v + h * p.cache.code_head;
  const uint8_t* const ksbase = p.cache.ks + h * p.cache.scale_head;
  const uint8_t* const vsbase = p.cache.vs + h * p.cache.scale_head;

  // Steps past the last one stand for it: what is loaded there is masked or never used.
  auto place = [&](int32_t t0) {
    const uint32_t t16 = static_cast<uint32_t>(min((t0 >> 4) + sub, last16));
    const uint32_t page = p.page_div ? __umulhi(t16, p.page_div) : t16;
    const uint32_t id = static_cast<uint32_t>(read_uniform(p.table, trow + page));
    return Place{id < p.cache.pages ? id : 0u, (t16 - page * page16) * 16u};
  };
  auto load_keys = [&](RawKeys<D>& w, Place at) {
    const uint8_t* kp = kbase + (at.id * p.cache.code_page + at.off * (D / 2)) +
                        (k16 * (D / 2) + kq * (D / 8));
    const uint8_t* sp = ksbase + (at.id * p.cache.scale_page + at.off * (D / 32)) +
                        (D == 64 ? (k16 >> 1) * 4 : D == 128 ? k16 * 4 : k16 * 8 + (kq >> 1) * 4);
    if constexpr (D == 64) {
      const uint2 t = *reinterpret_cast<const uint2*>(kp);
      w.k[0] = t.x; w.k[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 t = *reinterpret_cast<const uint4*>(kp + 16 * i);
        w.k[4 * i] = t.x; w.k[4 * i + 1] = t.y; w.k[4 * i + 2] = t.z; w.k[4 * i + 3] = t.w;
      }
    }
    w.s = *reinterpret_cast<const uint32_t*>(sp);
  };
  auto load_values = [&](RawValues<D>& w, Place at) {
    const uint8_t* vp = vbase + (at.id * p.cache.code_page + at.off * (D / 2)) +
                        (vh * 4 * (D / 2) + (vc * (EPI / 2) & ~3));
    const uint8_t* sp = vsbase + (at.id * p.cache.scale_page + at.off * (D / 32)) + vh * 4 * (D / 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w.v[i] = *reinterpret_cast<const uint32_t*>(vp + ((i >> 2) * 8 + (i & 3)) * (D / 2));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* a = sp + i * 8 * (D / 32);
      if constexpr (D == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(a);
        w.s[i][0] = x.x; w.s[i][1] = x.y;
      } else if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(a);
        w.s[i][0] = x.x; w.s[i][1] = x.y; w.s[i][2] = x.z; w.s[i][3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w.s[i][e] = *reinterpret_cast<const uint32_t*>(a + e * 8 + (vc >> 4) * 4);
      }
    }
  };
  auto decode_keys = [&](const RawKeys<D>& w, uint4* dst) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float sc = scale_of_byte(w.s, D == 256 && i >= 4 ? turn_k + 8 : turn_k);
      const int word = kq * (D / 32) + i;               // 8 codes: k step word / 2, half word % 2
      dst[((sub >> 1) * KS + (word >> 1)) * 64 + (word & 1) * 32 + (sub & 1) * 16 + k16] =
          decode8(w.k[i], sc);
    }
  };
  auto decode_values = [&](const RawValues<D>& w, int32_t t0, uint4* dst) {
    const uint32_t drop = D == 64 ? 8 * (vc & 3) : D == 128 ? 16 * (vc & 1) : 0;   // the lane's codes lowest
    const uint32_t turn = 9 + 8 * (D == 64 ? vc >> 4 : D == 128 ? vc >> 3 : (vc >> 2) & 3);
    float sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = scale_of_byte(D == 64 ? w.s[i >> 2][(i & 3) >> 1] : w.s[i >> 2][i & 3],
                            D == 64 && (i & 1) ? turn + 16 : turn);
    // What lies past the keys is given scale 1: finite, and its weight is 0.
    if (t0 + kTok > hi) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + sub * 16 + (i >> 2) * 8 + vh * 4 + (i & 3) >= hi) sc[i] = 1.f;
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int a = 0; a < EPI / 2; ++a) {
      uint32_t pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = decode2(D == 256 ? w.v[i] : w.v[i] >> drop, sc[i], a);
      uint4 x, y;
      x.x = __builtin_amdgcn_perm(pr[1], pr[0], kLowHalves);
      x.y = __builtin_amdgcn_perm(pr[3], pr[2], kLowHalves);
      x.z = __builtin_amdgcn_perm(pr[5], pr[4], kLowHalves);
      x.w = __builtin_amdgcn_perm(pr[7], pr[6], kLowHalves);
      y.x = __builtin_amdgcn_perm(pr[1], pr[0], kHighHalves);
      y.y = __builtin_amdgcn_perm(pr[3], pr[2], kHighHalves);
      y.z = __builtin_amdgcn_perm(pr[5], pr[4], kHighHalves);
      y.w = __builtin_amdgcn_perm(pr[7], pr[6], kHighHalves);
      dst[(sub * DT + 2 * a) * 64 + vh * 32 + vc] = x;
      dst[(sub * DT + 2 * a + 1) * 64 + vh * 32 + vc] = y;
    }
  };

  v16f acc[DT];
  float m = -kInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = v16f(0.f);

  // K steps [j0, j1) of the scores of 32-token half t.
  auto scores = [&](v16f (&s)[2], const uint4* kd, int t, int j0, int j1) {
#pragma unroll
    for (int j = j0; j < j1; ++j)
      s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8, kd[(t * KS + j) * 64 + lane]), qf[j], j == 0 ? v16f(0.f) : s[t],
          0, 0, 0);
  };

  RawKeys<D> rk;
  RawValues<D> rv;
  Place next_k, next_v;

  // Tile i: its scores `s` are there (kPipe) or made first; while its weights and products are made,
  // the next tile's scores are (kPipe: into `sn`), the keys and values that come next are decoded,
  // and the ones after them loaded.  One barrier a tile: what is decoded goes where a tile's keys
  // (values) were that every wavefront has read before the last barrier.
  auto step = [&](v16f (&s)[2], v16f (&sn)[2], auto odd, auto final, int32_t i) {
    constexpr int B = decltype(odd)::value;
    constexpr bool LAST = decltype(final)::value;
    const int32_t t0 = t_begin + i * kTok;
    if constexpr (!kPipe) {
#pragma unroll
      for (int t = 0; t < 2; ++t) scores(s, kl[B], t, 0, KS);
    }
    if (t0 + kTok > full_hi || t0 < full_lo) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int32_t key = t0 + (e >> 4) * 32 + (e & 3) + 8 * ((e & 15) >> 2) + 4 * hh;
        if (key >= row_hi || key < row_lo) s[e >> 4][e & 15] = -kInf;
        if (e % 8 == 7) __builtin_amdgcn_sched_barrier(0);
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
    top = max_halves(top) * p.scale_log2;
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
        for (int e = 0; e < 16; ++e) acc[d][e] *= f;
    }
    const float sub_m = m == -kInf ? 0.f : m;
#pragma unroll
    for (int q = 0; q < 4; ++q) {            // 16 tokens each
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[q >> 1][8 * (q & 1) + e], p.scale_log2, -sub_m));
        l += w[e];
      }
      const bf16x8 pf = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]),
                                                              pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])));
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, vl[B][(q * DT + d) * 64 + lane]), pf, acc[d], 0, 0, 0);
      if constexpr (!LAST && kPipe)
        scores(sn, kl[B ^ 1], q >> 1, (q & 1) * (KS / 2), ((q & 1) + 1) * (KS / 2));
    }
    if constexpr (!LAST) {
      if (keys) {
        decode_keys(rk, kl[kPipe ? B : B ^ 1]);
        load_keys(rk, next_k);
        next_k = place(t0 + (kPipe ? 4 : 3) * kTok);
      }
      if (values) {
        decode_values(rv, t0 + kTok, vl[B ^ 1]);
        load_values(rv, next_v);
        next_v = place(t0 + 3 * kTok);
      }
      lds_barrier();
    }
  };

  if (tiles > 0) {
    v16f sa[2], sb[2];
    if (keys) {
      load_keys(rk, place(t_begin));
      decode_keys(rk, kl[0]);
      load_keys(rk, place(t_begin + kTok));
      next_k = place(t_begin + 2 * kTok);
      if constexpr (kPipe) {
        decode_keys(rk, kl[1]);
        load_keys(rk, next_k);
        next_k = place(t_begin + 3 * kTok);
      }
    }
    if (values) {
      load_values(rv, place(t_begin));
      decode_values(rv, t_begin, vl[0]);
      load_values(rv, place(t_begin + kTok));
      next_v = place(t_begin + 2 * kTok);
    }
    lds_barrier();
    if constexpr (kPipe) {
#pragma unroll
      for (int t = 0; t < 2; ++t) scores(sa, kl[0], t, 0, KS);
      lds_barrier();                         // K(0) is read before K(2) overwrites it
    }
    int32_t i = 0;
    for (; i + 2 < tiles; i += 2) {
      step(sa, sb, IntC<0>{}, IntC<0>{}, i);
      step(sb, sa, IntC<1>{}, IntC<0>{}, i + 1);
    }
    if (i + 1 < tiles) {
      step(sa, sb, IntC<0>{}, IntC<0>{}, i);
      step(sb, sa, IntC<1>{}, IntC<1>{}, i + 1);
    } else {
      step(sa, sb, IntC<0>{}, IntC<1>{}, i);
    }
  }
  l += __shfl_xor(l, 32, 64);

  // Lane (c, hh) holds its row's head values DT (i % 4 + 8 (i / 4) + 4 hh) + d.
  auto write_row = [&]() {
    const int head = h * p.group + hg;
    const int64_t qrow = q0 + tok;
    const float inv = l == 0.f ? 0.f : 1.f / l;
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
          l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
  };
  if (parts == 1) {
    if (live) write_row();
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
  if (!arrive_last(p.counters + unit * kCounterStride, static_cast<uint32_t>(parts), &flag)) return;
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = v16f(0.f);
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
  if (live) write_row();
}

template <int D, int NW>
hipError_t launch(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  const int64_t grid = static_cast<int64_t>(plan.row_blocks) * plan.splits * p.batch * p.cache.heads;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((attn_many_kernel<D, NW>), dim3(static_cast<unsigned>(grid)), dim3(64 * NW), 0,
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
    a.groups = 256 * few_waves(head_dim, a.row_tiles);
    a.counter_bytes = (units * 4 * kCounterStride + 255) / 256 * 256;
    a.bytes = a.counter_bytes +
              2 * static_cast<int64_t>(a.groups) * 16 * a.row_tiles * (head_dim + 2) * 4;
    return a;
  }
  // Eight wavefronts of 32 rows share the decoding where there are rows for them (heads of 256 leave a
  // SIMD the registers for one wavefront only).
  a.row_tiles = head_dim == 256 || rows <= 128 ? 4 : 8;
  const int64_t block_rows = 32 * a.row_tiles;
  const int64_t blocks = (rows + block_rows - 1) / block_rows;
  a.row_blocks = static_cast<int>(blocks);
  const int64_t fit = 512 / (blocks * units);
  a.splits = static_cast<int>(fit < 1 ? 1 : fit > 64 ? 64 : fit);
  if (a.splits > 1) {
    a.counter_bytes = (blocks * units * 4 * kCounterStride + 255) / 256 * 256;
    a.bytes = a.counter_bytes +
              blocks * units * a.splits * block_rows * (head_dim + 2) * 4;
  }
  return a;
}

hipError_t launch_attn_many(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  const bool eight = plan.row_tiles == 8;
  if (p.cache.head_dim == 64) return eight ? launch<64, 8>(p, plan, stream) : launch<64, 4>(p, plan, stream);
  if (p.cache.head_dim == 128)
    return eight ? launch<128, 8>(p, plan, stream) : launch<128, 4>(p, plan, stream);
  return launch<256, 4>(p, plan, stream);
}

}  // namespace mx
