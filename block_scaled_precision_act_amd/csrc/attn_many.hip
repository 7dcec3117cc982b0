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
//
// Heads of 64 and 128 (attn_many_kernel): a wavefront has 32 rows to itself.  Heads of 256
// (attn_wide_kernel): the sums of 32 such rows fill half of a wavefront's registers, so two
// wavefronts share 32 rows, each scoring half of the tokens and summing half of the head's values;
// their weights pass through LDS.
#include "attn_common.h"

namespace mx {
namespace {

constexpr int kTok = 64;
constexpr float kLn2 = 0.6931471805599453f;
typedef float v16f __attribute__((ext_vector_type(16)));

// What a workgroup works on: a block of rows of a sequence and head, and a part of its keys.
struct Work {
  int32_t b, h, blk, part, parts;
  int32_t len, q0, rows, r0, first;       // first: the position of the sequence's first query
  int32_t hi, t_begin, tiles;             // keys end; this part's first token and tiles of 64
  int32_t full_hi, full_lo;               // tokens below and from which every row sees
  bool any;
};

__device__ __forceinline__ Work work_of(const AttnProblem& p, int block_rows, int row_blocks,
                                        int splits) {
  Work w;
  const uint32_t heads = p.cache.heads;
  // Heads fastest: with 8 of them a head's keys stay on one XCD's L2.  Late rows (the longest under
  // a causal mask) first.
  uint32_t idx = blockIdx.x;
  w.h = idx % heads;
  idx /= heads;
  w.b = idx % p.batch;
  idx /= p.batch;
  w.part = idx % splits;
  w.blk = row_blocks - 1 - static_cast<int>(idx / splits);
  const int64_t most = static_cast<int64_t>(p.table_width) * p.cache.page_size;
  const int32_t raw_len = read_uniform(p.lens, w.b);
  w.len = raw_len < 0 ? 0 : (raw_len < most ? raw_len : static_cast<int32_t>(most));
  int32_t q0 = w.b * p.max_q, q1 = q0 + p.max_q;
  if (p.starts) {
    q0 = min(max(read_uniform(p.starts, w.b), 0), p.total_q);
    q1 = min(max(read_uniform(p.starts, w.b + 1), q0), p.total_q);
  }
  const int32_t n = min(q1 - q0, p.max_q);
  w.q0 = q0;
  w.rows = n * p.group;
  w.r0 = w.blk * block_rows;
  w.any = w.r0 < w.rows;
  if (!w.any) return w;
  w.first = w.len - n;
  const int32_t tok_lo = w.r0 / p.group, tok_hi = (min(w.r0 + block_rows, w.rows) - 1) / p.group;
  w.hi = p.causal ? min(max(w.first + tok_hi + 1, 0), w.len) : w.len;
  const int32_t lo = p.window > 0 ? max(w.first + tok_lo + 1 - p.window, 0) & ~(kTok - 1) : 0;
  const int32_t all = max(0, (w.hi - lo + kTok - 1) / kTok);
  w.parts = max(1, min(splits, all / 4));
  w.any = w.part < w.parts;
  const int32_t tile0 = static_cast<int32_t>(static_cast<int64_t>(all) * w.part / w.parts);
  w.tiles = static_cast<int32_t>(static_cast<int64_t>(all) * (w.part + 1) / w.parts) - tile0;
  w.t_begin = lo + tile0 * kTok;
  w.full_hi = p.causal ? min(w.first + tok_lo + 1, w.len) : w.len;
  w.full_lo = p.window > 0 ? w.first + tok_hi + 1 - p.window : 0;
  return w;
}

// A lane's query row: lanes c and c + 32 of a wavefront share row r0 + 32 tile + c.
struct Row {
  bool live;
  int32_t tok, hg, lo, hi;                // query, grouped head, the keys it sees
};

__device__ __forceinline__ Row row_of(const AttnProblem& p, const Work& w, int tile) {
  Row r;
  const int32_t i = w.r0 + tile * 32 + (threadIdx.x & 31);
  r.live = i < w.rows;
  r.tok = r.live ? i / p.group : 0;
  r.hg = r.live ? i - r.tok * p.group : 0;
  r.hi = r.live && p.causal ? w.first + r.tok + 1 : w.len;
  r.lo = r.live && p.window > 0 ? w.first + r.tok + 1 - p.window : 0;
  return r;
}

// Its values, as B operands.
template <int KS>
__device__ __forceinline__ void load_query(const AttnProblem& p, const Work& w, const Row& r,
                                           bf16x8 (&qf)[KS]) {
  const uint16_t* row = p.q.p + static_cast<int64_t>(w.q0 + r.tok) * p.q.token_stride +
                        static_cast<int64_t>(w.h * p.group + r.hg) * p.q.head_stride +
                        8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 x = r.live ? *reinterpret_cast<const uint4*>(row + 16 * s) : make_uint4(0, 0, 0, 0);
    x.x ^= p.flip; x.y ^= p.flip; x.z ^= p.flip; x.w ^= p.flip;
    qf[s] = __builtin_bit_cast(bf16x8, x);
  }
}

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

// The wavefront's share of loading and decoding: the keys or values of one 16-token step `sub` of the
// tile (its page is the same for all lanes): of key lane % 16, codes [kq D / 4, (kq + 1) D / 4); of 8
// tokens (half vh), head values [EPI vc, EPI (vc + 1)).
template <int D>
struct Decoder {
  static constexpr int KS = D / 16, DT = D / 32, EPI = D / 32;
  const AttnProblem& p;
  const uint8_t *kbase, *vbase, *ksbase, *vsbase;
  int64_t trow;
  int32_t hi, last16;
  uint32_t page16, turn_k;
  int sub, k16, kq, vc, vh;

  __device__ __forceinline__ Decoder(const AttnProblem& p_, const Work& w, int sub_) : p(p_), sub(sub_) {
    const int lane = threadIdx.x & 63;
    kbase = p.cache.k + w.h * p.cache.code_head;
    vbase = p.cache.v + w.h * p.cache.code_head;
    ksbase = p.cache.ks + w.h * p.cache.scale_head;
    vsbase = p.cache.vs + w.h * p.cache.scale_head;
    trow = static_cast<int64_t>(w.b) * p.table_stride;
    hi = w.hi;
    last16 = (w.hi - 1) >> 4;
    page16 = p.cache.page_size >> 4;
    k16 = lane & 15;
    kq = lane >> 4;
    vc = lane & 31;
    vh = lane >> 5;
    turn_k = 9 + 8 * (D == 64 ? 2 * (k16 & 1) + (kq >> 1) : D == 128 ? kq : 2 * (kq & 1));
  }
  // Steps past the last one stand for it: what is loaded there is masked or never used.
  __device__ __forceinline__ Place place(int32_t t0) const {
    const uint32_t t16 = static_cast<uint32_t>(min((t0 >> 4) + sub, last16));
    const uint32_t page = p.page_div ? __umulhi(t16, p.page_div) : t16;
    const uint32_t id = static_cast<uint32_t>(read_uniform(p.table, trow + page));
    return Place{id < p.cache.pages ? id : 0u, (t16 - page * page16) * 16u};
  }
  __device__ __forceinline__ void load_keys(RawKeys<D>& w, Place at) const {
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
  }
  __device__ __forceinline__ void load_values(RawValues<D>& w, Place at) const {
    const uint8_t* vp = vbase + (at.id * p.cache.code_page + at.off * (D / 2)) +
                        (vh * 4 * (D / 2) + (vc * (EPI / 2) & ~3));
    const uint8_t* sp = vsbase + (at.id * p.cache.scale_page + at.off * (D / 32)) + vh * 4 * (D / 32);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w.v[i] = *reinterpret_cast<const uint32_t*>(vp + ((i >> 2) * 8 + (i & 3)) * (D / 2));
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
  }
  // Into [32-token half][k step][lane].
  __device__ __forceinline__ void decode_keys(const RawKeys<D>& w, uint4* dst) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float sc = scale_of_byte(w.s, D == 256 && i >= 4 ? turn_k + 8 : turn_k);
      const int word = kq * (D / 32) + i;               // 8 codes: k step word / 2, half word % 2
      dst[((sub >> 1) * KS + (word >> 1)) * 64 + (word & 1) * 32 + (sub & 1) * 16 + k16] =
          decode8(w.k[i], sc);
    }
  }
  // Of the tile from t0, into [16-token step][head value % DT][lane].
  __device__ __forceinline__ void decode_values(const RawValues<D>& w, int32_t t0, uint4* dst) const {
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
  }
};

// K steps [j0, j1) of the scores of one 32-token half.
template <int KS>
__device__ __forceinline__ void scores(v16f& s, const uint4* keys, const bf16x8 (&qf)[KS], int j0, int j1) {
#pragma unroll
  for (int j = j0; j < j1; ++j)
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(bf16x8, keys[j * 64 + (threadIdx.x & 63)]), qf[j], j == 0 ? v16f(0.f) : s, 0, 0, 0);
}

// Masks the lane's 16 scores of the 32 tokens from t0.
__device__ __forceinline__ void mask(v16f& s, const Row& r, int32_t t0) {
  const int32_t at = t0 + 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int32_t key = at + (e & 3) + 8 * (e >> 2);
    if (key >= r.hi || key < r.lo) s[e] = -kInf;
    if (e % 8 == 7) __builtin_amdgcn_sched_barrier(0);
  }
}

// The weights of 8 of the lane's scores as a B operand; their sum is added to l.
__device__ __forceinline__ bf16x8 weights(const v16f& s, int at, float scale, float sub, float& l) {
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[at + e], scale, -sub));
    l += w[e];
  }
  return __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]),
                                               pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])));
}

// The lane's sums are head values DT (i % 4 + 8 (i / 4) + 4 h) + d0 + d, d < N, h its half: the row
// is written, or (several parts) left in the workspace for the last part to join.
// Partial layout: values as the lanes hold them, 4 to a lane, lanes in a row; then m, then l.
template <int DT, int N>
__device__ __forceinline__ void write_row(const AttnProblem& p, const Work& w, const Row& r,
                                          const v16f (&acc)[N], float m, float l, int d0, bool lse) {
  const int hh = (threadIdx.x & 63) >> 5, head = w.h * p.group + r.hg;
  const int64_t qrow = w.q0 + r.tok;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* dst = p.out.p + qrow * p.out.token_stride + head * p.out.head_stride + d0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t x[N / 2];
#pragma unroll
    for (int d = 0; d < N / 2; ++d) x[d] = pack_bf16(acc[2 * d][i] * inv, acc[2 * d + 1][i] * inv);
    uint16_t* at = dst + DT * ((i & 3) + 8 * (i >> 2) + 4 * hh);
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(at) = x[0];
    else *reinterpret_cast<uint2*>(at) = make_uint2(x[0], x[1]);
  }
  if (lse && p.lse && hh == 0)
    p.lse[qrow * (static_cast<int64_t>(p.group) * p.cache.heads) + head] =
        l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int THREADS, int N>
__device__ __forceinline__ void store_part(float* part, const v16f (&acc)[N], float m, float l, int stat) {
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      store_shared4(part + ((d * 4 + i / 4) * THREADS + threadIdx.x) * 4, acc[d][i], acc[d][i + 1],
                    acc[d][i + 2], acc[d][i + 3]);
  if ((threadIdx.x & 32) == 0) {
    store_shared(part + N * 16 * THREADS + stat, m);
    store_shared(part + N * 16 * THREADS + THREADS / 2 + stat, l);
  }
}

// Joins `parts` partials, in order.  A part that saw nothing has m = -infinity and weight 0.
template <int THREADS, int N>
__device__ __forceinline__ void join_parts(const float* first, int64_t stride, int parts, int stat,
                                           v16f (&acc)[N], float& m, float& l) {
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int d = 0; d < N; ++d) acc[d] = v16f(0.f);
  for (int q = 0; q < parts; ++q) {
    const float* src = first + q * stride;
    const float pm = src[N * 16 * THREADS + stat], pl = src[N * 16 * THREADS + THREADS / 2 + stat];
    const float now = fmaxf(m, pm);
    const float fo = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
    const float fn = pm == -kInf ? 0.f : __builtin_amdgcn_exp2f(pm - now);
    m = now;
    l = l * fo + pl * fn;
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(src + ((d * 4 + i / 4) * THREADS + threadIdx.x) * 4);
        acc[d][i] = acc[d][i] * fo + x.x * fn;
        acc[d][i + 1] = acc[d][i + 1] * fo + x.y * fn;
        acc[d][i + 2] = acc[d][i + 2] * fo + x.z * fn;
        acc[d][i + 3] = acc[d][i + 3] * fo + x.w * fn;
      }
  }
}

// Floats of one partial: N sums of 16 a thread, m and l for each 2 threads.
constexpr int64_t part_floats(int threads, int n) { return static_cast<int64_t>(threads) * (16 * n + 1); }

// NW wavefronts of 32 query rows each.  Of 8, the first four decode keys and the others values (one
// of each to a SIMD); of 4, all decode both.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_many_kernel(const AttnProblem p, int row_blocks,
                                                               int splits) {
  constexpr int KS = D / 16, DT = D / 32, kThreads = 64 * NW;
  __shared__ uint4 kl[2][2 * KS * 64];
  __shared__ uint4 vl[2][4 * DT * 64];
  __shared__ uint32_t flag;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Work w = work_of(p, 32 * NW, row_blocks, splits);
  if (!w.any) return;
  const Row row = row_of(p, w, wave);
  bf16x8 qf[KS];
  load_query(p, w, row, qf);
  const bool keys = NW == 4 || wave < 4, values = NW == 4 || wave >= 4;
  const Decoder<D> dec(p, w, wave & 3);

  v16f acc[DT];
  float m = -kInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = v16f(0.f);
  RawKeys<D> rk;
  RawValues<D> rv;
  Place next_k, next_v;

  // Tile i: its scores `s` are there; while its weights and products are made, the next tile's scores
  // are (into `sn`), the keys after those and the next tile's values are decoded, and the ones after
  // them loaded.  One barrier a tile: K(i + 2) goes where K(i) was, V(i + 1) where V(i - 1) was, both
  // read by every wavefront before the last barrier.
  auto step = [&](v16f (&s)[2], v16f (&sn)[2], auto odd, auto final, int32_t i) {
    constexpr int B = decltype(odd)::value;
    constexpr bool LAST = decltype(final)::value;
    const int32_t t0 = w.t_begin + i * kTok;
    if (t0 + kTok > w.full_hi || t0 < w.full_lo) {
      mask(s[0], row, t0);
      mask(s[1], row, t0 + 32);
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
    const float sub = m == -kInf ? 0.f : m;
#pragma unroll
    for (int q = 0; q < 4; ++q) {            // 16 tokens each
      const bf16x8 pf = weights(s[q >> 1], 8 * (q & 1), p.scale_log2, sub, l);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, vl[B][(q * DT + d) * 64 + lane]), pf, acc[d], 0, 0, 0);
      if constexpr (!LAST)
        scores(sn[q >> 1], kl[B ^ 1] + (q >> 1) * KS * 64, qf, (q & 1) * (KS / 2), ((q & 1) + 1) * (KS / 2));
    }
    if constexpr (!LAST) {
      if (keys) {
        dec.decode_keys(rk, kl[B]);
        dec.load_keys(rk, next_k);
        next_k = dec.place(t0 + 4 * kTok);
      }
      if (values) {
        dec.decode_values(rv, t0 + kTok, vl[B ^ 1]);
        dec.load_values(rv, next_v);
        next_v = dec.place(t0 + 3 * kTok);
      }
      lds_barrier();
    }
  };

  if (w.tiles > 0) {
    v16f sa[2], sb[2];
    if (keys) {
      dec.load_keys(rk, dec.place(w.t_begin));
      dec.decode_keys(rk, kl[0]);
      dec.load_keys(rk, dec.place(w.t_begin + kTok));
      dec.decode_keys(rk, kl[1]);
      dec.load_keys(rk, dec.place(w.t_begin + 2 * kTok));
      next_k = dec.place(w.t_begin + 3 * kTok);
    }
    if (values) {
      dec.load_values(rv, dec.place(w.t_begin));
      dec.decode_values(rv, w.t_begin, vl[0]);
      dec.load_values(rv, dec.place(w.t_begin + kTok));
      next_v = dec.place(w.t_begin + 2 * kTok);
    }
    lds_barrier();
    scores(sa[0], kl[0], qf, 0, KS);
    scores(sa[1], kl[0] + KS * 64, qf, 0, KS);
    lds_barrier();                           // K(0) is read before K(2) overwrites it
    int32_t i = 0;
    for (; i + 2 < w.tiles; i += 2) {
      step(sa, sb, IntC<0>{}, IntC<0>{}, i);
      step(sb, sa, IntC<1>{}, IntC<0>{}, i + 1);
    }
    if (i + 1 < w.tiles) {
      step(sa, sb, IntC<0>{}, IntC<0>{}, i);
      step(sb, sa, IntC<1>{}, IntC<1>{}, i + 1);
    } else {
      step(sa, sb, IntC<0>{}, IntC<1>{}, i);
    }
  }
  l += __shfl_xor(l, 32, 64);

  if (w.parts > 1) {
    const int64_t unit = (static_cast<int64_t>(w.blk) * p.batch + w.b) * p.cache.heads + w.h;
    constexpr int64_t kPart = part_floats(kThreads, DT);
    float* const parts = p.parts + unit * splits * kPart;
    const int stat = wave * 32 + (lane & 31);
    store_part<kThreads>(parts + w.part * kPart, acc, m, l, stat);
    if (!arrive_last(p.counters + unit * kCounterStride, static_cast<uint32_t>(w.parts), &flag)) return;
    join_parts<kThreads>(parts, kPart, w.parts, stat, acc, m, l);
  }
  if (row.live) write_row<DT>(p, w, row, acc, m, l, 0, true);
}

// Heads of 256: eight wavefronts, the first four (half 0) and the last four (half 1) on the same four
// tiles of 32 rows.  Half h scores tokens [32 h, 32 h + 32) of a tile and sums head values
// 8 j + 4 h + (0..3).  Two barriers a tile:
//   first   half h's weights of tile i (from the scores of both halves' larger maximum) go to LDS; the
//           scores of tile i + 1 and their maxima are made; half 1 decodes the values of tile i
//   second  the products of tile i's weights and values; half 0 decodes the keys of tile i + 2
// so that each of the matrix runs has the other side's decoding beside it, and one buffer of keys,
// values and weights is enough.
__global__ __launch_bounds__(512, 2) void attn_wide_kernel(const AttnProblem p, int row_blocks, int splits) {
  constexpr int D = 256, KS = D / 16, DT = D / 32, N = DT / 2, kThreads = 512;
  __shared__ uint4 kl[2 * KS * 64];
  __shared__ uint4 vl[4 * DT * 64];
  __shared__ uint4 pl[4][4 * 64];           // [row tile][16-token step][lane]
  __shared__ float tops[2][4][2][32];       // [tile parity][row tile][half][row]
  __shared__ uint32_t flag;
  const int lane = threadIdx.x & 63, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = wave & 3, half = wave >> 2;
  const Work w = work_of(p, 128, row_blocks, splits);
  if (!w.any) return;
  const Row row = row_of(p, w, rt);
  bf16x8 qf[KS];
  load_query(p, w, row, qf);
  const Decoder<D> dec(p, w, rt);

  v16f acc[N];
  float m = -kInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < N; ++d) acc[d] = v16f(0.f);
  RawKeys<D> rk;
  RawValues<D> rv;
  Place next;

  // Scores of tile i, masked, and their maxima for the other half.
  auto score = [&](v16f& s, int32_t i) {
    const int32_t t0 = w.t_begin + i * kTok;
    scores(s, kl + half * KS * 64, qf, 0, KS);
    if (t0 + kTok > w.full_hi || t0 < w.full_lo) mask(s, row, t0 + half * 32);
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
    top = max_halves(top) * p.scale_log2;
    if (lane < 32) tops[i & 1][rt][half][c] = top;
  };
  auto step = [&](v16f& s, v16f& sn, auto final, int32_t i) {
    constexpr bool LAST = decltype(final)::value;
    const int32_t t0 = w.t_begin + i * kTok;
    const float top = fmaxf(tops[i & 1][rt][0][c], tops[i & 1][rt][1][c]);
    // As in attn_many_kernel; both halves see the same maxima and move together.
    if (__any(top > m + 8.f)) {
      const float now = fmaxf(m, top);
      const float f = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < N; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] *= f;
    }
    const float sub = m == -kInf ? 0.f : m;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      pl[rt][(half * 2 + u) * 64 + lane] = __builtin_bit_cast(uint4, weights(s, 8 * u, p.scale_log2, sub, l));
    if (half == 1) {
      dec.decode_values(rv, t0, vl);
      if constexpr (!LAST) {
        dec.load_values(rv, next);
        next = dec.place(t0 + 2 * kTok);
      }
    }
    if constexpr (!LAST) score(sn, i + 1);
    lds_barrier();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x8 pf = __builtin_bit_cast(bf16x8, pl[rt][q * 64 + lane]);
#pragma unroll
      for (int d = 0; d < N; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, vl[(q * DT + half * N + d) * 64 + lane]), pf, acc[d], 0, 0, 0);
    }
    if constexpr (!LAST) {
      if (half == 0) {
        dec.decode_keys(rk, kl);
        dec.load_keys(rk, next);
        next = dec.place(t0 + 4 * kTok);
      }
      lds_barrier();
    }
  };

  if (w.tiles > 0) {
    v16f sa, sb;
    if (half == 0) {
      dec.load_keys(rk, dec.place(w.t_begin));
      dec.decode_keys(rk, kl);
      dec.load_keys(rk, dec.place(w.t_begin + kTok));
    } else {
      dec.load_values(rv, dec.place(w.t_begin));
      next = dec.place(w.t_begin + kTok);
    }
    lds_barrier();
    score(sa, 0);
    lds_barrier();                           // K(0) is read before K(1) overwrites it
    if (half == 0) {
      dec.decode_keys(rk, kl);
      dec.load_keys(rk, dec.place(w.t_begin + 2 * kTok));
      next = dec.place(w.t_begin + 3 * kTok);
    }
    lds_barrier();
    int32_t i = 0;
    for (; i + 2 < w.tiles; i += 2) {
      step(sa, sb, IntC<0>{}, i);
      step(sb, sa, IntC<0>{}, i + 1);
    }
    if (i + 1 < w.tiles) {
      step(sa, sb, IntC<0>{}, i);
      step(sb, sa, IntC<1>{}, i + 1);
    } else {
      step(sa, sb, IntC<1>{}, i);
    }
  }
  // A row's sum is that of its two halves' shares.
  l += __shfl_xor(l, 32, 64);
  lds_barrier();
  if (lane < 32) tops[0][rt][half][c] = l;
  lds_barrier();
  l += tops[0][rt][half ^ 1][c];

  if (w.parts > 1) {
    const int64_t unit = (static_cast<int64_t>(w.blk) * p.batch + w.b) * p.cache.heads + w.h;
    constexpr int64_t kPart = part_floats(kThreads, N);
    float* const parts = p.parts + unit * splits * kPart;
    const int stat = wave * 32 + c;
    store_part<kThreads>(parts + w.part * kPart, acc, m, l, stat);
    if (!arrive_last(p.counters + unit * kCounterStride, static_cast<uint32_t>(w.parts), &flag)) return;
    join_parts<kThreads>(parts, kPart, w.parts, stat, acc, m, l);
  }
  if (row.live) write_row<DT>(p, w, row, acc, m, l, half * N, half == 0);
}

hipError_t grid_of(const AttnProblem& p, const AttnPlan& plan, dim3* grid) {
  const int64_t n = static_cast<int64_t>(plan.row_blocks) * plan.splits * p.batch * p.cache.heads;
  if (n > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  *grid = dim3(static_cast<unsigned>(n));
  return hipSuccess;
}

template <int D, int NW>
void launch(const AttnProblem& p, const AttnPlan& plan, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((attn_many_kernel<D, NW>), grid, dim3(64 * NW), 0, stream, p, plan.row_blocks,
                     plan.splits);
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
  // Eight wavefronts of 32 rows share the decoding where there are rows for them; with heads of 256,
  // eight share 128 rows.
  a.row_tiles = head_dim == 256 || rows <= 128 ? 4 : 8;
  const int64_t block_rows = 32 * a.row_tiles;
  const int64_t blocks = (rows + block_rows - 1) / block_rows;
  a.row_blocks = static_cast<int>(blocks);
  const int64_t fit = 512 / (blocks * units);
  a.splits = static_cast<int>(fit < 1 ? 1 : fit > 64 ? 64 : fit);
  if (a.splits > 1) {
    a.counter_bytes = (blocks * units * 4 * kCounterStride + 255) / 256 * 256;
    a.bytes = a.counter_bytes +
              blocks * units * a.splits * 4 *
                  (head_dim == 256 ? part_floats(512, 4) : part_floats(64 * a.row_tiles, head_dim / 32));
  }
  return a;
}

hipError_t launch_attn_many(const AttnProblem& p, const AttnPlan& plan, hipStream_t stream) {
  dim3 grid;
  const hipError_t e = grid_of(p, plan, &grid);
  if (e != hipSuccess) return e;
  const bool eight = plan.row_tiles == 8;
  if (p.cache.head_dim == 64) {
    eight ? launch<64, 8>(p, plan, grid, stream) : launch<64, 4>(p, plan, grid, stream);
  } else if (p.cache.head_dim == 128) {
    eight ? launch<128, 8>(p, plan, grid, stream) : launch<128, 4>(p, plan, grid, stream);
  } else {
    hipLaunchKernelGGL(attn_wide_kernel, grid, dim3(512), 0, stream, p, plan.row_blocks, plan.splits);
  }
  return hipGetLastError();
}

}  // namespace mx
