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
//
// Measured: a prompt of 8192 tokens, 32 heads of 128 on 8: 517 to 527 us (by box), 1045 TFLOP/s (a large
// library product reaches 1172, this library's own 8192^3 GEMM 1415), the matrix instructions busy 43% of
// the cycles; 512 and 386 queries of 16 heads of 256 on 2 against 32768 and 27891 tokens: 488 to 496 us,
// 910 TFLOP/s.  Power does not bound them (2.38 GHz after 200 calls): for every matrix instruction a
// wavefront reads 1 KB from LDS, which takes about as long, and decoding and softmax take as many cycles
// again; with the decoding left out the first takes 410 us and the second two thirds, without those reads
// the first takes 355.  More rows a wavefront would need fewer reads: 64 (four wavefronts, every register
// of the CU) leave one wavefront a SIMD and nothing to cover its waits with, 595 us.
//
// TREE: the queries are a tree's nodes, and a mask says which of the sequence's last tokens each sees; its words
// are read in the last tiles alone.  64 nodes of 4 sequences of up to 131073 tokens, 32 heads of 128 on 8: 533
// to 562 us (by box), 950 to 1003 TFLOP/s.  41 ragged trees of up to 12 nodes, 56 heads on 8: 99 us; 33 nodes of
// 16 heads of 256 on 2, 2 sequences: 71 us, a third of it for the 120 rows that 264 leave empty in three blocks.
#include "attn_common.h"

#include <algorithm>

namespace mx {
namespace {

constexpr int kTok = 64;
constexpr float kLn2 = 0.6931471805599453f;
typedef float v16f __attribute__((ext_vector_type(16)));

// What a workgroup works on at a time: a block of rows of a sequence and head (a unit), and a run of
// the 64-token tiles that some of its rows see.
struct Work {
  int32_t b, h, blk;
  int32_t len, q0, rows, r0, first;       // first: the position of the sequence's first query
  int32_t low, hi;                        // keys that any of its rows sees: [low, hi)
  int32_t t_begin, tiles;                 // the run's first token and tiles of 64
  int32_t full_hi, full_lo;               // tokens below and from which every row sees
  bool any;                               // the block has rows
};

// A whole unit.
template <bool TREE>
__device__ __forceinline__ Work unit_of(const AttnProblem& p, int block_rows, int h, int b, int blk) {
  Work w;
  w.h = h;
  w.b = b;
  w.blk = blk;
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
  w.tiles = 0;
  if (!w.any) return w;
  w.first = w.len - n;
  const int32_t tok_lo = w.r0 / p.group, tok_hi = (min(w.r0 + block_rows, w.rows) - 1) / p.group;
  w.hi = p.causal ? min(max(w.first + tok_hi + 1, 0), w.len) : w.len;
  w.low = p.window > 0 ? max(window_start(w.first + tok_lo, p.window), 0) : 0;
  w.t_begin = w.low & ~(kTok - 1);
  w.tiles = max(0, (w.hi - w.t_begin + kTok - 1) / kTok);
  w.full_hi = p.causal ? min(w.first + tok_lo + 1, w.len) : w.len;
  w.full_lo = p.window > 0 ? window_start(w.first + tok_hi, p.window) : 0;
  if constexpr (TREE) {                   // any of its queries may stand anywhere in the tree
    w.low = p.window > 0 ? max(window_start(w.first, p.window), 0) : 0;
    w.t_begin = w.low & ~(kTok - 1);
    w.tiles = max(0, (w.hi - w.t_begin + kTok - 1) / kTok);
    w.full_hi = w.first;
    w.full_lo = p.window > 0 ? window_start(w.len - 1, p.window) : 0;
  }
  return w;
}

// How units come to workgroups.
//
// As they are: a workgroup each, heads fastest (with 8 of them a head's keys stay on one XCD's L2), late
// rows, the longest under a causal mask, first.  Where they are fewer than the chip holds, each is cut
// into up to `splits` parts of its tiles, of 4 at least.
//
// Or dealt: sequences differ in length, and the longest unit's part lasts while other workgroups idle.
// All units' tiles, in the order (head, sequence, block), with kUnitSlots before each unit's for what it
// costs besides, are cut into equal runs, one a workgroup.  A run that would begin within kSnap tiles of
// a unit's ends begins there.  What a workgroup has of a unit that others share is a part: a workgroup
// has two at most (the end of a unit, the beginning of another).
//
// The lengths decide, on the device: a deal costs kDealCost tiles (more beginnings and parts), units as
// they are last as long as the longest one's part, or as the average in rounds.  One sequence is not
// dealt, nor are kDealUnits or more units a workgroup, which fill the chip evenly enough.  Dealt and not:
// 4 sequences of 5000 to 32768 tokens, up to 500 queries, 32 heads of 128 on 4: 515 and 915 us; 4 of 1000
// to 9000, up to 300, 16 of 256 on 2: 137 and 304 us; the two above with heads of 256: 495 and 545 (488
// since that kernel orders its reads).
// Looking at it costs about 5 us (4 x 300 queries of 200 to 300 tokens: 20 us, 25 when looked at), so the
// host spares it where the table is short.
//
// Parts are joined by attn_join_kernel.
constexpr int64_t kDealUnits = 4;
constexpr uint32_t kUnitSlots = 2, kSnap = 2, kLeastShare = 4, kDealCost = 8;      // tiles
constexpr int kLeastPart = 4;
constexpr int kMostEntries = 2048;         // (sequence, block) pairs of a deal
constexpr int kMostGroups = 512;
constexpr uint32_t kMixedSlots = AttnPlan::kMixedSlots;

__device__ __forceinline__ int parts_of(int tiles, int splits) {
  return max(1, min(splits, tiles / kLeastPart));
}

// Where a run begins, and the unit it begins in: its first slot and the one after its last, its number
// (head, sequence, block).  Left in the workspace for the join; the first run's holds the number of runs
// instead (0: no deal).
struct RunStart {
  uint32_t unit_first, unit_end, at, unit;
};
constexpr int64_t kStartFloats = kMostGroups * sizeof(RunStart) / 4;

// Whether two wavefronts share 32 of the unit's rows where a kernel takes such and others (MIXED).
__device__ __forceinline__ bool shares(const Work& w, int block_rows) { return w.rows - w.r0 <= block_rows / 2; }

// The slots of a tile: one; or, where units' tiles differ (MIXED), as many as their times are to each other.
// (Three of four: 5 or 7 of 8 and 2 of 3 leave the runs less even, by 0 to 8 us of 80 to 110.)
template <bool MIXED>
__device__ __forceinline__ uint32_t tile_slots(const Work& w, int block_rows) {
  return !MIXED ? 1 : shares(w, block_rows) ? kMixedSlots - 1 : kMixedSlots;
}

template <bool MIXED>
struct Deal {
  static constexpr uint32_t kScale = MIXED ? kMixedSlots : 1;
  const uint32_t* first;     // of each (sequence, block): its first slot in a head's, in LDS
  uint32_t entries, heads, groups;

  __device__ __forceinline__ uint32_t slot_of(uint32_t e) const {
    return __builtin_amdgcn_readfirstlane(first[e]);
  }
  __device__ __forceinline__ uint32_t per_head() const { return slot_of(entries); }
  // The entry that slot x of a head lies in: of the 64 runs of entries that the lanes stand for, then of
  // the run's entries.
  __device__ __forceinline__ uint32_t entry(uint32_t x) const {
    const uint32_t lane = threadIdx.x & 63, run = (entries + 63) / 64;
    const uint32_t next = (lane + 1) * run;
    const uint32_t e0 = run * __builtin_popcountll(__ballot(next < entries && first[min(next, entries)] <= x));
    const uint32_t e1 = e0 + lane + 1;
    return e0 + __builtin_popcountll(__ballot(lane + 1 < run && e1 < entries && first[min(e1, entries)] <= x));
  }
  __device__ __forceinline__ RunStart start(uint32_t g) const {
    const uint32_t per = per_head(), total = per * heads;
    const uint32_t whole = total / groups;
    const uint32_t x = g * whole + g * (total - whole * groups) / groups;      // g total / groups
    if (x >= total) return RunStart{total, total, total, 0};
    const uint32_t head = x / per, base = head * per, e = entry(x - base);
    const uint32_t s = base + slot_of(e), end = base + slot_of(e + 1);
    return RunStart{s, end, x <= s + kScale * (kUnitSlots + kSnap) ? s : x + kScale * kSnap >= end ? end : x,
                    head * entries + e};
  }
};

// Called by all THREADS of a workgroup; `first` has room for kMostEntries + 3.  The slots of all heads
// number less than 2^31.
template <int THREADS, bool TREE, bool MIXED>
__device__ __forceinline__ Deal<MIXED> deal(const AttnProblem& p, int block_rows, int row_blocks, int splits,
                                            int groups, uint32_t* first) {
  constexpr uint32_t kScale = Deal<MIXED>::kScale;
  Deal<MIXED> d;
  d.first = first;
  d.entries = p.batch * row_blocks;
  d.heads = p.cache.heads;
  for (uint32_t e = threadIdx.x; e < d.entries; e += THREADS) {
    const uint32_t b = e / row_blocks;
    const Work w = unit_of<TREE>(p, block_rows, 0, b, e - b * row_blocks);
    first[e + 1] =
        w.any ? static_cast<uint32_t>(w.tiles) * tile_slots<MIXED>(w, block_rows) + kScale * kUnitSlots : 0u;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t run = (d.entries + 63) / 64;
    const uint32_t e0 = min(threadIdx.x * run, d.entries), e1 = min(e0 + run, d.entries);
    uint32_t sum = 0, longest = 0, count = 0;
    for (uint32_t e = e0; e < e1; ++e) {
      const uint32_t n = first[e + 1];
      sum += n;
      longest = max(longest, n);
      count += n != 0;
    }
    uint32_t upto = sum;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) {
      const uint32_t v = __shfl_up(upto, i, 64);
      if (static_cast<int>(threadIdx.x) >= i) upto += v;
      longest = max(longest, static_cast<uint32_t>(__shfl_xor(longest, i, 64)));
      count += __shfl_xor(count, i, 64);
    }
    uint32_t at = upto - sum;
    for (uint32_t e = e0; e < e1; ++e) first[e + 1] = at += first[e + 1];
    if (threadIdx.x == 0) {
      first[0] = 0;
      first[d.entries + 1] = longest;
      first[d.entries + 2] = count;
    }
  }
  __syncthreads();
  const uint32_t total = d.per_head() * d.heads, units = max(1u, d.slot_of(d.entries + 2) * d.heads);
  const uint32_t longest = d.slot_of(d.entries + 1);
  const uint32_t span = max(longest / parts_of(static_cast<int>(longest / kScale), splits),
                            (units + groups - 1) / groups * (splits == 1 ? total / units : 0));
  d.groups = span <= total / groups + kScale * kDealCost
                 ? 0
                 : max(1u, min(static_cast<uint32_t>(groups), total / (kScale * kLeastShare)));
  return d;
}

// The kernel's first argument, read again from its place: what a workgroup derives from it for one
// unit is not kept in registers for the next (that cost spills in the loop over tokens).
template <bool TREE>
__device__ __forceinline__ ProblemOf<TREE> argument() {
  auto at = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(at));
  ProblemOf<TREE> p;
  __builtin_memcpy(&p, reinterpret_cast<const __attribute__((address_space(4))) ProblemOf<TREE>*>(at), sizeof(p));
  return p;
}

// The workgroup's number: a grid of more workgroups than one dimension holds has a second one, and then
// up to as many workgroups to spare.
__device__ __forceinline__ uint32_t group_number() { return blockIdx.y * gridDim.x + blockIdx.x; }

// A workgroup's units or parts, one after the other.  `groups`: runs of a deal (DEALT).
template <int THREADS, bool DEALT, bool TREE, bool MIXED = false>
struct Walk {
  uint32_t g, x, end;
  bool dealt;

  __device__ __forceinline__ Walk(const AttnProblem& p, int block_rows, int row_blocks, int splits,
                                  int groups, uint32_t* first) {
    x = 0;
    end = 1;
    dealt = false;
    if constexpr (DEALT) {
      const Deal<MIXED> d = deal<THREADS, TREE, MIXED>(p, block_rows, row_blocks, splits, groups, first);
      RunStart* const starts = reinterpret_cast<RunStart*>(p.parts);
      if (blockIdx.x == 0 && threadIdx.x == 0) starts[0] = RunStart{0, 0, 0, d.groups};
      if (d.groups == 0) {
        end = blockIdx.x < d.entries * d.heads * splits;
        return;
      }
      dealt = true;
      // Neighbouring runs (of one head's tokens) to one XCD.
      const uint32_t each = (d.groups + 7) / 8;
      g = blockIdx.x % 8 * each + blockIdx.x / 8;
      x = end = 0;
      if (blockIdx.x / 8 < each && g < d.groups) {
        const RunStart s = d.start(g);
        if (g > 0 && threadIdx.x == 0) starts[g] = s;
        x = s.at;
        end = d.start(g + 1).at;
      }
    }
  }
  // The next one and where its part goes (-1: it is whole); false: none is left.
  __device__ __forceinline__ bool next(const AttnProblem& p, int block_rows, int row_blocks, int splits,
                                       const uint32_t* first, Work* w, int* slot) {
    *slot = -1;
    if (x >= end) return false;
    if (!DEALT || !dealt) {
      x = end;
      const uint32_t id = DEALT ? blockIdx.x : group_number();       // a deal's grid has one dimension
      const uint32_t heads = p.cache.heads, h = id % heads, r = id / heads, b = r % p.batch;
      if (!DEALT && r / p.batch / splits >= static_cast<uint32_t>(row_blocks)) return false;
      const int part = r / p.batch % splits, blk = row_blocks - 1 - static_cast<int>(r / p.batch / splits);
      *w = unit_of<TREE>(p, block_rows, h, b, blk);
      const int parts = parts_of(w->tiles, splits);
      if (!w->any || part >= parts) return false;
      if (parts == 1) return true;
      *slot = ((blk * p.batch + b) * heads + h) * splits + part;
      const int32_t tile0 = static_cast<int32_t>(static_cast<int64_t>(w->tiles) * part / parts);
      w->tiles = static_cast<int32_t>(static_cast<int64_t>(w->tiles) * (part + 1) / parts) - tile0;
      w->t_begin += tile0 * kTok;
      return true;
    }
    constexpr uint32_t kScale = Deal<MIXED>::kScale;
    const Deal<MIXED> d = {first, static_cast<uint32_t>(p.batch * row_blocks), 0, 0};
    const uint32_t per = d.per_head(), head = x / per, base = head * per, e = d.entry(x - base);
    *w = unit_of<TREE>(p, block_rows, head, e / row_blocks, e % row_blocks);
    const uint32_t s = base + d.slot_of(e), stop = base + d.slot_of(e + 1), upto = min(end, stop);
    const uint32_t each = tile_slots<MIXED>(*w, block_rows);   // a tile that a run ends inside of is the next run's
    const uint32_t tile0 = x > s ? (x - s - kScale * kUnitSlots) / each : 0;
    if (x > s || upto < stop) *slot = 2 * g + (x == s);
    w->tiles = (upto - s - kScale * kUnitSlots) / each - tile0;
    w->t_begin += tile0 * kTok;
    x = upto;
    return true;
  }
};

// A lane's query row: lanes c and c + 32 of a wavefront share row r0 + 32 tile + c.
struct Row {
  bool live;
  int32_t tok, hg, lo, hi;                // query, grouped head, the keys it sees
};

template <bool TREE>
__device__ __forceinline__ Row row_of(const ProblemOf<TREE>& p, const Work& w, int tile,
                                      uint32_t thread = threadIdx.x) {
  Row r;
  const int32_t i = w.r0 + tile * 32 + (thread & 31);
  r.live = i < w.rows;
  r.tok = r.live ? i / p.group : 0;
  r.hg = r.live ? i - r.tok * p.group : 0;
  r.hi = r.live && p.causal ? w.first + r.tok + 1 : w.len;
  if constexpr (TREE) r.lo = p.window > 0 ? tree_window_start(p, w.q0 + r.tok, w.first, w.len) : 0;
  else r.lo = r.live && p.window > 0 ? window_start(w.first + r.tok, p.window) : 0;
  return r;
}

// Its values, as B operands.
template <int KS>
__device__ __forceinline__ void load_query(const AttnProblem& p, const Work& w, const Row& r,
                                           bf16x8 (&qf)[KS], uint32_t thread = threadIdx.x) {
  const uint16_t* row = p.q.p + static_cast<int64_t>(w.q0 + r.tok) * p.q.token_stride +
                        static_cast<int64_t>(w.h * p.group + r.hg) * p.q.head_stride +
                        8 * ((thread & 63) >> 5);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 x = r.live ? *reinterpret_cast<const uint4*>(row + 16 * s) : make_uint4(0, 0, 0, 0);
    x.x ^= p.flip; x.y ^= p.flip; x.z ^= p.flip; x.w ^= p.flip;
    qf[s] = __builtin_bit_cast(bf16x8, x);
  }
}

// A decoding thread's undecoded share of 64 tokens.  Of keys: a quarter of a token's codes (x[0 ..
// D / 32)) and the word that holds their scale byte(s) (x[15]).  Of values: the words of 8 tokens that
// hold its D / 32 codes (x[0 .. 8)), and those that hold their scale bytes (from x[8]: of the first
// four tokens, from x[12]: of the others).  Whole words: the widening of a loaded byte or half waits
// for the load at once, where these wait until the next tile needs them.
struct Raw {
  uint32_t x[16];
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

  __device__ __forceinline__ Decoder(const AttnProblem& p_, const Work& w, int sub_, uint32_t thread = threadIdx.x)
      : p(p_), sub(sub_) {
    const int lane = thread & 63;
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
  __device__ __forceinline__ void load_keys(Raw& w, Place at) const {
    const uint8_t* kp = kbase + (at.id * p.cache.code_page + at.off * (D / 2)) +
                        (k16 * (D / 2) + kq * (D / 8));
    const uint8_t* sp = ksbase + (at.id * p.cache.scale_page + at.off * (D / 32)) +
                        (D == 64 ? (k16 >> 1) * 4 : D == 128 ? k16 * 4 : k16 * 8 + (kq >> 1) * 4);
    if constexpr (D == 64) {
      const uint2 t = *reinterpret_cast<const uint2*>(kp);
      w.x[0] = t.x; w.x[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 t = *reinterpret_cast<const uint4*>(kp + 16 * i);
        w.x[4 * i] = t.x; w.x[4 * i + 1] = t.y; w.x[4 * i + 2] = t.z; w.x[4 * i + 3] = t.w;
      }
    }
    w.x[15] = *reinterpret_cast<const uint32_t*>(sp);
  }
  __device__ __forceinline__ void load_values(Raw& w, Place at) const {
    const uint8_t* vp = vbase + (at.id * p.cache.code_page + at.off * (D / 2)) +
                        (vh * 4 * (D / 2) + (vc * (EPI / 2) & ~3));
    const uint8_t* sp = vsbase + (at.id * p.cache.scale_page + at.off * (D / 32)) + vh * 4 * (D / 32);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w.x[i] = *reinterpret_cast<const uint32_t*>(vp + ((i >> 2) * 8 + (i & 3)) * (D / 2));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* a = sp + i * 8 * (D / 32);
      if constexpr (D == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(a);
        w.x[8 + 4 * i] = x.x; w.x[9 + 4 * i] = x.y;
      } else if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(a);
        w.x[8 + 4 * i] = x.x; w.x[9 + 4 * i] = x.y; w.x[10 + 4 * i] = x.z; w.x[11 + 4 * i] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w.x[8 + 4 * i + e] = *reinterpret_cast<const uint32_t*>(a + e * 8 + (vc >> 4) * 4);
      }
    }
  }
  // The same for what lies before the block's oldest window, of a run's first tile alone: here, as a test
  // of every tile in decode_values takes 25 us more of a chunk's 495 (heads of 256).
  __device__ __forceinline__ void load_first_values(Raw& w, const Work& u) const {
    load_values(w, place(u.t_begin));
    if (u.t_begin >= u.low) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (u.t_begin + sub * 16 + (i >> 2) * 8 + vh * 4 + (i & 3) >= u.low) continue;
      uint32_t& x = w.x[8 + (D == 64 ? 4 * (i >> 2) + ((i & 3) >> 1) : i)];
      const uint32_t mine = D == 64 ? 0xFFFFu << (16 * (i & 1)) : ~0u;      // heads of 64: two tokens a word
      x = (x & ~mine) | (kScalesOfOne & mine);
    }
  }
  // Into [32-token half][k step][lane].
  __device__ __forceinline__ void decode_keys(const Raw& w, uint4* dst) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float sc = scale_of_byte(w.x[15], D == 256 && i >= 4 ? turn_k + 8 : turn_k);
      const int word = kq * (D / 32) + i;               // 8 codes: k step word / 2, half word % 2
      dst[((sub >> 1) * KS + (word >> 1)) * 64 + (word & 1) * 32 + (sub & 1) * 16 + k16] =
          decode8(w.x[i], sc);
    }
  }
  // Of the tile from t0, into [16-token step][head value % DT][lane].
  __device__ __forceinline__ void decode_values(const Raw& w, int32_t t0, uint4* dst) const {
    const uint32_t drop = D == 64 ? 8 * (vc & 3) : D == 128 ? 16 * (vc & 1) : 0;   // the lane's codes lowest
    const uint32_t turn = 9 + 8 * (D == 64 ? vc >> 4 : D == 128 ? vc >> 3 : (vc >> 2) & 3);
    float sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = scale_of_byte(w.x[8 + (D == 64 ? 4 * (i >> 2) + ((i & 3) >> 1) : i)],
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
      for (int i = 0; i < 8; ++i) pr[i] = decode2(D == 256 ? w.x[i] : w.x[i] >> drop, sc[i], a);
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
__device__ __forceinline__ void scores(v16f& s, const uint4* keys, const bf16x8 (&qf)[KS], int j0, int j1,
                                       uint32_t thread = threadIdx.x) {
#pragma unroll
  for (int j = j0; j < j1; ++j)
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(bf16x8, keys[j * 64 + (thread & 63)]), qf[j], j == 0 ? v16f(0.f) : s, 0, 0, 0);
}

// Orders what follows in a block of code: N reads from LDS, or N matrix products.
constexpr int kLdsReads = 0x100, kProducts = 0x8;
template <int KIND, int N>
__device__ __forceinline__ void then() { __builtin_amdgcn_sched_group_barrier(KIND, N, 0); }

// Masks the lane's 16 scores of the 32 tokens from t0.  A tree's window takes of what lies before the
// tree; of the tree the mask alone does.
template <bool TREE>
__device__ __forceinline__ void mask(v16f& s, const ProblemOf<TREE>& p, const Work& w, const Row& r, int32_t t0,
                                     uint32_t thread = threadIdx.x) {
  const int32_t half = 4 * ((thread & 63) >> 5), at = t0 + half;
  uint32_t bits = ~0u;
  if constexpr (TREE) bits = tree_bits(p, w.q0 + r.tok, t0 - w.first) >> half;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int32_t o = (e & 3) + 8 * (e >> 2), key = at + o;
    bool hidden = key >= r.hi;
    if constexpr (TREE) hidden = hidden || !(bits >> o & 1) || (key < w.first && key < r.lo);
    else hidden = hidden || key < r.lo;
    if (hidden) s[e] = -kInf;
    if (e % 8 == 7) __builtin_amdgcn_sched_barrier(0);
  }
}

// The weights of 8 of the lane's scores as a B operand; their sum is added to l.  bf16 is the matrix
// instruction's type, the one that holds every decoded value exactly; the sum adds the weights unrounded,
// as the log-sum-exp needs them.  (Outputs are off from 64 bits by 0.0017 of their size, their own
// rounding; so they are with weights in fp32.)
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

// Writes N of the lane's sums of its row's head values DT (i % 4 + 8 (i / 4) + 4 h) + d0 + d, d < N,
// for i in [4 q0, 4 q1), h the lane's half.
template <int DT, int N, int Q0, int Q1>
__device__ __forceinline__ void write_values(const AttnProblem& p, const Work& w, const Row& r,
                                             const v4f (&acc)[N][Q1 - Q0], float l, int d0) {
  const int hh = (threadIdx.x & 63) >> 5;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* dst = p.out.p + static_cast<int64_t>(w.q0 + r.tok) * p.out.token_stride +
                  static_cast<int64_t>(w.h * p.group + r.hg) * p.out.head_stride + d0;
#pragma unroll
  for (int i = 4 * Q0; i < 4 * Q1; ++i) {
    uint32_t x[N / 2];
#pragma unroll
    for (int d = 0; d < N / 2; ++d)
      x[d] = pack_bf16(acc[2 * d][i / 4 - Q0][i % 4] * inv, acc[2 * d + 1][i / 4 - Q0][i % 4] * inv);
    uint16_t* at = dst + DT * ((i & 3) + 8 * (i >> 2) + 4 * hh);
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(at) = x[0];
    else *reinterpret_cast<uint2*>(at) = make_uint2(x[0], x[1]);
  }
}

__device__ __forceinline__ void write_lse(const AttnProblem& p, const Work& w, const Row& r, float m, float l) {
  if (p.lse && (threadIdx.x & 32) == 0)
    p.lse[static_cast<int64_t>(w.q0 + r.tok) * p.group * p.cache.heads + w.h * p.group + r.hg] =
        l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Floats of one part's partial result: a thread's N sums of 16, as 4 N units of 4, unit by unit, a
// thread after the other; then m, then l, of each row (a row is two threads').
constexpr int64_t part_floats(int threads, int n) { return static_cast<int64_t>(threads) * (16 * n + 1); }

// The rows are written, or a part of them left for the join.
template <int DT, int THREADS, bool TREE, int N>
__device__ __forceinline__ void finish(const AttnProblem& p, const Work& w, const Row& r, int slot,
                                       const v16f (&acc)[N], float m, float l, int d0) {
  if (TREE && !r.live) return;             // what the join does not read
  if (slot < 0) {
    if (!r.live) return;
    v4f x[N][4];
#pragma unroll
    for (int d = 0; d < N; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[d][i / 4][i % 4] = acc[d][i];
    write_values<DT, N, 0, 4>(p, w, r, x, l, d0);
    if (d0 == 0) write_lse(p, w, r, m, l);
    return;
  }
  float* const part = p.parts + kStartFloats + slot * part_floats(THREADS, N);
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(part + ((d * 4 + i) * THREADS + threadIdx.x) * 4) =
          make_float4(acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]);
  if ((threadIdx.x & 32) == 0) {
    const int row = threadIdx.x / 64 * 32 + (threadIdx.x & 31);
    part[N * 16 * THREADS + row] = m;
    part[N * 16 * THREADS + THREADS / 2 + row] = l;
  }
}

// Joins a unit's parts, in their order, whole rows at a time; a workgroup takes one of a thread's
// four lots of 4 for two of its N sums.  A launch of its own: the parts of one unit would be joined
// by one workgroup otherwise (128 rows of 60000 keys in 64 parts: 110 us, 63 us so).
// HALVES: 2 where two wavefronts share rows (attn_wide_kernel).
template <int DT, int THREADS, int N, int HALVES, bool TREE>
__global__ __launch_bounds__(THREADS) void attn_join_kernel(const ProblemOf<TREE> p, int row_blocks, int splits,
                                                            int groups) {
  constexpr int kSlices = 4 * N / 2, kTiles = THREADS / 64 / HALVES;
  const RunStart* const starts = reinterpret_cast<const RunStart*>(p.parts);
  const uint32_t slice = blockIdx.x % kSlices, lane = threadIdx.x & 63, runs = groups ? starts[0].unit : 0;
  uint32_t left = blockIdx.x / kSlices;
  // Part k lies at slot base + step k, the first at base + lead.
  int parts = 0, base, lead, step;
  Work w;
  if (runs == 0) {                           // the units as they are
    const uint32_t heads = p.cache.heads;
    if (splits == 1 || left >= heads * p.batch * row_blocks) return;
    w = unit_of<TREE>(p, 32 * kTiles, left % heads, left / heads % p.batch, left / heads / p.batch);
    parts = parts_of(w.tiles, splits);
    if (!w.any || parts == 1) return;
    base = left * splits;
    lead = 0;
    step = 1;
  } else {
    uint32_t g0 = 0, unit = ~0u;
    if constexpr (TREE) {
      // Those that runs begin inside of, each by the workgroups of the first of these runs: the part of the run
      // before it, and theirs.  (A run's neighbours are all it looks at: 41 sequences of up to 8192 tokens, 84
      // rows of 8 heads: 8 us; 14 where every workgroup counted the units before its own.)
      g0 = left + 1;
      if (g0 >= runs) return;
      for (uint32_t at = g0 - 1;; at += 64) {            // lane i: run at + i
        const uint32_t g = at + lane;
        const RunStart s = starts[min(g, runs - 1)];
        const bool in = g > 0 && g < runs && s.at > s.unit_first && s.at < s.unit_end;
        const uint32_t its = in ? s.unit : ~0u;
        uint64_t same;
        if (at < g0) {
          unit = __builtin_amdgcn_readlane(its, 1);
          if (unit == ~0u || static_cast<uint32_t>(__builtin_amdgcn_readlane(its, 0)) == unit) return;
          same = __ballot(its == unit) | 1u;             // lane 0: the part that begins the unit
        } else {
          same = __ballot(its == unit);
        }
        const int n = ~same ? __builtin_ctzll(~same) : 64;
        parts += n;
        if (n < 64) break;
      }
    } else {
      // Those that runs begin inside of, the i-th by the workgroups i of each slice: the part of the
      // workgroup before the first of these runs, and theirs.
      constexpr int kChunks = kMostGroups / 64;
      RunStart all[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) all[i] = starts[i * 64 + lane];
      uint32_t before = ~0u;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint32_t g = i * 64 + lane;
        const bool in = g > 0 && g < runs && all[i].at > all[i].unit_first && all[i].at < all[i].unit_end;
        const uint32_t its = in ? all[i].unit : ~0u;
        uint32_t prev = __shfl_up(its, 1, 64);
        if (lane == 0) prev = before;
        before = __builtin_amdgcn_readlane(its, 63);
        if (parts == 0) {
          uint64_t firsts = __ballot(in && prev != its);
          const uint32_t n = __builtin_popcountll(firsts);
          if (left < n) {
            for (; left > 0; --left) firsts &= firsts - 1;
            g0 = i * 64 + __builtin_ctzll(firsts);
            unit = __builtin_amdgcn_readlane(its, g0 & 63);
            parts = 1;
          } else {
            left -= n;
          }
        }
        if (parts > 0) parts += __builtin_popcountll(__ballot(its == unit));
      }
      if (parts == 0) return;
    }
    const uint32_t entries = p.batch * row_blocks, h = unit / entries, e = unit - h * entries;
    w = unit_of<TREE>(p, 32 * kTiles, h, e / row_blocks, e % row_blocks);
    base = 2 * (g0 - 1);
    lead = 1;
    step = 2;
  }
  const int wave = threadIdx.x / 64, row = wave * 32 + (threadIdx.x & 31);
  if constexpr (TREE)                      // a block of few rows: others leave nothing
    if (!row_of<TREE>(p, w, wave % kTiles).live) return;
  const int q = slice % 4, d = slice / 4 * 2;
  constexpr int64_t kPart = part_floats(THREADS, N);
  const float* src = p.parts + kStartFloats + base * kPart;
  float m = -kInf, l = 0.f;
  v4f acc[2][1] = {{v4f(0.f)}, {v4f(0.f)}};
  constexpr int kBatch = 8;
  for (int at = 0; at < parts; at += kBatch) {
    float pm[kBatch], pl[kBatch];
    v4f x[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {               // past the last part: that part, with no weight
      const int part = min(at + i, parts - 1);
      const float* from = src + (part == 0 ? lead : step * part) * kPart;
      pm[i] = at + i < parts ? from[N * 16 * THREADS + row] : -kInf;
      pl[i] = from[N * 16 * THREADS + THREADS / 2 + row];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        x[i][c] = *reinterpret_cast<const v4f*>(from + (((d + c) * 4 + q) * THREADS + threadIdx.x) * 4);
    }
    float now = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) now = fmaxf(now, pm[i]);
    const float fo = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
    m = now;
    l *= fo;
    acc[0][0] *= fo;
    acc[1][0] *= fo;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= parts) break;
      const float f = pm[i] == -kInf ? 0.f : __builtin_amdgcn_exp2f(pm[i] - now);
      l += pl[i] * f;
      acc[0][0] += x[i][0] * f;
      acc[1][0] += x[i][1] * f;
    }
  }
  const Row r = row_of<TREE>(p, w, wave % kTiles);
  if (!r.live) return;
  const int d0 = wave / kTiles * N + d;
  if (q == 0) write_values<DT, 2, 0, 1>(p, w, r, acc, l, d0);
  if (q == 1) write_values<DT, 2, 1, 2>(p, w, r, acc, l, d0);
  if (q == 2) write_values<DT, 2, 2, 3>(p, w, r, acc, l, d0);
  if (q == 3) write_values<DT, 2, 3, 4>(p, w, r, acc, l, d0);
  if (q == 0 && d0 == 0) write_lse(p, w, r, m, l);
}

// What two wavefronts that share rows have of them, put together in the first one's registers: the second
// leaves its share in LDS, half of the sums at a time (`room` holds that of every pair; nobody else uses it).
template <int DT, int PAIRS>
__device__ __forceinline__ void join_pair(bool second, int pair, v16f (&acc)[DT], float& m, float& l, float* room,
                                          float (*stats)[2][64]) {
  const int lane = threadIdx.x & 63;
  if (second) {
    stats[pair][0][lane] = m;
    stats[pair][1][lane] = l;
  }
  float mine = 1.f, its = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4* const at = reinterpret_cast<float4*>(room) + pair * (DT / 2 * 4 * 64) + lane;
    if (second) {
#pragma unroll
      for (int d = 0; d < DT / 2; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          at[(d * 4 + i) * 64] = make_float4(acc[k * (DT / 2) + d][4 * i], acc[k * (DT / 2) + d][4 * i + 1],
                                             acc[k * (DT / 2) + d][4 * i + 2], acc[k * (DT / 2) + d][4 * i + 3]);
    }
    lds_barrier();
    if (!second) {
      if (k == 0) {
        const float om = stats[pair][0][lane], now = fmaxf(m, om);
        mine = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
        its = om == -kInf ? 0.f : __builtin_amdgcn_exp2f(om - now);
        m = now;
        l = l * mine + stats[pair][1][lane] * its;
      }
#pragma unroll
      for (int d = 0; d < DT / 2; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = at[(d * 4 + i) * 64];
          v16f& a = acc[k * (DT / 2) + d];
          a[4 * i] = a[4 * i] * mine + x.x * its;
          a[4 * i + 1] = a[4 * i + 1] * mine + x.y * its;
          a[4 * i + 2] = a[4 * i + 2] * mine + x.z * its;
          a[4 * i + 3] = a[4 * i + 3] * mine + x.w * its;
        }
    }
    lds_barrier();
  }
}

// NW wavefronts.  Of 8, the first four decode keys and the others values (one of each to a SIMD); of 4,
// all decode both.  Each has 32 query rows and all 64 tokens of a tile (SPLIT 1); or two share 32 rows,
// with 32 tokens each (SPLIT 2), so that few rows keep every wavefront at work; or each unit in the way that
// its rows ask for (SPLIT kMixed).  The two ways' code is kept apart: what both derive from the argument and, for
// heads of 128, from the lane's number is derived twice, as kept for both it took registers from the loops (41 x
// 70 rows of up to 8192 tokens: 166 us, 129 so).
template <int D, int NW, bool DEALT, bool TREE, int SPLIT>
__global__ __launch_bounds__(64 * NW, 2) void attn_many_kernel(const ProblemOf<TREE> args, int row_blocks,
                                                               int splits, int groups) {
  constexpr int KS = D / 16, DT = D / 32, kThreads = 64 * NW;
  constexpr bool kMixed = SPLIT == AttnPlan::kMixed;
  constexpr int kBlock = SPLIT == 2 ? 16 * NW : 32 * NW;      // rows
  __shared__ uint4 kl[2][2 * KS * 64];
  __shared__ uint4 vl[2][4 * DT * 64];
  __shared__ float stats[SPLIT != 1 ? NW / 2 : 1][2][64];
  __shared__ uint32_t first[DEALT ? kMostEntries + 3 : 1];
  const int the_lane = threadIdx.x & 63;
  const int the_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Walk<kThreads, DEALT, TREE, kMixed> walk(args, kBlock, row_blocks, splits, groups, first);
  for (;;) {
    const ProblemOf<TREE> p = DEALT ? argument<TREE>() : args;
    Work w;
    int slot;
    if (!walk.next(p, kBlock, row_blocks, splits, first, &w, &slot)) return;
    auto attend = [&](auto sharing, const ProblemOf<TREE>& p) __attribute__((always_inline)) {
      constexpr int kShare = decltype(sharing)::value;
      constexpr int kTiles = NW / kShare, kHalves = 2 / kShare;   // of rows; of a tile's tokens, a wavefront's
      const uint32_t thread = kMixed && D == 128 ? again(threadIdx.x) : threadIdx.x;
      const int lane = kMixed ? thread & 63 : the_lane;
      const int wave = kMixed ? __builtin_amdgcn_readfirstlane(thread >> 6) : the_wave;
      const int rows_of = kShare == 1 ? wave : wave % kTiles, half = kShare == 1 ? 0 : wave / kTiles;
      const bool keys = NW == 4 || wave < 4, values = NW == 4 || wave >= 4;
      const Row row = row_of<TREE>(p, w, rows_of, thread);
      bf16x8 qf[KS];
      load_query(p, w, row, qf, thread);
      const Decoder<D> dec(p, w, wave & 3, thread);

      v16f acc[DT];
      float m = -kInf, l = 0.f;
      float slack = kSlack;                    // what a row's maximum may rise by before it is moved
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] = v16f(0.f);
      // A wavefront that decodes one of the two holds one share.
      Raw rk, rv_own;
      Raw& rv = NW == 4 ? rv_own : rk;
      Place next_k, next_v_own;
      Place& next_v = NW == 4 ? next_v_own : next_k;

      // Tile i: its scores `s` are there; while its weights and products are made, the next tile's scores
      // are (into `sn`), the keys after those and the next tile's values are decoded, and the ones after
      // them loaded.  One barrier a tile: K(i + 2) goes where K(i) was, V(i + 1) where V(i - 1) was, both
      // read by every wavefront before the last barrier.
      auto step = [&](v16f (&s)[kHalves], v16f (&sn)[kHalves], auto odd, auto final, int32_t i) {
        constexpr int B = decltype(odd)::value;
        constexpr bool LAST = decltype(final)::value;
        const int32_t t0 = w.t_begin + i * kTok;
        if (t0 + kTok > w.full_hi || t0 < w.full_lo) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) mask<TREE>(s[h], p, w, row, t0 + (half + h) * 32, thread);
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 16 * kHalves; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
        top = max_halves(top) * p.scale_log2;
        float scale = p.scale_log2;
        if (__any(top > m + slack)) {
          const float now = fmaxf(m, top);
          const float f = m == -kInf ? 0.f : __builtin_amdgcn_exp2f(m - now);
          m = now;
          l *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[d][e] *= f;
          slack = kSlack;
          if (large_scores(now)) {
#pragma unroll
            for (int e = 0; e < 16 * kHalves; ++e) s[e >> 4][e & 15] = rounded_product(s[e >> 4][e & 15], scale);
            scale = 1.f;
            slack = -kInf;
          }
        }
        const float sub = m == -kInf ? 0.f : m;
#pragma unroll
        for (int q = 0; q < 2 * kHalves; ++q) {  // 16 tokens each
          const bf16x8 pf = weights(s[q >> 1], 8 * (q & 1), scale, sub, l);
#pragma unroll
          for (int d = 0; d < DT; ++d)
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, vl[B][((2 * half + q) * DT + d) * 64 + lane]), pf, acc[d], 0, 0, 0);
          if constexpr (!LAST)
            scores(sn[q >> 1], kl[B ^ 1] + (half + (q >> 1)) * KS * 64, qf, (q & 1) * (KS / 2),
                   ((q & 1) + 1) * (KS / 2), thread);
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
        v16f sa[kHalves], sb[kHalves];
        if (keys) {
          dec.load_keys(rk, dec.place(w.t_begin));
          dec.decode_keys(rk, kl[0]);
          dec.load_keys(rk, dec.place(w.t_begin + kTok));
          dec.decode_keys(rk, kl[1]);
          dec.load_keys(rk, dec.place(w.t_begin + 2 * kTok));
          next_k = dec.place(w.t_begin + 3 * kTok);
        }
        if (values) {
          dec.load_first_values(rv, w);
          dec.decode_values(rv, w.t_begin, vl[0]);
          dec.load_values(rv, dec.place(w.t_begin + kTok));
          next_v = dec.place(w.t_begin + 2 * kTok);
        }
        lds_barrier();
#pragma unroll
        for (int h = 0; h < kHalves; ++h) scores(sa[h], kl[0] + (half + h) * KS * 64, qf, 0, KS, thread);
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

      if constexpr (kShare == 2) {
        lds_barrier();                         // the last tile's values are read
        join_pair<DT, kTiles>(half == 1, rows_of, acc, m, l, reinterpret_cast<float*>(vl), stats);
      }
      if (kShare == 1 || half == 0) finish<DT, 2 * kBlock, TREE>(p, w, row, slot, acc, m, l, 0);
    };
    if constexpr (!kMixed) attend(IntC<SPLIT>{}, p);
    else if (!shares(w, kBlock)) attend(IntC<1>{}, argument<TREE>());
    else attend(IntC<2>{}, argument<TREE>());
    if constexpr (!DEALT) return;
    lds_barrier();                           // before the next one's keys and values
  }
}

// Heads of 256: eight wavefronts, the first four (half 0) and the last four (half 1) on the same four
// tiles of 32 rows.  Half h scores tokens [32 h, 32 h + 32) of a tile and sums head values
// 8 j + 4 h + (0..3).  Two barriers a tile:
//   first   half h's weights of tile i (from the scores of both halves' larger maximum) go to LDS; the
//           scores of tile i + 1 and their maxima are made; half 1 decodes the values of tile i
//   second  the products of tile i's weights and values; half 0 decodes the keys of tile i + 2
// so that each of the matrix runs has the other side's decoding beside it, and one buffer of keys,
// values and weights is enough.
template <bool DEALT, bool TREE>
__global__ __launch_bounds__(512, 2) void attn_wide_kernel(const ProblemOf<TREE> args, int row_blocks, int splits,
                                                           int groups) {
  constexpr int D = 256, KS = D / 16, DT = D / 32, N = DT / 2, kThreads = 512;
  __shared__ uint4 kl[2 * KS * 64];
  __shared__ uint4 vl[4 * DT * 64];
  __shared__ uint4 pl[4][4 * 64];           // [row tile][16-token step][lane]
  __shared__ float tops[2][4][2][32];       // [tile parity][row tile][half][row]
  __shared__ uint32_t first[DEALT ? kMostEntries + 3 : 1];
  const int lane = threadIdx.x & 63, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = wave & 3, half = wave >> 2;
  Walk<kThreads, DEALT, TREE> walk(args, 128, row_blocks, splits, groups, first);
  for (;;) {
    const ProblemOf<TREE> p = DEALT ? argument<TREE>() : args;
    Work w;
    int slot;
    if (!walk.next(p, 128, row_blocks, splits, first, &w, &slot)) return;
    const Row row = row_of<TREE>(p, w, rt);
    bf16x8 qf[KS];
    load_query(p, w, row, qf);
    const Decoder<D> dec(p, w, rt);

    v16f acc[N];
    float m = -kInf, l = 0.f;
#pragma unroll
    for (int d = 0; d < N; ++d) acc[d] = v16f(0.f);
    Raw raw;
    Place next;

    // Scores of tile i, masked, and their maxima for the other half.
    auto score = [&](v16f& s, int32_t i) {
      const int32_t t0 = w.t_begin + i * kTok;
      scores(s, kl + half * KS * 64, qf, 0, KS);
      // Each operand is read a product ahead.  Left to the compiler that depends on the registers it has
      // over: where it reads into the same ones every time, a chunk takes 510 to 525 us for 495.
      then<kLdsReads, 2>();
#pragma unroll
      for (int j = 0; j < KS - 2; ++j) {
        then<kProducts, 1>();
        then<kLdsReads, 1>();
      }
      then<kProducts, 2>();
      // Multiplied at once, which large scores need (see kLargeScore): a chunk takes 488 us, 484 without.
      // (A branch for them, as in attn_many_kernel, takes 5% of a chunk in this loop, by its registers.)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = rounded_product(s[e], p.scale_log2);
      if (t0 + kTok > w.full_hi || t0 < w.full_lo) mask<TREE>(s, p, w, row, t0 + half * 32);
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
      top = max_halves(top);
      if (lane < 32) tops[i & 1][rt][half][c] = top;
    };
    auto step = [&](v16f& s, v16f& sn, auto final, int32_t i) {
      constexpr bool LAST = decltype(final)::value;
      const int32_t t0 = w.t_begin + i * kTok;
      const float top = fmaxf(tops[i & 1][rt][0][c], tops[i & 1][rt][1][c]);
      if (__any(top > m + kSlack)) {            // both halves see the same maxima and move together
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
        pl[rt][(half * 2 + u) * 64 + lane] = __builtin_bit_cast(uint4, weights(s, 8 * u, 1.f, sub, l));
      if (half == 1) {
        dec.decode_values(raw, t0, vl);
        if constexpr (!LAST) {
          dec.load_values(raw, next);
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
          dec.decode_keys(raw, kl);
          dec.load_keys(raw, next);
          next = dec.place(t0 + 4 * kTok);
        }
        lds_barrier();
      }
    };

    if (w.tiles > 0) {
      v16f sa, sb;
      if (half == 0) {
        dec.load_keys(raw, dec.place(w.t_begin));
        dec.decode_keys(raw, kl);
        dec.load_keys(raw, dec.place(w.t_begin + kTok));
      } else {
        dec.load_first_values(raw, w);
        next = dec.place(w.t_begin + kTok);
      }
      lds_barrier();
      score(sa, 0);
      lds_barrier();                           // K(0) is read before K(1) overwrites it
      if (half == 0) {
        dec.decode_keys(raw, kl);
        dec.load_keys(raw, dec.place(w.t_begin + 2 * kTok));
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

    // The row's numbers are worked out again: kept through the loop, they cost it registers.
    finish<DT, kThreads, TREE>(p, w, row_of<TREE>(p, w, rt, again(threadIdx.x)), slot, acc, m, l, half * N);
    if constexpr (!DEALT) return;
    lds_barrier();                           // before the next one's keys and values
  }
}

template <int D, int NW, bool TREE, int SPLIT = 1>
hipError_t launch(const ProblemOf<TREE>& p, const AttnPlan& plan, hipStream_t stream) {
  constexpr int DT = D / 32, kThreads = D == 256 ? 512 : 64 * NW, N = D == 256 ? DT / 2 : DT;
  constexpr int kOwners = SPLIT == 2 ? kThreads / 2 : kThreads;        // threads that a part's rows are left by
  const int64_t units = static_cast<int64_t>(plan.row_blocks) * p.batch * p.cache.heads;
  const int64_t most = std::max<int64_t>(units * plan.splits, plan.groups);
  if (most > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  // A deal and the join have few workgroups.
  const int64_t rows = (most + most_groups(kThreads) - 1) / most_groups(kThreads);
  const dim3 grid(static_cast<unsigned>((most + rows - 1) / rows), static_cast<unsigned>(rows));
  auto attend = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, plan.row_blocks, plan.splits, plan.groups);
  };
  if constexpr (D == 256) {
    if (plan.groups) attend(attn_wide_kernel<true, TREE>);
    else attend(attn_wide_kernel<false, TREE>);
  } else {
    if (plan.groups) attend(attn_many_kernel<D, NW, true, TREE, SPLIT>);
    else attend(attn_many_kernel<D, NW, false, TREE, SPLIT>);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (plan.splits == 1 && plan.groups == 0)) return e;
  // The units; of a deal those that have parts (there are no more of them than units, and a run begins inside
  // of each), or for a tree the runs but the first.
  const int64_t joined = !plan.groups ? units
                         : TREE ? std::max<int64_t>(plan.splits > 1 ? units : 0, plan.groups - 1)
                                : std::min<int64_t>(units, plan.groups - 1);
  hipLaunchKernelGGL((attn_join_kernel<DT, kOwners, N, D == 256 ? 2 : 1, TREE>),
                     dim3(static_cast<unsigned>(joined * (2 * N))), dim3(kOwners), 0, stream, p,
                     plan.row_blocks, plan.splits, plan.groups);
  return hipGetLastError();
}

}  // namespace

namespace {

constexpr int64_t few_part_bytes(int head_dim, int row_tiles) {
  return int64_t{2} * 256 * few_waves(head_dim, row_tiles) * 16 * row_tiles * (head_dim + 2) * 4;
}

// Threads that the chip holds of these kernels: eight wavefronts a CU.
constexpr int64_t kChipThreads = 256 * 512;

}  // namespace

AttnPlan plan_attn(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int head_dim, bool tree) {
  AttnPlan a = {};
  const int64_t rows = max_q * (q_heads / kv_heads), units = batch * kv_heads;
  a.few = rows <= 16 * (tree ? few_tree_tiles(head_dim) : few_tiles(head_dim));
  if (a.few) {
    a.row_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    a.groups = 256 * few_waves(head_dim, a.row_tiles);
    a.part_bytes = few_part_bytes(head_dim, a.row_tiles);
    return a;
  }
  // Eight wavefronts of 32 rows share the decoding where there are rows for them; with heads of 256,
  // eight share 128 rows.
  a.waves = head_dim == 256 || rows <= 128 ? 4 : 8;
  const int64_t block_rows = 32 * a.waves;
  a.split = 1;
  // Of a tree's blocks with half of their rows or fewer two wavefronts share 32: all blocks are (up to 64 rows, heads
  // of 128), or it is looked at, unit by unit.  Without and so, heads of 128: 41 sequences of up to 84 rows and 8192
  // tokens, 118 us and 99; 16 of up to 132 rows, 100 and 79; 16 of 264 rows, 174 and 157; full blocks 113 and 112.
  // Heads of 64: 24 sequences of up to 96 rows and 8192 tokens, 81 and 70; full blocks 85 and 87, 93 and 97.
  if (tree && head_dim == 128 && rows <= 64) a.split = 2;
  else if (tree && head_dim <= 128) a.split = AttnPlan::kMixed;
  const int64_t threads = head_dim == 256 ? 512 : 64 * a.waves, owners = a.split == 2 ? threads / 2 : threads;
  const int64_t blocks = a.split == 2 ? 1 : (rows + block_rows - 1) / block_rows;
  a.row_blocks = static_cast<int>(blocks);
  const int64_t groups = kChipThreads / threads, fit = groups / (blocks * units);
  a.splits = static_cast<int>(fit < 1 ? 1 : fit > 64 ? 64 : fit);
  if (batch > 1 && blocks * units < kDealUnits * groups) a.groups = static_cast<int>(groups);
  if (a.splits > 1 || a.groups > 0)
    a.part_bytes = 4 * (kStartFloats + (a.groups ? 2 : 1) * groups * part_floats(owners, head_dim == 64 ? 2 : 4));
  return a;
}

int64_t most_part_bytes(int64_t max_q, int64_t group, int head_dim) {
  const int64_t rows = max_q * group;
  int64_t most = 0;
  for (int t = 1; t <= few_tiles(head_dim); t *= 2)
    if (t == 1 || rows > 8 * t) most = std::max(most, few_part_bytes(head_dim, t));
  // A tree's rows go with the many from fewer on than others do; pairs of wavefronts leave half of the parts.
  if (rows > 16 * few_tree_tiles(head_dim))
    most = std::max(most, 4 * (kStartFloats + (head_dim == 128 && rows <= 64 ? 1 : 2) * kChipThreads *
                                                  (16 * (head_dim == 64 ? 2 : 4) + 1)));
  return most;
}

namespace {

template <bool TREE>
hipError_t launch_any(const ProblemOf<TREE>& p, const AttnPlan& plan, hipStream_t stream) {
  constexpr int kSplit = TREE ? AttnPlan::kMixed : 1;
  const bool eight = plan.waves == 8;
  if constexpr (TREE) {
    if (plan.split == 2) return launch<128, 4, true, 2>(p, plan, stream);
  }
  if (p.cache.head_dim == 64)
    return eight ? launch<64, 8, TREE, kSplit>(p, plan, stream) : launch<64, 4, TREE, kSplit>(p, plan, stream);
  if (p.cache.head_dim == 128)
    return eight ? launch<128, 8, TREE, kSplit>(p, plan, stream) : launch<128, 4, TREE, kSplit>(p, plan, stream);
  return launch<256, 4, TREE>(p, plan, stream);
}

}  // namespace

hipError_t launch_attn_many(const AttnTreeProblem& p, const AttnPlan& plan, hipStream_t stream) {
  return p.tree ? launch_any<true>(p, plan, stream) : launch_any<false>(p, plan, stream);
}

}  // namespace mx
