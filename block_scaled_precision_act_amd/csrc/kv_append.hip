// Appending keys and values to the paged MXFP4 cache for gfx950, the key rotated on the way.
//
// For a token and head: k' = R(position) k in fp32, each product rounded and then their sum (the
// stored codes are decided by comparisons, so the arithmetic is fixed and a plain program gets the
// same bytes), then per 32 values of k' and v the MXFP4 rule of mx_quant.h from the fp32 values.
//
// Bound by HBM.  D / 8 lanes own a token and head, 16 bytes of key and of value each, so four
// neighbouring lanes own a 32-block and its largest magnitude needs two quad permutes.  A rotated
// pair's other member, half a rotation away, is read again (it is another lane's 16 bytes of the
// same row, in the L1 by then).  16384 x 8 heads of 128, with the values as stored: 32 us for 161 MB,
// 5.0 TB/s, what a large copy reaches; one token for each of 41 sequences, 12 heads: 3.3 us, two
// thirds of it the launch.
#include "attn_common.h"

#include <algorithm>

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kLargest = 0x7F400000u;    // 6 * 2^125: what the largest finite code stands for

struct Quantized {
  uint32_t codes, byte;    // 8 E2M1 codes, and the 32-block's E8M0 byte
};

// Eight fp32 of the lane, the quad's 32 values a block: the rule of quant_chunk_fp4 on fp32.
// `top`: the block's largest |value| as fp32 bits.
__device__ __forceinline__ uint32_t block_top(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  return quad_max(m);
}

__device__ __forceinline__ Quantized quantize(const float (&x)[8], uint32_t top) {
  Quantized q;
  const uint32_t ab = __float_as_uint(fmaxf(__uint_as_float(top), 1e-4f));
  q.byte = (ab >> 23) - 2u + ((ab & 0x7FFFFFu) > 0x400000u);
  const float s = __uint_as_float(q.byte << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
  q.codes = c;
  return q;
}

__device__ __forceinline__ uint4 stored_values(const Quantized& q) {
  const float s = __uint_as_float(q.byte << 23);
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q.codes, s, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q.codes, s, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q.codes, s, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q.codes, s, 3));
  return o;
}

__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

// Past the caches: the values as stored are most of what is written (16384 x 8 heads of 128: 32 us, 39
// us without).
__device__ __forceinline__ void store_stream(uint16_t* p, uint4 v) {
  __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
}

// Values are read once (keys by two lanes, where they are rotated): 34 us without, there.
__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  const v4u t = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  return make_uint4(t[0], t[1], t[2], t[3]);
}

// (a, b) -> a c + b s with both products and the sum rounded (no fused multiply-add).
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
#pragma clang fp contract(off)
  const float ac = a * c;
  const float bs = b * s;
  return ac + bs;
}

// A row's owners handle U heads of one token, all loaded before the first is used; the token's slot and
// table entries are loaded once.
template <int LR, int U>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const KvAppendProblem p, uint32_t units) {
  constexpr int D = 8 * LR, RG = kThreads / LR;
  const int j = threadIdx.x % LR;
  const uint32_t unit = blockIdx.x * RG + threadIdx.x / LR;
  if (unit >= p.tokens * units) return;   // whole rows leave together
  const uint32_t t = unit / units, h0 = (unit - t * units) * U, heads = p.cache.heads;
  const uint16_t* const kt = p.k.p + t * p.k.token_stride + h0 * p.k.head_stride;
  const uint16_t* const vt = p.v.p + t * p.v.token_stride + h0 * p.v.head_stride;
  const int rot = p.rot.positions ? p.rot.rot : 0, half = rot >> 1;
  const bool turns = 8 * j < rot, halves = turns && !p.rot.interleaved;
  // rot % 16 == 0: the lane's 8 values lie on one side of rot / 2.
  const bool upper = 8 * j >= half;
  const int partner = upper ? 8 * j - half : 8 * j + half;
  uint4 kw[U], vw[U], ow[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = h0 + u < heads ? u : 0;
    const uint16_t* row = kt + at * p.k.head_stride;
    kw[u] = *reinterpret_cast<const uint4*>(row + 8 * j);
    ow[u] = halves ? *reinterpret_cast<const uint4*>(row + partner) : make_uint4(0, 0, 0, 0);
    vw[u] = load_stream(vt + at * p.v.head_stride + 8 * j);
  }
  const int64_t slot = p.slots[t];
  bool lost = false;                      // the position is outside the table
  float cc[8], ss[8];
  if (rot) {
    const uint32_t pos = static_cast<uint32_t>(p.rot.positions[t]);
    lost = pos >= p.rot.rows;
    if (turns && !lost) {
      const int64_t at = static_cast<int64_t>(pos) * half + (p.rot.interleaved ? 4 * j : upper ? 8 * j - half : 8 * j);
      const float4 c0 = *reinterpret_cast<const float4*>(p.rot.cos + at);
      const float4 s0 = *reinterpret_cast<const float4*>(p.rot.sin + at);
      float4 c1 = c0, s1 = s0;
      if (halves) {
        c1 = *reinterpret_cast<const float4*>(p.rot.cos + at + 4);
        s1 = *reinterpret_cast<const float4*>(p.rot.sin + at + 4);
      }
      cc[0] = c0.x; cc[1] = c0.y; cc[2] = c0.z; cc[3] = c0.w;
      cc[4] = c1.x; cc[5] = c1.y; cc[6] = c1.z; cc[7] = c1.w;
      ss[0] = s0.x; ss[1] = s0.y; ss[2] = s0.z; ss[3] = s0.w;
      ss[4] = s1.x; ss[5] = s1.y; ss[6] = s1.z; ss[7] = s1.w;
    }
  }
  if (slot < 0 || slot >= static_cast<int64_t>(p.cache.pages) * p.cache.page_size) return;
  const uint32_t page = static_cast<uint32_t>(slot) / p.cache.page_size;
  const uint32_t off = static_cast<uint32_t>(slot) - page * p.cache.page_size;
  const int64_t code0 = page * p.cache.code_page + static_cast<int64_t>(off) * (D / 2) + 4 * j;
  const int64_t scale0 = page * p.cache.scale_page + static_cast<int64_t>(off) * (D / 32) + j / 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t h = h0 + u;
    if (h >= heads) break;
    float k[8], v[8];
    widen(kw[u], k);
    widen(vw[u], v);
    if (turns && !lost) {
      if (p.rot.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = k[2 * i], b = k[2 * i + 1];
          k[2 * i] = turned(a, cc[i], b, -ss[i]);
          k[2 * i + 1] = turned(b, cc[i], a, ss[i]);
        }
      } else {
        float o[8];
        widen(ow[u], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = turned(k[e], cc[e], o[e], upper ? ss[e] : -ss[e]);
      }
    }
    // A value that no finite code stands for anywhere in the token's key or value (of this head) makes
    // the whole row NaN, through the key's scales.
    const uint32_t ktop = block_top(k), vtop = block_top(v);
    const uint64_t votes = __ballot(lost || ktop > kLargest || vtop > kLargest);
    constexpr uint64_t kMine = (uint64_t{1} << LR) - 1;
    const bool bad = ((votes >> (threadIdx.x % 64 / LR * LR)) & kMine) != 0;
    Quantized qk = quantize(k, ktop), qv = quantize(v, vtop);
    if (bad) {
      qk = {0u, 255u};
      qv = {0u, 127u};
    }
    const int64_t code = code0 + h * p.cache.code_head, scale = scale0 + h * p.cache.scale_head;
    *reinterpret_cast<uint32_t*>(p.cache.k + code) = qk.codes;
    *reinterpret_cast<uint32_t*>(p.cache.v + code) = qv.codes;
    if (j % 4 == 0) {
      p.cache.ks[scale] = static_cast<uint8_t>(qk.byte);
      p.cache.vs[scale] = static_cast<uint8_t>(qv.byte);
    }
    const int64_t out = (static_cast<int64_t>(t) * heads + h) * D + 8 * j;
    const uint4 nan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    if (p.k_out) store_stream(p.k_out + out, bad ? nan : stored_values(qk));
    if (p.v_out) store_stream(p.v_out + out, bad ? nan : stored_values(qv));
  }
}

template <int LR, int U>
hipError_t launch_u(KvAppendProblem p, hipStream_t stream) {
  constexpr int64_t RG = kThreads / LR;
  const uint32_t units = (p.cache.heads + U - 1) / U, tokens = p.tokens;
  const uint32_t most = static_cast<uint32_t>(std::min<int64_t>(tokens, most_groups(kThreads) * RG / units));
  for (uint32_t t = 0; t < tokens; t += most) {      // all at once, unless a grid does not hold them
    p.tokens = std::min(most, tokens - t);
    const int64_t all = static_cast<int64_t>(p.tokens) * units;
    hipLaunchKernelGGL((kv_append_kernel<LR, U>), dim3(static_cast<unsigned>((all + RG - 1) / RG)),
                       dim3(kThreads), 0, stream, p, units);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.k.p += p.tokens * p.k.token_stride;
    p.v.p += p.tokens * p.v.token_stride;
    p.slots += p.tokens;
    if (p.rot.positions) p.rot.positions += p.tokens;
    const int64_t values = static_cast<int64_t>(p.tokens) * p.cache.heads * (8 * LR);
    if (p.k_out) p.k_out += values;
    if (p.v_out) p.v_out += values;
  }
  return hipSuccess;
}

// From this many values on a row's owners take two heads at once; below, one, as the rows then do not
// fill the chip.  Two and one: 3.1 M values 7.6 and 7.5 us, 6.1 M 11.9 and 13.2 (heads of 128; 64 and
// 256 alike).
constexpr uint64_t kManyValues = uint64_t{1} << 22;

template <int LR>
hipError_t launch(const KvAppendProblem& p, hipStream_t stream) {
  return static_cast<uint64_t>(p.tokens) * p.cache.heads * (8 * LR) >= kManyValues
             ? launch_u<LR, 2>(p, stream)
             : launch_u<LR, 1>(p, stream);
}

}  // namespace

hipError_t launch_kv_append_fp4(const KvAppendProblem& p, hipStream_t stream) {
  if (p.cache.head_dim == 64) return launch<8>(p, stream);
  if (p.cache.head_dim == 128) return launch<16>(p, stream);
  return launch<32>(p, stream);
}

}  // namespace mx
