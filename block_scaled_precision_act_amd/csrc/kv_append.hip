// Appending keys and values to the paged MXFP4 cache for gfx950, the key rotated on the way.
//
// For a token and head: k' = R(position) k in fp32, each product rounded and then their sum (the
// stored codes are decided by comparisons, so the arithmetic is fixed and a plain program gets the
// same bytes), then per 32 values of k' and v the MXFP4 rule of mx_quant.h from the fp32 values.
//
// Bound by HBM.  D / 8 lanes own a token and head, 16 bytes of key and of value each, so four
// neighbouring lanes own a 32-block and its largest magnitude needs two quad permutes.  A rotated
// pair's other member, half a rotation away, is read again (it is another lane's 16 bytes of the
// same row, in the L1 by then).
#include "attn_common.h"

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

// (a, b) -> a c + b s with both products and the sum rounded (no fused multiply-add).
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
#pragma clang fp contract(off)
  const float ac = a * c;
  const float bs = b * s;
  return ac + bs;
}

template <int LR>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const KvAppendProblem p) {
  constexpr int D = 8 * LR, RG = kThreads / LR;
  const int j = threadIdx.x % LR;
  const uint32_t total = p.tokens * p.cache.heads;
  const uint32_t row = blockIdx.x * RG + threadIdx.x / LR;
  if (row >= total) return;               // whole rows leave together
  const uint32_t t = row / p.cache.heads, h = row - t * p.cache.heads;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= static_cast<int64_t>(p.cache.pages) * p.cache.page_size) return;
  const uint16_t* krow = p.k.p + t * p.k.token_stride + h * p.k.head_stride;
  const uint16_t* vrow = p.v.p + t * p.v.token_stride + h * p.v.head_stride;
  float k[8], v[8];
  widen(*reinterpret_cast<const uint4*>(krow + 8 * j), k);
  widen(*reinterpret_cast<const uint4*>(vrow + 8 * j), v);
  bool bad = false;
  if (p.rot.positions) {
    const uint32_t pos = static_cast<uint32_t>(p.rot.positions[t]);
    bad = pos >= p.rot.rows;
    const int rot = p.rot.rot, half = rot >> 1;
    if (!bad && 8 * j < rot) {
      const float* cs = p.rot.cos + static_cast<int64_t>(pos) * half;
      const float* sn = p.rot.sin + static_cast<int64_t>(pos) * half;
      if (p.rot.interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(cs + 4 * j);
        const float4 s = *reinterpret_cast<const float4*>(sn + 4 * j);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = k[2 * i], b = k[2 * i + 1];
          k[2 * i] = turned(a, cc[i], b, -ss[i]);
          k[2 * i + 1] = turned(b, cc[i], a, ss[i]);
        }
      } else {
        // rot % 16 == 0: the lane's 8 values lie on one side of rot / 2.
        const bool upper = 8 * j >= half;
        const int at = upper ? 8 * j - half : 8 * j;
        float o[8];
        widen(*reinterpret_cast<const uint4*>(krow + (upper ? 8 * j - half : 8 * j + half)), o);
        const float4 c0 = *reinterpret_cast<const float4*>(cs + at);
        const float4 c1 = *reinterpret_cast<const float4*>(cs + at + 4);
        const float4 s0 = *reinterpret_cast<const float4*>(sn + at);
        const float4 s1 = *reinterpret_cast<const float4*>(sn + at + 4);
        const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = turned(k[e], cc[e], o[e], upper ? ss[e] : -ss[e]);
      }
    }
  }
  // A value that no finite code stands for anywhere in the token's key or value (of this head)
  // makes the whole row NaN, through the key's scales.
  const uint32_t ktop = block_top(k), vtop = block_top(v);
  const uint64_t votes = __ballot(bad || ktop > kLargest || vtop > kLargest);
  const uint64_t mine = LR == 64 ? ~uint64_t{0} : ((uint64_t{1} << LR) - 1);
  bad = ((votes >> (threadIdx.x % 64 / LR * LR)) & mine) != 0;
  Quantized qk = quantize(k, ktop), qv = quantize(v, vtop);
  uint4 ko = stored_values(qk), vo = stored_values(qv);
  if (bad) {
    qk = {0u, 255u};
    qv = {0u, 127u};
    ko = vo = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
  }
  const uint32_t page = static_cast<uint32_t>(slot) / p.cache.page_size;
  const uint32_t off = static_cast<uint32_t>(slot) - page * p.cache.page_size;
  const int64_t code = page * p.cache.code_page + h * p.cache.code_head + off * (D / 2) + 4 * j;
  const int64_t scale = page * p.cache.scale_page + h * p.cache.scale_head + off * (D / 32) + j / 4;
  *reinterpret_cast<uint32_t*>(p.cache.k + code) = qk.codes;
  *reinterpret_cast<uint32_t*>(p.cache.v + code) = qv.codes;
  if (j % 4 == 0) {
    p.cache.ks[scale] = static_cast<uint8_t>(qk.byte);
    p.cache.vs[scale] = static_cast<uint8_t>(qv.byte);
  }
  const int64_t out = static_cast<int64_t>(row) * D + 8 * j;
  if (p.k_out) *reinterpret_cast<uint4*>(p.k_out + out) = ko;
  if (p.v_out) *reinterpret_cast<uint4*>(p.v_out + out) = vo;
}

template <int LR>
hipError_t launch(const KvAppendProblem& p, hipStream_t stream) {
  constexpr int RG = kThreads / LR;
  const uint64_t rows = static_cast<uint64_t>(p.tokens) * p.cache.heads;
  hipLaunchKernelGGL((kv_append_kernel<LR>), dim3(static_cast<unsigned>((rows + RG - 1) / RG)),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_fp4(const KvAppendProblem& p, hipStream_t stream) {
  if (p.cache.head_dim == 64) return launch<8>(p, stream);
  if (p.cache.head_dim == 128) return launch<16>(p, stream);
  return launch<32>(p, stream);
}

}  // namespace mx
