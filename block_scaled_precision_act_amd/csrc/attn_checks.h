// Checks of arguments shared by the C-ABI layers of the attention and draft operators.
#pragma once

#include "../../include/mx_attention.h"
#include "attn_internal.h"
#include "mx_internal.h"

#include <initializer_list>

namespace mx {

inline constexpr int64_t kMax31 = (int64_t{1} << 31) - 1;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

// a * b <= 2^31 - 1, both non-negative
inline bool fits31(int64_t a, int64_t b) { return a == 0 || b <= kMax31 / a; }

inline int device_status() {
  DeviceInfo dev;
  if (!current_device(&dev) || !dev.gfx950) return MX_ERR_DEVICE;
  return MX_OK;
}

// Rows of `unit` elements' alignment: base and strides.
inline int rows_status(const void* p, int64_t token_stride, int64_t head_stride, int64_t unit) {
  if (token_stride < 0 || head_stride < 0) return MX_ERR_STRIDE;
  if (!p) return MX_ERR_NULL;
  if (!aligned(p, 2 * unit) || token_stride % unit != 0 || head_stride % unit != 0)
    return MX_ERR_ALIGN;
  return MX_OK;
}

// Whether blocks of `size` at i a + j b, i < n and j < m, lie on each other.
inline bool blocks_meet(int64_t n, int64_t a, int64_t m, int64_t b, int64_t size) {
  if ((n > 1 && a < size) || (m > 1 && b < size)) return true;
  if (n <= 1 || m <= 1) return false;
  // The usual layouts: all of one index within a step of the other.
  if (a <= (b - size) / (n - 1) || b <= (a - size) / (m - 1)) return false;
  if (n > m) return blocks_meet(m, b, n, a, size);
  for (int64_t i = 1; i < n; ++i) {          // the j's whose steps end around those of i
    const __int128 at = static_cast<__int128>(i) * a, j = at / b;
    if (j >= 1 && j < m && at - j * b < size) return true;
    if (j + 1 < m && (j + 1) * b - at < size) return true;
  }
  return false;
}

// An output's rows must not lie on each other.
inline int output_status(const void* p, int64_t token_stride, int64_t head_stride, int64_t tokens,
                  int64_t heads, int64_t head_dim, int64_t unit) {
  const int st = rows_status(p, token_stride, head_stride, unit);
  if (st != MX_OK) return st;
  return blocks_meet(tokens, token_stride, heads, head_stride, head_dim) ? MX_ERR_STRIDE : MX_OK;
}

inline HeadRows rows(const void* p, int64_t token_stride, int64_t head_stride) {
  return HeadRows{static_cast<uint16_t*>(const_cast<void*>(p)), token_stride, head_stride};
}

inline int cache_status(const mx_kv_cache_fp4* c) {
  if (!c) return MX_ERR_NULL;
  if (!head_dim_ok(c->head_dim) || c->kv_heads <= 0 || c->kv_heads > 65535 || c->pages < 0 ||
      c->page_size <= 0 || c->page_size % 16 != 0 || !fits31(c->page_size, c->pages))
    return MX_ERR_SHAPE;
  if (c->code_page_stride < 0 || c->code_head_stride < 0 || c->scale_page_stride < 0 ||
      c->scale_head_stride < 0)
    return MX_ERR_STRIDE;
  const int64_t code_block = c->page_size * c->head_dim / 2;
  const int64_t scale_block = c->page_size * c->head_dim / 32;
  if ((c->pages > 1 && (c->code_page_stride < code_block || c->scale_page_stride < scale_block)) ||
      (c->kv_heads > 1 && (c->code_head_stride < code_block || c->scale_head_stride < scale_block)))
    return MX_ERR_STRIDE;
  if (c->pages > 0 && (!c->k || !c->k_scale || !c->v || !c->v_scale)) return MX_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->k_scale, 16) || !aligned(c->v, 16) ||
      !aligned(c->v_scale, 16) || c->code_page_stride % 16 != 0 || c->code_head_stride % 16 != 0 ||
      c->scale_page_stride % 16 != 0 || c->scale_head_stride % 16 != 0)
    return MX_ERR_ALIGN;
  return MX_OK;
}

inline KvCache cache_of(const mx_kv_cache_fp4& c) {
  return KvCache{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.k_scale),
                     static_cast<uint8_t*>(c.v), static_cast<uint8_t*>(c.v_scale),
                     c.code_page_stride, c.code_head_stride, c.scale_page_stride,
                     c.scale_head_stride, static_cast<uint32_t>(c.pages),
                     static_cast<uint32_t>(c.kv_heads), static_cast<uint32_t>(c.page_size),
                     static_cast<int>(c.head_dim)};
}

inline int first_error(std::initializer_list<int> all) {
  for (int s : all)
    if (s != MX_OK) return s;
  return MX_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

}  // namespace mx
