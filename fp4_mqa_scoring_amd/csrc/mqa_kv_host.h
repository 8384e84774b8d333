// Host-side checks of the key-value cache operators' entry points: sizes, heads and the
// strides of caches (internal to the library).
#pragma once

#include "mqa_fp4_topk.h"
#include "mqa_host.h"
#include "mqa_kv_cache.h"
#include "mqa_kv_fp4.h"

namespace mqa {
namespace host {

// A launch's threads are counted in 32 bits: at most 2^24 - 1 workgroups of 256.
constexpr int64_t kMaxItems = (1ll << 24) - 256;
constexpr int64_t kMaxPages = 0x7FFFFFFFll / 64;
constexpr int64_t kMaxLogical = (0x7FFFFFFFll - 512) / 64;

inline int64_t align_up(int64_t x) { return (x + 255) & ~255ll; }

inline int64_t element_bytes(int32_t type) { return type == MQA_KV_E4M3 ? 1 : 2; }

inline int32_t check_heads(int64_t num_rows, int32_t H, int32_t Hkv, int32_t D) {
  if (D != 64 && D != 128 && D != 256) return MQA_ERR_UNSUPPORTED;
  if (num_rows < 0 || H < 1 || H > 65536 || Hkv < 1 || H % Hkv) return MQA_ERR_BAD_SIZE;
  if (num_rows > kMaxItems / H) return MQA_ERR_BAD_SIZE;
  return MQA_OK;
}

// Strides of one tensor of the cache, checked and in bytes. Those of one page or one head are never taken, and
// may be anything (as torch's are): 0 in their place.
inline int32_t cache_strides(const int64_t* strides, const mqa_kv_cache& c, int64_t* page, int64_t* pos, int64_t* head) {
  const int64_t bytes = element_bytes(c.type), D = c.head_dim;
  const int64_t stride[3] = {c.num_phys_pages > 1 ? strides[0] : 0, strides[1], c.num_kv_heads > 1 ? strides[2] : 0};
  for (int i = 0; i < 3; ++i) {
    if (stride[i] < 0 || stride[i] >= (1ll << 35)) return MQA_ERR_BAD_SIZE;
    if (stride[i] * bytes % 16) return MQA_ERR_MISALIGNED;
  }
  // one page's extent, and every product of a stride in the kernels, fits
  const int64_t span = 63 * stride[1] * bytes;
  if (span >= 0x7FFFFFFFll - D * bytes) return MQA_ERR_BAD_SIZE;
  if (stride[2] * bytes > (0x7FFFFFFFll - D * bytes - span) / c.num_kv_heads) return MQA_ERR_BAD_SIZE;
  *page = stride[0] * bytes;
  *pos = stride[1] * bytes;
  *head = stride[2] * bytes;
  return MQA_OK;
}

// The same of one tensor of a cache in 4 bits: `row` bytes a head, strides multiples of `unit` bytes and below 2^36
// (of scales, whose unit is their row, 2^32).
inline int32_t fp4_strides(const int64_t* strides, const mqa_kv_cache_fp4& c, int64_t row, int64_t unit, int64_t* page,
                           int64_t* pos, int64_t* head) {
  const int64_t stride[3] = {c.num_phys_pages > 1 ? strides[0] : 0, strides[1], c.num_kv_heads > 1 ? strides[2] : 0};
  for (int i = 0; i < 3; ++i) {
    if (stride[i] < 0 || stride[i] >= (unit == row ? 1ll << 32 : 1ll << 36)) return MQA_ERR_BAD_SIZE;
    if (stride[i] % unit) return MQA_ERR_MISALIGNED;
  }
  const int64_t span = 63 * stride[1];
  if (span >= 0x7FFFFFFFll - row) return MQA_ERR_BAD_SIZE;
  if (stride[2] > (0x7FFFFFFFll - row - span) / c.num_kv_heads) return MQA_ERR_BAD_SIZE;
  *page = stride[0];
  *pos = stride[1];
  *head = stride[2];
  return MQA_OK;
}

}  // namespace host
}  // namespace mqa
