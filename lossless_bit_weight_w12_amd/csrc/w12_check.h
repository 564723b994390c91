// Checks shared by the host layers of the paged cache's calls.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "w12.h"

namespace w12 {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline w12_status hip_status(hipError_t e) { return e == hipSuccess ? W12_OK : W12_ERR_HIP; }

inline bool page_size_ok(uint32_t p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }

inline bool slots_ok(uint32_t pages, uint32_t page_size) {
  return pages > 0 && (uint64_t)pages * page_size < (1ull << 31);
}

// Tokens of one request: positions and the ends of 64-token units stay below 2^31.
inline bool length_ok(uint32_t pages, uint32_t page_size) {
  return pages > 0 && (uint64_t)pages * page_size <= (1ull << 30);
}

inline uint32_t log2u(uint32_t v) {
  uint32_t s = 0;
  while ((1u << s) < v) ++s;
  return s;
}

// Geometry and type of a cache, and the query heads that read it.
inline w12_status check_kv(const w12_kv* kv, uint32_t n_heads) {
  if (!kv->k || !kv->v) return W12_ERR_NULL;
  if (!page_size_ok(kv->page_size) || !slots_ok(kv->n_pages, kv->page_size)) return W12_ERR_SHAPE;
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256) return W12_ERR_SHAPE;
  if (n_heads < 1 || n_heads > W12_MAX_HEADS || kv->n_kv_heads < 1 || n_heads % kv->n_kv_heads)
    return W12_ERR_SHAPE;
  if (kv->dtype != W12_KV_BF16 && kv->dtype != W12_KV_E4M3) return W12_ERR_FORMAT;
  if (!(kv->k_scale > 0.f) || !(kv->v_scale > 0.f) || !isfinite(kv->k_scale) || !isfinite(kv->v_scale))
    return W12_ERR_FORMAT;
  if (kv->dtype == W12_KV_BF16 && (kv->k_scale != 1.f || kv->v_scale != 1.f)) return W12_ERR_FORMAT;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return W12_ERR_ALIGN;
  return W12_OK;
}

// Rows `stride` elements apart hold `heads` contiguous heads; m rows stay in 2^62 bytes.
inline bool stride_ok(uint64_t stride, uint32_t heads, uint32_t d) {
  return stride % 8 == 0 && stride >= (uint64_t)heads * d && stride < (1ull << 40);
}

}  // namespace w12
