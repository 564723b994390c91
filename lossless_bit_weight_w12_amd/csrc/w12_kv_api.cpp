// C-ABI host layer of the attention side of a decode step: argument validation (before any
// HIP call) and launch.
#include "w12.h"
#include "w12_check.h"
#include "w12_kv.h"

using namespace w12;

extern "C" {

w12_status w12_kv_plan(const w12_pages* p, const int32_t* len, const int32_t* req_off,
                       uint32_t n_req, uint32_t m, int32_t* kv_len, int32_t* pos,
                       int32_t* slot, void* stream) {
  if (!p || !len || !req_off || !kv_len || !p->table || !p->held || !p->ring || !p->state)
    return W12_ERR_NULL;
  if (m > 0 && (!pos || !slot)) return W12_ERR_NULL;
  if (!page_size_ok(p->page_size) || !slots_ok(p->n_pages, p->page_size) ||
      !length_ok(p->max_pages, p->page_size) || p->max_req < 1 || p->max_req > W12_MAX_REQ)
    return W12_ERR_SHAPE;
  if (n_req < 1 || n_req > p->max_req || m > W12_MAX_KV_ROWS) return W12_ERR_RANGE;
  for (const void* a : {(const void*)len, (const void*)req_off, (const void*)kv_len, (const void*)pos,
                        (const void*)slot, (const void*)p->table, (const void*)p->held,
                        (const void*)p->ring, (const void*)p->state})
    if (!aligned(a, 4)) return W12_ERR_ALIGN;
  PlanArgs a{};
  a.n_pages = p->n_pages;
  a.page_shift = log2u(p->page_size);
  a.max_pages = p->max_pages;
  a.table = p->table;
  a.held = p->held;
  a.ring = p->ring;
  a.state = p->state;
  a.len = len;
  a.req_off = req_off;
  a.n_req = n_req;
  a.m = m;
  a.kv_len = kv_len;
  a.pos = pos;
  a.slot = slot;
  return hip_status(launch_kv_plan(a, (hipStream_t)stream));
}

w12_status w12_qk_rope(const uint16_t* q, uint64_t q_stride, const uint16_t* k, uint64_t k_stride,
                       const uint16_t* v, uint64_t v_stride, uint32_t m, uint32_t n_heads,
                       const w12_kv* kv, const w12_rope* rope, const int32_t* pos,
                       const int32_t* slot, uint16_t* q_out, uint64_t q_out_stride, void* stream) {
  if (!kv || !rope) return W12_ERR_NULL;
  if (m > 0 && (!q || !k || !v || !pos || !slot || !q_out)) return W12_ERR_NULL;
  if (rope->rot_dim > 0 && !rope->inv_freq) return W12_ERR_NULL;
  const w12_status st = check_kv(kv, n_heads);
  if (st != W12_OK) return st;
  const uint32_t d = kv->head_dim;
  if (rope->rot_dim % 16 || rope->rot_dim > d) return W12_ERR_SHAPE;
  if (!stride_ok(q_stride, n_heads, d) || !stride_ok(q_out_stride, n_heads, d) ||
      !stride_ok(k_stride, kv->n_kv_heads, d) || !stride_ok(v_stride, kv->n_kv_heads, d))
    return W12_ERR_SHAPE;
  if (m > W12_MAX_KV_ROWS || (uint64_t)m * kv->n_kv_heads >= (1ull << 26)) return W12_ERR_RANGE;
  if (rope->interleaved > 1 || !(rope->eps >= 0.f) || !isfinite(rope->eps)) return W12_ERR_FORMAT;
  for (const void* a : {(const void*)q, (const void*)k, (const void*)v, (const void*)q_out,
                        (const void*)rope->q_norm, (const void*)rope->k_norm})
    if (!aligned(a, 16)) return W12_ERR_ALIGN;
  if (!aligned(pos, 4) || !aligned(slot, 4) || !aligned(rope->inv_freq, 8)) return W12_ERR_ALIGN;
  if (m == 0) return W12_OK;
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.m = m;
  a.n_heads = n_heads;
  a.n_kv_heads = kv->n_kv_heads;
  a.n_slots = kv->n_pages * kv->page_size;
  a.page_shift = log2u(kv->page_size);
  a.q_norm = rope->q_norm;
  a.k_norm = rope->k_norm;
  a.inv_freq = rope->inv_freq;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.eps = rope->eps;
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.pos = pos;
  a.slot = slot;
  a.q_out = q_out;
  a.kc = (uint8_t*)kv->k;
  a.vc = (uint8_t*)kv->v;
  return hip_status(launch_qk_rope(a, d, kv->dtype, (hipStream_t)stream));
}

w12_status w12_attn_paged(const uint16_t* q, uint64_t q_stride, uint32_t m, uint32_t n_heads,
                          const w12_kv* kv, const int32_t* table, uint32_t max_pages,
                          const int32_t* kv_len, const int32_t* req_off, uint32_t n_req,
                          float scale, uint16_t* out, uint64_t out_stride, void* ws,
                          size_t ws_bytes, void* stream) {
  if (!kv || !table || !kv_len || !req_off || !ws) return W12_ERR_NULL;
  if (m > 0 && (!q || !out)) return W12_ERR_NULL;
  const w12_status st = check_kv(kv, n_heads);
  if (st != W12_OK) return st;
  const uint32_t d = kv->head_dim;
  if (!length_ok(max_pages, kv->page_size)) return W12_ERR_SHAPE;
  if (!stride_ok(q_stride, n_heads, d) || !stride_ok(out_stride, n_heads, d)) return W12_ERR_SHAPE;
  if (n_req < 1 || n_req > W12_MAX_REQ || m > W12_MAX_KV_ROWS) return W12_ERR_RANGE;
  // Units of at least 32 tokens for tiles of at least 16 query rows, with up to 16 units of
  // overhead each: their number stays below 2^31.
  const uint64_t tokens = (uint64_t)max_pages * kv->page_size + 1024;   // <= 2^30 + 2^10
  const uint64_t qrows = (uint64_t)m * n_heads + 64ull * n_req * kv->n_kv_heads;   // < 2^31
  if (qrows * tokens >= (1ull << 40)) return W12_ERR_RANGE;
  // scores in powers of two: exp(scale q.k) = exp2(score_scale q.code)
  const float score_scale = (float)((double)scale * (double)kv->k_scale * 1.4426950408889634);
  if (!isfinite(score_scale)) return W12_ERR_FORMAT;
  if (ws_bytes < W12_ATTN_WS_BYTES) return W12_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 256) || !aligned(table, 4) ||
      !aligned(kv_len, 4) || !aligned(req_off, 4))
    return W12_ERR_ALIGN;
  if (m == 0) return W12_OK;
  AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.m = m;
  a.n_heads = n_heads;
  a.n_kv_heads = kv->n_kv_heads;
  a.group = n_heads / kv->n_kv_heads;
  a.group_inv = a.group == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / a.group);
  a.n_pages = kv->n_pages;
  a.page_shift = log2u(kv->page_size);
  a.kc = (const uint8_t*)kv->k;
  a.vc = (const uint8_t*)kv->v;
  a.table = table;
  a.max_pages = max_pages;
  a.kv_len = kv_len;
  a.req_off = req_off;
  a.n_req = n_req;
  a.score_scale = score_scale;
  a.v_scale = kv->v_scale;
  a.out = out;
  a.tickets = (uint32_t*)ws;
  a.partial = (float*)((uint8_t*)ws + 4096);
  return hip_status(launch_attn_paged(a, d, kv->dtype, (hipStream_t)stream));
}

}  // extern "C"
