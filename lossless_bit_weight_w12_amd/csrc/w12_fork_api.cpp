// C-ABI host layer of several continuations of one prompt (shared pages, the attention over
// them, the choice of beams):
// argument validation (before any HIP call) and launch.
#include "w12.h"
#include "w12_attn_shared.h"
#include "w12_beam.h"
#include "w12_check.h"
#include "w12_fork.h"

using namespace w12;

namespace {

w12_status check_pages(const w12_pages* p) {
  if (!p->table || !p->held || !p->ring || !p->state) return W12_ERR_NULL;
  if (!page_size_ok(p->page_size) || !slots_ok(p->n_pages, p->page_size) ||
      !length_ok(p->max_pages, p->page_size) || p->max_req < 1 || p->max_req > W12_MAX_REQ)
    return W12_ERR_SHAPE;
  return W12_OK;
}

bool aligned4(std::initializer_list<const void*> all) {
  for (const void* a : all)
    if (!aligned(a, 4)) return false;
  return true;
}

}  // namespace

extern "C" {

w12_status w12_kv_fork(const w12_pages* p, int32_t* refs, const int32_t* parent, const int32_t* len,
                       const int32_t* req_off, uint32_t n_req, uint32_t m, int32_t* kv_len,
                       int32_t* pos, int32_t* slot, int32_t* copies, void* stream) {
  if (!p || !refs || !len || !req_off || !kv_len || !copies) return W12_ERR_NULL;
  if (m > 0 && (!pos || !slot)) return W12_ERR_NULL;
  const w12_status st = check_pages(p);
  if (st != W12_OK) return st;
  if (n_req < 1 || n_req > p->max_req || m > W12_MAX_KV_ROWS) return W12_ERR_RANGE;
  if (!aligned4({p->table, p->held, p->ring, p->state, refs, parent, len, req_off, kv_len, pos, slot}) ||
      !aligned(copies, 16))
    return W12_ERR_ALIGN;
  ForkArgs a{};
  a.n_pages = p->n_pages;
  a.page_shift = log2u(p->page_size);
  a.max_pages = p->max_pages;
  a.max_req = p->max_req;
  a.table = p->table;
  a.held = p->held;
  a.ring = p->ring;
  a.state = p->state;
  a.refs = refs;
  a.parent = parent;
  a.len = len;
  a.req_off = req_off;
  a.n_req = n_req;
  a.m = m;
  a.kv_len = kv_len;
  a.pos = pos;
  a.slot = slot;
  a.copies = copies;
  return hip_status(launch_kv_fork(a, (hipStream_t)stream));
}

w12_status w12_kv_copy(const w12_kv* layers, uint32_t n_layers, const int32_t* copies,
                       uint32_t n_copies, void* stream) {
  if (!layers || (n_copies > 0 && !copies)) return W12_ERR_NULL;
  if (n_layers < 1 || n_layers > W12_MAX_LAYERS || n_copies > W12_MAX_COPIES) return W12_ERR_RANGE;
  for (uint32_t i = 0; i < n_layers; ++i) {
    const w12_status st = check_kv(layers + i, layers[i].n_kv_heads);
    if (st != W12_OK) return st;
    const w12_kv &a = layers[0], &b = layers[i];
    if (b.n_pages != a.n_pages || b.page_size != a.page_size || b.n_kv_heads != a.n_kv_heads ||
        b.head_dim != a.head_dim || b.dtype != a.dtype)
      return W12_ERR_SHAPE;
  }
  if (!aligned(copies, 16)) return W12_ERR_ALIGN;
  if (n_copies == 0) return W12_OK;
  const uint32_t es = layers[0].dtype == W12_KV_BF16 ? 2 : 1;
  CopyArgs a{};
  a.n_pages = layers[0].n_pages;
  a.page_shift = log2u(layers[0].page_size);
  a.page_bytes = layers[0].n_kv_heads * layers[0].page_size * layers[0].head_dim * es;
  a.key_shift = log2u(layers[0].head_dim * es / 16);
  a.vec_shift = log2u(16 / es);
  a.copies = copies;
  for (uint32_t i = 0; i < n_layers; i += kCopyLayers) {
    const uint32_t here = n_layers - i < kCopyLayers ? n_layers - i : kCopyLayers;
    for (uint32_t j = 0; j < here; ++j) {
      a.k[j] = layers[i + j].k;
      a.v[j] = layers[i + j].v;
    }
    const w12_status st = hip_status(launch_kv_copy(a, n_copies, here, (hipStream_t)stream));
    if (st != W12_OK) return st;
  }
  return W12_OK;
}

w12_status w12_kv_compact(const w12_pages* p, int32_t* refs, uint32_t first, uint32_t n_clear,
                          int32_t* moves, int32_t* moved, void* stream) {
  if (!p || !refs || !moves || !moved) return W12_ERR_NULL;
  const w12_status st = check_pages(p);
  if (st != W12_OK) return st;
  if (n_clear < 1 || n_clear > p->n_pages || first > p->n_pages - n_clear) return W12_ERR_RANGE;
  if (!aligned4({p->table, p->held, p->ring, p->state, refs, moved}) || !aligned(moves, 16))
    return W12_ERR_ALIGN;
  ClearArgs a{};
  a.n_pages = p->n_pages;
  a.page_size = p->page_size;
  a.max_pages = p->max_pages;
  a.max_req = p->max_req;
  a.first = first;
  a.n_clear = n_clear;
  a.table = p->table;
  a.held = p->held;
  a.ring = p->ring;
  a.state = p->state;
  a.refs = refs;
  a.moves = moves;
  a.moved = moved;
  return hip_status(launch_kv_compact(a, (hipStream_t)stream));
}

size_t w12_attn_shared_ws_bytes(uint32_t m, uint32_t n_heads, uint32_t head_dim) {
  if (n_heads < 1 || n_heads > W12_MAX_HEADS || (uint64_t)m * n_heads > W12_MAX_SHARED_ROWS) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return (size_t)shared_bytes(m, n_heads, head_dim);
}

w12_status w12_attn_shared(const uint16_t* q, uint64_t q_stride, uint32_t m, uint32_t n_heads,
                           const w12_kv* kv, const int32_t* table, uint32_t max_pages,
                           const int32_t* kv_len, const int32_t* req_off, uint32_t n_req,
                           const int32_t* grp_off, const int32_t* grp_len, uint32_t n_grp,
                           float scale, uint16_t* out, uint64_t out_stride, void* ws,
                           size_t ws_bytes, void* stream) {
  if (!kv || !table || !kv_len || !req_off || !grp_off || !grp_len || !ws) return W12_ERR_NULL;
  if (m > 0 && (!q || !out)) return W12_ERR_NULL;
  const w12_status st = check_kv(kv, n_heads);
  if (st != W12_OK) return st;
  const uint32_t d = kv->head_dim;
  if (!length_ok(max_pages, kv->page_size)) return W12_ERR_SHAPE;
  if (!stride_ok(q_stride, n_heads, d) || !stride_ok(out_stride, n_heads, d)) return W12_ERR_SHAPE;
  if (n_req < 1 || n_req > W12_MAX_REQ || n_grp < 1 || n_grp > W12_MAX_REQ) return W12_ERR_RANGE;
  if ((uint64_t)m * n_heads > W12_MAX_SHARED_ROWS) return W12_ERR_RANGE;
  // Units of at least 32 tokens by tiles of at least 16 query rows, a place each on the lines, with
  // the items' own places: their number stays below 2^31.
  const uint64_t tokens = (uint64_t)max_pages * kv->page_size + 1024;   // <= 2^30 + 2^10
  const uint64_t qrows = (uint64_t)m * n_heads + 64ull * n_req * kv->n_kv_heads;   // < 2^30
  if (qrows * tokens >= (1ull << 38)) return W12_ERR_RANGE;
  const float score_scale = (float)((double)scale * (double)kv->k_scale * 1.4426950408889634);
  if (!isfinite(score_scale)) return W12_ERR_FORMAT;
  if (ws_bytes < shared_bytes(m, n_heads, d)) return W12_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 256)) return W12_ERR_ALIGN;
  if (!aligned4({table, kv_len, req_off, grp_off, grp_len})) return W12_ERR_ALIGN;
  if (m == 0) return W12_OK;
  SharedArgs a{};
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
  a.grp_off = grp_off;
  a.grp_len = grp_len;
  a.n_req = n_req;
  a.n_grp = n_grp;
  a.score_scale = score_scale;
  a.v_scale = kv->v_scale;
  a.out = out;
  a.ws = (uint8_t*)ws;
  return hip_status(launch_attn_shared(a, d, kv->dtype, (hipStream_t)stream));
}

size_t w12_beam_ws_bytes(uint32_t n, uint32_t vocab, uint32_t k) {
  if (n > W12_MAX_REQ || vocab < 1 || vocab > W12_MAX_VOCAB || k < 1 || k > W12_MAX_BEAM_K) return 0;
  return (size_t)beam_bytes(n, vocab, k);
}

w12_status w12_beam_select(const void* logits, uint32_t dtype, uint64_t stride, uint32_t n,
                           uint32_t vocab, const float* scores, const int32_t* grp_off,
                           uint32_t n_grp, uint32_t k, int32_t* parent, int32_t* token,
                           float* score_out, void* ws, size_t ws_bytes, void* stream) {
  if (!grp_off || !parent || !token || !score_out || !ws) return W12_ERR_NULL;
  if (n > 0 && (!logits || !scores)) return W12_ERR_NULL;
  if (vocab < 1 || vocab > W12_MAX_VOCAB || k < 1 || k > W12_MAX_BEAM_K || k > vocab) return W12_ERR_SHAPE;
  if (stride < vocab || stride >= (1ull << 40)) return W12_ERR_SHAPE;
  if (n > W12_MAX_REQ || n_grp < 1 || n_grp > W12_MAX_REQ) return W12_ERR_RANGE;
  if (dtype != W12_LOGITS_BF16 && dtype != W12_LOGITS_F32) return W12_ERR_FORMAT;
  if (ws_bytes < beam_bytes(n, vocab, k)) return W12_ERR_WORKSPACE;
  if (!aligned(logits, dtype == W12_LOGITS_F32 ? 4 : 2) || !aligned(ws, 256)) return W12_ERR_ALIGN;
  if (!aligned4({scores, grp_off, parent, token, score_out})) return W12_ERR_ALIGN;
  BeamArgs a{};
  a.logits = logits;
  a.stride = stride;
  a.n = n;
  a.vocab = vocab;
  a.n_grp = n_grp;
  a.k = k;
  a.scores = scores;
  a.grp_off = grp_off;
  a.parent = parent;
  a.token = token;
  a.out = score_out;
  a.ws = (uint8_t*)ws;
  return hip_status(launch_beam_select(a, dtype == W12_LOGITS_F32, (hipStream_t)stream));
}

}  // extern "C"
