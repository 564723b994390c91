// The attention side of a decode step: launch arguments shared by its host layer
// (w12_kv_api.cpp) and its kernels (w12_kv.hip, w12_attn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

struct PlanArgs {
  uint32_t n_pages, page_shift, max_pages;   // page_shift: log2(page_size)
  int32_t* table;          // [max_req][max_pages]
  int32_t* held;           // [max_req]
  int32_t* ring;           // [n_pages]
  int32_t* state;          // [4]: head, count, ticket (zero before and after), 0
  const int32_t* len;      // [n_req]
  const int32_t* req_off;  // [n_req + 1]
  uint32_t n_req, m;
  int32_t* kv_len;         // [n_req]
  int32_t* pos;            // [m]
  int32_t* slot;           // [m]
};
hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s);

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint64_t q_stride, k_stride, v_stride, q_out_stride;   // elements
  uint32_t m, n_heads, n_kv_heads;
  uint32_t n_slots;        // n_pages * page_size
  uint32_t page_shift;     // log2(page_size)
  const uint16_t* q_norm;  // NULL: no norm
  const uint16_t* k_norm;
  const double* inv_freq;  // [rot_dim / 2]
  uint32_t rot_dim, interleaved;
  float eps;
  float k_scale, v_scale;  // E4M3 caches
  const int32_t* pos;
  const int32_t* slot;
  uint16_t* q_out;
  uint8_t* kc;
  uint8_t* vc;
};
// dtype: W12_KV_*
hipError_t launch_qk_rope(const RopeArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s);

struct AttnArgs {
  const uint16_t* q;
  uint64_t q_stride, out_stride;   // elements
  uint32_t m, n_heads, n_kv_heads, group;   // group = n_heads / n_kv_heads
  uint32_t group_inv;      // floor(2^32 / group), 2^32 - 1 for 1
  uint32_t n_pages, page_shift;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* table;    // [n_req][max_pages]
  uint32_t max_pages;
  const int32_t* kv_len;   // [n_req]
  const int32_t* req_off;  // [n_req + 1]
  uint32_t n_req;
  float score_scale;       // scale * k_scale * log2(e): scores in powers of two
  float v_scale;
  // set per kernel:
  float join_cost;         // of one more piece of an item, in units
  uint32_t grid, grid_inv; // workgroups, and their inverse as group_inv
  uint16_t* out;
  uint32_t* tickets;       // workspace: 1024 tickets (zero before and after) ...
  float* partial;          // ... then the partial results
};
hipError_t launch_attn_paged(const AttnArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s);

}  // namespace w12
