// Attention of requests that share their first tokens: launch arguments and the workspace's layout,
// common to the host layer (w12_fork_api.cpp) and the kernels (w12_attn_shared.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

struct SharedArgs {
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
  const int32_t* grp_off;  // [n_grp + 1]
  const int32_t* grp_len;  // [n_grp]
  uint32_t n_req, n_grp;
  float score_scale;       // scale * k_scale * log2(e): scores in powers of two
  float v_scale;
  uint16_t* out;
  uint8_t* ws;
  uint32_t grid;           // workgroups; set by the launch
};

// Workspace: lengths of the pieces; a record per request and per group; each row's request and
// group; then the partial results, a (maximum, sum) and head_dim values for each of the slots.
constexpr uint32_t kSharedGrid = 256;
constexpr uint32_t kRecWords = 8;
constexpr uint64_t kSharedReq = 256;                                      // bytes: records of requests,
constexpr uint64_t kSharedGrp = kSharedReq + 4096ull * kRecWords * 4;     // of groups,
constexpr uint64_t kSharedRow = kSharedGrp + 4096ull * kRecWords * 4;     // rows,
constexpr uint64_t kSharedMl = kSharedRow + (1ull << 17) * 8;             // partial maxima and sums
constexpr uint32_t shared_waves(uint32_t d) { return d == 256 ? 4 : 8; }  // of a workgroup
// Slots: every query row of an item has one per piece of the item; pieces (item i, worker w) come in
// the order of both, so the place "rows of the items before i, plus w times the largest item" is
// free of overlap.  One region for the items that workgroups take and one for those of waves; a row
// is in at most one item of the first and two of the second.
inline uint64_t shared_region(uint32_t m, uint32_t n_heads, uint32_t d) {
  return (uint64_t)m * n_heads + (uint64_t)kSharedGrid * 32 * shared_waves(d);
}
inline uint64_t shared_slots(uint32_t m, uint32_t n_heads, uint32_t d) {
  return shared_region(m, n_heads, d) + 2ull * m * n_heads + (uint64_t)kSharedGrid * shared_waves(d) * 32;
}
// (What heads of d values and narrower ones need: workgroups of heads of 256 have half the waves, and so, in
// calls of few rows, less to keep than those of 128.)
inline uint64_t shared_bytes(uint32_t m, uint32_t n_heads, uint32_t d) {
  uint64_t most = 0;
  for (uint32_t w = 64; w <= d; w *= 2) {
    const uint64_t bytes = kSharedMl + shared_slots(m, n_heads, w) * (8 + 4ull * w);
    most = bytes > most ? bytes : most;
  }
  return most;
}
hipError_t launch_attn_shared(const SharedArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s);

}  // namespace w12
