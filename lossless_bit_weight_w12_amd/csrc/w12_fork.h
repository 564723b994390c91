// Pages that requests share: launch arguments common to the host layer (w12_fork_api.cpp) and the
// kernels (w12_fork.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

struct ForkArgs {
  uint32_t n_pages, page_shift, max_pages, max_req;   // page_shift: log2(page_size)
  int32_t* table;          // [max_req][max_pages]
  int32_t* held;           // [max_req]
  int32_t* ring;           // [n_pages]
  int32_t* state;          // [4]
  int32_t* refs;           // W12_REFS_WORDS
  const int32_t* parent;   // [n_req], NULL: each request itself
  const int32_t* len;      // [n_req]
  const int32_t* req_off;  // [n_req + 1]
  uint32_t n_req, m;
  uint32_t grid, n_inv, at_once;   // workgroups, the inverse of n_req, columns in LDS; set by the launch
  int32_t* kv_len;         // [n_req]
  int32_t* pos;            // [m]
  int32_t* slot;           // [m]
  int32_t* copies;         // [n_req][4]
};
hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s);

constexpr uint32_t kCopyLayers = 128;   // of a launch, at most (their addresses are its arguments)
struct CopyArgs {
  uint32_t n_pages, page_shift, page_bytes;   // of K or V of a page
  uint32_t key_shift;      // log2 of the 16-byte vectors of a place of K
  uint32_t vec_shift;      // log2 of the places of a vector of V
  const int32_t* copies;
  void* k[kCopyLayers];
  void* v[kCopyLayers];
};
hipError_t launch_kv_copy(const CopyArgs& a, uint32_t n_copies, uint32_t n_layers, hipStream_t s);

struct ClearArgs {
  uint32_t n_pages, page_size, max_pages, max_req, first, n_clear;
  uint32_t per, blocks;    // pages of a workgroup, and their number (256 at most); set by the launch
  int32_t* table;
  const int32_t* held;
  int32_t* ring;
  int32_t* state;
  int32_t* refs;
  int32_t* moves;          // [n_clear][4]
  int32_t* moved;          // [1]
};
hipError_t launch_kv_compact(const ClearArgs& a, hipStream_t s);

}  // namespace w12
