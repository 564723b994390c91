// The choice of the beams that go on: launch arguments and the workspace's layout, common to the
// host layer (w12_fork_api.cpp) and the kernel (w12_beam.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

struct BeamArgs {
  const void* logits;
  uint64_t stride;         // elements
  uint32_t n, vocab, n_grp, k, splits;
  const float* scores;     // [n]
  const int32_t* grp_off;  // [n_grp + 1]
  int32_t* parent;         // [n_grp][k]
  int32_t* token;
  float* out;
  uint8_t* ws;
};

// A workgroup takes 256 threads' worth of 16 or 64 values each: the small share, whose many parts a
// row's join takes one by one, for few rows and short lists.
constexpr uint32_t kBeamT = 256, kBeamMany = 64, kBeamFew = 16, kBeamShort = 16;
inline uint32_t beam_values(uint32_t n, uint32_t vocab, uint32_t k) {
  const uint64_t many = (uint64_t)n * ((vocab + kBeamT * kBeamMany - 1) / (kBeamT * kBeamMany));
  return k > kBeamShort || vocab > (1u << 19) || many >= 512 ? kBeamMany : kBeamFew;
}
// (rows may begin anywhere in a 16-byte vector: up to 7 places more)
inline uint32_t beam_splits(uint32_t n, uint32_t vocab, uint32_t k) {
  const uint32_t per = kBeamT * beam_values(n, vocab, k);
  return (vocab + 7 + per - 1) / per;
}
// Workspace: a ticket per group; per row and part its maximum, its sum and its k best.
constexpr uint64_t kBeamTickets = 4096 * 4;
inline uint64_t beam_bytes(uint32_t n, uint32_t vocab, uint32_t k) {
  return kBeamTickets + (uint64_t)n * beam_splits(n, vocab, k) * (16 + 8ull * k);
}
hipError_t launch_beam_select(const BeamArgs& a, bool f32, hipStream_t s);

}  // namespace w12
