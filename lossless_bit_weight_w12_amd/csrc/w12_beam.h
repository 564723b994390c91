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

// A workgroup takes 256 threads' worth of 16, 32 or 64 values each: the smallest share that leaves
// at most four workgroups to a CU (us for 151936 BF16 logits, k = 8: 12 x 4 rows 19.9, 16.1, 16.1; 24 x 4
// rows 29.7, 22.1, 20.6), and the largest for long lists and rows, whose parts a join takes up to
// 256 of.
constexpr uint32_t kBeamT = 256, kBeamShort = 16, kBeamParts = 1024;
inline uint32_t beam_values(uint32_t n, uint32_t vocab, uint32_t k) {
  if (k > kBeamShort || vocab > (1u << 19)) return 64;
  for (uint32_t v = 16; v < 64; v *= 2)
    if ((uint64_t)n * ((vocab + kBeamT * v - 1) / (kBeamT * v)) <= kBeamParts) return v;
  return 64;
}
inline uint32_t beam_splits(uint32_t n, uint32_t vocab, uint32_t k) {
  const uint32_t per = kBeamT * beam_values(n, vocab, k);
  return (vocab + per - 1) / per;
}
// Workspace: a ticket per group; per row and part its maximum, its sum and its k best.  The size is what this
// call and every smaller one need, which may have smaller shares and so more parts: of either kind of
// those at most 1024 parts, and lists of kBeamShort at most.
constexpr uint64_t kBeamTickets = 4096 * 4;
inline uint64_t beam_bytes(uint32_t n, uint32_t vocab, uint32_t k) {
  uint64_t most = 0;
  for (uint32_t v = 16; v <= 64; v *= 2) {
    const uint64_t all = (uint64_t)n * ((vocab + kBeamT * v - 1) / (kBeamT * v));
    const uint64_t parts = v < 64 && all > kBeamParts ? kBeamParts : all, keys = v < 64 && k > kBeamShort ? kBeamShort : k;
    const uint64_t bytes = parts * (16 + 8 * keys);
    most = bytes > most ? bytes : most;
  }
  return kBeamTickets + most;
}
hipError_t launch_beam_select(const BeamArgs& a, bool f32, hipStream_t s);

}  // namespace w12
