// Device helpers of the block-table kernels (w12_kv.hip, w12_fork.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

constexpr uint32_t kPlanCap = 1u << 30;   // sums of pages saturate here, above any pool

// The ticket of a launch goes in steps of kTicket, so that the values a launch of G workgroups
// can leave it at, i kTicket with i < G, are told from what a state that is none may hold.
constexpr uint32_t kTicket = 0x9e3779b1u;
__host__ __device__ constexpr uint32_t inverse(uint32_t a) {   // modulo 2^32, of an odd a: five Newton steps
  uint32_t x = a;
  for (int i = 0; i < 5; ++i) x *= 2 - a * x;
  return x;
}
static_assert(inverse(kTicket) * kTicket == 1u, "kTicket's inverse");

// Smallest i in 1..n with a[i] > v, minus one: the segment of v in the ascending offsets
// a[0..n], for a[0] <= v < a[n] (segments may be empty).
__device__ __forceinline__ uint32_t segment(const uint32_t* a, uint32_t n, uint32_t v) {
  uint32_t lo = 1, hi = n;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) >> 1;
    if (a[mid] > v) hi = mid; else lo = mid + 1;
  }
  return lo - 1;
}

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kPlanCap); }

}  // namespace w12
