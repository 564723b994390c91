// Attention of a decode step's new rows over the paged cache (w12_attn_paged).
#include "w12.h"
#include "w12_kv.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

template <bool F8>
__device__ __forceinline__ float kv_value(const uint8_t* p, uint64_t i) {
  if constexpr (F8) return __builtin_amdgcn_cvt_f32_fp8((int)p[i], 0);
  else return bf(reinterpret_cast<const uint16_t*>(p)[i]);
}

// One wave per row and head: 64 tokens at a time, one per lane for the scores, then D / 64
// dimensions per lane for the weighted sum, with the running maximum and sum of the softmax.
template <int D, bool F8>
__global__ __launch_bounds__(64) void k_attn_simple(AttnArgs a) {
  __shared__ float s_q[D], s_p[64];
  const int lane = threadIdx.x;
  bool bad = false;
  for (uint32_t r = lane; r <= a.n_req; r += 64) {
    const int32_t o = a.req_off[r], before = r ? a.req_off[r - 1] : 0;
    bad |= o < before || o > (int32_t)a.m;
  }
  bad = __any(bad);
  const uint32_t ps = 1u << a.page_shift;
  for (uint64_t w = blockIdx.x; w < (uint64_t)a.m * a.n_heads; w += gridDim.x) {
    const uint32_t row = (uint32_t)(w / a.n_heads), h = (uint32_t)(w % a.n_heads), hk = h / a.group;
    uint32_t r = 0;
    int32_t len = -1, limit = 0;
    if (!bad) {
      if ((int32_t)row < a.req_off[0] || (int32_t)row >= a.req_off[a.n_req]) continue;
      uint32_t lo = 1, hi = a.n_req;
      while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.req_off[mid] > (int32_t)row) hi = mid; else lo = mid + 1;
      }
      r = lo - 1;
      len = a.kv_len[r];
      limit = len - (a.req_off[r + 1] - (int32_t)row) + 1;
    }
    const bool broken = len < 0 || (uint64_t)len > (uint64_t)a.max_pages * ps;
    if (broken) limit = 0;
    __syncthreads();
    for (int d = lane; d < D; d += 64) s_q[d] = bf(a.q[row * a.q_stride + (uint64_t)h * D + d]);
    __syncthreads();
    float top = -INFINITY, sum = 0.f, acc[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) acc[i] = 0.f;
    for (int32_t t0 = 0; t0 < limit; t0 += 64) {
      const int32_t t = t0 + lane;
      float s = -INFINITY;
      if (t < limit) {
        const int32_t page = a.table[(uint64_t)r * a.max_pages + ((uint32_t)t >> a.page_shift)];
        if (page < 0 || (uint32_t)page >= a.n_pages) {
          s = NAN;
        } else {
          const uint64_t at = (((uint64_t)page * a.n_kv_heads + hk) * ps + (t & (ps - 1))) * D;
          s = 0.f;
          for (int d = 0; d < D; ++d) s = fmaf(s_q[d], kv_value<F8>(a.kc, at + d), s);
          s *= a.score_scale;
        }
      }
      float mx = s;
#pragma unroll
      for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
      const float now = fmaxf(top, mx);
      const float base = now == -INFINITY ? 0.f : now;
      const float fade = exp2f(top - base), p = t < limit ? exp2f(s - base) : 0.f;
      top = now;
      sum = sum * fade + p;
      s_p[lane] = p;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < D / 64; ++i) acc[i] *= fade;
      const int32_t n = min(64, limit - t0);
      for (int32_t j = 0; j < n; ++j) {
        const int32_t page = a.table[(uint64_t)r * a.max_pages + ((uint32_t)(t0 + j) >> a.page_shift)];
        if (page < 0 || (uint32_t)page >= a.n_pages) continue;
        const uint64_t at = ((uint64_t)page * a.n_kv_heads + hk) * D * ps + ((t0 + j) & (ps - 1));
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          acc[i] = fmaf(s_p[j], kv_value<F8>(a.vc, at + (uint64_t)(lane + 64 * i) * ps), acc[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float y = bad || broken ? NAN : (limit > 0 ? acc[i] / sum * a.v_scale : 0.f);
      a.out[row * a.out_stride + (uint64_t)h * D + lane + 64 * i] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
  }
}

template <bool F8>
hipError_t attn_launch(const AttnArgs& a, uint32_t d, hipStream_t s) {
  const uint64_t all = (uint64_t)a.m * a.n_heads;
  const dim3 g((uint32_t)(all < 65536 ? all : 65536)), b(64);
  if (d == 64) hipLaunchKernelGGL((k_attn_simple<64, F8>), g, b, 0, s, a);
  else if (d == 128) hipLaunchKernelGGL((k_attn_simple<128, F8>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_attn_simple<256, F8>), g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_paged(const AttnArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s) {
  return dtype == W12_KV_E4M3 ? attn_launch<true>(a, head_dim, s) : attn_launch<false>(a, head_dim, s);
}

}  // namespace w12
