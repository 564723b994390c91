// Block tables of the paged cache (w12_kv_plan) and the norm, rotation and append of a
// decode step's heads (w12_qk_rope).
#include "w12.h"
#include "w12_kv.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kPlanT = 1024;                          // threads of the plan's workgroup
constexpr uint32_t kPlanPer = W12_MAX_REQ / kPlanT;   // requests per thread, at most
constexpr uint32_t kPlanCap = 1u << 30;               // sums of pages saturate here

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

// One request's page counts.
struct Want {
  bool valid;
  uint32_t want, held;     // pages it shall hold (held when invalid), pages it holds
};

__device__ __forceinline__ Want request_want(const PlanArgs& a, uint32_t r, uint32_t rows) {
  const int32_t len = a.len[r], held = a.held[r];
  const int64_t target = (int64_t)len + rows;
  Want w;
  w.valid = len >= 0 && held >= 0 && (uint32_t)held <= a.max_pages &&
            target <= (int64_t)a.max_pages * a.page_size;
  w.held = w.valid ? (uint32_t)held : 0u;
  w.want = w.valid ? (uint32_t)((target + a.page_size - 1) / a.page_size) : w.held;
  return w;
}

// Inclusive sum over the workgroup of one value per thread (saturating).
__device__ uint32_t plan_scan(uint32_t v, uint32_t* s_wave) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(v, o);
    if (lane >= o) v = sat_add(v, u);
  }
  __syncthreads();
  if (lane == 63) s_wave[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = sat_add(v, s_wave[w]);
  return v;
}

// The pool's bookkeeping in one workgroup: per-request page counts, their running sums in
// LDS, then every page that changes hands and every row as one flat list each.  Moved pages
// are found through the sums (a binary search), so long tables spread over all threads.
// Free pages are taken from the ring's start and given back at its end; the two ends never
// meet (count + freed <= n_pages is checked), and a page that is given back and taken in the
// same call is read from the table row that gave it, so nothing written here is read here.
__global__ __launch_bounds__(kPlanT) void k_kv_plan(PlanArgs a) {
  __shared__ uint32_t s_off[W12_MAX_REQ + 1], s_need[W12_MAX_REQ + 1], s_free[W12_MAX_REQ + 1];
  __shared__ uint32_t s_wave[kPlanT / 64];
  __shared__ uint32_t s_taken;
  const uint32_t t = threadIdx.x, n = a.n_req;
  if (t == 0) s_taken = 0u;
  const int32_t head0 = a.state[0], count0 = a.state[1];
  bool bad = head0 < 0 || (uint32_t)head0 >= a.n_pages || count0 < 0 || (uint32_t)count0 > a.n_pages;
  for (uint32_t r = t; r <= n; r += kPlanT) {
    const int32_t o = a.req_off[r];
    const int32_t before = r ? a.req_off[r - 1] : 0;
    bad |= o < before || o > (int32_t)a.m;
    s_off[r] = (uint32_t)o;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    for (uint32_t r = t; r < n; r += kPlanT) a.kv_len[r] = -1;
    for (uint32_t i = t; i < a.m; i += kPlanT) {
      a.pos[i] = -1;
      a.slot[i] = -1;
    }
    return;
  }
  // running sums of the pages that are missing and of those given back
  const uint32_t per = (n + kPlanT - 1) / kPlanT;
  uint32_t need[kPlanPer], freed[kPlanPer], nsum = 0, fsum = 0;
#pragma unroll
  for (uint32_t i = 0; i < kPlanPer; ++i) {
    const uint32_t r = t * per + i;
    need[i] = freed[i] = 0;
    if (i < per && r < n) {
      const Want w = request_want(a, r, s_off[r + 1] - s_off[r]);
      need[i] = w.want > w.held ? w.want - w.held : 0u;
      freed[i] = w.held > w.want ? w.held - w.want : 0u;
    }
    nsum = sat_add(nsum, need[i]);
    fsum = sat_add(fsum, freed[i]);
  }
  const uint32_t nend = plan_scan(nsum, s_wave), fend = plan_scan(fsum, s_wave);
  uint32_t ne = nend, fe = fend;
#pragma unroll
  for (int i = (int)kPlanPer - 1; i >= 0; --i) {
    const uint32_t r = t * per + i;
    if (i < (int)per && r < n) {
      s_need[r + 1] = ne;
      s_free[r + 1] = fe;
      ne -= need[i];
      fe -= freed[i];
    }
  }
  if (t == 0) s_need[0] = s_free[0] = 0u;
  __syncthreads();
  // a ring that would hold more pages than there are is no ring: nothing is given back or taken
  const uint32_t total_free = s_free[n];
  const bool ring_ok = (uint64_t)count0 + total_free <= a.n_pages;
  const uint32_t n_free = ring_ok ? total_free : 0u;
  const uint32_t head = (uint32_t)head0, count = (uint32_t)count0;
  const uint32_t avail = ring_ok ? count + n_free : 0u;

  auto freed_page = [&](uint32_t e) -> int32_t {
    const uint32_t r = segment(s_free, n, e);
    const Want w = request_want(a, r, s_off[r + 1] - s_off[r]);
    return a.table[(uint64_t)r * a.max_pages + w.want + (e - s_free[r])];
  };
  auto ring_at = [&](uint32_t j) -> uint32_t {   // j < 2 n_pages
    const uint32_t i = head + j;                 // head < n_pages < 2^27, j < 2^28
    return i % a.n_pages;
  };
  auto free_at = [&](uint32_t j) -> int32_t {
    return j < count ? a.ring[ring_at(j)] : freed_page(j - count);
  };
  // served: invalid requests are not; without missing pages always; else while they last
  auto served = [&](uint32_t r, const Want& w) {
    return w.valid && ring_ok && (s_need[r + 1] == s_need[r] || s_need[r + 1] <= avail);
  };
  // a saturated sum is above any avail, so differences are only taken of exact sums
  uint32_t taken = 0;
  for (uint32_t r = t; r < n; r += kPlanT)
    if (s_need[r + 1] > s_need[r] && s_need[r + 1] <= avail) taken = max(taken, s_need[r + 1]);
#pragma unroll
  for (int o = 32; o; o >>= 1) taken = max(taken, (uint32_t)__shfl_xor((int)taken, o));
  if ((t & 63) == 0 && taken) atomicMax(&s_taken, taken);
  __syncthreads();
  taken = s_taken;

  for (uint32_t i = t; i < a.m; i += kPlanT) {
    int32_t p = -1, s = -1;
    if (i >= s_off[0] && i < s_off[n]) {
      const uint32_t r = segment(s_off, n, i);
      const Want w = request_want(a, r, s_off[r + 1] - s_off[r]);
      if (served(r, w)) {
        p = a.len[r] + (int32_t)(i - s_off[r]);
        const uint32_t c = (uint32_t)p / a.page_size;
        const int32_t page = c < w.held ? a.table[(uint64_t)r * a.max_pages + c]
                                        : free_at(s_need[r] + (c - w.held));
        if (page >= 0 && (uint32_t)page < a.n_pages)
          s = page * (int32_t)a.page_size + p % (int32_t)a.page_size;
      }
    }
    a.pos[i] = p;
    a.slot[i] = s;
  }
  for (uint32_t e = t; e < n_free; e += kPlanT) a.ring[ring_at(count + e)] = freed_page(e);
  for (uint32_t e = t; e < taken; e += kPlanT) {
    const uint32_t r = segment(s_need, n, e);
    const Want w = request_want(a, r, s_off[r + 1] - s_off[r]);
    a.table[(uint64_t)r * a.max_pages + w.held + (e - s_need[r])] = free_at(e);
  }
  // counts last: every thread is through with the old ones
  bool keep[kPlanPer];
  Want ws[kPlanPer];
#pragma unroll
  for (uint32_t i = 0; i < kPlanPer; ++i) {
    const uint32_t r = t * per + i;
    keep[i] = true;
    if (i < per && r < n) {
      ws[i] = request_want(a, r, s_off[r + 1] - s_off[r]);
      const bool ok = served(r, ws[i]);
      keep[i] = !ok;
      a.kv_len[r] = ok ? a.len[r] + (int32_t)(s_off[r + 1] - s_off[r]) : -1;
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < kPlanPer; ++i) {
    const uint32_t r = t * per + i;
    if (!keep[i] && ws[i].want != ws[i].held) a.held[r] = (int32_t)ws[i].want;
  }
  if (t == 0 && ring_ok) {
    a.state[0] = (int32_t)ring_at(taken);
    a.state[1] = (int32_t)(avail - taken);
  }
}

// ------------------------------------------------------------------------ norm and rotation
constexpr int kRopeT = 256;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
  const __bf16 x = (__bf16)a, y = (__bf16)b;   // round to nearest even
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}

// E4M3 of x, saturating (NaN stays NaN).
__device__ __forceinline__ float sat_e4m3(float x) {
  return x != x ? x : fminf(fmaxf(x, -448.f), 448.f);
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat_e4m3(a), sat_e4m3(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(sat_e4m3(c), sat_e4m3(d), w, true);
  return (uint32_t)w;
}

// One workgroup per row: the row's sines and cosines once in LDS (the angle pos * inv_freq
// in FP64, brought to a fraction of a turn there, so far positions lose nothing), then each
// wave takes 64 / (D / 8) heads at a time, 8 dimensions per lane (16-byte loads).
template <int D, bool F8>
__global__ __launch_bounds__(kRopeT) void k_qk_rope(RopeArgs a) {
  constexpr int kSub = D / 8;          // lanes per head
  constexpr int kPar = 64 / kSub;      // heads per wave at a time
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const uint32_t row = blockIdx.x;
  const int32_t pos = a.pos[row];
  if (pos < 0) return;
  const uint32_t half = a.rot_dim / 2;
  if (threadIdx.x < half) {
    const double turns = (double)pos * a.inv_freq[threadIdx.x] * 0.15915494309189535;
    const float f = (float)(turns - rint(turns));
    float sn, cs;
    sincospif(2.f * f, &sn, &cs);
    s_cos[threadIdx.x] = cs;
    s_sin[threadIdx.x] = sn;
  }
  __syncthreads();
  const uint32_t slot = (uint32_t)a.slot[row];
  const bool store = slot < a.n_slots;
  const uint32_t page = slot >> a.page_shift, place = slot & ((1u << a.page_shift) - 1u);
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  const uint32_t sub = lane % kSub;
  const uint32_t heads = a.n_heads + 2 * a.n_kv_heads;
  for (uint32_t h0 = wave * kPar; h0 < heads; h0 += (kRopeT / 64) * kPar) {
    const uint32_t h = h0 + lane / kSub;
    const bool on = h < heads;
    const bool is_q = h < a.n_heads, is_v = h >= a.n_heads + a.n_kv_heads;
    const uint32_t hk = is_q ? 0u : (is_v ? h - a.n_heads - a.n_kv_heads : h - a.n_heads);
    const uint16_t* src = is_q ? a.q + row * a.q_stride + (uint64_t)h * D
                               : (is_v ? a.v + row * a.v_stride : a.k + row * a.k_stride) + (uint64_t)hk * D;
    u32x4 raw = {0u, 0u, 0u, 0u};
    if (on) raw = *reinterpret_cast<const u32x4*>(src + sub * 8);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf_lo(raw[i]);
      x[2 * i + 1] = bf_hi(raw[i]);
    }
    const uint16_t* w = is_q ? a.q_norm : a.k_norm;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < kSub; o <<= 1) ss += __shfl_xor(ss, o);
    if (on && !is_v && w) {
      const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
      const u32x4 g = *reinterpret_cast<const u32x4*>(w + sub * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = x[2 * i] * inv * bf_lo(g[i]);
        x[2 * i + 1] = x[2 * i + 1] * inv * bf_hi(g[i]);
      }
    }
    if (a.interleaved) {
      if (!is_v && sub * 8 < a.rot_dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = s_cos[sub * 4 + i], s = s_sin[sub * 4 + i];
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * c - v * s;
          x[2 * i + 1] = v * c + u * s;
        }
      }
    } else if (half) {
      const uint32_t hs = half / 8;   // lanes of one half
      const bool turn = sub < 2 * hs;
      const bool first = sub < hs;
      const int from = (lane - (int)sub) + (int)(turn ? (first ? sub + hs : sub - hs) : sub);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl(x[i], from);
        if (turn && !is_v) {
          const uint32_t f = (first ? sub : sub - hs) * 8 + i;
          x[i] = first ? x[i] * s_cos[f] - y * s_sin[f] : x[i] * s_cos[f] + y * s_sin[f];
        }
      }
    }
    if (!on) continue;
    if (is_q) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = bf_pack(x[2 * i], x[2 * i + 1]);
      *reinterpret_cast<u32x4*>(a.q_out + row * a.q_out_stride + (uint64_t)h * D + sub * 8) = o;
    } else if (store) {
      const uint64_t ph = (uint64_t)page * a.n_kv_heads + hk;   // this head's part of the page
      const uint32_t ps = 1u << a.page_shift;
      if constexpr (F8) {
        const float sc = is_v ? a.v_scale : a.k_scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] / sc;
        const uint32_t lo = pack_e4m3x4(x[0], x[1], x[2], x[3]), hi = pack_e4m3x4(x[4], x[5], x[6], x[7]);
        if (is_v) {
          uint8_t* d = a.vc + (ph * D + sub * 8) * ps + place;
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i * ps] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
        } else {
          *reinterpret_cast<u32x2*>(a.kc + (ph * ps + place) * D + sub * 8) = u32x2{lo, hi};
        }
      } else if (is_v) {
        uint16_t* d = reinterpret_cast<uint16_t*>(a.vc) + (ph * D + sub * 8) * ps + place;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i * ps] = (uint16_t)(raw[i / 2] >> (16 * (i & 1)));
      } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf_pack(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(a.kc) + (ph * ps + place) * D + sub * 8) = o;
      }
    }
  }
}

template <bool F8>
hipError_t rope_launch(const RopeArgs& a, uint32_t d, hipStream_t s) {
  const dim3 g(a.m), b(kRopeT);
  if (d == 64) hipLaunchKernelGGL((k_qk_rope<64, F8>), g, b, 0, s, a);
  else if (d == 128) hipLaunchKernelGGL((k_qk_rope<128, F8>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_qk_rope<256, F8>), g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_plan, dim3(1), dim3(kPlanT), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_qk_rope(const RopeArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s) {
  return dtype == W12_KV_E4M3 ? rope_launch<true>(a, head_dim, s) : rope_launch<false>(a, head_dim, s);
}

}  // namespace w12
