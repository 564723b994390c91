// Block tables of the paged cache (w12_kv_plan) and the norm, rotation and append of a
// decode step's heads (w12_qk_rope).
#include "w12.h"
#include "w12_kv.h"
#include "w12_plan.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The pool's bookkeeping.  Every workgroup forms the requests' page counts and their running
// sums in LDS; then every page that changes hands and every row is an entry of one flat list
// each, dealt to all threads and found through the sums (a binary search), so that long tables
// and long prompts spread evenly.  Free pages are taken from the ring's start and given back
// at its end; the two ends never meet (count + freed <= n_pages is checked), a page that is
// given back and taken in the same call is read from the table row that gives it, and new
// table entries are computed where rows need them, so nothing that is written here is
// read here, except held and state: those the workgroup that is through last writes.
//
// Bound by latency: two dependent reads (counts, then pages) behind a launch, 3 us.  Up to 256
// requests in workgroups of 256 threads: 200 requests of up to 5 rows 4.7 us, 6.2 us with 1024
// threads; several workgroups where many rows or pages can change hands (admitting 131k rows
// of 64 prompts and releasing them: 410 us in one workgroup, 16 us).
template <int T, int N>
__global__ __launch_bounds__(T) void k_kv_plan(PlanArgs a) {
  constexpr uint32_t kPer = N / T;   // requests of a thread, at most
  __shared__ uint32_t s_off[N + 1], s_need[N + 1], s_free[N + 1];
  __shared__ int32_t s_len[N], s_held[N];   // held: -1 for a request that is refused as it is
  __shared__ uint32_t s_wn[T / 64], s_wf[T / 64], s_wb[T / 64], s_last;
  const uint32_t t = threadIdx.x, n = a.n_req, lane = t & 63, wave = t >> 6;
  const uint32_t first = blockIdx.x * T + t, step = gridDim.x * T;   // of the flat lists
  const uint32_t shift = a.page_shift;
  const int32_t head0 = a.state[0], count0 = a.state[1];
  bool bad = head0 < 0 || (uint32_t)head0 >= a.n_pages || count0 < 0 || (uint32_t)count0 > a.n_pages;
  // A ticket that did not begin at zero would leave the counts as they were beside new tables.
  // (Workgroups that are through may have taken theirs already: any value a launch passes will do.)
  bad |= (uint32_t)a.state[2] * inverse(kTicket) >= gridDim.x;
  auto want_of = [&](int32_t len, uint32_t rows) { return (uint32_t)(((uint64_t)len + rows + (1u << shift) - 1) >> shift); };

  // page counts, and their running sums: missing ones and those given back
  const uint32_t per = (n + T - 1) / T;
  uint32_t need[kPer], freed[kPer], nsum = 0, fsum = 0;
#pragma unroll
  for (uint32_t i = 0; i < kPer; ++i) {
    const uint32_t r = t * per + i;
    need[i] = freed[i] = 0;
    if (i < per && r < n) {
      const int32_t lo = a.req_off[r], hi = a.req_off[r + 1], len = a.len[r], held = a.held[r];
      bad |= lo < 0 || hi < lo || hi > (int32_t)a.m;
      const int64_t target = (int64_t)len + (uint32_t)(hi - lo);
      const bool valid = len >= 0 && held >= 0 && (uint32_t)held <= a.max_pages && target <= (int64_t)a.max_pages << shift;
      s_off[r] = (uint32_t)lo;
      if (r + 1 == n) s_off[n] = (uint32_t)hi;
      s_len[r] = len;
      s_held[r] = valid ? held : -1;
      if (valid) {
        const uint32_t want = want_of(len, (uint32_t)(hi - lo)), have = (uint32_t)held;
        need[i] = want > have ? want - have : 0u;
        freed[i] = have > want ? have - want : 0u;
      }
    }
    nsum = sat_add(nsum, need[i]);
    fsum = sat_add(fsum, freed[i]);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(nsum, o), v = __shfl_up(fsum, o);
    if (lane >= (uint32_t)o) {
      nsum = sat_add(nsum, u);
      fsum = sat_add(fsum, v);
    }
  }
  bad = __any(bad);
  if (lane == 63) {
    s_wn[wave] = nsum;
    s_wf[wave] = fsum;
    s_wb[wave] = bad;
  }
  __syncthreads();
  uint32_t total_need = 0, total_free = 0;
#pragma unroll
  for (uint32_t w = 0; w < T / 64; ++w) {
    if (w < wave) {
      nsum = sat_add(nsum, s_wn[w]);
      fsum = sat_add(fsum, s_wf[w]);
    }
    total_need = sat_add(total_need, s_wn[w]);
    total_free = sat_add(total_free, s_wf[w]);
    bad |= s_wb[w] != 0;
  }
  // a ring that would hold more pages than there are is no ring
  bad |= (uint64_t)(uint32_t)count0 + total_free > a.n_pages;
  if (bad) {   // nothing changes
    for (uint32_t r = first; r < n; r += step) a.kv_len[r] = -1;
    for (uint32_t i = first; i < a.m; i += step) {
      a.pos[i] = -1;
      a.slot[i] = -1;
    }
    return;
  }
#pragma unroll
  for (int i = (int)kPer - 1; i >= 0; --i) {
    const uint32_t r = t * per + i;
    if (i < (int)per && r < n) {
      s_need[r + 1] = nsum;
      s_free[r + 1] = fsum;
      nsum -= need[i];   // (a saturated sum stays above any pool: kPer max_pages <= 2^28)
      fsum -= freed[i];
    }
  }
  if (t == 0) s_need[0] = s_free[0] = 0u;
  __syncthreads();
  const uint32_t head = (uint32_t)head0, count = (uint32_t)count0, avail = count + total_free;
  // requests are served while pages last: the largest sum that they cover is taken
  const uint32_t taken = total_need <= avail ? total_need : s_need[segment(s_need, n, avail)];

  auto rows_of = [&](uint32_t r) { return s_off[r + 1] - s_off[r]; };
  auto served = [&](uint32_t r) {   // (needs nothing, by its own count: saturated sums are equal too)
    return s_held[r] >= 0 && (s_need[r + 1] <= avail || want_of(s_len[r], rows_of(r)) <= (uint32_t)s_held[r]);
  };
  auto ring_at = [&](uint32_t j) {   // j <= n_pages
    const uint32_t i = head + j;
    return i >= a.n_pages ? i - a.n_pages : i;
  };
  auto freed_page = [&](uint32_t e) {
    const uint32_t r = segment(s_free, n, e);
    return a.table[(uint64_t)r * a.max_pages + want_of(s_len[r], rows_of(r)) + (e - s_free[r])];
  };
  auto free_at = [&](uint32_t j) { return j < count ? a.ring[ring_at(j)] : freed_page(j - count); };

  for (uint32_t i = first; i < a.m; i += step) {
    int32_t p = -1, s = -1;
    if (i >= s_off[0] && i < s_off[n]) {
      const uint32_t r = segment(s_off, n, i);
      if (served(r)) {
        p = s_len[r] + (int32_t)(i - s_off[r]);
        const uint32_t c = (uint32_t)p >> shift, held = (uint32_t)s_held[r];
        const int32_t page = c < held ? a.table[(uint64_t)r * a.max_pages + c] : free_at(s_need[r] + (c - held));
        if (page >= 0 && (uint32_t)page < a.n_pages) s = (page << shift) | (p & ((1 << shift) - 1));
      }
    }
    a.pos[i] = p;
    a.slot[i] = s;
  }
  for (uint32_t e = first; e < total_free; e += 4 * step) {   // four reads at once
    int32_t page[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (e + j * step < total_free) page[j] = freed_page(e + j * step);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (e + j * step < total_free) a.ring[ring_at(count + e + j * step)] = page[j];
  }
  for (uint32_t e = first; e < taken; e += 4 * step) {
    int32_t page[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (e + j * step < taken) page[j] = free_at(e + j * step);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (e + j * step < taken) {
        const uint32_t r = segment(s_need, n, e + j * step);
        a.table[(uint64_t)r * a.max_pages + (uint32_t)s_held[r] + (e + j * step - s_need[r])] = page[j];
      }
  }
  for (uint32_t r = first; r < n; r += step) a.kv_len[r] = served(r) ? s_len[r] + (int32_t)rows_of(r) : -1;

  // counts last: every workgroup is through with the old ones
  __syncthreads();
  if (gridDim.x > 1) {
    if (t == 0) {
      uint32_t* const ticket = reinterpret_cast<uint32_t*>(a.state + 2);
      s_last = __hip_atomic_fetch_add(ticket, kTicket, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (gridDim.x - 1) * kTicket;
      if (s_last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
  }
  for (uint32_t r = t; r < n; r += T)
    if (served(r)) a.held[r] = (int32_t)want_of(s_len[r], rows_of(r));
  if (t == 0) {
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

// q and k: a wave takes some heads of one row.  The row's sines and cosines once per wave (the
// angle pos * inv_freq in FP64, brought to a fraction of a turn there, so far positions lose
// nothing), handed to the lanes through LDS; then 64 / (D / 8) heads at a time, 8 dimensions
// per lane (16-byte loads and stores), the pair's other half from the lane that holds it.
// Bound by HBM for many rows; for few by one read, the arithmetic and one write behind it, so
// a row is split over as many waves as it has head groups.
template <int D, bool F8>
__device__ __forceinline__ void rope_heads(const RopeArgs& a, uint32_t row, uint32_t part, uint32_t parts,
                                           float2* s_turn) {
  constexpr int kSub = D / 8;          // lanes per head
  constexpr int kPar = 64 / kSub;      // heads per wave at a time
  const int lane = threadIdx.x & 63;
  // (Every read is requested before the first is waited for: 512 rows of 40 heads 6.8 -> 6.4 us,
  // 8192 rows 50.6 -> 49.4 us.)
  const int32_t pos = a.pos[row];
  const uint32_t slot = (uint32_t)a.slot[row];
  const uint32_t sub = lane % kSub, heads = a.n_heads + a.n_kv_heads, half = a.rot_dim / 2;
  auto load = [&](uint32_t h) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (h < heads)
      v = *reinterpret_cast<const u32x4*>((h < a.n_heads ? a.q + row * a.q_stride + (uint64_t)h * D
                                                         : a.k + row * a.k_stride + (uint64_t)(h - a.n_heads) * D) + sub * 8);
    return v;
  };
  const uint32_t h_first = part * kPar + lane / kSub;
  u32x4 next = load(h_first);
  double freq[(D / 2 + 63) / 64];
#pragma unroll
  for (int i = 0; i < (D / 2 + 63) / 64; ++i)
    freq[i] = lane + 64u * i < half ? a.inv_freq[lane + 64u * i] : 0.0;
  u32x4 wq = {0u, 0u, 0u, 0u}, wk = wq;
  if (a.q_norm) wq = *reinterpret_cast<const u32x4*>(a.q_norm + sub * 8);
  if (a.k_norm) wk = *reinterpret_cast<const u32x4*>(a.k_norm + sub * 8);
  if (pos < 0) return;
#pragma unroll
  for (int i = 0; i < (D / 2 + 63) / 64; ++i)
    if (lane + 64u * i < half) {
      const double turns = (double)pos * freq[i] * 0.15915494309189535;
      float sn, cs;
      sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
      s_turn[lane + 64u * i] = make_float2(cs, sn);
    }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();   // one wave writes and reads: LDS keeps the order
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  // this lane's pairs: interleaved 4 of them, else 8 whose other halves another lane holds
  float2 turn[8];
  const uint32_t hs = half / 8;   // lanes of one half
  const bool turned = sub * 8 < a.rot_dim, low = sub < hs;
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      turn[i] = a.interleaved ? s_turn[sub * 4 + i / 2] : s_turn[(low ? sub : sub - hs) * 8 + i];
  }
  const int from = lane - (int)sub + (int)(turned ? (low ? sub + hs : sub - hs) : sub);

  for (uint32_t h0 = h_first; h0 - lane / kSub < heads; h0 += parts * kPar) {
    const uint32_t h = h0;
    const u32x4 raw = next;
    next = load(h + parts * kPar);
    const bool is_q = h < a.n_heads;
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf_lo(raw[i]);
      x[2 * i + 1] = bf_hi(raw[i]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < kSub; o <<= 1) ss += __shfl_xor(ss, o);
    if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
      const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
      const u32x4 g = is_q ? wq : wk;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = x[2 * i] * inv * bf_lo(g[i]);
        x[2 * i + 1] = x[2 * i + 1] * inv * bf_hi(g[i]);
      }
    }
    if (a.interleaved) {
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float u = x[i], v = x[i + 1];
          x[i] = u * turn[i].x - v * turn[i].y;
          x[i + 1] = v * turn[i].x + u * turn[i].y;
        }
      }
    } else if (half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl(x[i], from);
        if (turned) x[i] = low ? x[i] * turn[i].x - y * turn[i].y : x[i] * turn[i].x + y * turn[i].y;
      }
    }
    if (h >= heads) continue;
    if (is_q) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = bf_pack(x[2 * i], x[2 * i + 1]);
      *reinterpret_cast<u32x4*>(a.q_out + row * a.q_out_stride + (uint64_t)h * D + sub * 8) = o;
    } else if (slot < a.n_slots) {
      const uint64_t ph = (uint64_t)(slot >> a.page_shift) * a.n_kv_heads + (h - a.n_heads);
      const uint64_t at = ((ph << a.page_shift) + (slot & ((1u << a.page_shift) - 1u))) * D + sub * 8;
      if constexpr (F8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] / a.k_scale;
        *reinterpret_cast<u32x2*>(a.kc + at) = u32x2{pack_e4m3x4(x[0], x[1], x[2], x[3]),
                                                     pack_e4m3x4(x[4], x[5], x[6], x[7])};
      } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf_pack(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(a.kc) + at) = o;
      }
    }
  }
}

// v: a workgroup takes one head of 16 rows.  Eight rows that fill an aligned group of 8 places
// are turned through LDS by the workgroup that holds the first of them (up to 7 rows are the
// next one's) and written with 16 bytes per dimension (E4M3: 8); the other rows value by value,
// each by its own workgroup.  8192 prompt rows take 98 us with every value on its own, 52 us so.
constexpr int kRowsV = 16;
template <int D, bool F8>
__device__ __forceinline__ void rope_values(const RopeArgs& a, uint32_t tile, uint32_t head, uint16_t* s_v) {
  constexpr int kSub = D / 8;
  const uint32_t t = threadIdx.x, lane = t & 63, ps = a.page_shift;
  // lanes 0..29 of every wave: the slots of the tile's rows (from lane 7) and of 7 on either side
  const int64_t near = (int64_t)tile * kRowsV + lane - 7;
  uint32_t slot = ~0u;   // none
  if (lane < kRowsV + 14 && near >= 0 && near < (int64_t)a.m) {
    const uint32_t s = (uint32_t)a.slot[near];
    if (a.pos[near] >= 0 && s < a.n_slots) slot = s;
  }
  constexpr int kEach = (kRowsV * kSub + kRopeT - 1) / kRopeT;   // 8 dimensions of a row per thread
  u32x4 own[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const uint32_t i = t + e * kRopeT;
    const uint64_t row = (uint64_t)tile * kRowsV + i / kSub;
    if (i < kRowsV * kSub && row < a.m)
      own[e] = *reinterpret_cast<const u32x4*>(a.v + row * a.v_stride + (uint64_t)head * D + i % kSub * 8);
  }
  const uint32_t after = __shfl_down(slot, 1);
  const uint64_t follows = __ballot(slot != ~0u && slot + 1 == after);
  const uint64_t full = __ballot(slot % 8 == 0 && ((follows >> lane) & 0x7f) == 0x7f);   // first rows of whole groups
  auto dest = [&](uint32_t s, uint32_t d) {
    return ((((uint64_t)(s >> ps) * a.n_kv_heads + head) * D + d) << ps) + (s & ((1u << ps) - 1u));
  };
  auto quot = [&](uint16_t x) { return __uint_as_float((uint32_t)x << 16) / a.v_scale; };

#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const uint32_t i = t + e * kRopeT, l = i / kSub + 7, d = i % kSub * 8;
    const uint32_t s = __shfl(slot, l & 63);
    if (i >= kRowsV * kSub || s == ~0u || (s % 8 <= l && ((full >> (l - s % 8)) & 1))) continue;
    const u32x4 x = own[e];
    const uint64_t at = dest(s, d);
    if constexpr (F8) {
      const uint32_t lo = pack_e4m3x4(quot(x[0]), quot(x[0] >> 16), quot(x[1]), quot(x[1] >> 16));
      const uint32_t hi = pack_e4m3x4(quot(x[2]), quot(x[2] >> 16), quot(x[3]), quot(x[3] >> 16));
#pragma unroll
      for (int j = 0; j < 8; ++j) a.vc[at + ((uint64_t)j << ps)] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<uint16_t*>(a.vc)[at + ((uint64_t)j << ps)] = (uint16_t)(x[j / 2] >> (16 * (j & 1)));
    }
  }

  uint32_t firsts = (uint32_t)(full >> 7) & 0xffffu;   // whole groups that begin in the tile
  if (!firsts) return;                                 // (the same in every wave)
  for (uint32_t i = t; i < (kRowsV + 7) * kSub; i += kRopeT) {
    const uint32_t r = i / kSub, c = i % kSub;
    const uint64_t row = (uint64_t)tile * kRowsV + r;
    if (row < a.m)
      *reinterpret_cast<u32x4*>(s_v + r * (D + 8) + c * 8) =
          *reinterpret_cast<const u32x4*>(a.v + row * a.v_stride + (uint64_t)head * D + c * 8);
  }
  __syncthreads();
  for (; firsts; firsts &= firsts - 1) {
    const uint32_t r = __ffs(firsts) - 1, s = __shfl(slot, r + 7);
    for (uint32_t d = t; d < D; d += kRopeT) {
      uint16_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = s_v[(r + j) * (D + 8) + d];
      const uint64_t at = dest(s, d);
      if constexpr (F8) {
        *reinterpret_cast<u32x2*>(a.vc + at) = u32x2{pack_e4m3x4(quot(v[0]), quot(v[1]), quot(v[2]), quot(v[3])),
                                                     pack_e4m3x4(quot(v[4]), quot(v[5]), quot(v[6]), quot(v[7]))};
      } else {
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(a.vc) + at) =
            u32x4{v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16, v[4] | (uint32_t)v[5] << 16,
                  v[6] | (uint32_t)v[7] << 16};
      }
    }
  }
}

// The first v_blocks workgroups take v, the others q and k.
template <int D, bool F8>
__global__ __launch_bounds__(kRopeT) void k_qk_rope(RopeArgs a, uint32_t v_blocks, uint32_t parts) {
  __shared__ __attribute__((aligned(16))) uint16_t s_v[(kRowsV + 7) * (D + 8)];
  if (blockIdx.x < v_blocks) {
    rope_values<D, F8>(a, blockIdx.x / a.n_kv_heads, blockIdx.x % a.n_kv_heads, s_v);
  } else {
    const uint64_t w = (uint64_t)(blockIdx.x - v_blocks) * (kRopeT / 64) + threadIdx.x / 64;
    if (w >= (uint64_t)a.m * parts) return;
    float2* const s_turn = reinterpret_cast<float2*>(s_v) + threadIdx.x / 64 * (D / 2);
    static_assert(sizeof(s_v) >= sizeof(float2) * (D / 2) * (kRopeT / 64), "four waves' turns");
    rope_heads<D, F8>(a, (uint32_t)(w / parts), (uint32_t)(w % parts), parts, s_turn);
  }
}

template <int D, bool F8>
void rope_go(const RopeArgs& a, hipStream_t s) {
  // A row over as many waves as it has head groups while there are fewer than 16384 (8192 rows
  // of 48 heads: 57 us on 8192 waves, 52 us on 16384 or 32768, 71 us on 98304, where every head
  // group pays for the row's sines).
  constexpr uint32_t kPar = 64 / (D / 8);
  const uint32_t groups = (a.n_heads + a.n_kv_heads + kPar - 1) / kPar;
  uint32_t parts = (16384 + a.m - 1) / a.m;
  if (parts > groups) parts = groups;
  const uint32_t v_blocks = (a.m + kRowsV - 1) / kRowsV * a.n_kv_heads;
  const uint64_t waves = (uint64_t)a.m * parts;
  const uint32_t blocks = v_blocks + (uint32_t)((waves + kRopeT / 64 - 1) / (kRopeT / 64));
  hipLaunchKernelGGL((k_qk_rope<D, F8>), dim3(blocks), dim3(kRopeT), 0, s, a, v_blocks, parts);
}

template <bool F8>
hipError_t rope_launch(const RopeArgs& a, uint32_t d, hipStream_t s) {
  if (d == 64) rope_go<64, F8>(a, s);
  else if (d == 128) rope_go<128, F8>(a, s);
  else rope_go<256, F8>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s) {
  // two rows per thread, or entries of the table that could all change hands
  const uint64_t rows = ((uint64_t)a.m + 511) / 512, pages = ((uint64_t)a.n_req * a.max_pages + 4095) / 4096;
  const uint64_t most = rows > pages ? rows : pages;
  if (a.n_req <= 256)
    hipLaunchKernelGGL((k_kv_plan<256, 256>), dim3((uint32_t)(most < 256 ? most : 256)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_plan<1024, W12_MAX_REQ>), dim3((uint32_t)(most < 64 ? most : 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_qk_rope(const RopeArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s) {
  return dtype == W12_KV_E4M3 ? rope_launch<true>(a, head_dim, s) : rope_launch<false>(a, head_dim, s);
}

}  // namespace w12
