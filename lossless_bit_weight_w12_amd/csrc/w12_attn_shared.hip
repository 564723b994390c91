// Attention of a decode step's new rows over the paged cache where requests share their first
// tokens (w12_attn_shared).
//
// Mathematics: the softmax of a row over its tokens is split at S, the shared tokens that every
// row of the group sees, rounded down to whole units: the rows of all the group's requests are query
// rows of one item over [0, S), which no mask touches, and each request's own rows go over [S, its
// length), as in w12_attn_paged.  Every part leaves values, maximum and sum in FP32; a second
// kernel joins a row's parts in a fixed order.
//
// Both kinds of items lie on lines that are cut into equal pieces (see w12_attn_paged).  Items of more query
// rows than a wave of the second line holds (32, 16 with heads of 256) are cut for workgroups: K and V pass
// through LDS once for up to 32 rows per wave, the waves taking rows, and, where there are fewer rows
// than waves, tokens too.  The others (the requests' own tokens, and shared ones of few rows) are cut for
// single waves, which read K and V straight into registers, so that many short requests run side by side.
//
// Bound by HBM where few rows share tokens: 24 prompts of up to 8000 tokens, 20 query rows a head (520 MB)
// 120 us at 87 of reading, of them 5 before the first load (tables, lines), 8 in the join; 80 rows a head over
// 131001 tokens (547 MB) 119 us at 91.  Bound by the matrix cores' neighbours where many do: 1600 rows a head
// over 8000 tokens in E4M3 116 us at 47 of products; by their counters the matrix cores have 30 us of work,
// the vector units some 45, the reads of LDS 15 to 30, and they overlap in part only.
#include <type_traits>

#include "w12.h"
#include "w12_attn.h"
#include "w12_attn_shared.h"
#include "w12_plan.h"

namespace w12 {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D, bool F8>
struct Shared {
  static constexpr int NW = (int)shared_waves(D), NT = D == 256 ? 1 : 2, T = 64 * NW;
  static constexpr int QT = 16 * NT;             // query rows of a wave on the waves' line
  static constexpr int RT = 32, QW = RT * NW;    // of a wave in a workgroup's item, of the item, at most
  static constexpr int UT = F8 ? 64 : 32;        // tokens of a wave's unit
  using Own = Tile<D, F8, NT, UT>;
  static constexpr int KS = D / 32, DT = D / 16;           // matrix steps and tiles of the waves' line,
  static constexpr int KR = D / 16, DR = D / 32;           // and of a workgroup's item
  static constexpr int SU = D == 256 ? 1 : 2;    // units of 64 tokens of a step through LDS
  static constexpr uint32_t kChunk = 1024;       // one operand of a wave
  static constexpr uint32_t kHalf = KR * kChunk;           // K, or V, of a span of 32 tokens
  static constexpr uint32_t kStep = SU * 2 * 2 * kHalf;
  static constexpr int NL = F8 ? D / 32 : D / 16;          // 16-byte loads of a wave per step
  // Places on the lines: per item, and per unit (of 64 tokens by row tiles of 32, of UT tokens).  Measured, us,
  // with 8 / 6 / 5, 8 / 5 / 5, 8 / 5 / 3 and 8 for all: 300 query rows a head over 20000 tokens in E4M3 68, 68, 66,
  // 72, 1600 over 8000 117, 118, 114, 118, 80 over 131001 in BF16 121, 119, 119, 122; with leads of 2, 8, 16
  // and 32 places: four groups of 50 rows over 20000 84, 79, 79, 79, 90 rows of heads of 256 100, 97, 98, 97.
  static constexpr uint32_t kLeadW = 8, kLeadV = 3;
  static __device__ __forceinline__ uint32_t cost(uint32_t row_tiles) {
    return row_tiles > 4 ? 8u : (row_tiles > 2 ? 6u : 5u);
  }

  // The running softmax of a query row in the staged loop.  Weights are 2^(c s + bias), the reference bias
  // following the maximum only when that has risen by a factor of 2^kRise (so the results are seldom
  // rescaled).  BF16 weights may reach 2^8.  FP16 ones begin at 2^15, as in the waves' path, so that as many
  // of the small ones are kept (11 bits down to 2^-29 of the largest, a part of them down to 2^-39), and
  // 2^15.9 is what the type leaves for them to rise to.  (From 2^7, with 2^8 to rise by, 1600 query rows a head over
  // 8000 tokens took 109 us in place of 115.5, and weights of 2^-32 were lost.)
  // c s + bias is one fused operation, exact but for its own rounding, and the bias is a number of its own, no
  // rounded product that would have to be the same elsewhere; where c s is so large (kFar) that the bias cannot
  // follow it (within a factor of 2, in FP16 2^(1/512)), `fine` takes the rest, and kUp is kept apart.
  static constexpr float kUp = F8 ? 15.f : 0.f, kRise = F8 ? 0.9f : 8.f, kFar = F8 ? 65536.f : 16777216.f;
  struct Row {
    float ref;    // raw score that the reference was taken from
    float bias;   // kUp - c ref, rounded; far out -c ref
    float fine;   // 0; far out what the rounding left, or kNothing
    float sum;    // this lane's part, of the weights as they enter the product
    __device__ __forceinline__ float up() const { return fine == 0.f ? 0.f : kUp; }
    __device__ __forceinline__ float power(float c, float x) const { return (fmaf(x, c, bias) - fine) + up(); }
  };
  static constexpr float kNothing = 1e-30f;
  static __device__ __forceinline__ Row row() { return Row{-INFINITY, kUp, 0.f, 0.f}; }
  // The reference brought up to a span's largest score mx.
  static __device__ __forceinline__ void rise(float c, float mx, Row& r, f32x16 (&o)[DR]) {
    const auto other = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
    mx = fmaxf(__uint_as_float(other[0]), __uint_as_float(other[1]));
    if (__any((mx - r.ref) * c > kRise)) {
      const bool none = r.ref == -INFINITY;
      if (mx > r.ref) {
        const float bias = r.bias, fine = r.fine, up = r.up(), to = -(mx * c), rest = fmaf(mx, c, to);
        const bool far = fabsf(to) >= kFar;
        r.ref = mx;
        r.bias = far ? to : fmaf(-mx, c, kUp);
        r.fine = far ? (rest == 0.f ? kNothing : rest) : 0.f;
        const float fade = none ? 0.f : pow2(((r.bias - bias) - (r.fine - fine)) + (r.up() - up));
        r.sum *= fade;
#pragma unroll
        for (int d = 0; d < DR; ++d) o[d] *= fade;
      }
    }
  }
  // Two scores to their weights 2^(c x + bias).
  static __device__ __forceinline__ uint32_t weigh(float c, float bias, float x, float y, float& sum) {
    const float u = pow2(fmaf(x, c, bias)), v = pow2(fmaf(y, c, bias));
    const uint32_t w = F8 ? f16_pack(u, v) : bf_pack(u, v);
    if constexpr (F8)
      sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2_t, w), f16x2_t{(_Float16)1.f, (_Float16)1.f}, sum, false);
    else
      sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), bf16x2_t{(__bf16)1.f, (__bf16)1.f}, sum, false);
    return w;
  }
  static __device__ __forceinline__ f32x16 mfma_k(u32x4 k, u32x4 q, f32x16 s) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, k), __builtin_bit_cast(bf16x8_t, q), s, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma_v(u32x4 v, u32x4 p, f32x16 o) {
    if constexpr (F8)
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, v), __builtin_bit_cast(f16x8_t, p), o, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, p), o, 0, 0, 0);
  }
  // What brings a row's results to the reference of the waves' path: weights 2^(c (s - ref) + Own::kUp).
  static __device__ __forceinline__ float adjust(float c, const Row& r) {
    return r.ref == -INFINITY ? pow2(Own::kUp - kUp) : pow2(Own::kUp - r.power(c, r.ref));
  }
};

// A group's shared tokens, or a request's own: query rows per key head, and units (of 64 tokens, of
// UT).
struct Part {
  uint32_t q, units;
  bool wide;   // on the workgroups' line
};
constexpr uint32_t kBroken = 0x80000000u;   // in place of what a row sees

__device__ __forceinline__ uint32_t pow2_above(uint32_t x) { return x <= 1 ? 1u : 1u << (32 - __clz((int)(x - 1))); }

// Places on the workgroups' line: for each head the items of QW rows, then that of what is left.
template <int D, bool F8>
__device__ __forceinline__ uint32_t places_w(const Part& p, uint32_t hkv) {
  using A = Shared<D, F8>;
  const uint32_t full = p.q / A::QW, rest = p.q - full * A::QW;
  return hkv * (full * (A::kLeadW + p.units * A::cost(A::NW)) +
                (rest ? A::kLeadW + p.units * A::cost((rest + A::RT - 1) / A::RT) : 0u));
}

// A group's shared tokens: units of 64 tokens for workgroups, of UT for waves.
template <int D, bool F8>
__device__ __forceinline__ Part part_shared(const SharedArgs& a, uint32_t rows, uint32_t shared) {
  using A = Shared<D, F8>;
  const uint32_t q = rows * a.group;
  const bool wide = q > (uint32_t)A::QT && shared;
  return Part{q, wide ? shared : shared * (64 / A::UT), wide};
}
// A request's own part: units from the shared ones on.
template <int D, bool F8>
__device__ __forceinline__ Part part_own(const SharedArgs& a, int32_t len, uint32_t rows, uint32_t shared) {
  using A = Shared<D, F8>;
  const bool broken = len < 0 || (uint64_t)len > ((uint64_t)a.max_pages << a.page_shift);
  const uint32_t upto = broken ? 0u : ((uint32_t)len + A::UT - 1) / A::UT, from = shared * (64 / A::UT);
  return Part{rows * a.group, rows && upto > from ? upto - from : 0u, false};
}

// How the items of the waves' line are cut: by the line's equal pieces, an item having a lead and a
// place per unit, or (shift > 0) each into pieces of 2^shift units, a place each.
struct Cut {
  uint32_t shift, lead;
  __device__ __forceinline__ uint32_t places(uint32_t units) const {   // of one item
    return shift ? (units + (1u << shift) - 1) >> shift : lead + units;
  }
  // units of the places [p0, p1) of an item; none: only its lead
  __device__ __forceinline__ void units_of(uint32_t units, uint32_t p0, uint32_t p1, uint32_t& ua, uint32_t& ub) const {
    ua = shift ? p0 << shift : (p0 > lead ? p0 - lead : 0u);
    ub = shift ? min(p1 << shift, units) : (p1 > lead ? p1 - lead : 0u);
  }
  // the places of an item's first and last unit
  __device__ __forceinline__ void ends(uint32_t units, uint32_t& first, uint32_t& last) const {
    first = shift ? 0u : lead;
    last = shift ? (units - 1) >> shift : lead + units - 1;
  }
};

// What a worker needs of the group or request at which its piece begins.
struct First {
  uint32_t at, start, slots;   // its place in the list, its first place on the line, the slots before it
  uint32_t row0, rows, shared; // batch rows, shared units of 64 tokens
  uint32_t lead;               // of a group: the request through whose table row the shared tokens are read
  int32_t len;                 // of a request
};

template <int D, bool F8>
__global__ __launch_bounds__((Shared<D, F8>::T)) void k_shared(SharedArgs a) {
  using A = Shared<D, F8>;
  using Own = typename A::Own;
  constexpr int NW = A::NW, NT = A::NT, T = A::T, KS = A::KS, DT = A::DT, UT = A::UT;
  constexpr uint32_t kMaxReq = W12_MAX_REQ;
  constexpr uint32_t kTables = 24 * (kMaxReq + 1), kBuf = 2 * A::kStep > kTables ? 2 * A::kStep : kTables;
  __shared__ __attribute__((aligned(16))) uint8_t s_buf[kBuf];
  __shared__ uint32_t s_from[kMaxReq];   // per request the units of 64 tokens its group shares
  __shared__ uint32_t s_w[5][NW];
  __shared__ First s_first[1 + NW];
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = uni(tid >> 6), b = blockIdx.x;
  const uint32_t hkv = a.n_kv_heads, n_req = a.n_req, n_grp = a.n_grp;
  // Workgroups of one XCD (b modulo 8) are neighbours on the lines: they read the same heads, and the
  // tiles of query rows that read the same tokens find them in the L2 that they share.
  const uint32_t at_line = a.grid % 8 ? b : (b & 7) * (a.grid >> 3) + (b >> 3);

  // ---- the tables in LDS, and what the groups share: the least that any of their rows sees
  // (Every phase is a short loop: what the kernel executes once it has to fetch first.)
  uint32_t* const s_off = reinterpret_cast<uint32_t*>(s_buf);      // [n_grp + 1]
  uint32_t* const s_req = s_off + kMaxReq + 1;                     // [n_req + 1]
  int32_t* const s_len = reinterpret_cast<int32_t*>(s_req + kMaxReq + 1);
  int32_t* const s_min = s_len + kMaxReq;
  uint32_t* const s_cnt = reinterpret_cast<uint32_t*>(s_min + kMaxReq);
  uint32_t* const s_lead = s_cnt + kMaxReq;
  auto usable = [&](int32_t len) { return len >= 0 && (uint64_t)len <= ((uint64_t)a.max_pages << a.page_shift); };
  uint32_t* const rec_r = reinterpret_cast<uint32_t*>(a.ws + kSharedReq);
  uint32_t* const rec_g = reinterpret_cast<uint32_t*>(a.ws + kSharedGrp);
  u32x2* const rec_row = reinterpret_cast<u32x2*>(a.ws + kSharedRow);
  bool bad = false;
#pragma nounroll
  for (uint32_t i = tid; i <= max(n_grp, n_req); i += T) {
    if (i <= n_grp) {
      const int32_t o = a.grp_off[i], next = i < n_grp ? a.grp_off[i + 1] : (int32_t)n_req;
      bad |= next < o || (i == 0 && o != 0) || (i == n_grp && o != next);
      s_off[i] = (uint32_t)o;
      if (i < n_grp) {
        s_min[i] = a.grp_len[i];
        s_cnt[i] = 0;
        s_lead[i] = ~0u;
      }
    }
    if (i <= n_req) {
      const int32_t o = a.req_off[i], next = i < n_req ? a.req_off[i + 1] : o;
      bad |= o < 0 || next < o || next > (int32_t)a.m;
      s_req[i] = (uint32_t)o;
      if (i < n_req) s_len[i] = a.kv_len[i];
    }
  }
  if (__syncthreads_or(bad)) {   // no request table, or no groups: NaN everywhere
    const uint64_t all = (uint64_t)a.m * a.n_heads * D;
    for (uint64_t i = (uint64_t)b * T + tid; i < all; i += (uint64_t)a.grid * T) {
      const uint64_t row = i / (a.n_heads * D);
      a.out[row * a.out_stride + i % (a.n_heads * D)] = 0x7fc0u;
    }
    if (b == 0 && tid == 0) *reinterpret_cast<uint32_t*>(a.ws) = 0u;   // nothing to join
    return;
  }
#pragma nounroll
  for (uint32_t r = tid; r < n_req; r += T) {
    const uint32_t g = segment(s_off, n_grp, r), rows = s_req[r + 1] - s_req[r];
    s_from[r] = g;
    if (rows && usable(s_len[r])) {
      atomicMin(&s_min[g], s_len[r] - (int32_t)rows + 1);
      atomicAdd(&s_cnt[g], 1u);
      atomicMin(&s_lead[g], r);
    }
  }
  __syncthreads();
#pragma nounroll
  for (uint32_t r = tid; r < n_req; r += T) {
    const uint32_t g = s_from[r];
    s_from[r] = s_cnt[g] > 1 && s_min[g] > 0 ? (uint32_t)s_min[g] / 64 : 0u;
    if (b == 0)   // (what the join needs: the first workgroup leaves it)
      for (uint32_t row = s_req[r]; row < s_req[r + 1]; ++row) rec_row[row] = u32x2{r, g};
  }
  __syncthreads();

  // ---- the lines, and this workgroup's and its waves' pieces of them
  const uint32_t n_all = n_grp + n_req, per_t = (n_all + T - 1) / T;   // groups, then requests
  auto part = [&](uint32_t e, First& f) {
    const bool own = e >= n_grp;
    const uint32_t r = own ? e - n_grp : s_off[e], r1 = own ? r + 1 : s_off[e + 1];
    f.at = e;
    f.row0 = s_req[r];
    f.rows = s_req[r1] - f.row0;
    f.shared = r1 > r ? s_from[r] : 0u;
    f.lead = own ? 0u : s_lead[e];
    f.len = own ? s_len[r] : 0;
    return own ? part_own<D, F8>(a, f.len, f.rows, f.shared) : part_shared<D, F8>(a, f.rows, f.shared);
  };
  // places and slots on the workgroups' line; units, items and slots on the waves'
  uint32_t sum[5] = {0, 0, 0, 0, 0};
#pragma nounroll
  for (uint32_t i = 0; i < per_t; ++i) {
    const uint32_t e = tid * per_t + i;
    if (e >= n_all) break;
    First f;
    const Part p = part(e, f);
    const uint32_t items = hkv * ((p.q + A::QT - 1) / A::QT), slots = p.units ? hkv * p.q : 0u;
    if (p.wide) {
      sum[0] += places_w<D, F8>(p, hkv);
      sum[1] += slots;
    } else if (p.units) {
      sum[2] += items * p.units;
      sum[3] += items;
      sum[4] += slots;
    }
  }
  uint32_t upto[5], total[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {   // sums before this thread, and of all
    upto[k] = wave_scan(sum[k]);
    if (lane == 63) s_w[k][wave] = upto[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    uint32_t v = lane < NW ? s_w[k][lane] : 0u;
    const uint32_t before = wave_scan(lane < (int)wave ? v : 0u);
    total[k] = (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(v), 63);
    upto[k] += (uint32_t)__builtin_amdgcn_readlane((int)before, 63) - sum[k];
  }
  const uint32_t all_w = total[0];
  // (pieces of a unit at least, so that every piece between an item's first and last unit has one)
  const uint32_t per_w = max((all_w + a.grid - 1) / a.grid, 2 * A::cost(NW));
  // The waves' line: equal pieces, wherever they cut the items; or, where there are so many waves that each
  // may have a piece of its own of few units, the items in pieces of two, four, eight or sixteen units.
  const uint32_t waves = a.grid * NW;
  Cut cut = {0u, A::kLeadV};
  if (2 * total[3] <= waves) {
    uint32_t shift = 1;
    while (shift < 5 && (total[2] >> shift) + total[3] > waves) ++shift;
    cut.shift = shift < 5 ? shift : 0u;
  }
  uint32_t all_v, start_v;
  if (cut.shift) {
    uint32_t pieces = 0;
#pragma nounroll
    for (uint32_t i = 0; i < per_t; ++i) {
      const uint32_t e = tid * per_t + i;
      if (e >= n_all) break;
      First f;
      const Part p = part(e, f);
      if (!p.wide) pieces += hkv * ((p.q + A::QT - 1) / A::QT) * cut.places(p.units);
    }
    start_v = wave_scan(pieces);
    __syncthreads();
    if (lane == 63) s_w[0][wave] = start_v;
    __syncthreads();
    const uint32_t v = lane < NW ? s_w[0][lane] : 0u, before = wave_scan(lane < (int)wave ? v : 0u);
    all_v = (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(v), 63);
    start_v += (uint32_t)__builtin_amdgcn_readlane((int)before, 63) - pieces;
  } else {
    all_v = total[2] + A::kLeadV * total[3];
    start_v = upto[2] + A::kLeadV * upto[3];
  }
  const uint32_t per_v = cut.shift ? 1u : max((all_v + waves - 1) / waves, 1u);
  // (pieces of few units go to as many workgroups as there are)
  const uint32_t next_wave = cut.shift ? a.grid : 1u, first_wave = cut.shift ? at_line : at_line * NW;
  const uint32_t wp = first_wave + wave * next_wave;   // this wave's place among all
#pragma nounroll
  for (uint32_t i = 0; i < per_t; ++i) {
    const uint32_t e = tid * per_t + i;
    if (e >= n_all) break;
    First f;
    const Part p = part(e, f);
    const uint32_t slots = p.units ? hkv * p.q : 0u;
    uint32_t places;
    if (p.wide) {
      places = places_w<D, F8>(p, hkv);
      f.start = upto[0];
      f.slots = upto[1];
      upto[0] += places;
      upto[1] += slots;
      if (at_line * per_w - f.start < places) s_first[0] = f;
    } else {
      places = p.units ? hkv * ((p.q + A::QT - 1) / A::QT) * cut.places(p.units) : 0u;
      f.start = start_v;
      f.slots = upto[4];
      start_v += places;
      upto[4] += slots;
#pragma nounroll
      for (uint32_t w = 0; w < (uint32_t)NW; ++w)
        if ((first_wave + w * next_wave) * per_v - f.start < places) s_first[1 + w] = f;
    }
    if (b == 0) {
      u32x4* const c = reinterpret_cast<u32x4*>(e < n_grp ? rec_g + kRecWords * e : rec_r + kRecWords * (e - n_grp));
      c[0] = u32x4{f.row0, p.q, p.units, f.start};
      // (of a request also what its first row sees)
      c[1] = u32x4{f.slots, e < n_grp ? (uint32_t)p.wide : (usable(f.len) ? (uint32_t)(f.len - (int32_t)f.rows + 1) : kBroken), 0u, 0u};
    }
  }
  if (b == 0) {
    if (tid == 0) *reinterpret_cast<u32x4*>(a.ws) = u32x4{1u, per_w, per_v, cut.shift};
    for (uint32_t i = tid; i < s_req[0]; i += T) rec_row[i] = u32x2{~0u, ~0u};
    for (uint32_t i = s_req[n_req] + tid; i < a.m; i += T) rec_row[i] = u32x2{~0u, ~0u};
  }
  __syncthreads();

  const float cs = fabsf(a.score_scale);
  const uint32_t flip = a.score_scale < 0.f ? 0x80008000u : 0u;
  const uint32_t mask = (1u << a.page_shift) - 1u;
  float2* const ml = reinterpret_cast<float2*>(a.ws + kSharedMl);
  const uint64_t region = (uint64_t)a.m * a.n_heads + (uint64_t)kSharedGrid * A::QW;
  float* const values = reinterpret_cast<float*>(ml + region + 2ull * a.m * a.n_heads + (uint64_t)kSharedGrid * NW * 32);
  auto per_group = [&](uint32_t x) { return div_by(x, a.group, a.group_inv); };
  auto load_q = [&](uint32_t row0, uint32_t head, uint32_t q0, uint32_t nw, bf16x8_t (&qf)[NT][KS]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t on = nt * 16 + (lane & 15) < (int)nw, qi = on ? q0 + nt * 16 + (lane & 15) : q0;
      const uint32_t row = per_group(qi), gq = qi - row * a.group;
      const uint16_t* p = a.q + (uint64_t)(row0 + row) * a.q_stride + (uint64_t)(head * a.group + gq) * D;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d = F8 ? 64 * (s / 2) + 16 * (lane >> 4) + 8 * (s & 1) : 32 * s + 8 * (lane >> 4);
        u32x4 w = *reinterpret_cast<const u32x4*>(p + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] ^= flip;
        qf[nt][s] = __builtin_bit_cast(bf16x8_t, w);
      }
    }
  };
  auto store = [&](uint64_t slot, uint32_t nw, const f32x4 (&o)[NT][DT], const float (&top)[NT], const float (&sum)[NT]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float l = group_sum(sum[nt]);
      const uint32_t qi = nt * 16 + (lane & 15);
      if (qi < nw) {
        if (lane < 16) ml[slot + qi] = make_float2(top[nt], l);
        float* const p = values + (slot + qi) * D + 4 * (lane >> 4);
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(p + 16 * d) = o[nt][d];
      }
    }
  };
  // a group's or request's values as the piece's first one has them in LDS
  auto first_of = [&](const First& s) {
    return First{uni(s.at), uni(s.start), uni(s.slots), uni(s.row0), uni(s.rows), uni(s.shared), uni(s.lead), (int32_t)uni((uint32_t)s.len)};
  };
  auto load_at = [&](First& f) {
    const bool own = f.at >= n_grp;
    const uint32_t r = own ? f.at - n_grp : (uint32_t)uniform_load(a.grp_off, f.at);
    const uint32_t r1 = own ? r + 1 : (uint32_t)uniform_load(a.grp_off, f.at + 1);
    f.row0 = (uint32_t)uniform_load(a.req_off, r);
    f.rows = (uint32_t)uniform_load(a.req_off, r1) - f.row0;
    f.shared = r1 > r ? uni(s_from[r]) : 0u;
    f.len = own ? uniform_load(a.kv_len, r) : 0;
    f.lead = r;
    if (!own && f.shared)   // the group's first request with rows and a length
      while (uniform_load(a.req_off, f.lead + 1) == uniform_load(a.req_off, f.lead) || !usable(uniform_load(a.kv_len, f.lead))) ++f.lead;
  };

  // ---- the workgroup's piece: shared tokens of many rows, through LDS
  if (at_line * per_w < all_w) {
    uint32_t pos = at_line * per_w;
    const uint32_t end = min(pos + per_w, all_w);
    First f = first_of(s_first[0]);
    while (pos < end) {
      const Part l = part_shared<D, F8>(a, f.rows, f.shared);
      const uint32_t nq_all = l.q, shared = l.units, row0 = f.row0;
      const uint32_t full = nq_all / A::QW, one = A::kLeadW + shared * A::cost(NW);
      const uint32_t rest = nq_all - full * A::QW, c_rest = A::cost((rest + A::RT - 1) / A::RT);
      const uint32_t per_head = full * one + (rest ? A::kLeadW + shared * c_rest : 0u);
      if (!l.wide || pos >= f.start + hkv * per_head) {
        if (l.wide) {
          f.start += hkv * per_head;
          f.slots += hkv * nq_all;
        }
        do {
          ++f.at;
          load_at(f);
        } while (f.rows == 0 || f.shared == 0);
        continue;
      }
      // the item: a tile of QW rows, or what is left, of a head
      const uint32_t head = (pos - f.start) / per_head, here = f.start + head * per_head;
      const uint32_t tile = min((pos - here) / one, full);
      const bool last = tile == full;
      const uint32_t first = here + tile * one, c = last ? c_rest : A::cost(NW), nq = last ? rest : (uint32_t)A::QW;
      const uint32_t len = A::kLeadW + shared * c, la = pos - first, n_here = min(len - la, end - pos);
      pos += n_here;
      if (la + n_here <= A::kLeadW) continue;   // only its lead falls into this piece
      const uint32_t ua = la > A::kLeadW ? (la - A::kLeadW + c - 1) / c : 0u;
      const uint32_t ub = (la + n_here - A::kLeadW + c - 1) / c;
      if (ua >= ub) continue;
      const uint64_t slot = f.slots + head * nq_all + tile * A::QW + (uint64_t)A::QW * at_line;
      const uint64_t trow = (uint64_t)f.lead * a.max_pages;
      // waves to row tiles, and those that are left to tokens
      const uint32_t tiles = pow2_above((nq + A::RT - 1) / A::RT), sub = wave & (tiles - 1), turn = wave / tiles;
      const uint32_t turns = min((uint32_t)NW / tiles, 2u * A::SU);
      const uint32_t nw = turn < turns && nq > sub * A::RT ? min((uint32_t)A::RT, nq - sub * A::RT) : 0u;
      const uint32_t r16 = lane & 15, g16 = lane >> 4, r32 = lane & 31, h32 = lane >> 5;
      u32x4 qf[A::KR];   // of query row r32: dimensions 16 s + 8 h32 .. + 7 of step s
      {
        const uint32_t qi = tile * A::QW + (r32 < nw ? sub * A::RT + r32 : 0u);
        const uint32_t row = per_group(qi), gq = qi - row * a.group;
        const uint16_t* const p = a.q + (uint64_t)(row0 + row) * a.q_stride + (uint64_t)(head * a.group + gq) * D + 8 * h32;
#pragma unroll
        for (int k = 0; k < A::KR; ++k) {
          qf[k] = *reinterpret_cast<const u32x4*>(p + 16 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[k][i] ^= flip;
        }
      }
      f32x16 o[A::DR];   // of query row r32: dimension 32 d + 8 j + 4 h32 + i in place 4 j + i
      typename A::Row soft = A::row();
#pragma unroll
      for (int d = 0; d < A::DR; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
      // Operands in LDS, 1 KB each, in the lanes' own order.  K of a span of 32 tokens: per 16 dimensions, lane
      // (row r32, half h32) 8 of them; row 8 j + 4 h + i is token 16 (j / 2) + 8 h + 4 (j % 2) + i, so that a lane's
      // scores, as the matrix core leaves them (rows 8 j + 4 h32 + i), are 8 consecutive tokens for each of
      // the two steps of the second product.  V: per 32 dimensions and 16 tokens, lane (dimension r32, half h32) 8
      // of those.
      // Fetching: of every step a wave takes K or V of a span: NL loads, half of them from each of the span's two
      // groups of 16 tokens, that lie in one page: 64 bytes of 16 keys, or 16 tokens of 32 (BF16) or 64
      // dimensions.  Their addresses are a base, the same for the wave, and a place of the lane that never
      // changes.  Units past the piece are fetched as its last one, so that nothing around the loads
      // depends on where the piece ends and the compiler waits for them where they are used.
      const uint32_t f_unit = wave >> 2, f_half = (wave >> 1) & 1;
      const bool f_v = wave & 1;
      constexpr uint32_t es = F8 ? 1 : 2;
      const uint32_t f_dist = f_v ? 64u << a.page_shift : 64u, f_place = f_v ? es : es * D;
      const uint32_t k_tok = 8 * ((r16 >> 2) & 1) + 4 * (r16 >> 3) + (r16 & 3);   // of row r16 among 16 tokens
      const uint32_t f_lane = f_v ? (F8 ? (uint32_t)lane << a.page_shift : ((r32 << a.page_shift) + 8 * h32) * 2)
                                  : k_tok * D * es + 16 * g16;
      const uint8_t* const f_cache = f_v ? a.vc : a.kc;
      u32x4 st[A::NL];
      uint32_t id_0 = 0, id_1 = 0, spoils = 0;
      auto pages_of = [&](uint32_t u0) {   // requested a step before they are needed
        const uint32_t t0 = min(u0 + f_unit, ub - 1) * 64 + 32 * f_half;
        id_0 = (uint32_t)uniform_load(a.table, trow + (t0 >> a.page_shift));
        id_1 = (uint32_t)uniform_load(a.table, trow + ((t0 + 16) >> a.page_shift));
      };
      auto fetch = [&](uint32_t u0) {
        const uint32_t t0 = min(u0 + f_unit, ub - 1) * 64 + 32 * f_half;
        const bool ok_0 = id_0 < a.n_pages, ok_1 = id_1 < a.n_pages;
        spoils = (ok_0 ? 0u : 1u) | (ok_1 ? 0u : 2u);   // (of values too: all bits set is NaN in either type)
        const uint64_t page = ((uint64_t)D * es) << a.page_shift;
        const uint8_t* const p = f_cache + ((uint64_t)(ok_0 ? id_0 : 0u) * hkv + head) * page + (uint64_t)(t0 & mask) * f_place;
        const uint8_t* const q = f_cache + ((uint64_t)(ok_1 ? id_1 : 0u) * hkv + head) * page + (uint64_t)((t0 + 16) & mask) * f_place;
#pragma unroll
        for (int i = 0; i < A::NL / 2; ++i) st[i] = Own::load16(p + i * f_dist + f_lane);
#pragma unroll
        for (int i = 0; i < A::NL / 2; ++i) st[A::NL / 2 + i] = Own::load16(q + i * f_dist + f_lane);
      };
      // In LDS the second group's keys lie 16 rows on, its values' step one operand; a load's 64 bytes of a key
      // are 2 (BF16) or 4 operands, its dimensions of V 2 or 4.
      const uint32_t put_0 = (2 * f_unit + f_half) * 2 * A::kHalf + (f_v ? A::kHalf : 0u) +
                             (f_v ? (F8 ? (uint32_t)h32 * 2048 + r32 * 16 : 16u * lane)
                                  : (F8 ? g16 * 1024 : (g16 >> 1) * 1024 + (g16 & 1) * 512) + r16 * 16);
      const uint32_t put_1 = put_0 + (f_v ? 1024 : 256);
      auto put = [&](uint32_t buf) {
        if (spoils) {   // keys in a page that is none: NaN, and so are the scores and the rows
#pragma unroll
          for (int i = 0; i < A::NL; ++i)
            if ((spoils >> (i < A::NL / 2 ? 0 : 1)) & 1u) st[i] = u32x4{~0u, ~0u, ~0u, ~0u};
        }
#pragma unroll
        for (int i = 0; i < A::NL; ++i) {
          uint8_t* const to = s_buf + buf * A::kStep + (i < A::NL / 2 ? put_0 : put_1) + (i % (A::NL / 2)) * (F8 ? 4096 : 2048);
          if constexpr (F8) {   // 16 dimensions of a token or tokens of a dimension: two operands' halves
            const u32x4 x[1] = {st[i]};
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<u32x4*>(to + 512 * h) = f_v ? Own::operand_v(x, h) : __builtin_bit_cast(u32x4, Own::operand(x, h));
          } else {
            *reinterpret_cast<u32x4*>(to) = st[i];
          }
        }
      };
      // The products of N spans of 32 tokens, one behind the other so that the matrix core works beside the
      // softmax: while the weights of a span are formed the next one's scores are, and while its maximum is
      // taken the values of the one before are summed: K0, K1, V0, K2, V1, K3, V2, V3.  (One after the other, a
      // wave's products and its softmax take the same time, 0.5 us per 64 tokens each, and the two waves
      // of a SIMD did not make up for it.)  The operands come through a ring of registers, requested
      // kRing operands before they are used: a matrix step on one takes 32 cycles, a read among eight
      // waves' some 200.
      constexpr int kRing = 8;
      auto run = [&](auto spans, uint32_t buf, uint32_t span) {
        constexpr int N = decltype(spans)::value, KR = A::KR, DR = A::DR;
        const uint8_t* const from = s_buf + buf * A::kStep + span * 2 * A::kHalf + 16 * lane;
        u32x4 ring[kRing];
        auto read = [&](int j) {   // operand j of the sequence
          if (j >= 2 * N * KR) return;
          const int n = j / KR, c = j % KR;
          const bool of_v = n == 2 * N - 1 || (n >= 2 && n % 2 == 0);
          const int sp = n == 2 * N - 1 ? N - 1 : (n < 2 ? n : (n % 2 ? (n + 1) / 2 : (n - 2) / 2));
          const int at = of_v ? (int)A::kHalf + ((c % DR) * 2 + c / DR) * (int)A::kChunk : c * (int)A::kChunk;   // V: tiles in turn
          ring[j % kRing] = *reinterpret_cast<const u32x4*>(from + sp * 2 * (int)A::kHalf + at);
        };
#pragma unroll
        for (int j = 0; j < kRing; ++j) read(j);
        f32x16 even, odd;   // scores of the spans in turn
        u32x4 p[2];
        auto score = [&](int i, int c, f32x16& s) {   // step c of span i
          const int j = (i < 2 ? i : 2 * i - 1) * KR + c;
          if (c == 0)
#pragma unroll
            for (int x = 0; x < 16; ++x) s[x] = 0.f;
          s = A::mfma_k(ring[j % kRing], qf[c], s);
          read(j + kRing);
        };
        auto value = [&](int i, int c) {
          const int j = (i == N - 1 ? 2 * N - 1 : 2 * i + 2) * KR + c;
          o[c % DR] = A::mfma_v(ring[j % kRing], p[c / DR], o[c % DR]);
          read(j + kRing);
        };
#pragma unroll
        for (int c = 0; c < KR; ++c) {
          score(0, c, even);
          fence();
        }
        // (the compiler's scheduler is told to deal the products, the reads and the rest out evenly)
        auto one = [&](auto index, f32x16& x, f32x16& y) {   // span `index`, its scores and those of the next
          constexpr int i = decltype(index)::value;
          fence();
          float m0 = x[0], m1 = x[1];
#pragma unroll
          for (int k = 2; k < 16; k += 4) {
            m0 = fmaxf(fmaxf(m0, x[k]), x[k + 1]);
            if (k + 2 < 16) m1 = fmaxf(fmaxf(m1, x[k + 2]), x[k + 3]);
          }
#pragma unroll
          for (int c = 0; c < KR; ++c)
            if (i) value(i - 1, c);
          if (i) {
#pragma unroll
            for (int c = 0; c < KR; ++c) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
          }
          fence();
          A::rise(cs, fmaxf(m0, m1), soft, o);
          float scale = cs, bias = soft.bias;
          if (__any(soft.fine != 0.f)) {   // scores far out
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = soft.power(cs, x[k]);
            scale = 1.f;
            bias = 0.f;
          }
          fence();
#pragma unroll
          for (int c = 0; c < KR; ++c)
            if (i + 1 < N) score(i + 1, c, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) p[k >> 2][k & 3] = A::weigh(scale, bias, x[2 * k], x[2 * k + 1], soft.sum);
          if (i + 1 < N) {
#pragma unroll
            for (int c = 0; c < KR; ++c) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 48 / KR, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
          }
          fence();
        };
        one(std::integral_constant<int, 0>{}, even, odd);
        if constexpr (N > 1) one(std::integral_constant<int, 1>{}, odd, even);
        if constexpr (N > 2) {
          one(std::integral_constant<int, 2>{}, even, odd);
          one(std::integral_constant<int, 3>{}, odd, even);
        }
#pragma unroll
        for (int c = 0; c < KR; ++c) {
          value(N - 1, c);
          fence();
        }
      };
      // (a loop for each number of spans: one loop with all would hold the results more than once)
      auto steps = [&](auto spans) {
        constexpr int N = decltype(spans)::value;
        __syncthreads();   // the buffers are free
        pages_of(ua);
        fetch(ua);
        pages_of(ua + A::SU);
        put(0);
        fetch(ua + A::SU);
        pages_of(ua + 2 * A::SU);
        uint32_t buf = 0;
        auto next = [&](uint32_t u0) {
          put(buf ^ 1);
          fetch(u0 + 2 * A::SU);
          pages_of(u0 + 3 * A::SU);
        };
        // While a step is worked on the next goes to the other half of the buffer, before the products in
        // one half of the waves and behind them in the other, so that the two waves of a SIMD do not want the
        // same at the same time.
        uint32_t u0 = ua;
#pragma nounroll
        for (; u0 + (N == 4 ? 1 : 0) < ub; u0 += A::SU) {
          __syncthreads();
          if (wave < NW / 2) next(u0);
          if (nw && (N == 4 || u0 + turn * N / 2 < ub)) run(spans, buf, N == 4 ? 0u : turn * N);
          if (wave >= NW / 2) next(u0);
          buf ^= 1;
        }
        if (N == 4 && u0 < ub) {   // the last step's one unit
          __syncthreads();
          if (nw) run(std::integral_constant<int, N == 4 ? 2 : N>{}, buf, 0);
        }
      };
      // spans of a step for each turn
      const uint32_t each = 2 * A::SU / turns;
      if (A::SU == 2 && each == 4) steps(std::integral_constant<int, 2 * A::SU>{});
      else if (each == 2) steps(std::integral_constant<int, 2>{});
      else steps(std::integral_constant<int, 1>{});
      float top = soft.ref, sum = soft.sum;
      {
        const float f = A::adjust(cs, soft);
        sum *= f;
#pragma unroll
        for (int d = 0; d < A::DR; ++d) o[d] *= f;
      }
      // the token turns joined, half of them at a time, through LDS in the lanes' own order
      f32x4* const s_o = reinterpret_cast<f32x4*>(s_buf);
      float2* const s_ml = reinterpret_cast<float2*>(s_buf + (uint32_t)(NW / 2) * A::DR * 4096);
      for (uint32_t h = turns / 2; h >= 1; h >>= 1) {
        __syncthreads();
        const uint32_t at = (turn % h) * tiles + sub;   // < NW / 2
        if (nw && turn >= h && turn < 2 * h) {
          s_ml[at * 64 + lane] = make_float2(top, sum);
#pragma unroll
          for (int d = 0; d < A::DR; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              s_o[((at * A::DR + d) * 4 + j) * 64 + lane] = f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        }
        __syncthreads();
        if (nw && turn < h) {
          const float2 x = s_ml[at * 64 + lane];
          const float m = fmaxf(top, x.x);
          const float f = top == -INFINITY ? 1.f : pow2((top - m) * cs);   // (without a maximum: 0, or NaN)
          const float e = x.x == -INFINITY ? 1.f : pow2((x.x - m) * cs);
          top = m;
          sum = sum * f + x.y * e;
#pragma unroll
          for (int d = 0; d < A::DR; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 y = s_o[((at * A::DR + d) * 4 + j) * 64 + lane];
#pragma unroll
              for (int i = 0; i < 4; ++i) o[d][4 * j + i] = o[d][4 * j + i] * f + y[i] * e;
            }
        }
      }
      if (turn == 0 && nw) {
        const auto other = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
        sum = __uint_as_float(other[0]) + __uint_as_float(other[1]);
        if (r32 < nw) {
          const uint64_t at = slot + sub * A::RT + r32;
          if (h32 == 0) ml[at] = make_float2(top, sum);
          float* const p = values + at * D + 4 * h32;
#pragma unroll
          for (int d = 0; d < A::DR; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<f32x4*>(p + 32 * d + 8 * j) = f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        }
      }
    }
  }

  // ---- the wave's piece: own tokens, and shared ones of few rows, straight from the cache
  uint32_t pos = wp * per_v;
  if (pos >= all_v) return;
  const uint32_t end = min(pos + per_v, all_v);
  First f = first_of(s_first[1 + wave]);
  while (pos < end) {
    const bool own = f.at >= n_grp;
    const Part l = own ? part_own<D, F8>(a, f.len, f.rows, f.shared) : part_shared<D, F8>(a, f.rows, f.shared);
    const uint32_t len1 = l.units && !l.wide ? cut.places(l.units) : 0u, places = hkv * ((l.q + A::QT - 1) / A::QT) * len1;
    if (pos >= f.start + places) {
      f.start += places;
      f.slots += len1 ? hkv * l.q : 0u;
      ++f.at;
      load_at(f);
      continue;
    }
    const uint32_t row0 = f.row0, req = own ? f.at - n_grp : f.lead, from = own ? f.shared * (64 / UT) : 0u;
    const int32_t base = own ? f.len - (int32_t)f.rows + 1 : (int32_t)(f.shared * 64);   // what row 0 sees
    const uint32_t item = (pos - f.start) / len1, first = f.start + item * len1;
    const uint32_t la = pos - first, n_here = min(len1 - la, end - pos);
    pos += n_here;
    uint32_t ua, ub;
    cut.units_of(l.units, la, la + n_here, ua, ub);
    if (ua >= ub) continue;
    ua += from;
    ub += from;
    const uint32_t tiles = (l.q + A::QT - 1) / A::QT, head = item / tiles, q0 = (item - head * tiles) * A::QT;
    const uint32_t nw = min((uint32_t)A::QT, l.q - q0);
    const uint64_t slot = region + f.slots + head * l.q + q0 + (uint64_t)A::QT * wp;
    const uint64_t trow = (uint64_t)req * a.max_pages;
    // all the wave's rows at once, or, where a value that is not finite lies among the tokens that some
    // of them see and some do not, one batch row after the other
    uint32_t qa = q0, qb = q0 + nw;
    bool apart = false;
    for (;;) {
      const int32_t see_min = own ? base + (int32_t)per_group(qa) : base;
      const int32_t see_max = own ? base + (int32_t)per_group(qb - 1) : base;
      const uint32_t see = see_max > 0 ? (uint32_t)see_max : 0u;
      const uint32_t uz = min(ub, (see + UT - 1) / UT);
      int32_t lim[NT];
      bf16x8_t qf[NT][KS];
      load_q(row0, head, qa, qb - qa, qf);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t qi = qa + nt * 16 + (lane & 15);
        lim[nt] = qi < qb ? (own ? base + (int32_t)per_group(qi) : base) : 0;
      }
      f32x4 o[NT][DT];
      float top[NT], sum[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = -INFINITY;
        sum[nt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[nt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      u32x4 kf[Own::TT][Own::KL], vf[DT][Own::VL];
      auto load_k = [&](const typename Own::Ids& x, uint32_t u) {
        Own::load_k(a, x, u, head, lane, [&](int t, int i, u32x4 v) { kf[t][i] = v; });
      };
      auto load_v = [&](const typename Own::Ids& x, uint32_t u) {
        Own::load_v(a, x, u, head, lane, [&](int d, int i, u32x4 v) { vf[d][i] = v; });
      };
      uint32_t u = ua;
      typename Own::Ids ids = {{0u, 0u, 0u, 0u}, 0u};
      if (u < uz) {
        ids = Own::load_ids(a, trow, u, see);
        load_k(ids, u);
        load_v(ids, u);
      }
      const uint32_t full = min(uz, see_min > 0 ? (uint32_t)see_min / UT : 0u);   // every row sees every token
      for (; u < full; ++u) {
        const bool more = u + 1 < uz;
        typename Own::Ids next = ids;
        if (more) next = Own::load_ids(a, trow, u + 1, see);
        f32x4 s[NT][Own::TT];
        Own::scores(kf, qf, s);
        fence();
        if (more) load_k(next, u + 1);
        fence();
        if (ids.bad) Own::spoil(ids.bad, lane, s);
        u32x4 p[NT][Own::PS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Own::template weights<false>(cs, 0u, s[nt], top[nt], sum[nt], o[nt], p[nt]);
        fence();
        Own::product(vf, p, o);
        fence();
        if (more) {
          load_v(next, u + 1);
          ids = next;
        }
      }
      bool odd = false;
      for (; u < uz; ++u) {
        const int32_t token = (int32_t)(u * UT);
        odd |= Own::odd_values(token, lane, see, see_min, see_max, vf);
        f32x4 s[NT][Own::TT];
        Own::scores(kf, qf, s);
        if (ids.bad) Own::spoil(ids.bad, lane, s);
        u32x4 p[NT][Own::PS];
        Own::ends_weights(cs, token, lane, lim, s, top, sum, o, p);
        Own::ends_product(token, lane, see_max, vf, p, o, [](int) { return true; });
        if (u + 1 < uz) {
          ids = Own::load_ids(a, trow, u + 1, see);
          load_k(ids, u + 1);
          load_v(ids, u + 1);
        }
      }
      if (odd && !apart) {
        apart = true;
        qb = q0;
      } else {
        store(slot + (qa - q0), qb - qa, o, top, sum);
        if (!apart || qb == q0 + nw) break;
      }
      qa = qb;
      qb = min(q0 + nw, (per_group(qa) + 1) * a.group);
    }
  }
}

// Largest value, and sum, over the wave.
__device__ __forceinline__ float wave_max(float v) {
  v = row_max(v);
  return group_max(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return group_sum(v);
}

// A wave joins the parts of one row and head: first those of the shared tokens, then its own, both
// in the order of their pieces.
template <int D, bool F8>
__global__ __launch_bounds__(256) void k_shared_join(SharedArgs a) {
  using A = Shared<D, F8>;
  constexpr int L = D / 4, SG = 64 / L;   // lanes of one part, parts at a time
  constexpr uint32_t kFlight = 8;         // reads of a lane at once
  const int lane = threadIdx.x & 63;
  const uint32_t id = uni(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (id >= a.m * a.n_heads) return;
  const uint32_t row = id / a.n_heads, h = id - row * a.n_heads;
  const int32_t* const hdr = reinterpret_cast<const int32_t*>(a.ws);
  const int32_t* const rows = reinterpret_cast<const int32_t*>(a.ws + kSharedRow);
  const uint32_t valid = (uint32_t)uniform_load(hdr, 0), per_w = (uint32_t)uniform_load(hdr, 1);
  const uint32_t per_v = (uint32_t)uniform_load(hdr, 2);
  const Cut cut = {(uint32_t)uniform_load(hdr, 3), A::kLeadV};
  const uint32_t req = (uint32_t)uniform_load(rows, 2ull * row), grp = (uint32_t)uniform_load(rows, 2ull * row + 1);
  if (!valid || req == ~0u) return;
  uint32_t r[6], g[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    r[i] = (uint32_t)uniform_load(reinterpret_cast<const int32_t*>(a.ws + kSharedReq), kRecWords * req + i);
    g[i] = (uint32_t)uniform_load(reinterpret_cast<const int32_t*>(a.ws + kSharedGrp), kRecWords * grp + i);
  }
  const uint32_t kvh = h / a.group, gq = h - kvh * a.group;
  const float2* const ml = reinterpret_cast<const float2*>(a.ws + kSharedMl);
  const uint64_t region = (uint64_t)a.m * a.n_heads + (uint64_t)kSharedGrid * A::QW;
  const float* const values =
      reinterpret_cast<const float*>(ml + region + 2ull * a.m * a.n_heads + (uint64_t)kSharedGrid * A::NW * 32);
  // the pieces with units of an item: workers w0 .. w0 + n - 1, slots `slot` + w step
  uint64_t g_slot = 0, r_slot = 0;
  uint32_t g_w0 = 0, g_n = 0, g_step = A::QT, r_w0 = 0, r_n = 0;
  if (g[2]) {
    const uint32_t nq_all = g[1], units = g[2], qi = (row - g[0]) * a.group + gq;
    g_slot = (uint64_t)g[4] + kvh * nq_all + qi;
    if (g[5]) {
      const uint32_t full = nq_all / A::QW, one = A::kLeadW + units * A::cost(A::NW), tile = qi / A::QW;
      const uint32_t rest = nq_all - full * A::QW, c_rest = A::cost((rest + A::RT - 1) / A::RT);
      const uint32_t per_head = full * one + (rest ? A::kLeadW + units * c_rest : 0u);
      const uint32_t c = tile == full ? c_rest : A::cost(A::NW), first = g[3] + kvh * per_head + tile * one + A::kLeadW;
      g_w0 = first / per_w;
      g_n = (first + (units - 1) * c) / per_w - g_w0 + 1;
      g_step = A::QW;
    } else {
      uint32_t p0, p1;
      cut.ends(units, p0, p1);
      const uint32_t first = g[3] + kvh * cut.places(units);
      g_w0 = (first + p0) / per_v;
      g_n = (first + p1) / per_v - g_w0 + 1;
      g_slot += region;
    }
    g_slot += (uint64_t)g_w0 * g_step;
  }
  if (r[2]) {
    const uint32_t q = r[1], units = r[2], qi = (row - r[0]) * a.group + gq, tiles = (q + A::QT - 1) / A::QT;
    uint32_t p0, p1;
    cut.ends(units, p0, p1);
    const uint32_t first = r[3] + (kvh * tiles + qi / A::QT) * cut.places(units);
    r_w0 = (first + p0) / per_v;
    r_n = (first + p1) / per_v - r_w0 + 1;
    r_slot = region + r[4] + kvh * q + qi + (uint64_t)r_w0 * A::QT;
  }
  const uint32_t n = g_n + r_n;
  auto slot_of = [&](uint32_t i) {
    return i < g_n ? g_slot + (uint64_t)i * g_step : r_slot + (uint64_t)(i - g_n) * A::QT;
  };
  const float cs = fabsf(a.score_scale);
  float m = -INFINITY, l = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  const uint32_t sg = lane / L, d = 4 * (lane % L);
  for (uint32_t i0 = 0; i0 < n; i0 += 64) {
    const uint32_t here = min(64u, n - i0);
    f32x4 x[kFlight];
    auto request = [&](uint32_t i) {   // (past the end: the last one again, unused)
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k)
        x[k] = *reinterpret_cast<const f32x4*>(values + slot_of(i0 + min(i + k * SG + sg, here - 1)) * D + d);
    };
    request(0);
    const float2 y = (uint32_t)lane < here ? ml[slot_of(i0 + lane)] : make_float2(-INFINITY, 0.f);
    const float mx = fmaxf(m, wave_max(y.x));
    const float fade = m == -INFINITY ? 1.f : pow2((m - mx) * cs);   // (without a maximum: 0, or NaN that stays)
    const float f = y.x == -INFINITY ? 1.f : pow2((y.x - mx) * cs);
    l = l * fade + wave_sum(y.y * f);
    v *= fade;
    m = mx;
    for (uint32_t i = 0; i < here; i += kFlight * SG) {
      if (i) request(i);
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k) {
        const uint32_t j = i + k * SG + sg;
        const float fk = __shfl(f, (int)min(j, 63u));
        if (j < here) v += x[k] * fk;
      }
    }
  }
#pragma unroll
  for (int o = L; o < 64; o <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], o);
  const bool broken = r[5] == kBroken;
  const int32_t sees = (int32_t)r[5] + (int32_t)(row - r[0]);
  const float f = broken ? NAN : (sees > 0 ? a.v_scale / l : 0.f);
  if (sg == 0) {
    if (broken || sees <= 0) v = f32x4{0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<u32x2*>(a.out + (uint64_t)row * a.out_stride + (uint64_t)h * D + d) =
        u32x2{bf_pack(v[0] * f, v[1] * f), bf_pack(v[2] * f, v[3] * f)};
  }
}

template <int D, bool F8>
hipError_t shared_go(const SharedArgs& given, hipStream_t s) {
  using A = Shared<D, F8>;
  SharedArgs a = given;
  // no more workgroups than the widest table could give pieces of the waves' line, and one for each
  // unit of shared tokens
  const uint64_t tokens = (uint64_t)a.max_pages << a.page_shift;
  const uint64_t units = (tokens + A::UT - 1) / A::UT;
  const uint64_t items = (((uint64_t)a.m * a.group + A::QT - 1) / A::QT + a.n_req + a.n_grp) * a.n_kv_heads;
  uint64_t grid = kSharedGrid;
  if (units < (1u << 20) && items < (1u << 20)) {
    const uint64_t wg = (items * (units / 2 + 1) + A::NW - 1) / A::NW;
    grid = wg < 1 ? 1 : (wg < grid ? wg : grid);
  }
  a.grid = (uint32_t)grid;
  hipLaunchKernelGGL((k_shared<D, F8>), dim3(a.grid), dim3(A::T), 0, s, a);
  hipLaunchKernelGGL((k_shared_join<D, F8>), dim3((a.m * a.n_heads + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <bool F8>
hipError_t shared_dim(const SharedArgs& a, uint32_t d, hipStream_t s) {
  if (d == 64) return shared_go<64, F8>(a, s);
  if (d == 128) return shared_go<128, F8>(a, s);
  return shared_go<256, F8>(a, s);
}

}  // namespace

hipError_t launch_attn_shared(const SharedArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s) {
  return dtype == W12_KV_E4M3 ? shared_dim<true>(a, head_dim, s) : shared_dim<false>(a, head_dim, s);
}

}  // namespace w12
