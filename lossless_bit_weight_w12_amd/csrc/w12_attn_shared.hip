// Attention of a decode step's new rows over the paged cache where requests share their first
// tokens (w12_attn_shared).
//
// Mathematics: the softmax of a row over its tokens is split at S, the shared tokens that every
// row of the group sees, rounded down to whole units: the rows of all the group's requests are query
// rows of one item over [0, S), which no mask touches, and each request's own rows go over [S, its
// length), as in w12_attn_paged.  Every part leaves values, maximum and sum in FP32; a second
// kernel joins a row's parts in a fixed order.
//
// Both kinds of items lie on lines that are cut into equal pieces (see w12_attn_paged).  Items of
// more than 32 query rows are cut for workgroups: K and V pass through LDS once for up to 32 rows
// per wave, the waves taking rows, and, where there are fewer rows than waves, tokens too.  The
// others (the requests' own tokens, and shared ones of few rows) are cut for single waves, which read
// K and V straight into registers, so that many short requests run side by side.
#include <type_traits>

#include "w12.h"
#include "w12_attn.h"
#include "w12_attn_shared.h"
#include "w12_plan.h"

namespace w12 {

namespace {

template <int D, bool F8>
struct Shared {
  static constexpr int NW = (int)shared_waves(D), NT = D == 256 ? 1 : 2, T = 64 * NW;
  static constexpr int QT = 16 * NT;             // query rows of a wave
  static constexpr int QW = QT * NW;             // of a workgroup's item, at most
  static constexpr int UT = F8 ? 64 : 32;        // tokens of a wave's unit
  using Own = Tile<D, F8, NT, UT>;
  static constexpr int KS = D / 32, DT = D / 16;
  static constexpr int SU = D == 256 ? 1 : 2;    // units of 64 tokens of a step through LDS
  static constexpr uint32_t kChunk = 1024;       // one operand of a wave
  static constexpr uint32_t kHalf = 2 * KS * kChunk;       // K, or V, of a span of 32 tokens
  static constexpr uint32_t kStep = SU * 2 * 2 * kHalf;
  static constexpr int NL = F8 ? D / 32 : D / 16;          // 16-byte loads of a wave per step
  // Places on the lines: per item, and per unit (of 64 tokens by row tiles of 32, of UT tokens)
  static constexpr uint32_t kLeadW = 8, kLeadV = 3, kLeastV = 6;
  static __device__ __forceinline__ uint32_t cost(uint32_t row_tiles) {
    return row_tiles > 4 ? 8u : (row_tiles > 2 ? 6u : 5u);
  }
};

// What the items of a group's shared tokens, or of a request's own, are.
struct Line {
  uint32_t q;        // query rows per key head
  uint32_t units;
  uint32_t places;   // on its line, all items
};

__device__ __forceinline__ uint32_t pow2_above(uint32_t x) { return x <= 1 ? 1u : 1u << (32 - __clz((int)(x - 1))); }

template <int D, bool F8>
__device__ __forceinline__ Line line_w(uint32_t q, uint32_t shared, uint32_t hkv) {   // q > QT
  using A = Shared<D, F8>;
  const uint32_t full = q / A::QW, rest = q - full * A::QW;
  Line l = {q, shared, hkv * full * (A::kLeadW + shared * A::cost(A::NW))};
  if (rest) l.places += hkv * (A::kLeadW + shared * A::cost((rest + A::QT - 1) / A::QT));
  return l;
}
template <int D, bool F8>
__device__ __forceinline__ Line line_v(uint32_t q, uint32_t units, uint32_t hkv) {
  using A = Shared<D, F8>;
  return Line{q, units, units ? hkv * ((q + A::QT - 1) / A::QT) * (A::kLeadV + units) : 0u};
}

// A request's own part: units from the shared ones on.
template <int D, bool F8>
__device__ __forceinline__ Line line_own(const SharedArgs& a, int32_t len, uint32_t rows, uint32_t shared) {
  using A = Shared<D, F8>;
  const bool broken = len < 0 || (uint64_t)len > ((uint64_t)a.max_pages << a.page_shift);
  const uint32_t upto = broken ? 0u : ((uint32_t)len + A::UT - 1) / A::UT, from = shared * (64 / A::UT);
  return line_v<D, F8>(rows * a.group, rows && upto > from ? upto - from : 0u, a.n_kv_heads);
}

template <int D, bool F8>
__global__ __launch_bounds__((Shared<D, F8>::T)) void k_shared(SharedArgs a) {
  using A = Shared<D, F8>;
  using Own = typename A::Own;
  constexpr int NW = A::NW, NT = A::NT, T = A::T, KS = A::KS, DT = A::DT, UT = A::UT;
  constexpr uint32_t kMaxReq = W12_MAX_REQ;
  constexpr uint32_t kBuf = 2 * A::kStep > 3 * 4 * (kMaxReq + 1) ? 2 * A::kStep : 3 * 4 * (kMaxReq + 1);
  __shared__ __attribute__((aligned(16))) uint8_t s_buf[kBuf];
  __shared__ uint32_t s_from[kMaxReq];   // per request the units of 64 tokens its group shares
  __shared__ uint32_t s_w[6][NW];
  __shared__ uint32_t s_spoil[2][2 * A::SU];
  __shared__ struct { uint32_t at, start, rows; } s_first[1 + NW];
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = uni(tid >> 6), b = blockIdx.x;
  const uint32_t hkv = a.n_kv_heads, n_req = a.n_req, n_grp = a.n_grp;

  // ---- what the groups share: the least that any of their rows sees
  bool bad = false;
  {
    uint32_t* const s_off = reinterpret_cast<uint32_t*>(s_buf);   // [n_grp + 1]
    int32_t* const s_min = reinterpret_cast<int32_t*>(s_off + kMaxReq + 1);
    uint32_t* const s_cnt = reinterpret_cast<uint32_t*>(s_min + kMaxReq);
    for (uint32_t g = tid; g <= n_grp; g += T) {
      const int32_t o = a.grp_off[g], next = g < n_grp ? a.grp_off[g + 1] : o;
      bad |= o < 0 || next < o || (g == 0 && o != 0) || (g == n_grp && o != (int32_t)n_req);
      s_off[g] = (uint32_t)o;
      if (g < n_grp) {
        s_min[g] = a.grp_len[g];
        s_cnt[g] = 0;
      }
    }
    bad = __syncthreads_or(bad);
    for (uint32_t r = tid; r < n_req && !bad; r += T) {
      const int32_t r0 = a.req_off[r], r1 = a.req_off[r + 1], len = a.kv_len[r];
      const uint32_t g = segment(s_off, n_grp, r);
      s_from[r] = g;
      if (r1 > r0 && len >= 0 && (uint64_t)len <= ((uint64_t)a.max_pages << a.page_shift)) {
        atomicMin(&s_min[g], len - (r1 - r0) + 1);
        atomicAdd(&s_cnt[g], 1u);
      }
    }
    __syncthreads();
    for (uint32_t r = tid; r < n_req && !bad; r += T) {
      const uint32_t g = s_from[r];
      s_from[r] = s_cnt[g] > 1 && s_min[g] > 0 ? (uint32_t)s_min[g] / 64 : 0u;
    }
    __syncthreads();
  }

  // ---- the lines, and this workgroup's and its waves' pieces of them
  const uint32_t per_g = (n_grp + T - 1) / T, per_r = (n_req + T - 1) / T;
  auto grp_line = [&](uint32_t g, uint32_t& rows, bool& wide) {   // (without shared tokens: no places)
    const uint32_t g0 = (uint32_t)a.grp_off[g], g1 = (uint32_t)a.grp_off[g + 1];
    const uint32_t shared = g1 > g0 ? s_from[g0] : 0u;
    rows = (uint32_t)(a.req_off[g1] - a.req_off[g0]);
    const uint32_t q = rows * a.group;
    wide = q > (uint32_t)A::QT;
    if (!shared) return Line{q, 0, 0};
    return wide ? line_w<D, F8>(q, shared, hkv) : line_v<D, F8>(q, shared * (64 / UT), hkv);
  };
  auto own_line = [&](uint32_t r) {
    const uint32_t rows = (uint32_t)(a.req_off[r + 1] - a.req_off[r]);
    return line_own<D, F8>(a, a.kv_len[r], rows, s_from[r]);
  };
  uint32_t sum[6] = {0, 0, 0, 0, 0, 0};   // places and rows: workgroups' line, waves' groups, requests
  if (!bad) {
    for (uint32_t i = 0; i < per_r; ++i) {
      const uint32_t r = tid * per_r + i;
      if (r < n_req) {
        const int32_t r0 = a.req_off[r], r1 = a.req_off[r + 1];
        bad |= r0 < 0 || r1 < r0 || r1 > (int32_t)a.m;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {   // no request table, or no groups: NaN everywhere
    const uint64_t all = (uint64_t)a.m * a.n_heads * D;
    for (uint64_t i = (uint64_t)b * T + tid; i < all; i += (uint64_t)a.grid * T) {
      const uint64_t row = i / (a.n_heads * D);
      a.out[row * a.out_stride + i % (a.n_heads * D)] = 0x7fc0u;
    }
    if (b == 0 && tid == 0) *reinterpret_cast<uint32_t*>(a.ws) = 0u;   // nothing to join
    return;
  }
  for (uint32_t i = 0; i < per_g; ++i) {
    const uint32_t g = tid * per_g + i;
    if (g < n_grp) {
      uint32_t rows;
      bool wide;
      const Line l = grp_line(g, rows, wide);
      sum[wide ? 0 : 2] += l.places;
      sum[wide ? 1 : 3] += l.places ? hkv * l.q : 0u;
    }
  }
  for (uint32_t i = 0; i < per_r; ++i) {
    const uint32_t r = tid * per_r + i;
    if (r < n_req) {
      const Line l = own_line(r);
      sum[4] += l.places;
      sum[5] += l.places ? hkv * l.q : 0u;
    }
  }
  uint32_t upto[6], total[6];
#pragma unroll
  for (int k = 0; k < 6; ++k) {
    upto[k] = wave_scan(sum[k]);
    if (lane == 63) s_w[k][wave] = upto[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 6; ++k) {
    total[k] = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const uint32_t v = uni(s_w[k][w]);
      if (w < (int)wave) upto[k] += v;
      total[k] += v;
    }
    upto[k] -= sum[k];   // before this thread's
  }
  upto[4] += total[2];
  upto[5] += total[3];
  const uint32_t all_w = total[0], all_v = total[2] + total[4];
  // (pieces of a unit at least, so that every piece between an item's first and last unit has one)
  const uint32_t per_w = max((all_w + a.grid - 1) / a.grid, 2 * A::cost(NW));
  const uint32_t per_v = max((all_v + a.grid * NW - 1) / (a.grid * NW), A::kLeastV);
  uint32_t* const rec_r = reinterpret_cast<uint32_t*>(a.ws + kSharedReq);
  uint32_t* const rec_g = reinterpret_cast<uint32_t*>(a.ws + kSharedGrp);
  u32x2* const rec_row = reinterpret_cast<u32x2*>(a.ws + kSharedRow);
  if (b == 0) {
    if (tid == 0) {
      uint32_t* const h = reinterpret_cast<uint32_t*>(a.ws);
      h[1] = per_w;
      h[2] = per_v;
      h[0] = 1u;
    }
    const uint32_t row_0 = (uint32_t)a.req_off[0], row_n = (uint32_t)a.req_off[n_req];
    for (uint32_t i = tid; i < row_0; i += T) rec_row[i] = u32x2{~0u, ~0u};
    for (uint32_t i = row_n + tid; i < a.m; i += T) rec_row[i] = u32x2{~0u, ~0u};
  }
  // the records for the join, each by one workgroup, and where the pieces begin
  auto starts = [&](uint32_t at, uint32_t start, uint32_t places, uint32_t rows, bool line) {
    if (line) {
      const uint32_t p = b * per_w;
      if (p >= start && p < start + places) s_first[0] = {at, start, rows};
    } else {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t p = (b * NW + w) * per_v;
        if (p >= start && p < start + places) s_first[1 + w] = {at, start, rows};
      }
    }
  };
  for (uint32_t i = 0; i < per_g; ++i) {
    const uint32_t g = tid * per_g + i;
    if (g < n_grp) {
      uint32_t rows;
      bool wide;
      const Line l = grp_line(g, rows, wide);
      const int k = wide ? 0 : 2;
      starts(g, upto[k], l.places, upto[k + 1], wide);
      if (g % a.grid == b) {
        uint32_t* const c = rec_g + kRecWords * g;
        c[0] = (uint32_t)a.req_off[a.grp_off[g]];
        c[1] = l.q;
        c[2] = l.places ? l.units : 0u;
        c[3] = upto[k];
        c[4] = upto[k + 1];
        c[5] = wide;
      }
      upto[k] += l.places;
      upto[k + 1] += l.places ? hkv * l.q : 0u;
    }
  }
  for (uint32_t i = 0; i < per_r; ++i) {
    const uint32_t r = tid * per_r + i;
    if (r < n_req) {
      const Line l = own_line(r);
      starts(n_grp + r, upto[4], l.places, upto[5], false);
      if (r % a.grid == b) {
        const uint32_t r0 = (uint32_t)a.req_off[r], r1 = (uint32_t)a.req_off[r + 1];
        const int32_t len = a.kv_len[r];
        uint32_t* const c = rec_r + kRecWords * r;
        c[0] = r0;
        c[1] = l.q;
        c[2] = l.units;
        c[3] = upto[4];
        c[4] = upto[5];
        const bool broken = len < 0 || (uint64_t)len > ((uint64_t)a.max_pages << a.page_shift);
        c[5] = broken ? 0x80000000u : (uint32_t)(len - (int32_t)(r1 - r0) + 1);   // what its first row sees
        uint32_t lo = 0, hi = n_grp;   // its group: the last that begins at or before it and is not empty
        while (hi - lo > 1) {
          const uint32_t mid = (lo + hi) >> 1;
          if ((uint32_t)a.grp_off[mid] <= r) lo = mid; else hi = mid;
        }
        for (uint32_t row = r0; row < r1; ++row) rec_row[row] = u32x2{r, lo};
      }
      upto[4] += l.places;
      upto[5] += l.places ? hkv * l.q : 0u;
    }
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
  // the table row that a group's shared tokens are read through: its first request with tokens
  auto lead_of = [&](uint32_t g0) {
    for (uint32_t r = g0;; ++r) {
      const int32_t len = uniform_load(a.kv_len, r);
      if (uniform_load(a.req_off, r + 1) > uniform_load(a.req_off, r) && len >= 0 &&
          (uint64_t)len <= ((uint64_t)a.max_pages << a.page_shift))
        return r;
    }
  };

  // ---- the workgroup's piece: shared tokens of many rows, through LDS
  if (b * per_w < all_w) {
    uint32_t pos = b * per_w;
    const uint32_t end = min(pos + per_w, all_w);
    uint32_t g = uni(s_first[0].at), start = uni(s_first[0].start), before = uni(s_first[0].rows);
    while (pos < end) {
      const uint32_t g0 = (uint32_t)uniform_load(a.grp_off, g), g1 = (uint32_t)uniform_load(a.grp_off, g + 1);
      const uint32_t shared = g1 > g0 ? uni(s_from[g0]) : 0u;
      const uint32_t row0 = (uint32_t)uniform_load(a.req_off, g0);
      const uint32_t nq_all = ((uint32_t)uniform_load(a.req_off, g1) - row0) * a.group;
      const Line l = shared && nq_all > (uint32_t)A::QT ? line_w<D, F8>(nq_all, shared, hkv) : Line{nq_all, 0, 0};
      if (pos >= start + l.places) {
        start += l.places;
        before += l.places ? hkv * nq_all : 0u;
        ++g;
        continue;
      }
      // the item: tiles of QW rows, all heads of one after the other, then what is left
      const uint32_t full = nq_all / A::QW, one = A::kLeadW + shared * A::cost(NW);
      uint32_t tile, head, first, len, c, nq;
      if (pos - start < full * hkv * one) {
        const uint32_t item = (pos - start) / one;
        tile = item / hkv;
        head = item - tile * hkv;
        first = start + item * one;
        len = one;
        c = A::cost(NW);
        nq = A::QW;
      } else {
        tile = full;
        nq = nq_all - full * A::QW;
        c = A::cost((nq + A::QT - 1) / A::QT);
        len = A::kLeadW + shared * c;
        head = (pos - start - full * hkv * one) / len;
        first = start + full * hkv * one + head * len;
      }
      const uint32_t la = pos - first, n_here = min(len - la, end - pos);
      pos += n_here;
      if (la + n_here <= A::kLeadW) continue;   // only its lead falls into this piece
      const uint32_t ua = la > A::kLeadW ? (la - A::kLeadW + c - 1) / c : 0u;
      const uint32_t ub = (la + n_here - A::kLeadW + c - 1) / c;
      if (ua >= ub) continue;
      const uint64_t slot = before + tile * A::QW * hkv + head * nq + (uint64_t)A::QW * b;
      const uint64_t trow = (uint64_t)lead_of(g0) * a.max_pages;
      // waves to row tiles, and those that are left to tokens
      const uint32_t tiles = pow2_above((nq + A::QT - 1) / A::QT), sub = wave & (tiles - 1), turn = wave / tiles;
      const uint32_t turns = min((uint32_t)NW / tiles, 2u * A::SU);
      const uint32_t nw = turn < turns && nq > sub * A::QT ? min((uint32_t)A::QT, nq - sub * A::QT) : 0u;
      const uint32_t q0 = tile * A::QW + sub * A::QT;
      bf16x8_t qf[NT][KS];
      load_q(row0, head, nw ? q0 : 0u, nw, qf);
      f32x4 o[NT][DT];
      float top[NT], sum[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = -INFINITY;
        sum[nt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[nt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      // fetching: a wave takes K or V of a span of 32 tokens (BF16), or of a unit half of K's tokens or
      // of V's dimensions (E4M3, decoded on the way into LDS)
      u32x4 st[A::NL];
      uint32_t ids[F8 ? 4 : 2] = {}, spoils = 0;
      const uint32_t f_unit = F8 ? wave >> 2 : wave >> 2, f_half = F8 ? wave & 1 : (wave >> 1) & 1;
      const bool f_v = F8 ? (wave >> 1) & 1 : wave & 1;
      const uint32_t r16 = lane & 15, g16 = lane >> 4;
      auto pages_of = [&](uint32_t u0) {   // requested a step before they are needed
        const uint32_t u = u0 + f_unit;
        if (u >= ub) return;
#pragma unroll
        for (int j = 0; j < (F8 ? 4 : 2); ++j)
          ids[j] = (uint32_t)uniform_load(a.table, trow + ((u * 64 + (F8 ? 16 * j : 32 * f_half + 16 * j)) >> a.page_shift));
      };
      auto fetch = [&](uint32_t u0) {
        const uint32_t u = u0 + f_unit;
        if (u >= ub) return;
        spoils = 0;
#pragma unroll
        for (int j = 0; j < (F8 ? 4 : 2); ++j) {
          const bool ok = ids[j] < a.n_pages;
          spoils |= ok ? 0u : 1u << j;
          ids[j] = ok ? ids[j] : 0u;
        }
        if constexpr (F8) {
          if (f_v) {
            const uint32_t lo = (g16 & 1) ? ids[1] : ids[0], hi = (g16 & 1) ? ids[3] : ids[2];
            const uint32_t id = (g16 & 2) ? hi : lo, place = (u * 64 + 16 * g16) & mask;
            const uint8_t* p = a.vc + ((((uint64_t)id * hkv + head) * D + f_half * (D / 2) + r16) << a.page_shift) + place;
            const uint32_t next = 16u << a.page_shift;
#pragma unroll
            for (int i = 0; i < A::NL; ++i) st[i] = Own::load16(p + (uint64_t)i * next);
          } else {
            const uint32_t lo = (r16 & 4) ? ids[1] : ids[0], hi = (r16 & 4) ? ids[3] : ids[2];
            const uint32_t id = (r16 & 8) ? hi : lo;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t place = (u * 64 + 16 * (r16 >> 2) + 4 * (2 * f_half + t) + (r16 & 3)) & mask;
              const uint8_t* p = a.kc + ((((uint64_t)id * hkv + head) << a.page_shift) + place) * D + 16 * g16;
#pragma unroll
              for (int i = 0; i < A::NL / 2; ++i) st[t * (A::NL / 2) + i] = Own::load16(p + 64 * i);
            }
          }
        } else {
          const uint32_t t0 = u * 64 + 32 * f_half;
          if (f_v) {
            const uint32_t id = (g16 & 2) ? ids[1] : ids[0], place = (t0 + 8 * g16) & mask;
            const uint8_t* p = a.vc + (((((uint64_t)id * hkv + head) * D + r16) << a.page_shift) + place) * 2;
            const uint32_t next = 32u << a.page_shift;
#pragma unroll
            for (int i = 0; i < A::NL; ++i) st[i] = Own::load16(p + (uint64_t)i * next);
          } else {
            const uint32_t id = (r16 & 8) ? ids[1] : ids[0];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t place = (t0 + 8 * (r16 >> 2) + 4 * t + (r16 & 3)) & mask;
              const uint8_t* p = a.kc + ((((uint64_t)id * hkv + head) << a.page_shift) + place) * (D * 2) + 16 * g16;
#pragma unroll
              for (int i = 0; i < KS; ++i) st[t * KS + i] = Own::load16(p + 64 * i);
            }
          }
        }
      };
      auto put = [&](uint32_t u0, uint32_t buf) {
        if (u0 + f_unit >= ub) return;
        uint8_t* const step = s_buf + buf * A::kStep + 16 * lane;
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < A::NL; ++i) {
            const u32x4 x[1] = {st[i]};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (f_v) {   // tokens 8h .. 8h + 7 of the lane's 16: span h
                u32x4* const to = reinterpret_cast<u32x4*>(step + (2 * f_unit + h) * 2 * A::kHalf + A::kHalf + (f_half * (DT / 2) + i) * A::kChunk);
                *to = Own::operand_v(x, h);
              } else {     // dimensions 8h .. 8h + 7 of the lane's 16: matrix step 2 i + h
                const int t = i / (A::NL / 2), k = 2 * (i % (A::NL / 2)) + h;
                u32x4* const to = reinterpret_cast<u32x4*>(step + (2 * f_unit + f_half) * 2 * A::kHalf + (t * KS + k) * A::kChunk);
                *to = __builtin_bit_cast(u32x4, Own::operand(x, h));
              }
            }
          }
        } else {
          uint8_t* const to = step + (2 * f_unit + f_half) * 2 * A::kHalf + (f_v ? A::kHalf : 0u);
#pragma unroll
          for (int i = 0; i < A::NL; ++i) *reinterpret_cast<u32x4*>(to + i * A::kChunk) = st[i];
        }
        if (!f_v && lane == 0) s_spoil[buf][2 * f_unit + f_half] = spoils;
      };
      // the products of NS spans of 32 tokens
      auto unit = [&](auto spans, uint32_t buf, uint32_t span) {
        constexpr int NS = decltype(spans)::value;
        using Part = Tile<D, F8, NT, 32 * NS>;
        const uint8_t* const from = s_buf + buf * A::kStep + span * 2 * A::kHalf + 16 * lane;
        f32x4 s[NT][2 * NS];
#pragma unroll
        for (int t = 0; t < 2 * NS; ++t) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const bf16x8_t kk = *reinterpret_cast<const bf16x8_t*>(from + (t / 2) * 2 * A::kHalf + ((t & 1) * KS + i) * A::kChunk);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              s[nt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, qf[nt][i], s[nt][t], 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const uint32_t spoilt = uni(s_spoil[buf][span + k]);
          if (spoilt && ((spoilt >> (F8 ? g16 : g16 >> 1)) & 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][2 * k] = s[nt][2 * k + 1] = f32x4{NAN, NAN, NAN, NAN};
          }
        }
        u32x4 p[NT][NS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Part::template weights<false>(cs, 0u, s[nt], top[nt], sum[nt], o[nt], p[nt]);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            const u32x4 vv = *reinterpret_cast<const u32x4*>(from + k * 2 * A::kHalf + A::kHalf + d * A::kChunk);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[nt][d] = Own::mfma_v(vv, p[nt][k], o[nt][d]);
          }
      };
      __syncthreads();   // the buffers are free
      pages_of(ua);
      fetch(ua);
      pages_of(ua + A::SU);
      // (a loop for each form of a unit: one loop with both would hold the results twice)
      auto steps = [&](auto&& work) {
        uint32_t buf = 0;
        for (uint32_t u0 = ua; u0 < ub; u0 += A::SU) {
          put(u0, buf);
          fetch(u0 + A::SU);
          pages_of(u0 + 2 * A::SU);
          __syncthreads();
          work(u0, buf);
          buf ^= 1;
        }
      };
      if (!nw)
        steps([](uint32_t, uint32_t) {});
      else if (turns <= (uint32_t)A::SU)
        steps([&](uint32_t u0, uint32_t buf) {
#pragma nounroll
          for (uint32_t k = turn; k < (uint32_t)A::SU && u0 + k < ub; k += turns)
            unit(std::integral_constant<int, 2>{}, buf, 2 * k);
        });
      else
        steps([&](uint32_t u0, uint32_t buf) {
          if (u0 + (turn >> 1) < ub) unit(std::integral_constant<int, 1>{}, buf, turn);
        });
      // the token turns joined, half of them at a time, through LDS in the lanes' own order
      f32x4* const s_o = reinterpret_cast<f32x4*>(s_buf);
      float2* const s_ml = reinterpret_cast<float2*>(s_buf + (uint32_t)(NW / 2) * NT * DT * 1024);
      for (uint32_t h = turns / 2; h >= 1; h >>= 1) {
        __syncthreads();
        const uint32_t at = (turn % h) * tiles + sub;   // < NW / 2
        if (nw && turn >= h && turn < 2 * h) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s_ml[(at * NT + nt) * 64 + lane] = make_float2(top[nt], sum[nt]);
#pragma unroll
            for (int d = 0; d < DT; ++d) s_o[((at * NT + nt) * DT + d) * 64 + lane] = o[nt][d];
          }
        }
        __syncthreads();
        if (nw && turn < h) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 x = s_ml[(at * NT + nt) * 64 + lane];
            const float m = fmaxf(top[nt], x.x);
            const float f = top[nt] == -INFINITY ? 1.f : pow2((top[nt] - m) * cs);   // (without a maximum: 0, or NaN)
            const float e = x.x == -INFINITY ? 1.f : pow2((x.x - m) * cs);
            top[nt] = m;
            sum[nt] = sum[nt] * f + x.y * e;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[nt][d] = o[nt][d] * f + s_o[((at * NT + nt) * DT + d) * 64 + lane] * e;
          }
        }
      }
      if (turn == 0 && nw) store(slot + sub * A::QT, nw, o, top, sum);
    }
  }

  // ---- the wave's piece: own tokens, and shared ones of few rows, straight from the cache
  const uint32_t wp = b * NW + wave;
  uint32_t pos = wp * per_v;
  if (pos >= all_v) return;
  const uint32_t end = min(pos + per_v, all_v);
  uint32_t at = uni(s_first[1 + wave].at), start = uni(s_first[1 + wave].start), before = uni(s_first[1 + wave].rows);
  while (pos < end) {
    const bool own = at >= n_grp;
    uint32_t row0, rows, from = 0;
    int32_t base;   // what row 0 sees
    uint32_t req, g0 = 0;
    Line l;
    if (own) {
      req = at - n_grp;
      row0 = (uint32_t)uniform_load(a.req_off, req);
      rows = (uint32_t)uniform_load(a.req_off, req + 1) - row0;
      const int32_t len = uniform_load(a.kv_len, req);
      const uint32_t shared = uni(s_from[req]);
      l = line_own<D, F8>(a, len, rows, shared);
      from = shared * (64 / UT);
      base = len - (int32_t)rows + 1;
    } else {
      g0 = (uint32_t)uniform_load(a.grp_off, at);
      const uint32_t g1 = (uint32_t)uniform_load(a.grp_off, at + 1);
      row0 = (uint32_t)uniform_load(a.req_off, g0);
      rows = (uint32_t)uniform_load(a.req_off, g1) - row0;
      const uint32_t shared = g1 > g0 ? uni(s_from[g0]) : 0u;
      l = shared && rows * a.group <= (uint32_t)A::QT ? line_v<D, F8>(rows * a.group, shared * (64 / UT), hkv) : Line{0, 0, 0};
      base = (int32_t)(shared * 64);
      req = 0;
    }
    if (pos >= start + l.places) {
      start += l.places;
      before += l.places ? hkv * l.q : 0u;
      ++at;
      continue;
    }
    if (!own) req = lead_of(g0);
    const uint32_t len1 = A::kLeadV + l.units, item = (pos - start) / len1, first = start + item * len1;
    const uint32_t la = pos - first, n_here = min(len1 - la, end - pos);
    pos += n_here;
    if (la + n_here <= A::kLeadV) continue;
    const uint32_t ua = from + (la > A::kLeadV ? la - A::kLeadV : 0u), ub = from + la + n_here - A::kLeadV;
    const uint32_t tiles = (l.q + A::QT - 1) / A::QT, head = item / tiles, q0 = (item - head * tiles) * A::QT;
    const uint32_t nw = min((uint32_t)A::QT, l.q - q0);
    const uint64_t slot = region + before + head * l.q + q0 + (uint64_t)A::QT * wp;
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
  const int lane = threadIdx.x & 63;
  const uint32_t id = uni(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (id >= a.m * a.n_heads) return;
  const uint32_t row = id / a.n_heads, h = id - row * a.n_heads;
  const uint32_t* const hdr = reinterpret_cast<const uint32_t*>(a.ws);
  const u32x2 where = reinterpret_cast<const u32x2*>(a.ws + kSharedRow)[row];
  const uint32_t valid = hdr[0], per_w = hdr[1], per_v = hdr[2];
  if (!valid || where[0] == ~0u) return;
  const uint32_t* const r = reinterpret_cast<const uint32_t*>(a.ws + kSharedReq) + kRecWords * where[0];
  const uint32_t* const g = reinterpret_cast<const uint32_t*>(a.ws + kSharedGrp) + kRecWords * where[1];
  const uint32_t hkv = a.n_kv_heads, kvh = h / a.group, gq = h - kvh * a.group;
  const float2* const ml = reinterpret_cast<const float2*>(a.ws + kSharedMl);
  const uint64_t region = (uint64_t)a.m * a.n_heads + (uint64_t)kSharedGrid * A::QW;
  const float* const values =
      reinterpret_cast<const float*>(ml + region + 2ull * a.m * a.n_heads + (uint64_t)kSharedGrid * A::NW * 32);
  // the pieces with units of an item: workers w0 .. w0 + n - 1, slots `slot` + w step
  uint64_t g_slot = 0, r_slot = 0;
  uint32_t g_w0 = 0, g_n = 0, g_step = A::QT, r_w0 = 0, r_n = 0;
  if (g[2]) {
    const uint32_t nq_all = g[1], units = g[2], qi = (row - g[0]) * a.group + gq;
    if (g[5]) {
      const uint32_t full = nq_all / A::QW, one = A::kLeadW + units * A::cost(A::NW), tile = qi / A::QW;
      const bool last = tile == full;
      const uint32_t nq = last ? nq_all - full * A::QW : (uint32_t)A::QW, c = last ? A::cost((nq + A::QT - 1) / A::QT) : A::cost(A::NW);
      const uint32_t first = g[3] + (last ? full * hkv * one + kvh * (A::kLeadW + units * c) : (tile * hkv + kvh) * one);
      g_w0 = (first + A::kLeadW) / per_w;
      g_n = (first + A::kLeadW + (units - 1) * c) / per_w - g_w0 + 1;
      g_slot = (uint64_t)g[4] + tile * A::QW * hkv + kvh * nq + (qi - tile * A::QW);
      g_step = A::QW;
    } else {
      const uint32_t first = g[3] + kvh * (A::kLeadV + units);
      g_w0 = (first + A::kLeadV) / per_v;
      g_n = (first + A::kLeadV + units - 1) / per_v - g_w0 + 1;
      g_slot = region + g[4] + kvh * nq_all + qi;
    }
  }
  if (r[2]) {
    const uint32_t q = r[1], units = r[2], qi = (row - r[0]) * a.group + gq, tiles = (q + A::QT - 1) / A::QT;
    const uint32_t first = r[3] + (kvh * tiles + qi / A::QT) * (A::kLeadV + units);
    r_w0 = (first + A::kLeadV) / per_v;
    r_n = (first + A::kLeadV + units - 1) / per_v - r_w0 + 1;
    r_slot = region + r[4] + kvh * q + qi;
  }
  const uint32_t n = g_n + r_n;
  auto slot_of = [&](uint32_t i) {
    return i < g_n ? g_slot + (uint64_t)(g_w0 + i) * g_step : r_slot + (uint64_t)(r_w0 + i - g_n) * A::QT;
  };
  const float cs = fabsf(a.score_scale);
  float m = -INFINITY, l = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  const uint32_t sg = lane / L, d = 4 * (lane % L);
  for (uint32_t i0 = 0; i0 < n; i0 += 64) {
    float2 x = make_float2(-INFINITY, 0.f);
    if (i0 + lane < n) x = ml[slot_of(i0 + lane)];
    const float mx = fmaxf(m, wave_max(x.x));
    const float fade = m == -INFINITY ? 1.f : pow2((m - mx) * cs);   // (without a maximum: 0, or NaN that stays)
    const float f = x.x == -INFINITY ? 1.f : pow2((x.x - mx) * cs);
    l = l * fade + wave_sum(x.y * f);
    v *= fade;
    m = mx;
    const uint32_t here = min(64u, n - i0);
    for (uint32_t i = 0; i < here; i += SG) {
      const uint32_t k = i + sg;
      const float fk = __shfl(f, (int)min(k, 63u));
      if (k < here) v += *reinterpret_cast<const f32x4*>(values + slot_of(i0 + k) * D + d) * fk;
    }
  }
#pragma unroll
  for (int o = L; o < 64; o <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], o);
  const bool broken = r[5] == 0x80000000u;
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
    const uint64_t wg = (items * (units + A::kLeadV) / A::kLeastV + A::NW - 1) / A::NW;
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
