// Attention of a decode step's new rows over the paged cache (w12_attn_paged).
//
// Mathematics: per request, key head and tile of query rows (a query row is a pair of a batch
// row and one of the group's query heads), one pass over the tokens with the running maximum
// and sum of the softmax.  Both products run on the matrix cores with the tokens as the
// rows of the first and the summed index of the second:
//   S^T [token][query] = K Q^T,   O^T [dim][query] += V^T P^T,
// so that a lane keeps one query row (column l % 16) through both, and the scores it computes
// are the weights it feeds back: the matrix core leaves lane group g = l / 16 with rows 4g ..
// 4g + 3 of each 16-token tile and wants 8 consecutive summed indices of it, and since the
// order in which tokens are dealt to tile rows is free, tile row 4a + i takes the token that
// makes a lane's scores 8 (BF16) or 16 (E4M3) consecutive tokens: the ones its 16-byte loads
// of V^T hold.  Nothing has to pass through LDS inside the loop, and every load is 16 bytes
// used as it comes.
//
// Where several tiles of query rows read the same keys, their waves can read K and V from LDS
// instead: a step of 64 KB, in the operands' own order (so the reads have no conflicts), which
// the waves fetch together while they work on the step before it.
//
// Split: the work of all requests, heads and tiles is one line of units of UT tokens, cut into
// equal pieces, one per workgroup; inside a piece each wave takes every NW-th unit.  Lengths
// can be as uneven as they like and a single long request still fills the chip.  A workgroup
// joins its waves in LDS; an item (request, tile, head) cut by a piece's border is joined by
// the workgroup that finishes it last, in piece order, so the result does not depend on
// which that is.
//
// Bound by HBM where there is enough to read (24 requests, 98k tokens, 8 key heads of 128 in
// BF16, 423 MB: 84 us, 5.0 TB/s over the call and 5.9 in the loop; one request of 131k tokens,
// 537 MB: 105 us, 5.1 TB/s), else by the dependent steps around the loop (one request of 17
// tokens: 6 us; of 4096: 13 us).
#include "w12.h"
#include "w12_attn.h"
#include "w12_kv.h"

namespace w12 {

namespace {

// Workgroups of a launch, at most (one ticket each): one per CU; with one tile of query rows, so
// that the registers allow it, two or four where a unit's K and V (`bytes`) are so small that
// four waves do not keep enough reads in flight (64 requests of up to 8191 tokens with heads of
// 64: in BF16 117 -> 109 us with two, in E4M3 90 -> 71 us with two, 68 us with four).
constexpr uint32_t workgroups(int nt, int bytes) {
  return nt > 1 || bytes > 16384 ? 256 : (bytes > 8192 ? 512 : 1024);
}
constexpr uint32_t kTicketBytes = 4096;

// Partial results pass between workgroups on any XCD, whose L2 caches are not coherent for
// plain accesses: stores and loads at device scope (sc1), a ticket taken after the stores
// are complete.
constexpr int kCpolDevice = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ws_rsrc(const float* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), (short)0,
                                           (int)(W12_ATTN_WS_BYTES - kTicketBytes), 0x00020000);
}
__device__ __forceinline__ void st_dev4(__amdgpu_buffer_rsrc_t rs, uint32_t off, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, off, 0, kCpolDevice);
}
__device__ __forceinline__ void st_dev2(__amdgpu_buffer_rsrc_t rs, uint32_t off, float a, float b) {
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(a), __float_as_uint(b)}, rs, off, 0, kCpolDevice);
}
__device__ __forceinline__ f32x4 ld_dev4(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, kCpolDevice));
}
__device__ __forceinline__ u32x2 ld_dev2(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, kCpolDevice);
}

// One request: its rows and what it lays on the line.
struct Req {
  int32_t row0, len;
  uint32_t rows;
  bool broken;       // len is none
  uint32_t units;    // units of UT tokens of an item (at least one, which may be empty)
  uint32_t tiles;    // tiles of query rows, per key head
};

// One item (request, tiles, head) as its output needs it, and its pieces if it is cut.
struct Item {
  int32_t row0;          // the request's first row
  int32_t base;          // tokens that row sees
  bool broken;
  uint32_t head, q0, nq; // query rows q0 .. q0 + nq - 1 of the head
  uint32_t w0, w1, late; // workgroups with a piece; 1: the first one's second partial
};

template <int D, bool F8, int NT, int NW, int UT, bool ST>
struct Attn : Tile<D, F8, NT, UT> {
  static constexpr int ES = F8 ? 1 : 2;          // bytes per cached value
  static constexpr int ROW = D + 4;              // LDS row of the join, padded
  static constexpr int T = 64 * NW;
  // Staged (ST): a step of SU units (64 KB) passes through LDS, CB wave loads of K and of V per
  // unit; a wave fetches K or V of one unit.
  static constexpr uint32_t SU = NW / 2;
  static constexpr uint32_t CB = UT * D * 2 / 1024;
  static_assert(!ST || (!F8 && UT * D == 8192), "64 KB per step");
  static constexpr uint32_t kWG = workgroups(NT, 2 * UT * D * ES);
  // What an item costs a workgroup beside its units (its queries' load, the join, the writes:
  // about 15000 cycles under load, the time of 128 KB), in units.
  static constexpr uint32_t kLead = 131072 / (2 * UT * D * ES);
};

template <int D, bool F8, int NT, int NW, int UT, bool ST>
__global__ __launch_bounds__(64 * NW, workgroups(NT, 2 * UT * D * (F8 ? 1 : 2)) / 256) void k_attn(AttnArgs given) {
  using A = Attn<D, F8, NT, NW, UT, ST>;
  constexpr int QT = A::QT, KS = A::KS, DT = A::DT, TT = A::TT, PS = A::PS, T = A::T;
  // the waves' results, and later the (max, sum) pairs of an item's pieces
  constexpr uint32_t kJoin = sizeof(float) * NT * NW * 16 * A::ROW, kStep = A::SU * 2 * A::CB * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t s_buf[ST && 2 * kStep > kJoin ? 2 * kStep : kJoin];
  constexpr uint32_t kPairs = sizeof(s_buf) / sizeof(float2);
  static_assert(kPairs >= A::kWG, "one row of every piece");
  auto& s_o = *reinterpret_cast<float (*)[NT][NW][16][A::ROW]>(s_buf);
  float2* const s_ml = reinterpret_cast<float2*>(s_buf);
  __shared__ float s_m[NW][QT], s_l[NW][QT];
  __shared__ uint32_t s_scan[NW], s_line[NW], s_few[NW], s_items[NW], s_bad[NW];
  __shared__ uint32_t s_start[5];
  __shared__ uint32_t s_last[2];
  __shared__ uint32_t s_spoil[2][A::SU];   // staged: Ids::bad of the step's units
  __shared__ Item s_cut[2];   // (in LDS: scalar registers are short)
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = uni(tid >> 6);
  const uint32_t hkv = given.n_kv_heads, n_req = given.n_req;

  auto request = [&](int32_t row0, int32_t row1, int32_t len) {
    Req q;
    q.row0 = row0;
    q.len = len;
    q.rows = (uint32_t)(row1 - row0);
    q.broken = len < 0 || (uint64_t)len > ((uint64_t)given.max_pages << given.page_shift);
    q.units = q.broken || len == 0 ? 1u : ((uint32_t)len + UT - 1) / UT;
    q.tiles = (q.rows * given.group + QT - 1) / QT;
    return q;
  };

  // ---- the line, and this workgroup's piece of it
  const uint32_t per_t = (n_req + T - 1) / T;
  auto mine_at = [&](uint32_t i) {   // this thread's i-th request
    const uint32_t r = tid * per_t + i;
    return r < n_req ? request(given.req_off[r], given.req_off[r + 1], given.kv_len[r]) : Req{0, 0, 0, false, 1, 0};
  };
  const Req mine_0 = mine_at(0);   // the only one up to T requests: loaded once
  auto mine = [&](uint32_t i) { return i == 0 ? mine_0 : mine_at(i); };
  uint32_t all_units = 0, few_units = 0, all_items = 0;   // with items of one tile, of NW tiles
  // (the host layer keeps the whole line below 2^31)
  bool bad = false;
  for (uint32_t i = 0; i < per_t; ++i) {
    const Req q = mine(i);
    bad |= q.row0 < 0 || (int32_t)q.rows < 0 || (int64_t)q.row0 + q.rows > (int64_t)given.m;
    all_units += q.tiles * hkv * q.units;
    few_units += (q.tiles + NW - 1) / NW * hkv * q.units;
    all_items += q.tiles * hkv;
  }
  all_units = wave_scan(all_units);
  few_units = wave_scan(few_units);
  all_items = wave_scan(all_items);
  bad = __any(bad);
  if (lane == 63) {
    s_scan[wave] = all_units;
    s_few[wave] = few_units;
    s_items[wave] = all_items;
    s_bad[wave] = bad;
  }
  __syncthreads();
  all_units = few_units = all_items = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    all_units += uni(s_scan[w]);
    few_units += uni(s_few[w]);
    all_items += uni(s_items[w]);
    bad |= uni(s_bad[w]) != 0;
  }
  if (bad) {   // no request table: NaN everywhere
    const uint64_t all = (uint64_t)given.m * given.n_heads * D;
    for (uint64_t i = (uint64_t)blockIdx.x * T + tid; i < all; i += (uint64_t)given.grid * T) {
      const uint64_t row = i / (given.n_heads * D);
      given.out[row * given.out_stride + i % (given.n_heads * D)] = 0x7fc0u;
    }
    return;
  }
  // A long item is a tile, or, where there is work for every workgroup anyway, up to NW tiles of
  // one head, one for each wave, so that K and V are read once for all of them (16 rows of 5
  // heads each against 98k tokens: 202 us apart, 146 us together; but 8 heads of 1 to 4 rows
  // against 10k tokens, 2 units per workgroup: 22 us apart, 29 us together).
  auto per_grid = [&](uint32_t x) { return div_by(x, given.grid, given.grid_inv); };
  const uint32_t span = all_units >= 16 * given.grid ? NW : 1u;   // tiles of a long item, at most
  const uint32_t mean = min(per_grid((span > 1 ? few_units : all_units) + given.grid - 1), 1u << 20);
  auto wide = [&](const Req& q) { return span > 1 ? (q.tiles + NW - 1) / NW : q.tiles; };   // long items per head
  // A long item has a lead of kLead places on the line, then one per unit; its units may fall
  // into several pieces.  A brief one (few enough units that a wave does better with an
  // item of its own than all waves one after the other: with k = mean / units items per
  // piece, (k - 1) kLead >= units) is never cut: it belongs to the piece it begins in.
  auto brief = [&](const Req& q) { return !ST && q.units < 4096 && q.units * (q.units + A::kLead) <= A::kLead * mean; };
  auto lead = [&](const Req& q) { return brief(q) ? (A::kLead + NW - 1) / NW : A::kLead; };
  auto places = [&](const Req& q) { return lead(q) + q.units; };   // of one item
  auto items = [&](const Req& q) { return (brief(q) ? q.tiles : wide(q)) * hkv; };
  uint32_t line = 0;
  for (uint32_t i = 0; i < per_t; ++i) {
    const Req q = mine(i);
    line += items(q) * places(q);
  }
  uint32_t upto = wave_scan(line);
  if (lane == 63) s_line[wave] = upto;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t v = uni(s_line[w]);
    if (w < (int)wave) upto += v;
    total += v;
  }
  // Equal pieces.  While there are more workgroups than needed a piece is as long as the join
  // of an item's pieces pays for (with p of them the item takes units / p + p join_cost), and
  // of at least 4 units, so that a workgroup's waves share an item before it is cut; but of
  // no more than the mean item.
  const float units = all_items ? (float)all_units / (float)all_items : 1.f;   // of the mean item
  const uint32_t least = (uint32_t)fminf(units, fmaxf(4.f, __builtin_amdgcn_sqrtf(units * given.join_cost)));
  const uint32_t per = uni(max(per_grid(total + given.grid - 1), least));
  const uint32_t here = blockIdx.x * per;   // where the piece begins
  uint32_t pos = here;
  const uint32_t end = min(pos + per, total);
  if (pos >= total) return;
  // What the line does not need is read from the arguments here: the compiler would load it at
  // the kernel's entry, have no scalar registers for it, and wait for it three times before the
  // first request is read (one request of 17 tokens 6.35 us, 6.2 us so).
  AttnArgs a = given;
  {
    auto late = (const __attribute__((address_space(4))) AttnArgs*)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(late));
    a.q = late->q;
    a.q_stride = late->q_stride;
    a.out_stride = late->out_stride;
    a.n_pages = late->n_pages;
    a.kc = late->kc;
    a.vc = late->vc;
    a.table = late->table;
    a.score_scale = late->score_scale;
    a.v_scale = late->v_scale;
    a.out = late->out;
    a.tickets = late->tickets;
    a.partial = late->partial;
  }
  if (pos >= upto - line && pos < upto) {   // one thread: the request it starts in
    uint32_t at = upto - line;
    uint32_t i = 0;
    Req q = mine(0);
    while (pos >= at + items(q) * places(q)) {
      at += items(q) * places(q);
      q = mine(++i);
    }
    s_start[0] = tid * per_t + i;
    s_start[1] = at;
    s_start[2] = (uint32_t)q.row0;
    s_start[3] = q.rows;
    s_start[4] = (uint32_t)q.len;
  }
  __syncthreads();
  uint32_t r = uni(s_start[0]), start = uni(s_start[1]);   // a request and its place on the line

  const float cs = fabsf(a.score_scale);
  const uint32_t flip = a.score_scale < 0.f ? 0x80008000u : 0u;
  const __amdgpu_buffer_rsrc_t rs = ws_rsrc(a.partial);
  constexpr uint32_t kSlot = NW * QT * (D + 2) * 4;   // bytes of one partial: values, then (max, sum)
  auto per_group = [&](uint32_t x) { return div_by(x, a.group, a.group_inv); };
  auto out_at = [&](const Item& t, uint32_t qi) {   // query row qi of the item
    const uint32_t row = per_group(t.q0 + qi), gq = t.q0 + qi - row * a.group;
    return a.out + (uint64_t)(t.row0 + row) * a.out_stride + (uint64_t)(t.head * a.group + gq) * D;
  };
  auto scale_of = [&](const Item& t, uint32_t qi, float l) {
    const int32_t sees = t.base + (int32_t)per_group(t.q0 + qi);
    return t.broken ? NAN : (sees > 0 ? a.v_scale / l : 0.f);   // (without a token the values are 0)
  };
  auto put = [](uint16_t* p, f32x4 v, float f) {
    *reinterpret_cast<u32x2*>(p) = u32x2{bf_pack(v[0] * f, v[1] * f), bf_pack(v[2] * f, v[3] * f)};
  };
  uint32_t n_cut = 0;   // items that the piece's borders cut: two at most
  auto load_req = [&](uint32_t i) {
    return request(uniform_load(a.req_off, i), uniform_load(a.req_off, i + 1), uniform_load(a.kv_len, i));
  };
  Req now = request((int32_t)uni(s_start[2]), (int32_t)(uni(s_start[2]) + uni(s_start[3])), (int32_t)uni(s_start[4]));
  // From item i of request r (which begins at place s): on to the k-th brief item, over
  // requests without items; false if the piece or the run of brief items ends before.
  auto skip = [&](uint32_t& i_r, uint32_t& s, Req& q, uint32_t& i, uint32_t k) {
    i += k;
    while (i >= items(q)) {
      i -= items(q);
      s += items(q) * places(q);
      if (s >= end) return false;
      q = load_req(++i_r);
      if (q.tiles && !brief(q)) {
        i = 0;
        return false;
      }
    }
    return s + i * places(q) < end;
  };

  while (pos < end) {
    while (pos >= start + items(now) * places(now)) {
      start += items(now) * places(now);
      now = load_req(++r);
    }
    const bool alone = brief(now);   // a wave takes an item by itself
    Req q = now;
    uint32_t r_item, item, first = 0, ua = 0, ub;
    if (alone) {
      uint32_t at = start;
      r_item = r;
      item = (pos - start + places(now) - 1) / places(now);
      uint32_t next = item;
      const bool have = skip(r_item, at, q, item, wave);
      skip(r, start, now, next, NW);
      pos = start + next * places(now);
      if (!have) continue;
      ub = q.units;
    } else {
      const uint32_t len1 = places(now), ld = lead(now);
      item = pos - start < len1 ? 0u : (pos - start) / len1;
      first = start + item * len1;
      const uint32_t la = pos - first, n_here = min(len1 - la, end - pos);
      pos += n_here;
      if (la + n_here <= ld) continue;   // only its lead falls into this piece
      r_item = r;
      ua = la > ld ? la - ld : 0u;
      ub = la + n_here - ld;
    }
    {
      // ---- units [ua, ub) of item (r_item, tile, head)
      const int32_t row0 = q.row0;
      const bool broken = q.broken;
      // a wave's rows: a tile of its own; a long item of up to NW tiles deals its waves out to
      // them, and waves of the same tile take units in turn
      const uint32_t per_head = alone ? q.tiles : wide(q);
      const uint32_t head = per_head == 1 ? item : item / per_head, q0 = (item - head * per_head) * (alone ? 1u : span) * QT;
      const uint32_t nq = min((alone ? 1u : span) * QT, q.rows * a.group - q0);
      const uint32_t deal = alone || nq <= (uint32_t)QT ? 1u : (nq <= 2u * QT ? 2u : (uint32_t)NW);   // tiles dealt to
      const uint32_t sub = alone ? 0u : wave & (deal - 1), turn = alone ? 0u : wave / deal;
      const uint32_t stride = alone ? 1u : NW / deal;
      const uint32_t qw = q0 + sub * QT, nw = nq > sub * QT ? min((uint32_t)QT, nq - sub * QT) : 0u;   // the wave's rows
      const int32_t base = broken ? -(1 << 30) : q.len - (int32_t)q.rows + 1;   // what the request's row 0 sees
      const int32_t see_min = base + (int32_t)per_group(qw);
      const int32_t see_max = nw ? base + (int32_t)per_group(qw + nw - 1) : 0;
      // units past what the tile's last row sees are passed over
      const uint32_t see = see_max > 0 ? (uint32_t)see_max : 0u;
      const uint32_t uz = min(ub, (see + UT - 1) / UT);

      int32_t lim[NT];
      bf16x8_t qf[NT][KS];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t qi = qw + nt * 16 + (lane & 15);
        const uint32_t row = per_group(qi), gq = qi - row * a.group;
        const bool on = nt * 16 + (lane & 15) < (int)nw;
        lim[nt] = on ? base + (int32_t)row : 0;
        const uint16_t* p = a.q + (uint64_t)(row0 + (on ? row : 0u)) * a.q_stride +
                            (uint64_t)(head * a.group + (on ? gq : 0u)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int d = F8 ? 64 * (s / 2) + 16 * (lane >> 4) + 8 * (s & 1) : 32 * s + 8 * (lane >> 4);
          u32x4 w = *reinterpret_cast<const u32x4*>(p + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] ^= flip;
          qf[nt][s] = __builtin_bit_cast(bf16x8_t, w);
        }
      }
      f32x4 o[NT][DT];
      float top[NT], sum[NT];   // running maximum of the raw scores, this lane's part of the sum
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = -INFINITY;
        sum[nt] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[nt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
      }

      const uint64_t trow = (uint64_t)r_item * a.max_pages;
      u32x4 kf[TT][A::KL], vf[DT][A::VL];
      // a unit (kf, vf) in which some row's tokens end
      auto ends_in = [&](uint32_t u, uint32_t spoilt, auto&& values) {
        f32x4 s[NT][TT];
        A::scores(kf, qf, s);
        values();
        if (spoilt) A::spoil(spoilt, lane, s);
        A::ends(cs, (int32_t)(u * UT), lane, lim, see, see_min, see_max, vf, s, top, sum, o);
      };
      if constexpr (ST) {
        // A step ahead: while the waves work on a step in one half of the buffer, the next is on
        // its way to their registers and goes to the other half.
        const uint32_t see_all = (uint32_t)max(base + (int32_t)per_group(q0 + nq - 1), 0);
        const uint32_t uz_all = min(ub, (see_all + UT - 1) / UT);
        const uint32_t of_step = wave / 2;   // the step's unit that this wave fetches
        const bool of_v = wave & 1;          // its V, or its K
        u32x4 st[A::CB];
        uint32_t spoils = 0;
        auto fetch = [&](uint32_t u0) {
          const uint32_t u = u0 + of_step;
          if (u >= uz_all) return;
          const typename A::Ids x = A::load_ids(a, trow, u, see_all);
          spoils = x.bad;
          if (of_v) A::load_v(a, x, u, head, lane, [&](int d, int i, u32x4 v) { st[d * A::VL + i] = v; });
          else A::load_k(a, x, u, head, lane, [&](int t, int i, u32x4 v) { st[t * A::KL + i] = v; });
        };
        __syncthreads();   // the buffer is free
        fetch(ua);
        uint32_t u0 = ua, b = 0;
        auto step = [&](auto&& unit) {
          if (u0 + of_step < uz_all) {
            u32x4* const to = reinterpret_cast<u32x4*>(s_buf + b * kStep) + wave * A::CB * 64 + lane;
#pragma unroll
            for (uint32_t c = 0; c < A::CB; ++c) to[c * 64] = st[c];
            if (lane == 0) s_spoil[b][of_step] = spoils;
          }
          fetch(u0 + A::SU);
          __syncthreads();
          for (uint32_t k = turn; k < A::SU && u0 + k < uz; k += stride) {
            const u32x4* const from = reinterpret_cast<const u32x4*>(s_buf + b * kStep) + k * 2 * A::CB * 64 + lane;
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
              for (int i = 0; i < KS; ++i) kf[t][i] = from[(t * KS + i) * 64];
            unit(u0 + k, uni(s_spoil[b][k]), [&] {   // (not before: the registers of K are free then)
              fence();
#pragma unroll
              for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < PS; ++i) vf[d][i] = from[(A::CB + d * PS + i) * 64];
              fence();
            });
          }
          u0 += A::SU;
          b ^= 1;
        };
        // (one loop with both forms of a unit would hold the results twice)
        const int32_t see_first = base + (int32_t)per_group(q0);   // what the item's first row sees
        const uint32_t full_all = min(uz_all, see_first > 0 ? (uint32_t)see_first / UT : 0u);
        while (u0 + A::SU <= full_all)
          step([&](uint32_t, uint32_t spoilt, auto&& values) {
            f32x4 s[NT][TT];
            A::scores(kf, qf, s);
            values();
            if (spoilt) A::spoil(spoilt, lane, s);
            u32x4 p[NT][PS];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) A::template weights<false>(cs, 0u, s[nt], top[nt], sum[nt], o[nt], p[nt]);
            A::product(vf, p, o);
          });
        while (u0 < uz_all) step(ends_in);
      } else {
        auto load_k = [&](const typename A::Ids& x, uint32_t u) {
          A::load_k(a, x, u, head, lane, [&](int t, int i, u32x4 v) { kf[t][i] = v; });
        };
        auto load_v = [&](const typename A::Ids& x, uint32_t u) {
          A::load_v(a, x, u, head, lane, [&](int d, int i, u32x4 v) { vf[d][i] = v; });
        };
        uint32_t u = ua + turn;
        typename A::Ids ids = {{0u, 0u, 0u, 0u}, 0u};
        if (u < uz) {
          ids = A::load_ids(a, trow, u, see);
          load_k(ids, u);
          load_v(ids, u);
        }
        // full units: every row sees every token; the next unit's pages, K and V are requested as
        // soon as the registers they go to are free
        const uint32_t full = min(uz, see_min > 0 ? (uint32_t)see_min / UT : 0u);
        for (; u < full; u += stride) {
          const bool more = u + stride < uz;
          typename A::Ids next = ids;
          if (more) next = A::load_ids(a, trow, u + stride, see);
          f32x4 s[NT][TT];
          A::scores(kf, qf, s);
          fence();
          if (more) load_k(next, u + stride);
          fence();
          if (ids.bad) A::spoil(ids.bad, lane, s);
          u32x4 p[NT][PS];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) A::template weights<false>(cs, 0u, s[nt], top[nt], sum[nt], o[nt], p[nt]);
          fence();
          A::product(vf, p, o);
          fence();
          if (more) {
            load_v(next, u + stride);
            ids = next;
          }
        }
        for (; u < uz; u += stride) {
          ends_in(u, ids.bad, [] {});
          if (u + stride < uz) {
            ids = A::load_ids(a, trow, u + stride, see);
            load_k(ids, u + stride);
            load_v(ids, u + stride);
          }
        }
      }

      // (values of the thread's place, hidden from the optimiser: it would compute what the
      // join needs before the loops above and keep it there, in registers they have not got)
      const int tj = opaque(tid), lj = tj & 63;
      Item it = {row0, base, broken, head, q0, nq, 0, 0, 0};
      if (alone) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float l = group_sum(sum[nt]);
          const uint32_t qi = nt * 16 + (lj & 15);
          if (qi < nq) {
            uint16_t* const p = out_at(it, qi) + 4 * (lj >> 4);
            const float f = scale_of(it, qi, l);
#pragma unroll
            for (int d = 0; d < DT; ++d) put(p + 16 * d, o[nt][d], f);
          }
        }
        continue;
      }

      // ---- the waves' results joined in LDS
      const uint32_t real = first + lead(q);   // the item's first unit on the line
      const uint32_t w0 = real >= here ? blockIdx.x : real / per;   // (it reaches into this piece)
      const uint32_t w1 = real + q.units <= end ? blockIdx.x : (real + q.units - 1) / per;
      const bool whole = w0 == w1;
      const uint32_t late = first > w0 * per ? 1u : 0u;   // the first piece's second partial
      const uint32_t my_slot = (blockIdx.x * 2 + (blockIdx.x == w0 ? late : 0u)) * kSlot;
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float l = group_sum(sum[nt]);
        if (lj < 16) {
          s_m[wave][nt * 16 + lj] = top[nt];
          s_l[wave][nt * 16 + lj] = l;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<f32x4*>(&s_o[nt][wave][lj & 15][16 * d + 4 * (lj >> 4)]) = o[nt][d];
      }
      __syncthreads();
      // a row's factors once, in place of the maxima
      for (uint32_t row = tj; row < nq; row += T) {
        const uint32_t tile = row / QT, n = row % QT;
        float t[NW], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int j = 0; j < NW; ++j)   // the waves that share the tile
          t[j] = j < (int)stride ? s_m[tile + j * deal][n] : -INFINITY;
#pragma unroll
        for (int j = 0; j < NW; ++j) m = fmaxf(m, t[j]);
#pragma unroll
        for (int j = 0; j < NW; ++j)
          if (j < (int)stride) {
            const float f = t[j] == -INFINITY ? 1.f : pow2((t[j] - m) * cs);   // (without a maximum: 0, or NaN that stays)
            l += s_l[tile + j * deal][n] * f;
            s_m[tile + j * deal][n] = f;
          }
        s_l[tile][n] = l;
        if (!whole) st_dev2(rs, my_slot + (NW * QT * D + 2 * row) * 4, m, l);
      }
      __syncthreads();
#pragma unroll 2
      for (uint32_t e = tj; e < nq * (D / 4); e += T) {
        const uint32_t row = e / (D / 4), d = 4 * (e % (D / 4));   // of the item
        const uint32_t tile = row / QT, nt = row % QT / 16, n = row % 16;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NW; ++j)
          if (j < (int)stride)
            v += *reinterpret_cast<const f32x4*>(&s_o[nt][tile + j * deal][n][d]) * s_m[tile + j * deal][nt * 16 + n];
        if (whole) put(out_at(it, row) + d, v, scale_of(it, row, s_l[tile][nt * 16 + n]));
        else st_dev4(rs, my_slot + (row * D + d) * 4, v);
      }
      if (!whole) {   // its values are on their way to the workspace
        it.w0 = w0;
        it.w1 = w1;
        it.late = late;
        if (tid == 0) s_cut[n_cut] = it;
        ++n_cut;
      }
    }
  }

  // ---- the items that the piece's borders cut: the workgroup that is through with one last
  // joins its pieces in order
  if (n_cut == 0) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid < (int)n_cut) {
    uint32_t* const ticket = a.tickets + s_cut[tid].w0;
    const uint32_t old = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last[tid] = old == s_cut[tid].w1 - s_cut[tid].w0;
    if (s_last[tid]) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  for (uint32_t i = 0; i < n_cut; ++i) {
    if (!uni(s_last[i])) continue;
    const Item& t = s_cut[i];
    const Item c = {(int32_t)uni(t.row0), (int32_t)uni(t.base), uni(t.broken) != 0, uni(t.head), uni(t.q0),
                    uni(t.nq), uni(t.w0), uni(t.w1), uni(t.late)};
    // as many rows at a time as the pieces' maxima and sums leave room for in LDS
    const uint32_t pieces = c.w1 - c.w0 + 1;   // at most A::kWG
    const uint32_t most = min(c.nq, kPairs / pieces);
    auto slot_of = [&](uint32_t w) { return ((c.w0 + w) * 2 + (w == 0 ? c.late : 0u)) * kSlot; };
    // the values, PU places of a thread and B pieces of each in flight: another
    // workgroup's write takes about 5000 cycles to read, and only the number of reads at
    // once helps; the first ones are requested together with the maxima
    constexpr uint32_t PU = QT * (D / 4) / T < 4 ? 1 : (NT == 1 ? 2 : 4), B = 16 / PU;
    for (uint32_t n0 = 0; n0 < c.nq; n0 += most) {
      const uint32_t rows = min(most, c.nq - n0), n_places = rows * (D / 4);
      f32x4 x[PU][B];
      auto request_values = [&](uint32_t e, uint32_t w) {
        // (places and pieces past the end: an offset past the buffer, which reads as zero)
#pragma unroll
        for (uint32_t i = 0; i < PU; ++i)
#pragma unroll
          for (uint32_t b = 0; b < B; ++b) {
            const bool on = e + i * T < n_places && w + b < pieces;
            x[i][b] = ld_dev4(rs, on ? slot_of(w + b) + (n0 * (D / 4) + e + i * T) * 16 : 0x7ffffff0u);
          }
      };
      request_values(tid, 0);
      // 16 lanes per row: its pieces' maxima and sums, each lane's own kept in LDS, and
      // turned into factors there; two rows at once
      for (uint32_t n1 = tid >> 4; n1 < rows; n1 += 2 * T / 16) {
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 2
        for (uint32_t w = tid & 15; w < pieces; w += 16) {
          u32x2 ml[2];
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k)
            if (n1 + k * (T / 16) < rows)
              ml[k] = ld_dev2(rs, slot_of(w) + (NW * QT * D + 2 * (n0 + n1 + k * (T / 16))) * 4);
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k)
            if (n1 + k * (T / 16) < rows) {
              s_ml[w * rows + n1 + k * (T / 16)] = make_float2(__uint_as_float(ml[k][0]), __uint_as_float(ml[k][1]));
              m[k] = fmaxf(m[k], __uint_as_float(ml[k][0]));
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) m[k] = row_max(m[k]);
        for (uint32_t w = tid & 15; w < pieces; w += 16)
#pragma unroll
          for (uint32_t k = 0; k < 2; ++k)
            if (n1 + k * (T / 16) < rows) {
              const float2 ml = s_ml[w * rows + n1 + k * (T / 16)];
              const float f = ml.x == -INFINITY ? 1.f : pow2((ml.x - m[k]) * cs);
              l[k] += ml.y * f;
              s_ml[w * rows + n1 + k * (T / 16)].x = f;
            }
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
          const float all = row_sum(l[k]);
          if ((tid & 15) == 0 && n1 + k * (T / 16) < rows) (&s_l[0][0])[n1 + k * (T / 16)] = all;
        }
      }
      __syncthreads();
      bool there = true;   // the first values were requested above
      for (uint32_t e = tid; e < n_places; e += PU * T) {
        f32x4 v[PU];
#pragma unroll
        for (uint32_t i = 0; i < PU; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (uint32_t w = 0; w < pieces; w += B) {
          if (!there) request_values(e, w);
          there = false;
#pragma unroll
          for (uint32_t i = 0; i < PU; ++i) {
            const uint32_t n = min(e + i * T, n_places - 1) / (D / 4);
#pragma unroll
            for (uint32_t b = 0; b < B; ++b) v[i] += x[i][b] * s_ml[min(w + b, pieces - 1) * rows + n].x;
          }
        }
#pragma unroll
        for (uint32_t i = 0; i < PU; ++i)
          if (e + i * T < n_places) {
            const uint32_t n = (e + i * T) / (D / 4);
            put(out_at(c, n0 + n) + 4 * ((e + i * T) % (D / 4)), v[i], scale_of(c, n0 + n, (&s_l[0][0])[n]));
          }
      }
      __syncthreads();
    }
  }
}

template <int D, bool F8, int NT, int NW, int UT, bool ST = false>
hipError_t attn_go(const AttnArgs& a, hipStream_t s) {
  using A = Attn<D, F8, NT, NW, UT, ST>;
  // no more workgroups than units that the widest table could fill
  const uint64_t tiles = ((uint64_t)a.m * a.group + (uint64_t)a.n_req * (16 * NT - 1)) / (16 * NT) + 1;
  const uint64_t units = (((uint64_t)a.max_pages << a.page_shift) + UT - 1) / UT;
  uint64_t wg = A::kWG;
  if (units < wg && tiles * a.n_kv_heads * units < wg) wg = tiles * a.n_kv_heads * units;
  // What one more piece costs the join of an item, in units: a read's latency, and the values
  // of its rows at 30 bytes per cycle against a unit's at 10.
  const uint64_t mean = ((uint64_t)a.m + a.n_req - 1) / a.n_req * a.group;
  AttnArgs b = a;
  b.join_cost = 0.3f + (float)(mean < 16 * NT * NW ? mean : 16 * NT * NW) * 4.f / (6.f * UT * (F8 ? 1 : 2));
  static_assert(A::kWG * 2ull * NW * 16 * NT * (D + 2) * 4 <= W12_ATTN_WS_BYTES - kTicketBytes, "workspace");
  static_assert(A::kWG * 4 <= kTicketBytes, "tickets");
  b.grid = (uint32_t)wg;
  b.grid_inv = wg == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / wg);
  hipLaunchKernelGGL((k_attn<D, F8, NT, NW, UT, ST>), dim3((uint32_t)wg), dim3(64 * NW), 0, s, b);
  return hipGetLastError();
}

// Tile of query rows by the mean number per request: 16 while it holds them, else 32 (what the
// registers hold; with a head_dim of 256 that is 16).  Units of 64 tokens in E4M3 (16 bytes of
// V^T).  In BF16 of 32 where 64 do not fit (256), and at 128, where a short request's one unit
// is half the work (300 requests of up to 100 tokens 24 us with 64, 19 us with 32; one of 17
// tokens 7.7 and 6.2 us; 98k tokens in 24 requests 83 and 84 us, 131k in one 103 and 105 us; 25
// query rows each 94 us with 64, 91 us with 32); 64 for more than two tiles, whose waves take a
// tile each and read the same unit at once (80 query rows each 165 us with 32, 146 us with 64).
// Staged through LDS (BF16) where several waves read a tile of K and V often enough.  How long the
// requests are is not known here, only how wide the table is, and on short ones staging loses
// (the step's barriers, no items of a wave's own, and where the work does not suffice for items of
// several tiles nothing is shared): so it is taken where long ones gain more than that.
// With a head_dim of 256, whose waves hold 16 rows, from the second tile on (24 requests of up to
// 8000 tokens, 4 key heads, 32 / 48 / 64 / 128 / 256 query rows each: 110 -> 98, 139 -> 111, 163 ->
// 123, 303 -> 207 and 583 -> 364 us; 8 of up to 500, 32 / 64 / 128 rows 16.4 -> 16.8, 24 -> 26, 29 ->
// 31 us; one of 4096, 64 / 128 rows 22.5 -> 25, 52 -> 44 us; prompts of 64 to 300 tokens, 512 rows
// each, 38 -> 45 us).  With 128 for more than one item's tiles and pages of 64 or more, where a load
// of V^T touches 16 lines (24 requests of up to 8000 tokens, 256 rows each 215 -> 157 us, four prompts
// 244 -> 169 us; one of 4096 30 -> 32 us, 8 of up to 500 28 -> 31 us); below, the long ones gain less
// (128 rows, pages of 64, 121 -> 101 us, 80 rows 95 -> 87 us; 256 rows, pages of 32, 174 -> 154 us, of
// 16, 166 -> 154 us) and the short ones lose as much (256 rows, pages of 16, one of 4096 tokens 29 ->
// 32 us, 8 of up to 500 26 -> 30 us).  With 64 prompts lose (four of 256 rows and up to 4096 tokens
// 119 -> 124 us), and in E4M3, whose decoding costs a wave as much as the wait, 80 rows take 129
// us either way.
template <int D, bool F8>
hipError_t attn_rows(const AttnArgs& a, hipStream_t s) {
  const uint64_t rows = ((uint64_t)a.m + a.n_req - 1) / a.n_req * a.group;
  // Can there be items of several tiles?  With tables as wide as they are, as the kernel decides
  // it: 16 units for each of 256 workgroups.
  [[maybe_unused]] auto shared = [&](uint64_t tile, uint64_t unit) {
    const uint64_t tiles = ((uint64_t)a.m * a.group + a.n_req * (tile - 1)) / tile * a.n_kv_heads;
    return tiles * ((((uint64_t)a.max_pages << a.page_shift) + unit - 1) / unit) >= 16 * 256;
  };
  if constexpr (D < 256) {
    if (rows > 16) {
      if constexpr (D == 128 && !F8)
        if (rows <= 32) return attn_go<D, F8, 2, 4, 32>(a, s);
      if constexpr (D == 128 && !F8)
        if (rows > 128 && a.page_shift >= 6 && shared(32, 64)) return attn_go<D, F8, 2, 4, 64, true>(a, s);
      return attn_go<D, F8, 2, 4, 64>(a, s);
    }
  }
  if constexpr (D == 256 && !F8)
    if (rows > 16 && shared(16, 32)) return attn_go<D, F8, 1, 4, 32, true>(a, s);
  return attn_go<D, F8, 1, 4, F8 || D < 128 ? 64 : 32>(a, s);
}

template <bool F8>
hipError_t attn_dim(const AttnArgs& a, uint32_t d, hipStream_t s) {
  if (d == 64) return attn_rows<64, F8>(a, s);
  if (d == 128) return attn_rows<128, F8>(a, s);
  return attn_rows<256, F8>(a, s);
}

}  // namespace

hipError_t launch_attn_paged(const AttnArgs& a, uint32_t head_dim, uint32_t dtype, hipStream_t s) {
  return dtype == W12_KV_E4M3 ? attn_dim<true>(a, head_dim, s) : attn_dim<false>(a, head_dim, s);
}

}  // namespace w12
