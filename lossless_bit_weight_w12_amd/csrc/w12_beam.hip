// The choice of the beams that go on (w12_beam_select).
//
// Mathematics: score(row, token) = scores[row] + logit - lse(row), lse the logarithm of the row's sum
// of exponentials, in FP64; a group's k best.  Within a row the order is the logits' own, so a part
// of a row needs no lse to give its k best: one pass reads the logits into registers, once, takes
// the part's maximum, its sum of exponentials and its k best, and the workgroup of a group that is
// through last joins the rows' parts and then the rows.
//
// The k best of a part: of its threads' largest values about the k-th, by bisection with the counts of
// ballots; whatever reaches that is a candidate (slightly more than k of them, as a rule), and the
// candidates' ranks among themselves give their order.  Where equal values make them too many,
// the k are taken one after the other.
//
// Exponentials: exp2 of the hardware, whose own error is the only one that is left (see Exps); sums in FP64.
// That keeps lse within 1e-7 whatever the logits are, so the choice is that of FP64 unless scores are as close
// as that.  (Terms are alike in a row of few values, and behind one that stands out, and then so are their
// roundings: sums of a thread in FP32 were off by up to 2.5e-6.  They took 19.6 us in place of 20.3 for 96 rows
// in BF16; terms of exactly reduced arguments 23.0.)
//
// Bound by the dependent steps behind the reads: 4 rows of 151936 FP32 logits 12.3 us, of them 4 for the
// part, 1.2 for the ticket, 5 for the join; 96 rows in BF16 (29 MB, 4.9 us of reading) 20.3, of them 8 to
// 13 for the part; k = 64 takes 24 to 28 us more.  Tickets of a call lie as far apart as their 16 KB allow: beside
// each other in one line they passed one after the other, 18 ns each (38 us in place of 20).
#include "w12.h"
#include "w12_beam.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // in memory, at an element's alignment

constexpr uint32_t kCand = 1024;   // candidates of a part, at most
constexpr uint32_t kRanked = 128;  // of a row

// Values as whole numbers of the same order: -0 as 0, NaN as -inf; nothing gives 0.
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x == x ? x + 0.f : -INFINITY);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t order64(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x == x ? x + 0.0 : -(double)INFINITY);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) { return (uint64_t)order(x) << 32 | (uint32_t)~token; }

// Over the wave's lanes, the result in all of them: maxima of whole numbers, sums of FP64.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));   // within rows of 16 lanes
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xf, 0xf, false));   // a row's last lane to the next row
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xf, 0xf, false));   // lane 31 to the upper half
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint64_t with = __ballot((uint32_t)(v >> 32) == hi);
  if ((with & (with - 1)) == 0)   // one lane alone, as a rule
    return (uint64_t)hi << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, __ffsll((unsigned long long)with) - 1);
  return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
template <int C, int Rows>
__device__ __forceinline__ double add_from(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, Rows, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), C, Rows, 0xf, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v = add_from<0x111, 0xf>(v);
  v = add_from<0x112, 0xf>(v);
  v = add_from<0x114, 0xf>(v);
  v = add_from<0x118, 0xf>(v);
  v = add_from<0x142, 0xa>(v);
  v = add_from<0x143, 0xc>(v);
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 63) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63));
}

// What a part's exponentials are relative to: exp(0), so that nothing is lost in a difference, or, where the
// largest value is far from 0, that.  (From 64 on, FP32 values less than 32 below it differ from it by 24 bits at
// most, BF16 values from 32 on, and below -24 those less than 24 below it, so that the difference is exact; what
// lies lower is 2^21 values of e^-24 at most.)
template <bool F32>
__device__ __forceinline__ float base_of(float top) {
  return (top >= -24.f && top < (F32 ? 64.f : 32.f)) || top == -INFINITY ? 0.f : top;
}

// Sum of exp(x).  x log2(e) is taken as h + l, h in FP32: exp2 of the hardware of h (off by 8.5e-8 of itself at
// most, over all h), and what l makes of it to first order, l exp2(h), in a sum of its own.  With log2(e) in 24
// bits, h is rounded and l what that leaves out, 2^-18 at most; for BF16 values below 32, in 16 bits, h is exact
// and l the rest of log2(e), 7.1e-6 of x (whose second order is 1.3e-8 of a term where x is 32).  Below -150 a
// term is nothing (the largest is 2^-35 at least), -inf among them.
template <bool Bits16>
struct Exps {
  static constexpr float kL = Bits16 ? 1.44268798828125f : 1.44269502f;
  static constexpr float kLow = Bits16 ? 7.05260771e-6f : 1.92596299e-8f;   // log2(e) - kL
  double sum = 0;
  float rest = 0.f;
  __device__ __forceinline__ void add(float given) {
    const float x = __builtin_elementwise_maximum(given, -150.f);   // (NaN stays)
    const float h = x * kL, e = __builtin_amdgcn_exp2f(h);
    sum += (double)e;
    rest = fmaf(e, Bits16 ? x : fmaf(x, kLow, fmaf(x, kL, -h)), rest);
  }
  __device__ __forceinline__ double all() const {
    return sum + (double)rest * ((Bits16 ? (double)kLow : 1.0) * 0.6931471805599453);
  }
};

// LDS that the wave has written and reads: it keeps the order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct Part {   // of a row, in the workspace
  float top;
  uint32_t pad;
  double sum;
};

template <class F>
__device__ __forceinline__ F load_dev(const F* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <class F>
__device__ __forceinline__ void store_dev(F* p, F v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// V values per vector of 16 bytes, N values of a thread, lists of up to K.
template <bool F32, int N, int K>
__global__ __launch_bounds__(kBeamT, K > 16 ? 2 : 4) void k_beam(BeamArgs a) {
  constexpr int V = F32 ? 4 : 8, U = N / V, T = (int)kBeamT, W = T / 64;
  constexpr uint32_t kKeys = K > 16 ? 1024 : 640;   // keys of one row in a wave's registers
  __shared__ union {
    struct {
      uint64_t cand[kCand];
      float most[T];
    } part;
    struct {
      uint64_t keys[W][kRanked];
      uint64_t rows[W12_MAX_BEAMS][K];
      double lse[W12_MAX_BEAMS];
    } join;
  } s;
  __shared__ uint64_t s_best[W];
  __shared__ double s_sum[W];
  __shared__ uint32_t s_count, s_grp, s_last;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const uint32_t split = blockIdx.x, row = blockIdx.y, k = a.k, S = a.splits;
  Part* const parts = reinterpret_cast<Part*>(a.ws + kBeamTickets);
  uint64_t* const lists = reinterpret_cast<uint64_t*>(parts + (uint64_t)a.n * S);

  // ---- the part's values, requested first
  // (Dealt by token, wherever the row begins: rows with the same logits have the same sums, bit for bit, and
  // so the same scores.  Rows that begin inside a vector take loads across lines for it.)
  u32x4 raw[U];
  const uint32_t es = F32 ? 4 : 2;
  const uint8_t* const base = reinterpret_cast<const uint8_t*>(a.logits) + row * a.stride * es;
  const uint32_t token_0 = split * T * N + t * V;   // of this thread
  constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;   // -inf
  if (row < a.n) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t e = token_0 + i * T * V;
      raw[i] = u32x4{kNone, kNone, kNone, kNone};
      if (e + V <= a.vocab) {
        raw[i] = *reinterpret_cast<const u32x4_any*>(base + (uint64_t)e * es);
      } else if (e < a.vocab) {   // at the row's end
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (e + j < a.vocab) {
            if constexpr (F32) {
              raw[i][j] = reinterpret_cast<const uint32_t*>(base)[e + j];
            } else {
              const uint32_t x = reinterpret_cast<const uint16_t*>(base)[e + j];
              raw[i][j / 2] = j & 1 ? (raw[i][j / 2] & 0xffffu) | x << 16 : (raw[i][j / 2] & 0xffff0000u) | x;
            }
          }
      }
    }
  }
  auto at = [&](int i, int j) {
    if constexpr (F32) return __uint_as_float(raw[i][j]);
    else return __uint_as_float(j & 1 ? raw[i][j / 2] & 0xffff0000u : raw[i][j / 2] << 16);
  };
  auto token = [&](int i, int j) { return token_0 + i * T * V + j; };

  // ---- the row's group
  if (t == 0) s_grp = s_count = 0;
  __syncthreads();
  {
    bool bad = false;
    uint32_t before = 0;   // groups that begin at this row or before it
    for (uint32_t g0 = 0; g0 <= a.n_grp; g0 += T) {
      const uint32_t g = g0 + t;
      bool here = false;
      if (g <= a.n_grp) {
        const int32_t o = a.grp_off[g], next = a.grp_off[g < a.n_grp ? g + 1 : g];
        bad |= o < 0 || next < o || o > (int32_t)a.n || next - o > W12_MAX_BEAMS;
        here = o <= (int32_t)row;
      }
      before += (uint32_t)__popcll(__ballot(here));
    }
    if (lane == 0 && before) atomicAdd(&s_grp, before);
    bad = __syncthreads_or(bad);
    if (split == 0 && row == 0)   // groups without rows, and a table that is none
      for (uint64_t i = t; i < (uint64_t)a.n_grp * k; i += T) {
        const uint32_t g = (uint32_t)(i / k);
        if (!bad && a.grp_off[g] < a.grp_off[g + 1]) continue;
        a.parent[i] = a.token[i] = -1;
        a.out[i] = bad ? NAN : -INFINITY;
      }
    if (bad || row >= a.n || s_grp == 0 || s_grp > a.n_grp) return;
  }
  const uint32_t grp = s_grp - 1, r0 = (uint32_t)a.grp_off[grp], rows = (uint32_t)a.grp_off[grp + 1] - r0;

  // ---- maximum, sum, and a bound that at least k values reach
  const bool any = token_0 < a.vocab;
  float most = -INFINITY, vec[U];   // of the vectors too
#pragma unroll
  for (int i = 0; i < U; ++i) {
    vec[i] = at(i, 0);
#pragma unroll
    for (int j = 1; j < V; ++j) vec[i] = fmaxf(vec[i], at(i, j));
    most = fmaxf(most, vec[i]);
  }
  s.part.most[t] = any ? most : NAN;
  __syncthreads();
  uint32_t o[4];   // of all threads, four a lane: every wave does the same
  {
    const float4 x = reinterpret_cast<const float4*>(s.part.most)[lane];
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = f[i] == f[i] ? order(f[i]) : 0u;
      most = fmaxf(most, f[i]);
    }
  }
  const uint32_t top = wave_max(order(most));
  most = value(top);
  auto reach = [&](uint32_t v) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += (uint32_t)__popcll(__ballot(o[i] >= v));
    return c;
  };
  uint32_t bound = 1;
  if (reach(1) > k) {
    uint32_t hi = top + 1;
    const uint32_t low = min(min(o[0] - 1, o[1] - 1), min(o[2] - 1, o[3] - 1));   // (0, none, wraps round)
    bound = ~wave_max(~low) + 1;
    while (hi - bound > 1) {
      const uint32_t mid = bound + (hi - bound) / 2, c = reach(mid);
      if (c < k) {
        hi = mid;
      } else {
        bound = mid;
        if (c <= k + k / 4 + 1) break;
      }
    }
  }
  auto packed = [&] {   // values are taken from the vectors anew, rather than held
#pragma unroll
    for (int i = 0; i < U; ++i) asm volatile("" : "+v"(raw[i]));
  };
  packed();
  const float from = base_of<F32>(most);
  double all;
  if (from == 0.f) {
    Exps<!F32> exps;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) exps.add(at(i, j));
    all = wave_sum(exps.all());
  } else {
    Exps<false> exps;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) exps.add(at(i, j) - from);
    all = wave_sum(exps.all());
  }
  if (lane == 0) s_sum[wave] = all;

  // ---- candidates, and the k best of them in order
  packed();
  auto found = [&](float x, uint32_t tok) {
    const uint32_t c = atomicAdd(&s_count, 1u);
    if (c < kCand) s.part.cand[c] = key_of(x, tok);
  };
  if (bound > order(-INFINITY)) {   // no NaN, no place outside the row reaches it
    const float at_least = value(bound);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (vec[i] >= at_least) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (at(i, j) >= at_least) found(at(i, j), token(i, j));
      }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (token(i, j) < a.vocab && order(at(i, j)) >= bound) found(at(i, j), token(i, j));
  }
  __syncthreads();
  const uint64_t mine = (uint64_t)row * S + split;
  uint64_t* const list = lists + mine * k;
  if (t == 0) {
    double v = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) v += s_sum[w];
    store_dev(&parts[mine].top, most);
    store_dev(&parts[mine].sum, v);
  }
  const uint32_t count = s_count;
  if (count <= kCand) {
    for (uint32_t c = t; c < count; c += T) {
      const uint64_t key = s.part.cand[c];
      uint32_t rank = 0;
      for (uint32_t i = 0; i < count; ++i) rank += s.part.cand[i] > key;
      if (rank < k) store_dev(list + rank, key);
    }
    for (uint32_t c = count + t; c < k; c += T) store_dev(list + c, (uint64_t)0);
  } else {   // too many equal values: one after the other
    uint64_t last = ~0ull;
    for (uint32_t r = 0; r < k; ++r) {
      uint64_t best = 0;
      packed();
      uint32_t tok = token_0;
      asm volatile("" : "+v"(tok));   // (nor are the tokens held)
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint64_t key = key_of(at(i, j), tok + i * T * V + j);
          if (tok + i * T * V + j < a.vocab && key < last && key > best) best = key;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      best = wave_max64(best);
      if (lane == 0) s_best[wave] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) best = s_best[w] > best ? s_best[w] : best;
      if (t == 0) store_dev(list + r, best);
      last = best;
      __syncthreads();
    }
  }

  // ---- the group's last workgroup joins
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (t == 0) {
    uint32_t* const ticket = reinterpret_cast<uint32_t*>(a.ws) + grp * (4096 / a.n_grp);
    s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == rows * S - 1;
    if (s_last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!s_last) return;
  // a wave per row: its lse, and its k best of the parts' lists
  const double base_score = lane < rows ? (double)a.scores[r0 + lane] : 0.0;   // (of the last step, requested now)
  for (uint32_t b = wave; b < rows; b += W) {
    const uint64_t first = (uint64_t)(r0 + b) * S;
    const uint64_t* const from = lists + first * k;
    const uint32_t all = S * k;
    uint64_t v[kKeys / 64];
    if (all <= kKeys) {
#pragma unroll
      for (uint32_t i = 0; i < kKeys / 64; ++i) v[i] = lane + 64 * i < all ? load_dev(from + lane + 64 * i) : (uint64_t)0;
    }
    float tops[4];
    double sums[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const bool on = lane + 64 * i < S;
      tops[i] = on ? load_dev(&parts[first + lane + 64 * i].top) : -INFINITY;
      sums[i] = on ? load_dev(&parts[first + lane + 64 * i].sum) : 0.0;
    }
    const uint32_t top_order = wave_max(order(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]))));
    const float top = value(top_order);
    const double to = base_of<F32>(top);
    double all_sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (64u * i < S)   // (without a maximum: 0, or NaN that stays)
        all_sum += tops[i] == -INFINITY ? sums[i] : sums[i] * exp((double)base_of<F32>(tops[i]) - to);
    all_sum = wave_sum(all_sum);
    if (lane == 0) s.join.lse[b] = to + log(all_sum);
    // As in a part: a bound that at least k keys reach and not many more, and those by their ranks among
    // themselves.  (Taking the largest head of the lists k times took 0.2 us a time.)
    uint32_t count = kRanked + 1;
    if (all <= kKeys) {
      auto reach = [&](uint32_t x) {
        uint32_t c = 0;
#pragma unroll
        for (uint32_t i = 0; i < kKeys / 64; ++i)
          if (64 * i < all) c += (uint32_t)__popcll(__ballot((uint32_t)(v[i] >> 32) >= x));
        return c;
      };
      uint32_t low = 1;
      count = reach(1);
      if (count > k + k / 2 + 8) {
        uint32_t mine = 0;   // (64 keys at least reach the least of the lanes' largest)
#pragma unroll
        for (uint32_t i = 0; i < kKeys / 64; ++i) mine = max(mine, (uint32_t)(v[i] >> 32));
        uint32_t high = top_order + 1;
        low = max(~wave_max(~mine), 1u);
        count = reach(low);
        while (high - low > 1 && count > k + k / 2 + 8) {
          const uint32_t mid = low + (high - low) / 2, c = reach(mid);
          if (c < k) {
            high = mid;
          } else {
            low = mid;
            count = c;
          }
        }
      }
      if (count <= kRanked) {
        uint64_t* const list = s.join.keys[wave];
        uint32_t at = 0;
#pragma unroll
        for (uint32_t i = 0; i < kKeys / 64; ++i)
          if (64 * i < all) {
            const bool in = (uint32_t)(v[i] >> 32) >= low;
            const uint64_t with = __ballot(in);
            if (in) list[at + (uint32_t)__popcll(with & ((1ull << lane) - 1ull))] = v[i];
            at += (uint32_t)__popcll(with);
          }
        wave_sync();
        const uint64_t x = lane < count ? list[lane] : 0, y = lane + 64 < count ? list[lane + 64] : 0;
        uint32_t rx = 0, ry = 0;
        for (uint32_t i = 0; i < count; ++i) {
          const uint64_t z = list[i];
          rx += z > x;
          ry += z > y;
        }
        if (lane < count && rx < k) s.join.rows[b][rx] = x;
        if (lane + 64 < count && ry < k) s.join.rows[b][ry] = y;
        if (lane >= count && lane < k) s.join.rows[b][lane] = 0;   // (there are no more)
      }
    }
    if (count > kRanked) {   // more keys than that, or too many equal logits: one after the other
      auto key = [&](uint32_t l, uint32_t p) { return l < S && p < k ? load_dev(from + l * k + p) : (uint64_t)0; };
      uint64_t head[4], next[4], mine = 0;
      uint32_t pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        head[i] = key(lane + 64 * i, 0u);
        next[i] = key(lane + 64 * i, 1u);
        pos[i] = 1;
      }
      for (uint32_t r = 0; r < k; ++r) {
        uint64_t best = head[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) best = head[i] > best ? head[i] : best;
        const uint64_t won = wave_max64(best);
        mine = lane == r ? won : mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool here = head[i] == won;   // keys are distinct but for 0, which nothing follows
          head[i] = here ? next[i] : head[i];
          pos[i] += here;
          next[i] = key(lane + 64 * i, pos[i]);
        }
      }
      if (lane < k) s.join.rows[b][lane] = mine;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  auto score_of = [&](uint64_t key, double base, double lse) {
    const double score = base + ((double)value((uint32_t)(key >> 32)) - lse);
    return score == score ? score : -(double)INFINITY;
  };
  if (rows * k <= 64) {   // a lane per pair, by its rank; equal scores in the order of the lanes
    const uint32_t r = lane / k, p = lane - r * k;
    const bool on = r < rows;
    const uint64_t key = on ? s.join.rows[on ? r : 0][p] : 0;
    const uint64_t bits = __builtin_bit_cast(uint64_t, base_score);
    const double base = __builtin_bit_cast(double, (uint64_t)(uint32_t)__shfl((int)(bits >> 32), (int)(r & 63)) << 32 |
                                                       (uint32_t)__shfl((int)(uint32_t)bits, (int)(r & 63)));
    const double score = score_of(key, base, on ? s.join.lse[r] : 0.0);
    const uint64_t ord = key ? order64(score) : 0;
    uint32_t rank = 0;
    for (uint32_t i = 0; i < rows * k; ++i) {
      const uint64_t z = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(ord >> 32), (int)i) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)ord, (int)i);
      rank += z > ord || (z == ord && i < lane);
    }
    const uint32_t found = (uint32_t)__popcll(__ballot(ord != 0));
    const uint64_t at_out = (uint64_t)grp * k;
    if (ord && rank < k) {
      a.parent[at_out + rank] = (int32_t)(r0 + r);
      a.token[at_out + rank] = (int32_t)~(uint32_t)key;
      a.out[at_out + rank] = (float)score;
    }
    if (lane >= found && lane < k) {
      a.parent[at_out + lane] = a.token[at_out + lane] = -1;
      a.out[at_out + lane] = -INFINITY;
    }
    return;
  }
  // a lane per row: the best score of all, lower rows first
  const bool on = lane < rows;
  const double lse = on ? s.join.lse[lane] : 0.0;
  uint32_t pos = 1;
  auto ahead = [&](uint32_t p) {
    const uint64_t v = s.join.rows[on ? lane : 0u][p < k ? p : 0u];
    return on && p < k ? v : (uint64_t)0;
  };
  uint64_t key = ahead(0), next = ahead(1);
  int32_t parent = -1, tok = -1;   // of the lane's place in the answer
  float out = -INFINITY;
  for (uint32_t r = 0; r < k; ++r) {
    const double score = score_of(key, base_score, lse);
    const uint64_t ord = key ? order64(score) : 0, won = wave_max64(ord);
    if (won == 0) break;
    const int w = __ffsll((unsigned long long)__ballot(ord == won)) - 1;
    const int32_t token_w = (int32_t)~(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, w);
    const float score_w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint((float)score), w));
    if (lane == r) {
      parent = (int32_t)r0 + w;
      tok = token_w;
      out = score_w;
    }
    const bool here = (int)lane == w;
    key = here ? next : key;
    pos += here;
    next = ahead(pos);
  }
  if (lane < k) {
    const uint64_t at_out = (uint64_t)grp * k + lane;
    a.parent[at_out] = parent;
    a.token[at_out] = tok;
    a.out[at_out] = out;
  }
}

template <bool F32, int N>
hipError_t beam_go(const BeamArgs& a, hipStream_t s) {
  const dim3 grid(a.splits, a.n ? a.n : 1);
  if (N < 64 || a.k <= kBeamShort) hipLaunchKernelGGL((k_beam<F32, N, (int)kBeamShort>), grid, dim3(kBeamT), 0, s, a);
  else if constexpr (N == 64) hipLaunchKernelGGL((k_beam<F32, N, W12_MAX_BEAM_K>), grid, dim3(kBeamT), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_select(const BeamArgs& given, bool f32, hipStream_t s) {
  BeamArgs a = given;
  a.splits = beam_splits(a.n, a.vocab, a.k);
  switch (beam_values(a.n, a.vocab, a.k)) {
    case 16: return f32 ? beam_go<true, 16>(a, s) : beam_go<false, 16>(a, s);
    case 32: return f32 ? beam_go<true, 32>(a, s) : beam_go<false, 32>(a, s);
    default: return f32 ? beam_go<true, 64>(a, s) : beam_go<false, 64>(a, s);
  }
}

}  // namespace w12
