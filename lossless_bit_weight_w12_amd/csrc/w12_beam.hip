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
// Exponentials: exp2 of the hardware on the rounded product with log2(e), and the product's
// remainder to first order; sums of a thread in FP32, of threads and parts in FP64.  That keeps lse
// within about 1e-8, so the choice is that of FP64 unless scores are as close as that.
//
// Bound by HBM for many rows, else by the dependent steps behind the reads.
#include "w12.h"
#include "w12_beam.h"

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kCand = 1024;   // candidates of a part, at most

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

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) {
  return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), o) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)v, o);
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t u = shfl_xor64(v, o);
    v = u > v ? u : v;
  }
  return v;
}
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// exp(t), t <= 0.
__device__ __forceinline__ float exp_of(float t) {
  constexpr float kL = 1.44269502f, kLow = 1.92596299e-8f;   // log2(e)
  const float h = t * kL, r = fmaf(t, kL, -h) + t * kLow;
  const float e = __builtin_amdgcn_exp2f(h);
  return t > -100.f ? fmaf(e, r * 0.693147181f, e) : e;   // (t = -inf has no remainder)
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
__global__ __launch_bounds__(kBeamT) void k_beam(BeamArgs a) {
  constexpr int V = F32 ? 4 : 8, U = N / V, T = (int)kBeamT, W = T / 64;
  constexpr uint32_t kKeys = K > 16 ? 1024 : 640;   // keys of one row in LDS, per wave
  __shared__ union {
    struct {
      uint64_t cand[kCand];
      float most[T];
    } part;
    struct {
      uint64_t keys[W][kKeys];
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
  u32x4 raw[U];
  const uint32_t es = F32 ? 4 : 2;
  const uint8_t* const base = reinterpret_cast<const uint8_t*>(a.logits) + row * a.stride * es;
  const uint32_t skew = (uint32_t)((uintptr_t)base / es % V);   // the row's first value within its vector
  const uint32_t token_0 = split * T * N + t * V - skew;        // of this thread (below zero: before the row)
  constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;   // -inf
  if (row < a.n) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t e = token_0 + i * T * V;
      raw[i] = u32x4{kNone, kNone, kNone, kNone};
      if (e < a.vocab && e + V <= a.vocab) {
        raw[i] = *reinterpret_cast<const u32x4*>(base + (uint64_t)e * es);
      } else if ((int32_t)e > -V && (int32_t)e < (int32_t)a.vocab) {   // at an end of the row
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (e + j < a.vocab) {
            if constexpr (F32) {
              raw[i][j] = reinterpret_cast<const uint32_t*>(base)[(int32_t)(e + j)];
            } else {
              const uint32_t x = reinterpret_cast<const uint16_t*>(base)[(int32_t)(e + j)];
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
    uint32_t before = 0;
    for (uint32_t g = t; g <= a.n_grp; g += T) {
      const int32_t o = a.grp_off[g], next = g < a.n_grp ? a.grp_off[g + 1] : o;
      bad |= o < 0 || next < o || o > (int32_t)a.n || next - o > W12_MAX_BEAMS;
      before += o <= (int32_t)row;
    }
    before = wave_sum(before);
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
  const uint32_t grp = s_grp - 1;

  // ---- maximum, sum, and a bound that at least k values reach
  bool any = false;
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    any |= (int32_t)token(i, 0) > -V && (int32_t)token(i, 0) < (int32_t)a.vocab;   // (a vector may hold more than the row)
#pragma unroll
    for (int j = 0; j < V; ++j) most = fmaxf(most, at(i, j));
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
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) most = fmaxf(most, __shfl_xor(most, i));
  auto reach = [&](uint32_t v) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += (uint32_t)__popcll(__ballot(o[i] >= v));
    return c;
  };
  uint32_t bound = 1;
  if (reach(1) > k) {
    uint32_t hi = order(most) + 1;
    bound = min(min(o[0] ? o[0] : ~0u, o[1] ? o[1] : ~0u), min(o[2] ? o[2] : ~0u, o[3] ? o[3] : ~0u));
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) bound = min(bound, (uint32_t)__shfl_xor((int)bound, i));
    bound = __builtin_amdgcn_readfirstlane((int)bound);
    hi = __builtin_amdgcn_readfirstlane((int)hi);
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
  const float shift = most == -INFINITY ? 0.f : most;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) sum += exp_of(at(i, j) - shift);
  const double all = wave_sum((double)sum);
  if (lane == 0) s_sum[wave] = all;

  // ---- candidates, and the k best of them in order
  const bool plain = bound > order(-INFINITY);   // no NaN, no place outside the row reaches it
  const float at_least = value(bound);
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = at(i, j);
      const bool on = plain ? x >= at_least : token(i, j) < a.vocab && order(x) >= bound;
      if (on) {
        const uint32_t c = atomicAdd(&s_count, 1u);
        if (c < kCand) s.part.cand[c] = key_of(x, token(i, j));
      }
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
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint64_t key = key_of(at(i, j), token(i, j));
          if (token(i, j) < a.vocab && key < last && key > best) best = key;
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
  const uint32_t r0 = (uint32_t)a.grp_off[grp], rows = (uint32_t)a.grp_off[grp + 1] - r0;
  if (t == 0) {
    uint32_t* const ticket = reinterpret_cast<uint32_t*>(a.ws) + grp;
    s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == rows * S - 1;
    if (s_last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!s_last) return;
  // a wave per row: its lse, and its k best of the parts' lists (four at most a lane)
  for (uint32_t b = wave; b < rows; b += W) {
    const uint64_t first = (uint64_t)(r0 + b) * S;
    const uint64_t* const from = lists + first * k;
    const bool in_lds = S * k <= kKeys;
    if (in_lds)
      for (uint32_t i = lane; i < S * k; i += 64) s.join.keys[wave][i] = load_dev(from + i);
    float top = -INFINITY;
    for (uint32_t i = lane; i < S; i += 64) top = fmaxf(top, load_dev(&parts[first + i].top));
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    const double to = top == -INFINITY ? 0.0 : (double)top;
    double v = 0;
    for (uint32_t i = lane; i < S; i += 64) {
      const float x = load_dev(&parts[first + i].top);
      const double y = load_dev(&parts[first + i].sum);
      v += x == -INFINITY ? y : y * exp((double)x - to);   // (0, or NaN that stays)
    }
    v = wave_sum(v);
    if (lane == 0) s.join.lse[b] = (top == -INFINITY ? -(double)INFINITY : to) + log(v);
    auto key = [&](uint32_t l, uint32_t p) -> uint64_t {
      if (l >= S || p >= k) return 0;
      return in_lds ? s.join.keys[wave][l * k + p] : load_dev(from + l * k + p);
    };
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();   // one wave writes and reads: LDS keeps the order
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    uint64_t head[4];
    uint32_t pos[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) head[i] = key(lane + 64 * i, 0);
    for (uint32_t r = 0; r < k; ++r) {
      uint64_t best = head[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) best = head[i] > best ? head[i] : best;
      const uint64_t won = wave_max64(best);
      if (lane == 0) s.join.rows[b][r] = won;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (won && head[i] == won) head[i] = key(lane + 64 * i, ++pos[i]);   // keys are distinct
    }
  }
  __syncthreads();
  if (wave != 0) return;
  // a lane per row: the best score of all, lower rows first
  const bool on = lane < rows;
  const double base_score = on ? (double)a.scores[r0 + lane] : 0.0;
  uint32_t pos = 0;
  uint64_t key = 0, ord = 0;
  double score = 0;
  auto next = [&] {
    key = on && pos < k ? s.join.rows[lane][pos] : 0;
    score = base_score + ((double)value((uint32_t)(key >> 32)) - s.join.lse[lane]);
    score = score == score ? score : -(double)INFINITY;
    ord = key ? order64(score) : 0;
    ++pos;
  };
  next();
  for (uint32_t r = 0; r < k; ++r) {
    const uint64_t won = wave_max64(ord), tied = __ballot(ord == won);
    const uint64_t out = (uint64_t)grp * k + r;
    if (won == 0) {
      if (lane == 0) {
        a.parent[out] = a.token[out] = -1;
        a.out[out] = -INFINITY;
      }
    } else if ((int)lane == __ffsll((unsigned long long)tied) - 1) {
      a.parent[out] = (int32_t)(r0 + lane);
      a.token[out] = (int32_t)~(uint32_t)key;
      a.out[out] = (float)score;
      next();
    }
  }
}

template <bool F32, int N>
hipError_t beam_go(const BeamArgs& a, hipStream_t s) {
  const dim3 grid(a.splits, a.n ? a.n : 1);
  if (a.k <= kBeamShort) hipLaunchKernelGGL((k_beam<F32, N, (int)kBeamShort>), grid, dim3(kBeamT), 0, s, a);
  else hipLaunchKernelGGL((k_beam<F32, N, W12_MAX_BEAM_K>), grid, dim3(kBeamT), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_select(const BeamArgs& given, bool f32, hipStream_t s) {
  BeamArgs a = given;
  a.splits = beam_splits(a.n, a.vocab, a.k);
  const bool many = beam_values(a.n, a.vocab, a.k) == kBeamMany;
  if (f32) return many ? beam_go<true, (int)kBeamMany>(a, s) : beam_go<true, (int)kBeamFew>(a, s);
  return many ? beam_go<false, (int)kBeamMany>(a, s) : beam_go<false, (int)kBeamFew>(a, s);
}

}  // namespace w12
