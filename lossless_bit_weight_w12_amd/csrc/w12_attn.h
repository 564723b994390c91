// Attention over the paged cache: what a wave does with a unit of tokens, shared by the kernels of
// w12_attn_paged (w12_attn.hip) and w12_attn_shared (w12_attn_shared.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace w12 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int32_t uniform_load(const int32_t* p, uint64_t i) {
  // read through the constant address space (a scalar load): nothing here writes it
  return reinterpret_cast<const __attribute__((address_space(4))) int32_t*>((uintptr_t)p)[i];
}
__device__ __forceinline__ uint32_t uni(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ uint32_t bf_pack(float a, float b) {   // round to nearest even, one instruction
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

__device__ __forceinline__ uint32_t f16_pack(float a, float b) {   // round to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, f16x2_t));
}

// 2^x as the hardware has it (one ulp; results below 2^-126 are zero, far below any rounding
// of a sum that holds the weight 1 of the maximum).
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Nothing is scheduled across: a load stays behind the products that free its registers.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Largest value (sum) over the four lanes that share a query row (l % 16).
__device__ __forceinline__ float group_max(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float group_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Inclusive sum over the wave, lane 63 with all of it (row shifts by 1, 2, 4, 8, then the rows'
// last lanes broadcast on).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

// Largest value (sum) over 16 lanes (a row of the wave), by rotations.
template <int R>
__device__ __forceinline__ float row_turn(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + R, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_turn<8>(v));
  v = fmaxf(v, row_turn<4>(v));
  v = fmaxf(v, row_turn<2>(v));
  return fmaxf(v, row_turn<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_turn<8>(v);
  v += row_turn<4>(v);
  v += row_turn<2>(v);
  return v + row_turn<1>(v);
}

// x / d from inv = floor(2^32 / d) (2^32 - 1 for d = 1): the product is x / d or one below.
__device__ __forceinline__ uint32_t div_by(uint32_t x, uint32_t d, uint32_t inv) {
  const uint32_t q = (uint32_t)(((uint64_t)x * inv) >> 32);
  return q + (x - q * d >= d ? 1u : 0u);
}

// One wave's work on a unit of UT tokens: NT tiles of 16 query rows, heads of D values.  (Of Args
// the cache's fields are read: table, page_shift, n_pages, n_kv_heads, kc, vc.)
template <int D, bool F8, int NT, int UT>
struct Tile {
  static constexpr int ES = F8 ? 1 : 2;          // bytes per cached value
  static constexpr int QT = 16 * NT;             // query rows of a tile
  static constexpr int KS = D / 32;              // matrix steps of a score
  static constexpr int KL = F8 ? KS / 2 : KS;    // 16-byte loads of one key per lane
  static constexpr int DT = D / 16;              // 16-dimension tiles of the output
  static constexpr int TT = UT / 16;             // 16-token tiles of a unit
  static constexpr int PS = UT / 32;             // matrix steps over a unit's tokens
  static constexpr int VL = F8 ? PS / 2 : PS;    // 16-byte loads of one dimension of V per lane
  // Weights of E4M3 values are times 2^15 (and so are their sums and products: the quotient is the
  // same), 32768 at most: FP16 keeps 11 bits of them down to 2^-29 of the largest, and a part of
  // them down to 2^-39.
  static constexpr float kUp = F8 ? 15.f : 0.f;

  // Page ids of a unit's 16-token groups; groups past `end` read page 0 (masked).
  struct Ids {
    u32x4 id;          // (a vector and no array: it has to stay in registers)
    uint32_t bad;      // bit j: group j holds tokens the tile sees and a page that is none
  };
  template <class Args>
  static __device__ __forceinline__ Ids load_ids(const Args& a, uint64_t trow, uint32_t u, uint32_t end) {
    Ids x = {{0u, 0u, 0u, 0u}, 0u};
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint32_t t = u * UT + 16 * j;
      const bool need = t < end;
      const uint32_t p = need ? (uint32_t)uniform_load(a.table, trow + (t >> a.page_shift)) : 0u;
      const bool ok = p < a.n_pages;
      x.bad |= ok ? 0u : 1u << j;
      x.id[j] = ok ? p : 0u;
    }
    return x;
  }

  static __device__ __forceinline__ u32x4 load16(const uint8_t* p) {
    return *reinterpret_cast<const u32x4*>(p);
  }

  // K of a unit: lane (row r = l % 16 of each token tile, group g) the 16 bytes g of each
  // 64-byte step of its token's key.
  template <class Args, class P>
  static __device__ __forceinline__ void load_k(const Args& a, const Ids& x, uint32_t u, uint32_t head,
                                                int lane, P&& put) {
    static_assert(!F8 || UT == 64, "an E4M3 lane load holds 16 tokens of a 64-token unit");
    const uint32_t r = lane & 15, g = lane >> 4, mask = (1u << a.page_shift) - 1u;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t tok = F8 ? 16 * (r >> 2) + 4 * t + (r & 3) : 32 * (t / 2) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3);
      uint32_t id;
      if constexpr (F8) {
        const uint32_t lo = (r & 4) ? x.id[1] : x.id[0], hi = (r & 4) ? x.id[3] : x.id[2];
        id = (r & 8) ? hi : lo;
      } else {
        id = (r & 8) ? x.id[2 * (t / 2) + 1] : x.id[2 * (t / 2)];
      }
      const uint32_t place = (u * UT + tok) & mask;
      const uint8_t* p = a.kc + ((((uint64_t)id * a.n_kv_heads + head) << a.page_shift) + place) * (D * ES) + 16 * g;
#pragma unroll
      for (int i = 0; i < KL; ++i) put(t, i, load16(p + 64 * i));
    }
  }

  // V^T of a unit: lane (dimension l % 16 of each dimension tile, group g) 16 bytes of
  // consecutive tokens: 32 s + 8 g .. + 7 (BF16), 16 g .. + 15 (E4M3).
  template <class Args, class P>
  static __device__ __forceinline__ void load_v(const Args& a, const Ids& x, uint32_t u, uint32_t head,
                                                int lane, P&& put) {
    static_assert(!F8 || UT == 64, "an E4M3 lane load holds 16 tokens of a 64-token unit");
    const uint32_t g = lane >> 4, mask = (1u << a.page_shift) - 1u;
#pragma unroll
    for (int s = 0; s < VL; ++s) {
      uint32_t id, tok;
      if constexpr (F8) {
        const uint32_t lo = (g & 1) ? x.id[1] : x.id[0], hi = (g & 1) ? x.id[3] : x.id[2];
        id = (g & 2) ? hi : lo;
        tok = 16 * g;
      } else {
        id = (g & 2) ? x.id[2 * s + 1] : x.id[2 * s];
        tok = 32 * s + 8 * g;
      }
      const uint32_t place = (u * UT + tok) & mask;
      const uint8_t* p = a.vc + (((((uint64_t)id * a.n_kv_heads + head) * D + (lane & 15)) << a.page_shift) + place) * ES;
      const uint32_t step = (16u * ES) << a.page_shift;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        put(d, s, load16(p));
        p += step;
      }
    }
  }

  // Operands of step s (32 dimensions or tokens) from the lane's loads: of the first product in
  // BF16, the type of q, of the second in BF16, or in FP16 for E4M3.
  template <int L>
  static __device__ __forceinline__ bf16x8_t operand(const u32x4 (&x)[L], int s) {
    if constexpr (F8) {
      u32x4 o;   // every E4M3 value is a BF16 value
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = x[s / 2][2 * (s & 1) + h];
        o[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
        o[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
      }
      return __builtin_bit_cast(bf16x8_t, o);
    } else {
      return __builtin_bit_cast(bf16x8_t, x[s]);
    }
  }

  template <int L>
  static __device__ __forceinline__ u32x4 operand_v(const u32x4 (&x)[L], int s) {
    if constexpr (F8) {
      u32x4 o;   // every E4M3 value is an FP16 value
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = x[s / 2][2 * (s & 1) + h];
        o[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        o[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
      }
      return o;
    } else {
      return x[s];
    }
  }
  static __device__ __forceinline__ f32x4 mfma_v(u32x4 v, u32x4 p, f32x4 o) {
    if constexpr (F8)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, v), __builtin_bit_cast(f16x8_t, p), o, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, p), o, 0, 0, 0);
  }

  // S^T of a unit.
  static __device__ __forceinline__ void scores(const u32x4 (&kf)[TT][KL], const bf16x8_t (&q)[NT][KS],
                                                f32x4 (&s)[NT][TT]) {
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const bf16x8_t kk = operand(kf[t], i);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[nt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[nt][i], s[nt][t], 0, 0, 0);
      }
      fence();
    }
  }

  // O^T += V^T P^T.
  static __device__ __forceinline__ void product(const u32x4 (&vf)[DT][VL], const u32x4 (&p)[NT][PS],
                                                 f32x4 (&o)[NT][DT]) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
#pragma unroll
      for (int i = 0; i < PS; ++i) {
        const u32x4 vv = operand_v(vf[d], i);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[nt][d] = mfma_v(vv, p[nt][i], o[nt][d]);
      }
      fence();
    }
  }

  // Scores of tokens in pages that are none.
  static __device__ __forceinline__ void spoil(uint32_t bad, int lane, f32x4 (&s)[NT][TT]) {
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t grp = F8 ? lane >> 4 : 2 * (t / 2) + (lane >> 5);
      if ((bad >> grp) & 1u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][t] = f32x4{NAN, NAN, NAN, NAN};
      }
    }
  }

  // One step of the running softmax of a query row: raw scores s to weights exp2(c (s - top)) for
  // the second product, their FP32 sum, and the old results faded where the maximum rose.
  // A weight enters the product in the type of V's operand.  BF16, 2^-8 of it at most: the sum is
  // that of the rounded weights, so that they add up to the divisor and the result is a mean of
  // the values seen (with the unrounded sum 64 equal values came back 2^-8 too small; no case's
  // time differs).  E4M3 values go in FP16, with 2^-11 of each weight, and their sum is taken as
  // it comes: 24 draft blocks 0.0017 of the norm from 64 bits, the rounding of the result alone, in
  // place of 0.0020, and 80 query rows 133 -> 130 us for the shorter sum.  BF16 weights in two parts
  // and a third product would bring the rest there too, 0.0016 in place of 0.0017, for 80 query
  // rows 146 -> 154 us and for prompts 169 -> 189 us: not taken.
  // top is the same in the four lanes of a row, sum is each lane's own part.  A NaN score leaves
  // the maximum alone and makes the sum NaN.
  template <bool EDGE>
  static __device__ __forceinline__ void weights(float c, uint32_t seen, f32x4 (&s)[TT], float& top, float& sum,
                                                 f32x4 (&o)[DT], u32x4 (&p)[PS]) {
    float mx = top;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, !EDGE || ((seen >> (4 * t + i)) & 1u) ? s[t][i] : -INFINITY);
    mx = group_max(mx);
    if (__any(mx > top)) {
      const float fade = top == -INFINITY ? 0.f : pow2((top - mx) * c);
      sum *= fade;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= fade;
      top = mx;
    }
    // (the distance from the maximum first, then its scaling: with c s - c top in one step and c top
    // rounded, scores past 2^22 gave weights that differed between units, past 2^31 NaN; it costs 1 %
    // at most: 24 requests with heads of 128 83.9 -> 84.9 us)
    const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = pow2(F8 ? fmaf(s[t][i] - base, c, kUp) : (s[t][i] - base) * c);
        s[t][i] = !EDGE || ((seen >> (4 * t + i)) & 1u) ? e : 0.f;
      }
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const f32x4 x = s[2 * i], y = s[2 * i + 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = (j < 2 ? x : y)[2 * (j & 1)], v = (j < 2 ? x : y)[2 * (j & 1) + 1];
        if constexpr (F8) {
          p[i][j] = f16_pack(u, v);
          sum += u;
          sum += v;
        } else {
          p[i][j] = bf_pack(u, v);
          sum += __uint_as_float(p[i][j] << 16);
          sum += __uint_as_float(p[i][j] & 0xffff0000u);
        }
      }
    }
    fence();
  }

  // Bytes of the lane's dword w (0..3) of load s that hold tokens below `end` (from the
  // lane's first token of the load).
  static __device__ __forceinline__ uint32_t token_mask(int32_t left, int w) {
    const int32_t n = left - (F8 ? 4 : 2) * w;   // tokens of this dword below the end
    constexpr int per = F8 ? 4 : 2;
    return n >= per ? 0xffffffffu : (n <= 0 ? 0u : (1u << (n * (F8 ? 8 : 16))) - 1u);
  }

  // The lane's first token of a unit that begins at `token`.
  static __device__ __forceinline__ int32_t lane_token(int32_t token, int lane) {
    return token + (F8 ? 16 : 8) * (lane >> 4);
  }

  // Weights of a unit (scores s, its first token) in which some row's tokens end, of the tokens
  // that each row sees, lim[nt] in all.
  static __device__ __forceinline__ void ends_weights(float cs, int32_t token, int lane, const int32_t (&lim)[NT],
                                                      f32x4 (&s)[NT][TT], float (&top)[NT], float (&sum)[NT],
                                                      f32x4 (&o)[NT][DT], u32x4 (&p)[NT][PS]) {
    const int32_t t_lane = lane_token(token, lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t seen = 0;   // bit 4t + i: the row sees the token
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t tok = t_lane + (F8 ? 4 * t + i : 32 * (t / 2) + 4 * (t & 1) + i);
          seen |= tok < lim[nt] ? 1u << (4 * t + i) : 0u;
        }
      weights<true>(cs, seen, s[nt], top[nt], sum[nt], o[nt], p[nt]);
    }
  }

  // Is a value of the tokens see_min .. see - 1, which some of the wave's rows see and some do not,
  // not finite?  In the product it would reach those that do not (0 * inf).
  static __device__ __forceinline__ bool odd_values(int32_t token, int lane, uint32_t see, int32_t see_min,
                                                    int32_t see_max, const u32x4 (&vf)[DT][VL]) {
    const int32_t t_lane = lane_token(token, lane);
    uint32_t odd = 0;
    if (see_min < see_max) {
#pragma unroll
      for (int l = 0; l < VL; ++l)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t look = token_mask((int32_t)see - (t_lane + 32 * l), w) &
                                ~token_mask(see_min - (t_lane + 32 * l), w) & (F8 ? 0x7f7f7f7fu : 0x7f807f80u);
#pragma unroll
          for (int d = 0; d < DT; ++d)   // E4M3 NaN: S.1111.111; BF16: exponent all ones
            odd |= (vf[d][l][w] & look) + (F8 ? 0x01010101u : 0x00800080u);
        }
      odd &= F8 ? 0x80808080u : 0x80008000u;
    }
    return __any(odd != 0);
  }

  // The product with the values of tokens below `upto`; zeros in the others' place, which may hold
  // anything.  take(nt): rows that it is for.
  template <class Take>
  static __device__ __forceinline__ void ends_product(int32_t token, int lane, int32_t upto, const u32x4 (&vf)[DT][VL],
                                                      const u32x4 (&p)[NT][PS], f32x4 (&o)[NT][DT], Take&& take) {
    const int32_t t_lane = lane_token(token, lane);
    uint32_t keep[VL][4];
#pragma unroll
    for (int l = 0; l < VL; ++l)
#pragma unroll
      for (int w = 0; w < 4; ++w) keep[l][w] = token_mask(upto - (t_lane + 32 * l), w);
    fence();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      u32x4 x[VL];
#pragma unroll
      for (int l = 0; l < VL; ++l)
#pragma unroll
        for (int w = 0; w < 4; ++w) x[l][w] = vf[d][l][w] & keep[l][w];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 sum_d = o[nt][d];
#pragma unroll
        for (int i = 0; i < PS; ++i)
          sum_d = mfma_v(operand_v(x, i), p[nt][i], sum_d);
        if (take(nt)) o[nt][d] = sum_d;   // a lane holds one row's sums
      }
      fence();
    }
  }

  // A unit (scores s, values vf) in which some row's tokens end.  see_min .. see_max: what the wave's
  // rows see, see: the last of that, or 0.  With odd values each row takes a product of its own.
  static __device__ __forceinline__ void ends(float cs, int32_t token, int lane, const int32_t (&lim)[NT], uint32_t see,
                                              int32_t see_min, int32_t see_max, const u32x4 (&vf)[DT][VL],
                                              f32x4 (&s)[NT][TT], float (&top)[NT], float (&sum)[NT],
                                              f32x4 (&o)[NT][DT]) {
    u32x4 p[NT][PS];
    ends_weights(cs, token, lane, lim, s, top, sum, o, p);
    const bool apart = odd_values(token, lane, see, see_min, see_max, vf);
    for (int32_t row = apart ? max(see_min, 1) : see_max; row <= see_max; ++row)
      ends_product(token, lane, row, vf, p, o, [&](int nt) { return !apart || lim[nt] == row; });
  }
};

}  // namespace

}  // namespace w12
