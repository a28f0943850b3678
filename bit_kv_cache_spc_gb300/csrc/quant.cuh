// The quantiser's rules, shared by the kernels that code groups
// (quantize.cu, extend.cu): parameters, codes and thresholds of a group, and
// where its (min, max) words lie in the record.
#pragma once

#include "common.cuh"

namespace spc {

// z and s from the group's min and max, in binary32 exactly as written
// (the __f*_rn intrinsics are never contracted into FMA).
__device__ __forceinline__ void quant_params(int bits, float lo, float hi, float& z, float& s) {
  if (bits == 1) {
    z = __fmul_rn(__fadd_rn(__fmul_rn(3.0f, lo), hi), 0.25f);
    s = __fmul_rn(__fsub_rn(hi, lo), 0.5f);
  } else {
    z = lo;
    s = __fdiv_rn(__fsub_rn(hi, lo), 3.0f);
  }
}

// The multiplier that stands in for a division by s: the correctly rounded
// reciprocal; 0 when s == 0 (the code is then 0); NaN when 1/s overflows
// binary32 (s below about 2^-128, a subnormal range), so that every quotient
// of such a group is settled by the IEEE division in quant_code.
__device__ __forceinline__ float quant_recip(float s) {
  if (s == 0.0f) return 0.0f;
  const float rs = __frcp_rn(s);
  return isinf(rs) ? __int_as_float(0x7FC00000) : rs;
}

// clamp(rint(fl((x - z) / s)), 0, 2^bits - 1), 0 when s == 0 (rs == 0 then).
// The product with the correctly rounded reciprocal rs is within 1e-6 of the
// IEEE quotient for the quotients that occur (|q| <= 3), so it decides every
// value whose quotient is farther than 1e-5 from a rounding boundary k + 1/2;
// the IEEE division settles the rest, and every product that is not a number
// (a NaN rs, or an infinite x - z times a zero rs).  At 1 bit the code is 1
// exactly when the quotient exceeds 1/2 (1/2 itself rounds to even, 0); a
// quotient that is not a number gets code 0.
template <int BITS>
__device__ __forceinline__ uint32_t quant_code(float x, float z, float s, float rs) {
  const float d = __fsub_rn(x, z);
  float t = __fmul_rn(d, rs);
  if (BITS == 1) {
    if (!(fabsf(__fsub_rn(t, 0.5f)) >= 1e-5f) && s != 0.0f) t = __fdiv_rn(d, s);
    return t > 0.5f ? 1u : 0u;
  } else {
    const float fr = __fsub_rn(t, floorf(t));
    if (!(fabsf(__fsub_rn(fr, 0.5f)) >= 1e-5f) && s != 0.0f) t = __fdiv_rn(d, s);
    return (uint32_t)fminf(fmaxf(rintf(t), 0.0f), 3.0f);  // fmaxf(NaN, 0) = 0
  }
}

// bf16 bit patterns in value order and back: ord increases with the value
// (-0 just below +0, NaN patterns outside every finite and infinite value).
__device__ __forceinline__ uint32_t bf16_ord(uint32_t b) { return (b & 0x8000u) ? (b ^ 0xFFFFu) : (b | 0x8000u); }
__device__ __forceinline__ uint32_t bf16_unord(uint32_t o) { return (o & 0x8000u) ? (o & 0x7FFFu) : (o ^ 0xFFFFu); }

// The smallest bf16 value x of a group's range [lo, hi] whose code
// quant_code<BITS>(x, z, s, rs) is at least `level` (1 .. 2^BITS - 1), as a
// float; NaN when no x of the range reaches it.  quant_code is the code of
// the IEEE quotient fl(fl(x - z) / s), a non-decreasing function of x, so an
// element of the group has code >= level exactly when x >= the threshold (a
// NaN element compares false, code 0, as quant_code gives it).  Checked at
// both ends of the range first (lo's code is not always 0: when 3 min + max
// overflows binary32, z = -inf and every element codes 1), then in the
// bracket (lo, hi]: the bf16 value at the analytic point z + (level - 1/2) s
// and its two neighbours settle it unless binary32 absorbs x - z over a run
// of bf16 values there (tiny x near a zero midpoint), which bisection then
// resolves.
template <int BITS>
__device__ __forceinline__ float code_threshold(float lo, float hi, float z, float s, float rs, uint32_t level) {
  auto ge = [&](uint32_t o) {
    return quant_code<BITS>(__uint_as_float(bf16_unord(o) << 16), z, s, rs) >= level;
  };
  uint32_t a = bf16_ord(__float_as_uint(lo) >> 16), b = bf16_ord(__float_as_uint(hi) >> 16);
  if (!(a <= b) || !ge(b)) return __int_as_float(0x7FC00000);
  if (ge(a)) return __uint_as_float(bf16_unord(a) << 16);
  // invariant: code(a) < level <= code(b)
  const float guess = __fadd_rn(z, __fmul_rn((float)level - 0.5f, s));
  const uint32_t og = min(max(bf16_ord(__float_as_uint(guess) >> 16), a + 1u), b);
  if (ge(og)) {
    b = og;
    if (og - 1u > a) {
      if (!ge(og - 1u)) return __uint_as_float(bf16_unord(og) << 16);
      b = og - 1u;
    }
  } else {
    a = og;
    if (og + 1u < b) {
      if (ge(og + 1u)) return __uint_as_float(bf16_unord(og + 1u) << 16);
      a = og + 1u;
    }
  }
  while (b - a > 1u) {
    const uint32_t m = (a + b) >> 1;
    if (ge(m)) b = m; else a = m;
  }
  return __uint_as_float(bf16_unord(b) << 16);
}

// Whether an x with d = fl(x - z) has a code of at least `level`, for s in
// [2^-100, 2^100], without the quotient.  fl(d / s) is above 1/2 exactly when 2
// d > s; at least 3/2 when d / s >= 3/2 - 2^-24 and above 5/2 when d / s > 5/2
// + 2^-23 (the ties at those half steps round to the even 3/2 and 5/2).  Both
// sides of those comparisons are multiples of half an ulp of s and, where they
// are close, a few of them, so one rounding decides them exactly.
template <int BITS>
__device__ __forceinline__ bool code_reaches(float d, float s, int level) {
  if (BITS == 1 || level == 1) return __fadd_rn(d, d) > s;
  if (level == 2) return __fmaf_rn(-1.5f, s, d) >= s * -5.9604644775390625e-8f;
  return __fmaf_rn(-2.5f, s, d) > s * 1.1920928955078125e-7f;
}

// The bf16 patterns of code_threshold for every level at once: the bf16 value
// nearest to z + (level - 1/2) s or one of its neighbours, where code_reaches
// says so (a threshold below lo or above hi serves as well: no element lies
// there); else (a range near zero or overflow, binary32 absorbing x - z over a
// run of bf16 values) by code_threshold's search.
template <int BITS>
__device__ __forceinline__ void code_thresholds(float lo, float hi, float z, float s, uint32_t* thr) {
  bool found = s >= 7.888609052210118e-31f && s <= 1.2676506002282294e30f;
#pragma unroll
  for (int l = 1; l < (1 << BITS); ++l) {
    float guess = __fmaf_rn((float)l - 0.5f, s, z);
    // Where the guess is near zero (lo = -hi) the bf16 values about it are far finer than x - z: the threshold
    // is half an ulp below the first difference that reaches the level.
    if (BITS == 1) {
      guess += __uint_as_float((__float_as_uint(s) & 0x7F800000u) - (25u << 23));  // the one above s / 2
    } else if (l == 2) {
      const float d = __fsub_rn(guess, z);
      const float half_ulp = __uint_as_float((__float_as_uint(d) & 0x7F800000u) - (24u << 23));
      const float at = code_reaches<BITS>(d, s, l) ? 1.0f : -1.0f;
      guess = __fadd_rn(z, d) - half_ulp * (code_reaches<BITS>(d - 2.0f * half_ulp, s, l) ? 3.0f : at);
    }
    uint16_t b;
    asm("cvt.rn.bf16.f32 %0, %1;\n" : "=h"(b) : "f"(guess));
    const bool at = code_reaches<BITS>(__fsub_rn(bf16_to_f32(b), z), s, l);
    // x - z and what it reaches do not decrease with x: one neighbour settles it
    const uint32_t next = bf16_unord(bf16_ord(b) + (at ? ~0u : 1u));
    thr[l - 1] = at ? b : next;
    found = found && code_reaches<BITS>(__fsub_rn(bf16_to_f32(next), z), s, l) != at;
  }
  if (found) return;
  const float rs = quant_recip(s);
#pragma unroll 1
  for (int l = 1; l < (1 << BITS); ++l) {
    const uint32_t t = __float_as_uint(code_threshold<BITS>(lo, hi, z, s, rs, (uint32_t)l)) >> 16;
    if (l == 1) thr[0] = t;
    if (BITS == 2 && l == 2) thr[BITS - 1] = t;
    if (BITS == 2 && l == 3) thr[2 * BITS - 2] = t;
  }
}

// min/max of bf16 values carried as floats; -0.0 is stored as +0.0.
__device__ __forceinline__ uint32_t bf16_bits_canonical(float f) {
  return f == 0.0f ? 0u : (__float_as_uint(f) >> 16);
}

// Token pair p of a group (tokens 2p, 2p+1) is where value code words
// (a, t = p & 3, j = 2 * (p >> 3) + ((p >> 2) & 1)) take their bits; the
// (min, max) of token n, channel group cg is value-minmax word 32 t' + m with
// t' = (n & 7) >> 1, m = 16 (n >> 4) + 4 (2 ((n & 15) >> 3) + (n & 1)) + cg.
__device__ __forceinline__ int vmeta_word(int n, int cg) {
  const int n16 = n & 15;
  return 32 * ((n16 & 7) >> 1) + 16 * (n >> 4) + 4 * (2 * (n16 >> 3) + (n16 & 1)) + cg;
}
// At g = 64 a half's 64 value-minmax words hold token n's (min, max) of
// channels 64c .. 64c+63 at word 2m + c, where m = 8 ((n >> 1) & 3) +
// 4 (n >> 4) + 2 ((n >> 3) & 1) + (n & 1) is the lane that reads token n.
__device__ __forceinline__ int vmeta64_word(int n, int c) {
  return 2 * (8 * ((n >> 1) & 3) + 4 * (n >> 4) + 2 * ((n >> 3) & 1) + (n & 1)) + c;
}

}  // namespace spc
