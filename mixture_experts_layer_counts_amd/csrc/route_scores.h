// Arithmetic of routing from scores, shared by the standalone kernels
// (route_scored.hip) and the layer for a few tokens (few.hip): scores in fp64,
// candidates that carry their expert's id, and butterflies over lanes.
#pragma once

#include "common.h"

namespace moe {

constexpr double kLast = -1e300;  // choosing value of an expert whose c is NaN or -inf

// A constant that stays in scalar registers: a plain one is copied into vector
// registers before every step of a polynomial, two moves each.
__device__ __forceinline__ double scalar(double c) {
  asm("" : "+s"(c));
  return c;
}

// exp(x) for |x| <= 750, relative error about 1e-14: x = n ln 2 + r with
// |r| <= ln(2) / 2, and the Taylor polynomial of degree 11 (the next term is
// below 7e-15 of the result).
__device__ __forceinline__ double exp64(double x) {
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -0.6931471805599453, x);
  double p = fma(r, scalar(1.0 / 39916800.0), scalar(1.0 / 3628800.0));
  p = fma(p, r, scalar(1.0 / 362880.0));
  p = fma(p, r, scalar(1.0 / 40320.0));
  p = fma(p, r, scalar(1.0 / 5040.0));
  p = fma(p, r, scalar(1.0 / 720.0));
  p = fma(p, r, scalar(1.0 / 120.0));
  p = fma(p, r, scalar(1.0 / 24.0));
  p = fma(p, r, scalar(1.0 / 6.0));
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, static_cast<int>(n));
}

// A logit as a number: NaN as -inf, +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  l = __builtin_isnan(l) ? -INFINITY : l;
  return l > 3.402823466e38f ? 3.402823466e38f : l;
}

// 1 / d for 1 <= d < 2^1020: two Newton steps from the hardware's estimate
// (some 2^-26), exact to the last place or two.
__device__ __forceinline__ double recip64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

// 1 / (1 + exp(-l)); exp(700) is still finite.
__device__ __forceinline__ double sigmoid64(float l) {
  const float c = fminf(fmaxf(l, -700.f), 700.f);
  const double s = recip64(1.0 + exp64(-static_cast<double>(c)));
  return l == -INFINITY ? 0.0 : s;
}

// exp(l - m) for l <= m; 0 where it is below exp(-700), and for l = -inf.
__device__ __forceinline__ double exp_below(float l, float m) {
  const double d = static_cast<double>(l) - static_cast<double>(m);
  const double e = exp64(d > -700.0 ? d : -700.0);  // no branch: neighbours' chains interleave
  return d > -700.0 ? e : 0.0;
}

// A chosen expert's score for renormalised gates, which depend on the ratios of
// the chosen scores alone: `top` is the largest of the chosen logits, and where
// the scores lie far below fp64's range (masked experts that a bias chose) this
// is their multiple exp(l - top).  Below -500 a sigmoid is exp(l) to 1e-217.
__device__ __forceinline__ double chosen_score(bool sigmoid, float l, float top) {
  return sigmoid && top >= -500.f ? sigmoid64(l) : exp_below(l, top);
}

// Maximum and minimum of two candidates (never NaN).  As instructions of their
// own: fmax would first quieten each operand that comes from a bit pattern.
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// ---- the lanes of one token: LPT = 16 (a DPP row), 32 or 64 consecutive ones ----
// Step d of a butterfly over them: the pair (this lane's value, its partner's),
// in either order.  Steps 0 .. 3 pair lanes of a row (lane ^ 1, lane ^ 2, the
// mirror in 8 lanes and the mirror in 16, each of which joins two halves that
// agree within themselves), step 4 two rows, step 5 two halves of the wave.
template <int STEP>
__device__ __forceinline__ void partner32(uint32_t x, uint32_t& a, uint32_t& b) {
  constexpr int kDpp[4] = {0xB1, 0x4E, 0x141, 0x140};
  if constexpr (STEP < 4) {
    a = x;
    constexpr int kCtrl = kDpp[STEP < 4 ? STEP : 0];
    b = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), kCtrl, 0xF, 0xF, false));
  } else if constexpr (STEP == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int STEP>
__device__ __forceinline__ void partner64(double x, double& a, double& b) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  uint32_t al, bl, ah, bh;
  partner32<STEP>(static_cast<uint32_t>(u), al, bl);
  partner32<STEP>(static_cast<uint32_t>(u >> 32), ah, bh);
  a = __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(ah) << 32 | al));
  b = __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(bh) << 32 | bl));
}

template <int LPT, int STEP = 0>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr ((1 << STEP) < LPT) {
    uint32_t a, b;
    partner32<STEP>(__float_as_uint(v), a, b);
    return lanes_max<LPT, STEP + 1>(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  return v;
}
template <int LPT, int STEP = 0>
__device__ __forceinline__ double lanes_sum(double v) {
  if constexpr ((1 << STEP) < LPT) {
    double a, b;
    partner64<STEP>(v, a, b);
    return lanes_sum<LPT, STEP + 1>(a + b);
  }
  return v;
}
template <int LPT, int STEP = 0>
__device__ __forceinline__ uint32_t lanes_or(uint32_t v) {
  if constexpr ((1 << STEP) < LPT) {
    uint32_t a, b;
    partner32<STEP>(v, a, b);
    return lanes_or<LPT, STEP + 1>(a | b);
  }
  return v;
}

template <int LPT, int STEP = 0>
__device__ __forceinline__ double lanes_best64(double v) {  // the largest candidate
  if constexpr ((1 << STEP) < LPT) {
    double a, b;
    partner64<STEP>(v, a, b);
    return lanes_best64<LPT, STEP + 1>(max64(a, b));
  }
  return v;
}

// Candidate of expert e, and the id back from it.
__device__ __forceinline__ double candidate(double c, int e) {
  c += 0.0;  // -0 as +0
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(c)) & ~uint64_t(1023);
  return __longlong_as_double(static_cast<long long>(b | (c < 0.0 ? e : 1023 - e)));
}
__device__ __forceinline__ int candidate_id(double key) {
  const int low = static_cast<int>(__double_as_longlong(key)) & 1023;
  return key < 0.0 ? low : 1023 - low;
}

}  // namespace moe
