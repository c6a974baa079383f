// Routing from scores, and its gradient, on gfx950 (moe_route_scored and
// moe_route_backward in include/moe.h).
//
// Scores are formed in fp64: with a bias the choice compares s_e + b_e, which
// lie within [0, 1] and next to each other more often than fp32 can tell apart
// (256 scores per token, millions per call), and gfx950 runs fp64 vector
// arithmetic at the rate of unpacked fp32.  A candidate is one double, the
// choosing value with its 10 low mantissa bits replaced by the expert id, so
// that a maximum of doubles is the arg-max with ties to the lower id.

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr double kLast = -1e300;  // choosing value of an expert whose c is NaN or -inf

// exp(x) for |x| <= 750, relative error about 1e-14: x = n ln 2 + r with
// |r| <= ln(2) / 2, and the Taylor polynomial of degree 11 (the next term is
// below 7e-15 of the result).
__device__ __forceinline__ double exp64(double x) {
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -0.6931471805599453, x);
  double p = 1.0 / 39916800.0;
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
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

// 1 / (1 + exp(-l)); exp(700) is still finite.
__device__ __forceinline__ double sigmoid64(float l) {
  const double x = static_cast<double>(l);
  const double c = x < -700.0 ? -700.0 : (x > 700.0 ? 700.0 : x);
  return l == -INFINITY ? 0.0 : 1.0 / (1.0 + exp64(-c));
}

// exp(l - m) for l <= m; 0 where it is below exp(-700).
__device__ __forceinline__ double exp_below(float l, float m) {
  const double d = static_cast<double>(l) - static_cast<double>(m);
  return d > -700.0 ? exp64(d) : 0.0;
}

// Reductions over the LPT consecutive lanes of one token; every lane gets the result.
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < LPT; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <int LPT>
__device__ __forceinline__ double group_max(double v) {
#pragma unroll
  for (int d = 1; d < LPT; d *= 2) v = fmax(v, __shfl_xor(v, d));
  return v;
}
template <int LPT>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
  for (int d = 1; d < LPT; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Candidate of expert e, and the id back from it.
__device__ __forceinline__ double candidate(double c, int e) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(c)) & ~uint64_t(1023);
  return __longlong_as_double(static_cast<long long>(b | (c < 0.0 ? e : 1023 - e)));
}
__device__ __forceinline__ int candidate_id(double key) {
  const int low = static_cast<int>(__double_as_longlong(key)) & 1023;
  return key < 0.0 ? low : 1023 - low;
}

// LPT lanes per token, EPL logits per lane (LPT * EPL >= E): lane j holds
// experts 4 (LPT q + j) .. + 3 for q = 0, 1, ...
template <int LPT, int EPL>
__device__ __forceinline__ int expert_of(int j, int i) {
  return ((i >> 2) * LPT + j) * 4 + (i & 3);
}

template <int LPT, int EPL>
__global__ __launch_bounds__(256) void route_scored_kernel(RouterArgs r, const float* __restrict__ planes, int parts,
                                                           int64_t part_stride, const float* __restrict__ bias,
                                                           float* __restrict__ logits, int T, int E, int k,
                                                           int32_t* __restrict__ idx, float* __restrict__ gate,
                                                           int* err) {
  constexpr int TPB = 256 / LPT;  // tokens per block
  __shared__ double c_s[TPB][LPT * EPL];
  __shared__ float l_s[TPB][LPT * EPL];
  __shared__ double g_s[TPB][kMaxGroups];
  const int tok_b = static_cast<int>(threadIdx.x) / LPT, j = static_cast<int>(threadIdx.x) % LPT;
  const int token = blockIdx.x * TPB + tok_b;
  const bool live = token < T;
  const int64_t row = static_cast<int64_t>(live ? token : T - 1) * E;

  float l[EPL];
  double c[EPL];
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<LPT, EPL>(j, i);
    float v = -INFINITY;
    if (e < E) {
      v = planes[row + e];
      for (int p = 1; p < parts; ++p) v += planes[row + p * part_stride + e];
      if (planes != logits && live) logits[row + e] = v;
      bad |= !__builtin_isfinite(v);
    }
    l[i] = clean_logit(v);
    l_s[tok_b][e] = l[i];
    m = fmaxf(m, l[i]);
  }
  double sum = 0.0;
  if (!r.sigmoid) {
    m = group_max<LPT>(m);
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += exp_below(l[i], m);
    sum = group_sum<LPT>(sum);
  }
  // score of a logit (0 for every expert of a token whose logits are all -inf)
  auto score = [&](float v) { return r.sigmoid ? sigmoid64(v) : (v == -INFINITY ? 0.0 : exp_below(v, m) / sum); };
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<LPT, EPL>(j, i);
    c[i] = kLast;
    if (e < E) {
      const float b = bias ? bias[e] : 0.f;
      bad |= !__builtin_isfinite(b);
      const double v = score(l[i]) + b;
      c[i] = v > kLast ? (v < -kLast ? v : -kLast) : kLast;
    }
    c_s[tok_b][e] = c[i];
  }
  if (live && bad) raise_error(err, kErrNonFinite);

  // groups: each lane ranks some of them by counting the better ones
  uint64_t kept = ~uint64_t(0);
  const int size = E / r.groups;
  if (r.kept_groups < r.groups) {
    __syncthreads();
    for (int g = j; g < r.groups; g += LPT) {
      double a = -INFINITY, b = -INFINITY;
      for (int e = g * size; e < (g + 1) * size; ++e) {
        const double v = c_s[tok_b][e];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      g_s[tok_b][g] = r.top2 && size > 1 ? a + b : a;
    }
    __syncthreads();
    uint64_t mine = 0;
    for (int g = j; g < r.groups; g += LPT) {
      int better = 0;
      const double v = g_s[tok_b][g];
      for (int o = 0; o < r.groups; ++o) {
        const double u = g_s[tok_b][o];
        better += u > v || (u == v && o < g);
      }
      mine |= better < r.kept_groups ? uint64_t(1) << g : 0;
    }
#pragma unroll
    for (int d = 1; d < LPT; d *= 2) mine |= __shfl_xor(mine, d);
    kept = mine;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<LPT, EPL>(j, i);
    c[i] = e < E && (kept >> (r.groups > 1 ? e / size : 0)) & 1 ? candidate(c[i], e) : -INFINITY;
  }

  // k rounds of a maximum over the token's lanes; lane s keeps slot s
  int my_id = 0;
  for (int s = 0; s < k; ++s) {
    double best = c[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = fmax(best, c[i]);
    best = group_max<LPT>(best);
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = c[i] == best ? -INFINITY : c[i];
    if (j == s) my_id = candidate_id(best);
  }
  __syncthreads();  // l_s is whole
  double w = j < k ? score(l_s[tok_b][my_id]) : 0.0;
  if (r.renorm) {
    const double W = group_sum<LPT>(w);
    w = W > 0.0 ? w / W : 0.0;
  }
  if (live && j < k) {
    idx[static_cast<int64_t>(token) * k + j] = my_id;
    gate[static_cast<int64_t>(token) * k + j] = static_cast<float>(w * r.scale);
  }
}

// One token per LPT lanes; the row of dlogits is put together in LDS.
template <int LPT, int EPL, bool BF16>
__global__ __launch_bounds__(256) void route_backward_kernel(RouterArgs r, const float* __restrict__ logits,
                                                             const int32_t* __restrict__ idx,
                                                             const float* __restrict__ dgate, int T, int E, int k,
                                                             float* __restrict__ out32, uint16_t* __restrict__ out16,
                                                             int ld, int* err) {
  constexpr int TPB = 256 / LPT;
  __shared__ float dw_s[TPB][LPT * EPL];  // dw of the chosen experts, 0 elsewhere
  const int tok_b = static_cast<int>(threadIdx.x) / LPT, j = static_cast<int>(threadIdx.x) % LPT;
  const int token = blockIdx.x * TPB + tok_b;
  const bool live = token < T;
  const int64_t row = static_cast<int64_t>(live ? token : T - 1) * E;
  const int64_t krow = static_cast<int64_t>(live ? token : T - 1) * k;
#pragma unroll
  for (int i = 0; i < EPL; ++i) dw_s[tok_b][expert_of<LPT, EPL>(j, i)] = 0.f;

  int id = j < k ? idx[krow + j] : -1;
  if (j < k && (id < 0 || id >= E)) {
    if (live) raise_error(err, kErrExpertRange);
    id = -1;
  }
  const float lj = id >= 0 ? clean_logit(logits[row + id]) : -INFINITY;
  const double dg = id >= 0 ? static_cast<double>(dgate[krow + j]) : 0.0;

  // softmax scores that are not renormalised need the maximum and the sum of
  // the whole row; renormalised ones only their ratios among the chosen
  const bool dense = !r.sigmoid && !r.renorm;
  float l[EPL];
  float m = lj;
  if (dense) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = expert_of<LPT, EPL>(j, i);
      l[i] = e < E ? clean_logit(logits[row + e]) : -INFINITY;
      m = fmaxf(m, l[i]);
    }
  }
  m = group_max<LPT>(m);
  double sum = 1.0;
  if (dense) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += exp_below(l[i], m);
    sum = group_sum<LPT>(sum);
  }
  auto score = [&](float v) { return r.sigmoid ? sigmoid64(v) : (v == -INFINITY ? 0.0 : exp_below(v, m) / sum); };
  const double s = id >= 0 ? score(lj) : 0.0;
  double dw = dg * r.scale;
  if (r.renorm) {
    const double W = group_sum<LPT>(s);
    const double mean = W > 0.0 ? group_sum<LPT>(dw * s) / W : 0.0;
    dw = W > 0.0 ? (dw - mean) / W : 0.0;
  }
  // the softmax's own mean, sum_s s_s dw_s: zero for renormalised gates
  const double mean = dense ? group_sum<LPT>(s * dw) : 0.0;
  __syncthreads();
  if (id >= 0) atomicAdd(&dw_s[tok_b][id], static_cast<float>(dense ? dw : r.sigmoid ? s * (1.0 - s) * dw : s * dw));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<LPT, EPL>(j, i);
    if (!live || e >= (BF16 ? ld : E)) continue;
    float v = dw_s[tok_b][e];
    if (dense) v = static_cast<float>(score(l[i]) * (v - mean));
    if constexpr (BF16)
      out16[static_cast<int64_t>(token) * ld + e] = f32_to_bf16(v);
    else
      out32[static_cast<int64_t>(token) * ld + e] = v;
  }
}

}  // namespace

hipError_t launch_route_scored(const RouterArgs& r, const float* planes, int parts, int64_t part_stride,
                               const float* bias, float* logits, int T, int E, int k, int32_t* idx, float* gate,
                               int* err, hipStream_t stream) {
  if (T <= 0) return hipSuccess;
  if (parts < 1 || parts > kMaxRouterParts || E > 1024 || k > 16 || r.groups > kMaxGroups) return hipErrorInvalidValue;
#define MOE_RUN(LPT, EPL)                                                                                          \
  route_scored_kernel<LPT, EPL><<<(T + 256 / LPT - 1) / (256 / LPT), 256, 0, stream>>>(                            \
      r, planes, parts, part_stride, bias, logits, T, E, k, idx, gate, err)
  if (E <= 256)
    MOE_RUN(64, 4);
  else if (E <= 512)
    MOE_RUN(64, 8);
  else
    MOE_RUN(64, 16);
#undef MOE_RUN
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouterArgs& r, const float* logits, const int32_t* idx, const float* dgate,
                                 int T, int E, int k, float* out32, uint16_t* out16, int ld, int* err,
                                 hipStream_t stream) {
  if (T <= 0) return hipSuccess;
  if (E > 1024 || ld < E || ld > 1024 || k > 16 || !out32 == !out16) return hipErrorInvalidValue;
#define MOE_RUN(LPT, EPL, BF16)                                                                                    \
  route_backward_kernel<LPT, EPL, BF16><<<(T + 256 / LPT - 1) / (256 / LPT), 256, 0, stream>>>(                    \
      r, logits, idx, dgate, T, E, k, out32, out16, ld, err)
  if (out16) {
    if (ld <= 256)
      MOE_RUN(64, 4, true);
    else if (ld <= 512)
      MOE_RUN(64, 8, true);
    else
      MOE_RUN(64, 16, true);
  } else {
    if (ld <= 256)
      MOE_RUN(64, 4, false);
    else if (ld <= 512)
      MOE_RUN(64, 8, false);
    else
      MOE_RUN(64, 16, false);
  }
#undef MOE_RUN
  return hipGetLastError();
}

}  // namespace moe
