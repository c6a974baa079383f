// Routing from scores, and its gradient, on gfx950 (moe_route_scored and
// moe_route_backward in include/moe.h).
//
// Scores are formed in fp64: with a bias the choice compares s_e + b_e, which
// lie within [0, 1] and next to each other more often than fp32 can tell apart
// (256 scores per token, millions per call), and gfx950 runs fp64 vector
// arithmetic at the rate of unpacked fp32.  A candidate is one double, the
// choosing value with its 10 low mantissa bits replaced by the expert id, so
// that a maximum of doubles is the arg-max with ties to the lower id.
//
// What bounds the choice is arithmetic (a row of 256 logits is 1 KB, and 8192
// of them a microsecond or two of memory), so a wave takes four tokens: 16 lanes
// and, at 256 experts, 16 registers each.  A lane sorts its candidates once; then
// the sorted lists of two lanes meet log2(16) times, each time keeping the 8 (or
// 16) largest of both by one bitonic merge, with the partner's list coming by
// DPP inside the 16-lane row.  Rounds of a wave-wide arg-max (a token a wave,
// k rounds of six crossbar steps) took 26 us for 8192 tokens where this takes
// 9.9, and 10.0 for one where this takes 4.7 (sigmoid, 256 experts in 8 groups).

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

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

// The two largest of `lanes` (a power of two) neighbouring lanes' pairs, for N
// pairs side by side.
template <int LPT, int N, int STEP = 0>
__device__ __forceinline__ void lanes_two(double (&best)[N], double (&next)[N], int lanes) {
  if constexpr ((1 << STEP) < LPT) {
    if ((1 << STEP) >= lanes) return;  // uniform
#pragma unroll
    for (int i = 0; i < N; ++i) {
      double a, b, c, d;
      partner64<STEP>(best[i], a, b);
      partner64<STEP>(next[i], c, d);
      best[i] = max64(a, b);
      next[i] = max64(min64(a, b), max64(c, d));
    }
    lanes_two<LPT, N, STEP + 1>(best, next, lanes);
  }
}

// ---- sorted lists in registers (falling order) ----
__device__ __forceinline__ void order(double& hi, double& lo) {
  const double a = hi, b = lo;
  hi = max64(a, b);
  lo = min64(a, b);
}
// A bitonic list of N into falling order.
template <int N>
__device__ __forceinline__ void bitonic(double* v) {
#pragma unroll
  for (int d = N / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) order(v[i], v[i + d]);
}
// Any list of N (a power of two) into falling order: runs of 1, 2, 4, ... merged,
// every other run turned round by the index it is compared at.
template <int N>
__device__ __forceinline__ void sort_list(double* v) {
#pragma unroll
  for (int run = 2; run <= N; run *= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & (run / 2)) == 0) {
        const int o = (i & ~(run - 1)) + (run - 1) - (i & (run - 1));  // mirror in the run
        order(v[i], v[o]);
      }
#pragma unroll
    for (int d = run / 4; d > 0; d /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & d) == 0) order(v[i], v[i + d]);
  }
}
// The K largest of every lane's list of K, in falling order, on all LPT lanes.
template <int K, int LPT, int STEP = 0>
__device__ __forceinline__ void lanes_best(double (&v)[K]) {
  if constexpr ((1 << STEP) < LPT) {
    double a[K], b[K];
#pragma unroll
    for (int i = 0; i < K; ++i) partner64<STEP>(v[i], a[i], b[i]);
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = max64(a[i], b[K - 1 - i]);
    bitonic<K>(v);
    lanes_best<K, LPT, STEP + 1>(v);
  }
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

// EPL experts per lane (LPT * EPL >= E): lane j holds experts 4 (LPT q + j) ..
// + 3 for q = 0, 1, ...
template <int LPT, int EPL>
__device__ __forceinline__ int expert_of(int j, int i) {
  return ((i >> 2) * LPT + j) * 4 + (i & 3);
}
// A row of E floats into that layout (past E: `fill`), in 16-byte pieces if VEC.
template <int LPT, int EPL, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int j, int E, float fill, float (&v)[EPL]) {
#pragma unroll
  for (int q = 0; q < EPL / 4; ++q) {
    const int e = expert_of<LPT, EPL>(j, 4 * q);
    if (VEC) {
      f32x4_t x = {fill, fill, fill, fill};
      if (e < E) x = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = x[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = e + i < E ? row[e + i] : fill;
    }
  }
}

template <int K, int LPT, int EPL, bool VEC>
__global__ __launch_bounds__(256) void route_scored_kernel(RouterArgs r, const float* __restrict__ planes, int parts,
                                                           int64_t part_stride, const float* __restrict__ bias,
                                                           float* __restrict__ logits, int T, int E, int k,
                                                           int32_t* __restrict__ idx, float* __restrict__ gate,
                                                           int* err) {
  constexpr int TPB = 256 / LPT;  // tokens per block
  extern __shared__ double c_s[];  // [TPB][LPT * EPL], only for groups that are read from LDS
  __shared__ float l_s[TPB][LPT * EPL];
  __shared__ double g_s[TPB][kMaxGroups];  // padded to a multiple of four groups
  const int tok_b = static_cast<int>(threadIdx.x) / LPT, j = static_cast<int>(threadIdx.x) % LPT;
  const int token = blockIdx.x * TPB + tok_b;
  const bool live = token < T;
  const int64_t row = static_cast<int64_t>(live ? token : T - 1) * E;

  float l[EPL];
  load_row<LPT, EPL, VEC>(planes + row, j, E, 0.f, l);
  for (int p = 1; p < parts; ++p) {
    float more[EPL];
    load_row<LPT, EPL, VEC>(planes + row + p * part_stride, j, E, 0.f, more);
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] += more[i];
  }
  float b[EPL];
  if (bias) load_row<LPT, EPL, VEC>(bias, j, E, 0.f, b);
  if (planes != logits && live) {
#pragma unroll
    for (int q = 0; q < EPL / 4; ++q) {
      const int e = expert_of<LPT, EPL>(j, 4 * q);
      if constexpr (VEC) {
        const f32x4_t v = {l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]};
        if (e < E) *reinterpret_cast<f32x4_t*>(logits + row + e) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < E) logits[row + e + i] = l[4 * q + i];
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<LPT, EPL>(j, i);
    bad |= !__builtin_isfinite(l[i]);
    if (!bias) b[i] = 0.f;
    bad |= !__builtin_isfinite(b[i]);
    l[i] = e < E ? clean_logit(l[i]) : -INFINITY;
  }
#pragma unroll
  for (int q = 0; q < EPL / 4; ++q)
    *reinterpret_cast<f32x4_t*>(&l_s[tok_b][expert_of<LPT, EPL>(j, 4 * q)]) =
        f32x4_t{l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]};
  if (live && bad) raise_error(err, kErrNonFinite);

  // choosing values.  Without a bias, and with groups that rank by their
  // largest, scores order as their logits do, and only a sum needs the row's
  // exponentials.
  double c[EPL];
  float m = 0.f;
  double inv = 1.0;  // softmax: 1 / sum (renormalised gates do not need it)
  const bool by_logit = !bias && (r.kept_groups == r.groups || !r.top2 || r.group_size == 1);
  if (r.sigmoid && !by_logit) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = sigmoid64(l[i]);
  } else if (!r.sigmoid && !(by_logit && r.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
    m = lanes_max<LPT>(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] = exp_below(l[i], m);
      sum += c[i];
    }
    sum = lanes_sum<LPT>(sum);
    inv = sum > 0.0 ? recip64(sum) : 0.0;  // at least 1, or 0 for a token whose logits are all -inf
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const double v = by_logit ? static_cast<double>(l[i]) : c[i] * inv + static_cast<double>(b[i]);
    c[i] = v > kLast ? (v < -kLast ? v : -kLast) : kLast;
    if (expert_of<LPT, EPL>(j, i) >= E) c[i] = -INFINITY;
  }

  // e / size
  auto group_of = [&](int e) { return __umul24(static_cast<uint32_t>(e), r.group_magic) >> 20; };
  // groups: their scores into g_s, then each is ranked by counting the better ones
  uint64_t kept = ~uint64_t(0);
  if (r.kept_groups < r.groups) {
    const int size = r.group_size;
    if (r.group_lanes == 0) {
      // a group is 1, 2, 4, ... neighbouring lanes' quads: the two largest by
      // the first steps of the butterfly, in registers
      double best[EPL / 4], next[EPL / 4];
#pragma unroll
      for (int q = 0; q < EPL / 4; ++q) {
        const double h0 = max64(c[4 * q], c[4 * q + 1]), l0 = min64(c[4 * q], c[4 * q + 1]);
        const double h1 = max64(c[4 * q + 2], c[4 * q + 3]), l1 = min64(c[4 * q + 2], c[4 * q + 3]);
        best[q] = max64(h0, h1);
        next[q] = max64(min64(h0, h1), max64(l0, l1));
      }
      lanes_two<LPT>(best, next, size / 4);
      if ((j & (size / 4 - 1)) == 0) {  // a group's first lane
#pragma unroll
        for (int q = 0; q < EPL / 4; ++q) {
          const int e = expert_of<LPT, EPL>(j, 4 * q);
          if (e < E) g_s[tok_b][group_of(e)] = r.top2 ? best[q] + next[q] : best[q];
        }
      }
    } else {
      // any other size: group_lanes lanes read one together
#pragma unroll
      for (int i = 0; i < EPL; ++i) c_s[tok_b * LPT * EPL + expert_of<LPT, EPL>(j, i)] = c[i];
      __syncthreads();
      const int sub = r.group_lanes, part = j & (sub - 1);
      for (int g = j / sub; g < r.groups; g += LPT / sub) {
        const double* cg = &c_s[tok_b * LPT * EPL + g * size];
        double best = -INFINITY, next = -INFINITY;
        for (int e = part; e < size; e += sub) {
          const double v = cg[e];
          next = max64(next, min64(best, v));
          best = max64(best, v);
        }
        for (int d = 1; d < sub; d *= 2) {
          const double ob = __shfl_xor(best, d), on = __shfl_xor(next, d);
          next = max64(min64(best, ob), max64(next, on));
          best = max64(best, ob);
        }
        if (part == 0) g_s[tok_b][g] = r.top2 && size > 1 ? best + next : best;
      }
    }
    for (int g = r.groups + j; g < (r.groups + 3) / 4 * 4; g += LPT) g_s[tok_b][g] = -INFINITY;
    __syncthreads();
    uint32_t lo = 0, hi = 0;
    for (int g = j; g < r.groups; g += LPT) {
      int better = 0;
      const double v = g_s[tok_b][g];
      for (int o = 0; o < r.groups; o += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double u = g_s[tok_b][o + i];
          better += u > v || (u == v && o + i < g);
        }
      }
      const uint32_t bit = better < r.kept_groups ? 1u << (g & 31) : 0u;
      lo |= g < 32 ? bit : 0u;
      hi |= g < 32 ? 0u : bit;
    }
    lo = lanes_or<LPT>(lo);
    hi = r.groups > 32 ? lanes_or<LPT>(hi) : 0u;
    kept = static_cast<uint64_t>(hi) << 32 | lo;
  }
  auto in = [&](int e) { return (kept >> (group_of(e) & 63)) & 1; };  // past E: any bit
#pragma unroll
  for (int q = 0; q < EPL / 4; ++q) {
    const int e = expert_of<LPT, EPL>(j, 4 * q);
    const bool quad = in(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = r.group_size % 4 == 0 ? quad : in(e + i);  // uniform: a quad lies in one group
      const double v = c[4 * q + i];
      c[4 * q + i] = ok && v > -INFINITY ? candidate(v, e + i) : -INFINITY;
    }
  }

  // the K largest: each lane's own, then the lanes'
  double best[K];
  if constexpr (EPL <= K) {
    constexpr int N = EPL <= 4 ? 4 : (EPL <= 8 ? 8 : 16);
    double list[N];
#pragma unroll
    for (int i = 0; i < N; ++i) list[i] = i < EPL ? c[i < EPL ? i : 0] : -INFINITY;
    sort_list<N>(list);
#pragma unroll
    for (int i = 0; i < K; ++i) best[i] = i < N ? list[i < N ? i : 0] : -INFINITY;
  } else {
    static_assert(EPL <= 2 * K, "two lists a lane");
    double more[K];
#pragma unroll
    for (int i = 0; i < K; ++i) best[i] = c[i];
#pragma unroll
    for (int i = 0; i < K; ++i) more[i] = K + i < EPL ? c[K + i < EPL ? K + i : 0] : -INFINITY;
    sort_list<K>(best);
    sort_list<K>(more);
#pragma unroll
    for (int i = 0; i < K; ++i) best[i] = max64(best[i], more[K - 1 - i]);
    bitonic<K>(best);
  }
  lanes_best<K, LPT>(best);

  // lane s takes slot s
  double mine = best[0];
#pragma unroll
  for (int i = 1; i < K; ++i) mine = j == i ? best[i] : mine;
  const int my_id = candidate_id(mine);
  __syncthreads();  // l_s is whole
  const float my_l = j < k ? l_s[tok_b][my_id] : -INFINITY;
  double w;
  if (r.renorm) {
    w = chosen_score(r.sigmoid, my_l, lanes_max<LPT>(my_l));
    const double W = lanes_sum<LPT>(w);
    w = W > 0.0 ? w / W : 0.0;
  } else {
    w = r.sigmoid ? sigmoid64(my_l) : exp_below(my_l, m) * inv;
  }
  if (live && j < k) {
    idx[static_cast<int64_t>(token) * k + j] = my_id;
    gate[static_cast<int64_t>(token) * k + j] = static_cast<float>(w * r.scale);
  }
}

// One token per LPT lanes; the chosen experts' terms are put in their places in LDS.
template <int LPT, int EPL, bool BF16, bool VEC>
__global__ __launch_bounds__(256) void route_backward_kernel(RouterArgs r, const float* __restrict__ logits,
                                                             const int32_t* __restrict__ idx,
                                                             const float* __restrict__ dgate, int T, int E, int k,
                                                             float* __restrict__ out32, uint16_t* __restrict__ out16,
                                                             int ld, int* err) {
  constexpr int TPB = 256 / LPT;
  __shared__ double dw_s[TPB][LPT * EPL];  // the chosen experts' terms, 0 elsewhere
  const int tok_b = static_cast<int>(threadIdx.x) / LPT, j = static_cast<int>(threadIdx.x) % LPT;
  const int token = blockIdx.x * TPB + tok_b;
  const bool live = token < T;
  const int64_t row = static_cast<int64_t>(live ? token : T - 1) * E;
  const int64_t krow = static_cast<int64_t>(live ? token : T - 1) * k;

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
  double z[EPL];
  float m = 0.f;
  double inv = 1.0;
  if (dense) {
    float l[EPL];
    load_row<LPT, EPL, VEC>(logits + row, j, E, -INFINITY, l);
    m = lj;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = clean_logit(l[i]);
      m = fmaxf(m, l[i]);
    }
    m = lanes_max<LPT>(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      z[i] = exp_below(l[i], m);
      sum += z[i];
    }
    sum = lanes_sum<LPT>(sum);
    inv = sum > 0.0 ? recip64(sum) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) dw_s[tok_b][expert_of<LPT, EPL>(j, i)] = 0.0;
  double s;  // 0 for a lane without an expert (lj is -inf there)
  double dw = dg * r.scale;
  if (r.renorm) {
    s = chosen_score(r.sigmoid, lj, lanes_max<LPT>(lj));
    const double W = lanes_sum<LPT>(s);
    const double mean = W > 0.0 ? lanes_sum<LPT>(dw * s) / W : 0.0;
    // (a single expert's gate is `scale` whatever its score: no rounding left over)
    dw = W > 0.0 && k > 1 ? (dw - mean) / W : 0.0;
  } else {
    s = r.sigmoid ? sigmoid64(lj) : exp_below(lj, m) * inv;
  }
  // the softmax's own mean, sum_s s_s dw_s: zero for renormalised gates
  const double mean = dense ? lanes_sum<LPT>(s * dw) : 0.0;
  __syncthreads();
  // (1 - s as a score of its own: from l of about 20 the difference is worth less than an fp32 step)
  if (id >= 0) atomicAdd(&dw_s[tok_b][id], dense ? dw : r.sigmoid ? s * sigmoid64(-lj) * dw : s * dw);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < EPL / 4; ++q) {
    const int e = expert_of<LPT, EPL>(j, 4 * q);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double t = dw_s[tok_b][e + i];
      v[i] = static_cast<float>(dense ? z[4 * q + i] * inv * (t - mean) : t);
    }
    if (!live) continue;
    const int64_t at = static_cast<int64_t>(token) * ld + e;
    if constexpr (BF16) {  // rows of ld, a multiple of 64
      if (e < ld) *reinterpret_cast<uint2*>(out16 + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else if constexpr (VEC) {
      if (e < E) *reinterpret_cast<f32x4_t*>(out32 + at) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) out32[at + i] = v[i];
    }
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// What the kernels need of the groups.
RouterArgs with_groups(RouterArgs r, int E, int lanes) {
  r.group_size = E / r.groups;
  r.group_magic = (1u << 20) / static_cast<uint32_t>(r.group_size) + 1;  // exact for e < 1024
  const int quads = r.group_size / 4;
  if (r.group_size % 4 == 0 && (quads & (quads - 1)) == 0 && quads <= lanes) {
    r.group_lanes = 0;  // in registers
    return r;
  }
  // lanes that read one group together: a power of two that divides its size
  r.group_lanes = 1;
  while (2 * r.group_lanes * r.groups <= lanes && r.group_size % (2 * r.group_lanes) == 0) r.group_lanes *= 2;
  return r;
}

// Experts a lane holds at most, and the lanes of a token for them.
int lanes_for(int E) { return E <= 256 ? 16 : (E <= 512 ? 32 : 64); }
// For few tokens a whole wave takes one, four or eight experts a lane: its chain
// of fp64 instructions is shorter, and that counts while SIMDs have one wave or
// none (1024 tokens), for 129 to 256 experts while they have two.  256 experts in
// 8 groups: one token 4.7 us against 6.8 with 16 lanes, 2048 tokens 6.0 against
// 7.1, 4096 tokens 8.6 against 7.3; 128 experts: 1024 tokens 3.7 against 3.9,
// 1536 4.5 against 3.9; 384 in 12 groups: 6.2 against 6.7 and 7.4 against 6.8.
bool wave_a_token(int T, int E) { return E <= 512 && T <= (E > 128 && E <= 256 ? 2048 : 1024); }

}  // namespace

hipError_t launch_route_scored(const RouterArgs& args, const float* planes, int parts, int64_t part_stride,
                               const float* bias, float* logits, int T, int E, int k, int32_t* idx, float* gate,
                               int* err, hipStream_t stream) {
  if (T <= 0) return hipSuccess;
  if (parts < 1 || parts > kMaxRouterParts || E > 1024 || k > 16 || args.groups > kMaxGroups || E % args.groups)
    return hipErrorInvalidValue;
  const bool wave = wave_a_token(T, E);
  const int lanes = wave ? 64 : lanes_for(E);
  const RouterArgs r = with_groups(args, E, lanes);
  const bool vec = E % 4 == 0 && part_stride % 4 == 0 && aligned16(planes) && aligned16(bias) && aligned16(logits);
  const int blocks = (T - 1) / (256 / lanes) + 1;
#define MOE_RUN(K, LPT, EPL)                                                                                        \
  (vec ? route_scored_kernel<K, LPT, EPL, true> : route_scored_kernel<K, LPT, EPL, false>)                          \
      <<<blocks, 256, r.group_lanes ? sizeof(double) * 256 * EPL : 0, stream>>>(                                    \
          r, planes, parts, part_stride, bias, logits, T, E, k, idx, gate, err)
#define MOE_RUN_K(LPT, EPL) \
  if (k <= 8)               \
    MOE_RUN(8, LPT, EPL);   \
  else                      \
    MOE_RUN(16, LPT, EPL)
  if (wave && E <= 256) {
    MOE_RUN_K(64, 4);
  } else if (wave) {
    MOE_RUN_K(64, 8);
  } else if (E <= 128) {
    MOE_RUN_K(16, 8);
  } else if (lanes == 16) {
    MOE_RUN_K(16, 16);
  } else if (E <= 384) {
    MOE_RUN_K(32, 12);
  } else if (lanes == 32) {
    MOE_RUN_K(32, 16);
  } else {
    MOE_RUN_K(64, 16);
  }
#undef MOE_RUN_K
#undef MOE_RUN
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouterArgs& r, const float* logits, const int32_t* idx, const float* dgate,
                                 int T, int E, int k, float* out32, uint16_t* out16, int ld, int* err,
                                 hipStream_t stream) {
  if (T <= 0) return hipSuccess;
  if (E > 1024 || ld < E || ld > 1024 || k > 16 || !out32 == !out16) return hipErrorInvalidValue;
  if (out16 && (ld % 4 || reinterpret_cast<uintptr_t>(out16) % 8)) return hipErrorInvalidValue;
  const bool vec = E % 4 == 0 && aligned16(logits) && aligned16(out32);
  const int lanes = lanes_for(ld), blocks = (T - 1) / (256 / lanes) + 1;
#define MOE_RUN(LPT, EPL)                                                                                         \
  (out16 ? (vec ? route_backward_kernel<LPT, EPL, true, true> : route_backward_kernel<LPT, EPL, true, false>)     \
         : (vec ? route_backward_kernel<LPT, EPL, false, true> : route_backward_kernel<LPT, EPL, false, false>))  \
      <<<blocks, 256, 0, stream>>>(r, logits, idx, dgate, T, E, k, out32, out16, ld, err)
  if (ld <= 128)
    MOE_RUN(16, 8);
  else if (lanes == 16)
    MOE_RUN(16, 16);
  else if (ld <= 384)
    MOE_RUN(32, 12);
  else if (lanes == 32)
    MOE_RUN(32, 16);
  else
    MOE_RUN(64, 16);
#undef MOE_RUN
  return hipGetLastError();
}

}  // namespace moe
