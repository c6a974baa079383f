// Rows to 8-bit integers, device pieces shared by the quantiser and the products
// that quantise their own activations.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kI8Chunk = 8;  // elements per thread and step: 8 bytes of q, 16 or 32 bytes read

__device__ __forceinline__ float i8_as_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float i8_as_f32(float v) { return v; }

template <bool VEC, typename T>
__device__ __forceinline__ void i8_load_chunk(const T* __restrict__ src, int64_t c, int64_t K, float (&v)[kI8Chunk]) {
  const int64_t k0 = c * kI8Chunk;
  if (VEC && k0 + kI8Chunk <= K) {
    T t[kI8Chunk];
    constexpr int kWords = kI8Chunk * sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      reinterpret_cast<u32x4_t*>(t)[i] = reinterpret_cast<const u32x4_t*>(src + k0)[i];
#pragma unroll
    for (int i = 0; i < kI8Chunk; ++i) v[i] = i8_as_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kI8Chunk; ++i) v[i] = k0 + i < K ? i8_as_f32(src[k0 + i]) : 0.f;
  }
}

// round(127 v / m), ties to even, exactly: the remainder 127 v - q m is exact in
// fp64 and decides the values whose quotient is next to a half.
__device__ __forceinline__ int i8_exact_quotient(float v, float m) {
  const double x = 127.0 * static_cast<double>(v);
  double q = rint(x / static_cast<double>(m));
  const double d2 = 2.0 * fma(-q, static_cast<double>(m), x);
  const bool odd = static_cast<int>(q) & 1;
  if (d2 > m || (d2 == m && odd)) q += 1.0;
  if (d2 < -m || (d2 == -m && odd)) q -= 1.0;
  return static_cast<int>(q);
}

// Eight quotients as bytes.  In fp32 the quotient v r, with r the float above
// 127 / m rounded, is off by at most 127 1.5 2^-23, so it is right unless it lies
// within 2^-14 of a half; adding 1.5 2^23 rounds it to an integer in the sum's
// low bits.  The one exact half there is among bf16 values, |v| = m / 2 (127 has
// to divide the other factor), comes out as 64, the even side, since r is not
// below 127 / m.  A chunk that holds another value so close is settled by the
// remainder d = 127 v - q m: 127 v = hi + lo exactly, hi - q m is exact (a
// multiple of half m's last place, at most about m / 2), and 2 |d| against m,
// with lo, says on which side of the half it lies.  (Settling m / 2 there as
// well took 42 us for 8192 x 7168 bf16, without any check 34.)
// `exact`: rows whose r or 127 m would leave fp32's range.
__device__ __forceinline__ uint2 i8_quotients(const float (&v)[kI8Chunk], float m, float r, bool exact) {
  constexpr float kMagic = 12582912.f;
  uint32_t b[kI8Chunk];
  float near = 1.f;
  const float half = 0.5f * m;
#pragma unroll
  for (int e = 0; e < kI8Chunk; ++e) {
    const float y = fmaf(v[e], r, kMagic);
    b[e] = __float_as_uint(y);
    const float f = fmaf(v[e], r, kMagic - y);  // the fraction, in [-0.5, 0.5]
    near = fminf(near, fabsf(v[e]) == half ? 1.f : 0.5f - fabsf(f));
  }
  if (exact) {
#pragma unroll
    for (int e = 0; e < kI8Chunk; ++e) b[e] = static_cast<uint32_t>(i8_exact_quotient(v[e], m));
  } else if (near < 0x1p-14f) {
#pragma unroll
    for (int e = 0; e < kI8Chunk; ++e) {
      const float q = __uint_as_float(b[e]) - kMagic;
      const float hi = 127.f * v[e], lo = fmaf(127.f, v[e], -hi);
      const float d = fmaf(-q, m, hi);
      const float over = fmaf(2.f, fabsf(d), -m) + 2.f * (d < 0.f ? -lo : lo);  // 2 |127 v - q m| - m
      const bool step = over > 0.f || (over == 0.f && (b[e] & 1u));
      b[e] += step ? (d < 0.f ? 0xffffffffu : 1u) : 0u;
    }
  }
  auto pack = [&](int i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0c0c0400u);
    return lo | (hi << 16);
  };
  return make_uint2(pack(0), pack(4));
}

// Largest |v| of a chunk as bits, against `bits`: NaN above infinity above every number.
__device__ __forceinline__ uint32_t i8_max_bits(const float (&v)[kI8Chunk], uint32_t bits) {
#pragma unroll
  for (int e = 0; e < kI8Chunk; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
    bits = b > bits ? b : bits;
  }
  return bits;
}

// How a row with the largest magnitude `bits` is quantised.
struct I8RowScale {
  float m, r, scale;
  bool some, exact;
  __device__ __forceinline__ explicit I8RowScale(uint32_t bits) {
    const bool finite = bits < 0x7f800000u;
    some = bits && finite;  // neither all zero nor not finite
    m = __uint_as_float(bits);
    scale = finite ? m / 127.f : __uint_as_float(0x7fc00000u);
    r = some ? __uint_as_float(__float_as_uint(127.f / m) + 1u) : 0.f;
    exact = some && (m < 0x1p-100f || m > 0x1p119f);  // r or 127 m past fp32's range, or close
  }
  __device__ __forceinline__ uint2 operator()(const float (&v)[kI8Chunk]) const {
    return some ? i8_quotients(v, m, r, exact) : make_uint2(0, 0);
  }
};

constexpr int kI8Held = 4;  // chunks a thread keeps; longer rows are read twice

// Row i by `TH` threads: a wave of its own for rows of up to 2048 (no barrier,
// four rows a workgroup), a whole workgroup for longer ones.
template <int TH, bool VEC, typename T>
__device__ __forceinline__ void i8_quantize_row(const QuantI8Args& a, int64_t i) {
  int64_t from = i, to = i;
  if (a.limit && a.p_begin + i >= *a.limit) return;  // behind the last routed row
  const int tid = static_cast<int>(threadIdx.x) % TH;
  if (a.routes && tid == 0) {
    const int32_t route = a.routes[a.p_begin + i];
    if (route < 0 || route >= a.n_routes) raise_error(a.err, kErrExpertRange);  // a table of the caller's own
  }
  if (a.sched) {
    const int64_t p = a.p_begin + i;
    const int32_t route = a.sched[p];
    from = route / a.k;
    to = p % a.ring_rows;
    if (route < 0 || from >= a.src_rows) {  // a table not built by the schedule kernels
      if (tid == 0) raise_error(a.err, kErrExpertRange);
      return;
    }
  }
  const T* __restrict__ src = static_cast<const T*>(a.src) + from * a.K;
  int8_t* __restrict__ q = a.q + to * a.Kp;
  const int64_t chunks = a.Kp / kI8Chunk;

  float v[kI8Held][kI8Chunk];
  uint32_t bits = 0;
#pragma unroll
  for (int h = 0; h < kI8Held; ++h) {
    const int64_t c = tid + h * TH;
    if (c < chunks)
      i8_load_chunk<VEC>(src, c, a.K, v[h]);
    else
#pragma unroll
      for (int e = 0; e < kI8Chunk; ++e) v[h][e] = 0.f;
    bits = i8_max_bits(v[h], bits);
  }
  for (int64_t c = tid + kI8Held * TH; c < chunks; c += TH) {
    float w[kI8Chunk];
    i8_load_chunk<VEC>(src, c, a.K, w);
    bits = i8_max_bits(w, bits);
  }
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t o = __shfl_xor(bits, d);
    bits = o > bits ? o : bits;
  }
  if constexpr (TH > kWave) {
    __shared__ uint32_t part[TH / kWave];
    if (lane_id() == 0) part[tid / kWave] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TH / kWave; ++w) bits = part[w] > bits ? part[w] : bits;
  }

  const I8RowScale quant(bits);
  if (tid == 0) a.scale[to] = quant.scale;
  auto put = [&](int64_t c, const float(&w)[kI8Chunk]) { *reinterpret_cast<uint2*>(q + c * kI8Chunk) = quant(w); };
#pragma unroll
  for (int h = 0; h < kI8Held; ++h) {
    const int64_t c = tid + h * TH;
    if (c < chunks) put(c, v[h]);
  }
  for (int64_t c = tid + kI8Held * TH; c < chunks; c += TH) {
    float w[kI8Chunk];
    i8_load_chunk<VEC>(src, c, a.K, w);
    put(c, w);
  }
}

}  // namespace moe
