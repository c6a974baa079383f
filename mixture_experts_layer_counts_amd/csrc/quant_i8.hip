// Rows to 8-bit integers with one scale per row, on gfx950 (moe_quantize_int8
// in include/moe.h; also the int8 layer's activations and its gather).
//
//   m = max |v|,  scale = m / 127,  q = round(127 v / m), ties to even
//
// A row of zeros has scale 0; a row with an infinity or a NaN has q = 0 and
// scale NaN, so that every product with it is NaN.  One workgroup per row: the
// row stays in registers between its maximum and its quotients.

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8;  // elements per thread and step: 8 bytes of q, 16 or 32 bytes read
constexpr int kHeld = 4;   // chunks a thread keeps; longer rows (over 8192) are read twice

__device__ __forceinline__ float as_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float as_f32(float v) { return v; }

template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* __restrict__ src, int64_t c, int64_t K, float (&v)[kChunk]) {
  const int64_t k0 = c * kChunk;
  if (VEC && k0 + kChunk <= K) {
    T t[kChunk];
    constexpr int kWords = kChunk * sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      reinterpret_cast<u32x4_t*>(t)[i] = reinterpret_cast<const u32x4_t*>(src + k0)[i];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = as_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = k0 + i < K ? as_f32(src[k0 + i]) : 0.f;
  }
}

// round(127 v / m), ties to even, exactly: the remainder 127 v - q m is exact in
// fp64 and decides the values whose quotient is next to a half.
__device__ __forceinline__ int exact_quotient(float v, float m) {
  const double x = 127.0 * static_cast<double>(v);
  double q = rint(x / static_cast<double>(m));
  const double d2 = 2.0 * fma(-q, static_cast<double>(m), x);
  const bool odd = static_cast<int>(q) & 1;
  if (d2 > m || (d2 == m && odd)) q += 1.0;
  if (d2 < -m || (d2 == -m && odd)) q -= 1.0;
  return static_cast<int>(q);
}

// Eight quotients as bytes.  In fp32 the quotient v r with r = 127 / m is off by
// at most 127 2^-23 (r's rounding and the product's), so it is right unless it
// lies within 2^-15 of a half; adding 1.5 2^23 rounds it to an integer in the
// sum's low bits.  The exact form then redoes the chunks that hold such a
// value, one in a thousand or so, and rows whose r would leave fp32's range.
// (fp64 throughout took 59 us for 8192 x 7168 bf16, bound by arithmetic.)
__device__ __forceinline__ uint2 quotients(const float (&v)[kChunk], float m, float r, bool exact) {
  constexpr float kMagic = 12582912.f;
  uint32_t b[kChunk];
  float near = 1.f;
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    const float y = fmaf(v[e], r, kMagic);
    b[e] = __float_as_uint(y);
    const float f = fmaf(v[e], r, kMagic - y);  // the fraction, in [-0.5, 0.5]
    near = fminf(near, 0.5f - fabsf(f));
  }
  if (exact || near < 0x1p-15f) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) b[e] = static_cast<uint32_t>(exact_quotient(v[e], m));
  }
  auto pack = [&](int i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0c0c0400u);
    return lo | (hi << 16);
  };
  return make_uint2(pack(0), pack(4));
}

template <bool VEC, typename T>
__device__ __forceinline__ void quantize_row(const QuantI8Args& a, int64_t i) {
  int64_t from = i, to = i;
  if (a.limit && a.p_begin + i >= *a.limit) return;  // behind the last routed row
  if (a.sched) {
    const int64_t p = a.p_begin + i;
    const int32_t route = a.sched[p];
    from = route / a.k;
    to = p % a.ring_rows;
    if (route < 0 || from >= a.src_rows) {  // a table not built by the schedule kernels
      if (threadIdx.x == 0) raise_error(a.err, kErrExpertRange);
      return;
    }
  }
  const T* __restrict__ src = static_cast<const T*>(a.src) + from * a.K;
  int8_t* __restrict__ q = a.q + to * a.Kp;
  const int64_t chunks = a.Kp / kChunk;
  const int tid = threadIdx.x;

  float v[kHeld][kChunk];
  uint32_t bits = 0;  // largest |v| as bits: NaN above infinity above every number
  auto take = [&](const float(&w)[kChunk]) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const uint32_t b = __float_as_uint(w[e]) & 0x7fffffffu;
      bits = b > bits ? b : bits;
    }
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int64_t c = tid + h * kThreads;
    if (c < chunks)
      load_chunk<VEC>(src, c, a.K, v[h]);
    else
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[h][e] = 0.f;
    take(v[h]);
  }
  for (int64_t c = tid + kHeld * kThreads; c < chunks; c += kThreads) {
    float w[kChunk];
    load_chunk<VEC>(src, c, a.K, w);
    take(w);
  }
  __shared__ uint32_t part[kThreads / kWave];
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t o = __shfl_xor(bits, d);
    bits = o > bits ? o : bits;
  }
  if (lane_id() == 0) part[tid / kWave] = bits;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) bits = part[w] > bits ? part[w] : bits;

  const bool some = bits && bits < 0x7f800000u;  // neither all zero nor not finite
  const float m = __uint_as_float(bits);
  if (tid == 0) a.scale[to] = bits < 0x7f800000u ? m / 127.f : __uint_as_float(0x7fc00000u);
  const float r = some ? 127.f / m : 0.f;
  const bool exact = some && m < 0x1p-100f;  // r past fp32's range, or close
  auto put = [&](int64_t c, const float(&w)[kChunk]) {
    *reinterpret_cast<uint2*>(q + c * kChunk) = some ? quotients(w, m, r, exact) : make_uint2(0, 0);
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int64_t c = tid + h * kThreads;
    if (c < chunks) put(c, v[h]);
  }
  for (int64_t c = tid + kHeld * kThreads; c < chunks; c += kThreads) {
    float w[kChunk];
    load_chunk<VEC>(src, c, a.K, w);
    put(c, w);
  }
}

template <bool VEC, typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_i8_kernel(const QuantI8Args a) {
  quantize_row<VEC, T>(a, blockIdx.x);
}

// The rows of two matrices in one launch: the first rows0 workgroups take a's.
__global__ __launch_bounds__(kThreads) void quantize_two_i8_kernel(const QuantI8Args a, const QuantI8Args b,
                                                                   int rows0) {
  const int i = blockIdx.x;
  if (i < rows0)
    quantize_row<true, float>(a, i);
  else
    quantize_row<true, float>(b, i - rows0);
}

bool valid(const QuantI8Args& a) {
  return a.K > 0 && a.Kp >= a.K && a.Kp % 16 == 0 && reinterpret_cast<uintptr_t>(a.q) % 8 == 0;
}

}  // namespace

hipError_t launch_quantize_two_i8(const QuantI8Args& a, int64_t rows_a, const QuantI8Args& b, int64_t rows_b,
                                  hipStream_t stream) {
  if (rows_a <= 0 || rows_b <= 0 || rows_a + rows_b > 0x7fffffff || !valid(a) || !valid(b)) return hipErrorInvalidValue;
  for (const QuantI8Args* x : {&a, &b})
    if (x->K % 4 || reinterpret_cast<uintptr_t>(x->src) % 16) return hipErrorInvalidValue;
  quantize_two_i8_kernel<<<static_cast<unsigned>(rows_a + rows_b), kThreads, 0, stream>>>(a, b,
                                                                                          static_cast<int>(rows_a));
  return hipGetLastError();
}

hipError_t launch_quantize_rows_i8(const QuantI8Args& a, bool src_f32, int64_t rows, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  if (rows > 0x7fffffff || !valid(a)) return hipErrorInvalidValue;
  const int64_t per16 = src_f32 ? 4 : 8;  // elements in 16 bytes
  const bool vec = a.K % per16 == 0 && reinterpret_cast<uintptr_t>(a.src) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(rows)), block(kThreads);
  if (src_f32) {
    if (vec)
      quantize_rows_i8_kernel<true, float><<<grid, block, 0, stream>>>(a);
    else
      quantize_rows_i8_kernel<false, float><<<grid, block, 0, stream>>>(a);
  } else {
    if (vec)
      quantize_rows_i8_kernel<true, uint16_t><<<grid, block, 0, stream>>>(a);
    else
      quantize_rows_i8_kernel<false, uint16_t><<<grid, block, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
