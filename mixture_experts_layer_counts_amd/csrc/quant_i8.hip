// Rows to 8-bit integers with one scale per row, on gfx950 (moe_quantize_int8
// in include/moe.h; also the int8 layer's activations and its gather).
//
//   m = max |v|,  scale = m / 127,  q = round(127 v / m), ties to even
//
// A row of zeros has scale 0; a row with an infinity or a NaN has q = 0 and
// scale NaN, so that every product with it is NaN.  One workgroup per row: the
// row stays in registers between its maximum and its quotients.

#include "common.h"
#include "i8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kHeld = 4;  // chunks a thread keeps; longer rows are read twice

// Row i by `TH` threads: a wave of its own for rows of up to 2048 (no barrier,
// four rows a workgroup), a whole workgroup for longer ones.
template <int TH, bool VEC, typename T>
__device__ __forceinline__ void quantize_row(const QuantI8Args& a, int64_t i) {
  int64_t from = i, to = i;
  if (a.limit && a.p_begin + i >= *a.limit) return;  // behind the last routed row
  if (a.sched) {
    const int64_t p = a.p_begin + i;
    const int32_t route = a.sched[p];
    from = route / a.k;
    to = p % a.ring_rows;
    if (route < 0 || from >= a.src_rows) {  // a table not built by the schedule kernels
      if (static_cast<int>(threadIdx.x) % TH == 0) raise_error(a.err, kErrExpertRange);
      return;
    }
  }
  const T* __restrict__ src = static_cast<const T*>(a.src) + from * a.K;
  int8_t* __restrict__ q = a.q + to * a.Kp;
  const int64_t chunks = a.Kp / kI8Chunk;
  const int tid = static_cast<int>(threadIdx.x) % TH;

  float v[kHeld][kI8Chunk];
  uint32_t bits = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int64_t c = tid + h * TH;
    if (c < chunks)
      i8_load_chunk<VEC>(src, c, a.K, v[h]);
    else
#pragma unroll
      for (int e = 0; e < kI8Chunk; ++e) v[h][e] = 0.f;
    bits = i8_max_bits(v[h], bits);
  }
  for (int64_t c = tid + kHeld * TH; c < chunks; c += TH) {
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
  for (int h = 0; h < kHeld; ++h) {
    const int64_t c = tid + h * TH;
    if (c < chunks) put(c, v[h]);
  }
  for (int64_t c = tid + kHeld * TH; c < chunks; c += TH) {
    float w[kI8Chunk];
    i8_load_chunk<VEC>(src, c, a.K, w);
    put(c, w);
  }
}

template <int TH, bool VEC, typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_i8_kernel(const QuantI8Args a, int rows) {
  const int i = static_cast<int>(blockIdx.x) * (kThreads / TH) + static_cast<int>(threadIdx.x) / TH;
  if (i < rows) quantize_row<TH, VEC, T>(a, i);
}

// The rows of two matrices in one launch: the first rows0 workgroups take a's.
__global__ __launch_bounds__(kThreads) void quantize_two_i8_kernel(const QuantI8Args a, const QuantI8Args b,
                                                                   int rows0) {
  const int i = blockIdx.x;
  if (i < rows0)
    quantize_row<kThreads, true, float>(a, i);
  else
    quantize_row<kThreads, true, float>(b, i - rows0);
}

template <bool VEC, typename T>
hipError_t run_rows(const QuantI8Args& a, int rows, hipStream_t stream) {
  if (a.Kp <= kWave * kHeld * kI8Chunk) {
    constexpr int per = kThreads / kWave;
    quantize_rows_i8_kernel<kWave, VEC, T><<<(rows - 1) / per + 1, kThreads, 0, stream>>>(a, rows);
  } else {
    quantize_rows_i8_kernel<kThreads, VEC, T><<<rows, kThreads, 0, stream>>>(a, rows);
  }
  return hipGetLastError();
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
  const int n = static_cast<int>(rows);
  if (src_f32) return vec ? run_rows<true, float>(a, n, stream) : run_rows<false, float>(a, n, stream);
  return vec ? run_rows<true, uint16_t>(a, n, stream) : run_rows<false, uint16_t>(a, n, stream);
}

}  // namespace moe
