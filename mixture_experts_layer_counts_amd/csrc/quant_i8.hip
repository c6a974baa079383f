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
constexpr int kWaveRow = kWave * kI8Held * kI8Chunk;  // longest row that a wave holds
constexpr int64_t kLaunchRows = int64_t(1) << 23;     // a launch's threads stay below 2^32

template <int TH, bool VEC, typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_i8_kernel(const QuantI8Args a, int rows) {
  const int i = static_cast<int>(blockIdx.x) * (kThreads / TH) + static_cast<int>(threadIdx.x) / TH;
  if (i < rows) i8_quantize_row<TH, VEC, T>(a, i);
}

// The rows of two matrices in one launch: the first rows0 workgroups take a's.
__global__ __launch_bounds__(kThreads) void quantize_two_i8_kernel(const QuantI8Args a, const QuantI8Args b,
                                                                   int rows0) {
  const int i = blockIdx.x;
  if (i < rows0)
    i8_quantize_row<kThreads, true, float>(a, i);
  else
    i8_quantize_row<kThreads, true, float>(b, i - rows0);
}

template <bool VEC, typename T>
hipError_t run_rows(const QuantI8Args& a, int rows, hipStream_t stream) {
  if (a.Kp <= kWaveRow) {
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
  for (int64_t at = 0; at < rows; at += kLaunchRows) {
    QuantI8Args part = a;
    part.p_begin += at;
    if (!a.sched) {
      part.src = static_cast<const char*>(a.src) + at * a.K * (src_f32 ? 4 : 2);
      part.q += at * a.Kp;
      part.scale += at;
    }
    const int n = static_cast<int>(rows - at < kLaunchRows ? rows - at : kLaunchRows);
    hipError_t e;
    if (src_f32)
      e = vec ? run_rows<true, float>(part, n, stream) : run_rows<false, float>(part, n, stream);
    else
      e = vec ? run_rows<true, uint16_t>(part, n, stream) : run_rows<false, uint16_t>(part, n, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
