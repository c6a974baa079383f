// Products in 8-bit integers for few rows, on gfx950: C[r, n] = sa[r] sb[n]
// sum_k A[r, k] B[n, k], dense (moe_matmul_int8) or over the experts' tile
// lists (moe_forward).
//
// With few rows the weights' bytes are the time, so they go from memory
// straight to the matrix core's registers: no LDS, no barrier in the K loop.
// v_mfma_i32_16x16x64_i8 takes 16 weight rows as its row operand and 16
// activation rows as its column operand; lane l supplies row l % 16, bytes
// 16 (l / 16) .. + 15 of the 64-byte step, and ends up with four consecutive
// output columns of one activation row.  The four waves of a workgroup take
// every fourth 128-byte stage of K and meet in LDS, in integers, so the split
// changes no bit.

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kStage = 128;  // bytes of K per stage

// NBL blocks of 16 columns (SwiGLU: of gate and of up) by RB blocks of 16 rows.
template <int NBL, int RB, int EPI>
__device__ __forceinline__ void rows_item(const I8GemmArgs& a, int e, int64_t p0, int nrows, int n0, i32x4_t* red) {
  constexpr int NB = EPI == kEpiSwiGLU ? 2 : 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r16 = lane & 15, kq = lane >> 4;

  int64_t arow[RB];
  const int8_t* ap[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = rb * 16 + r16;
    arow[rb] = i8_a_row(a, p0 + (row < nrows ? row : nrows - 1));
    ap[rb] = a.A + arow[rb] * a.K + kq * 16;
  }
  // weights: row n of stage st at n * row_b + st * stage_b
  const int64_t row_b = a.b_plane ? kStage : a.K, stage_b = a.b_plane ? a.b_plane * kStage : kStage;
  const int64_t expert = static_cast<int64_t>(e) * a.N * a.K;
  const int8_t* bp[NB][NBL];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int b = 0; b < NBL; ++b) {
      int n = n0 + b * 16 + r16;
      n = n < a.N ? n : a.N - 1;
      bp[h][b] = (h ? a.B1 : a.B0) + expert + n * row_b + kq * 16;
    }
  i32x4_t acc[NB][NBL][RB];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int b = 0; b < NBL; ++b)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) acc[h][b][rb] = i32x4_t{};

  const int nk = a.K / kStage;
  for (int st = wave; st < nk; st += kWaves) {
    i32x4_t av[RB][2], bv[NB][NBL][2];
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
      for (int b = 0; b < NBL; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          bv[h][b][s] = *reinterpret_cast<const i32x4_t*>(bp[h][b] + st * stage_b + s * 64);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        av[rb][s] = *reinterpret_cast<const i32x4_t*>(ap[rb] + static_cast<int64_t>(st) * kStage + s * 64);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int b = 0; b < NBL; ++b)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            acc[h][b][rb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[h][b][s], av[rb][s], acc[h][b][rb], 0, 0, 0);
  }

  constexpr int BLK = NB * NBL * RB;
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int b = 0; b < NBL; ++b)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) red[(wave * BLK + (h * NBL + b) * RB + rb) * kWave + lane] = acc[h][b][rb];
  __syncthreads();
  // each wave finishes some of the (column block, row block) pairs
  for (int pair = wave; pair < NBL * RB; pair += kWaves) {
    const int b = pair / RB, rb = pair % RB;
    i32x4_t sum[NB];
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      sum[h] = red[(h * NBL * RB + pair) * kWave + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum[h] += red[(w * BLK + h * NBL * RB + pair) * kWave + lane];
    }
    const int row = rb * 16 + r16, col = n0 + b * 16 + kq * 4;
    if (row >= nrows || col >= a.N) continue;
    const int64_t p = p0 + row;
    const float sa = a.As[arow[rb]];
    const int64_t crow = i8_c_row(a, p);
    if (crow < 0) continue;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = col + i < a.N ? col + i : a.N - 1;
      const int64_t at = static_cast<int64_t>(e) * a.N + n;
      v[i] = static_cast<float>(sum[0][i]) * sa * a.Bs0[at];
      if constexpr (EPI == kEpiSwiGLU) v[i] = silu_mul(v[i], static_cast<float>(sum[1][i]) * sa * a.Bs1[at]);
    }
    const int64_t at = crow * a.ldc + col;
    const bool whole = col + 4 <= a.N && a.ldc % 4 == 0;
    if constexpr (EPI == kEpiBF16) {
      uint16_t* c = static_cast<uint16_t*>(a.C) + at;
      if (whole)
        *reinterpret_cast<uint2*>(c) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      else
        for (int i = 0; i < 4 && col + i < a.N; ++i) c[i] = f32_to_bf16(v[i]);
    } else {
      float* c = static_cast<float*>(a.C) + at;
      if (whole)
        *reinterpret_cast<f32x4_t*>(c) = f32x4_t{v[0], v[1], v[2], v[3]};
      else
        for (int i = 0; i < 4 && col + i < a.N; ++i) c[i] = v[i];
    }
  }
}

template <int NBL, int EPI>
__global__ __launch_bounds__(kWaves * kWave) void gemm_i8_rows_kernel(const I8GemmArgs a, int n_blocks) {
  constexpr int NB = EPI == kEpiSwiGLU ? 2 : 1;
  __shared__ i32x4_t red[kWaves * NB * NBL * 2 * kWave];
  const int ti = static_cast<int>(blockIdx.x) / n_blocks, n0 = static_cast<int>(blockIdx.x) % n_blocks * 16 * NBL;
  int e = 0, nrows;
  int64_t p0;
  if (a.tiles) {
    if (ti >= *a.tile_count) return;
    const int4 t = a.tiles[ti];
    e = t.x & 1023;
    p0 = t.y;
    nrows = t.z;
  } else {
    p0 = static_cast<int64_t>(ti) * kI8RowsBM;
    nrows = static_cast<int>(min(static_cast<int64_t>(kI8RowsBM), a.dense_rows - p0));
  }
  if (nrows <= 16)
    rows_item<NBL, 1, EPI>(a, e, p0, nrows, n0, red);
  else
    rows_item<NBL, 2, EPI>(a, e, p0, nrows, n0, red);
}

template <int NBL, int EPI>
hipError_t run_rows(const I8GemmArgs& a, hipStream_t stream) {
  const int64_t tiles = a.tiles ? a.max_tiles : (a.dense_rows + kI8RowsBM - 1) / kI8RowsBM;
  const int64_t n_blocks = (a.N + 16 * NBL - 1) / (16 * NBL), work = tiles * n_blocks;
  if (work <= 0) return hipSuccess;
  if (work > 0x7fffffff) return hipErrorInvalidValue;
  gemm_i8_rows_kernel<NBL, EPI>
      <<<static_cast<unsigned>(work), kWaves * kWave, 0, stream>>>(a, static_cast<int>(n_blocks));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const I8GemmArgs& a, int epilogue, hipStream_t stream) {
  if (a.K <= 0 || a.K % kStage || a.K > 65536 || a.N <= 0 || a.a_rows <= 0) return hipErrorInvalidValue;
  if (a.a_rows * a.K >= (int64_t(1) << 31) || static_cast<int64_t>(a.N) * a.K >= (int64_t(1) << 31))
    return hipErrorInvalidValue;
  if (a.b_plane != 0 && a.b_plane != a.N) return hipErrorInvalidValue;
  if (a.tiles && !a.tile_count) return hipErrorInvalidValue;
  for (const void* p : {static_cast<const void*>(a.A), static_cast<const void*>(a.B0),
                        static_cast<const void*>(epilogue == kEpiSwiGLU ? a.B1 : a.B0), static_cast<const void*>(a.C)})
    if (!p || reinterpret_cast<uintptr_t>(p) % 16) return hipErrorInvalidValue;
  if (a.tile_rows != kI8RowsBM) return launch_gemm_i8_tiles(a, epilogue, stream);
  switch (epilogue) {
    case kEpiSwiGLU:
      return run_rows<2, kEpiSwiGLU>(a, stream);
    case kEpiBF16:
      return run_rows<4, kEpiBF16>(a, stream);
    case kEpiF32:
      return run_rows<4, kEpiF32>(a, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace moe
