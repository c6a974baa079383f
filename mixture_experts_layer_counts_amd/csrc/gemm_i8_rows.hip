// Products in 8-bit integers for few rows, on gfx950: C[r, n] = sa[r] sb[n]
// sum_k A[r, k] B[n, k], dense (moe_matmul_int8) or over the experts' tile
// lists (moe_forward).
//
// With few rows the weights' bytes are the time, so they go from memory
// straight to the matrix core's registers: no LDS, no barrier in the K loop.
// v_mfma_i32_16x16x64_i8 takes 16 weight rows as its row operand and 16
// activation rows as its column operand; lane l supplies row l % 16, bytes
// 16 (l / 16) .. + 15 of the 64-byte step, and ends up with four consecutive
// output columns of one activation row.  The waves of a workgroup take the
// 128-byte stages of K in turn and meet in LDS, in integers, so the split
// changes no bit.
//
// One launch can hold two products (the routed experts' and the shared one's,
// which at a few tokens would each leave most of the chip idle).

#include <utility>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStage = 128;  // bytes of K per stage

// NBL blocks of 16 columns (SwiGLU: of gate and of up) by RB blocks of 16 rows.
template <int NBL, int RB, int WAVES, int EPI>
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
  for (int st = wave; st < nk; st += WAVES) {
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
  for (int pair = wave; pair < NBL * RB; pair += WAVES) {
    const int b = pair / RB, rb = pair % RB;
    i32x4_t sum[NB];
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      sum[h] = red[(h * NBL * RB + pair) * kWave + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum[h] += red[(w * BLK + h * NBL * RB + pair) * kWave + lane];
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

template <int NBL, int WAVES, int EPI>
__device__ __forceinline__ void rows_block(const I8GemmArgs& a, int block, i32x4_t* red) {
  const int n_blocks = (a.N + 16 * NBL - 1) / (16 * NBL);
  const int ti = block / n_blocks, n0 = block % n_blocks * 16 * NBL;
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
    rows_item<NBL, 1, WAVES, EPI>(a, e, p0, nrows, n0, red);
  else
    rows_item<NBL, 2, WAVES, EPI>(a, e, p0, nrows, n0, red);
}

// Workgroups below blocks0 work on `a`, the others on `b`.
template <int NBL, int WAVES, int EPI0, int EPI1>
__global__ __launch_bounds__(WAVES* kWave) void gemm_i8_rows_kernel(const I8GemmArgs a, const I8GemmArgs b,
                                                                    int blocks0) {
  constexpr int NB = EPI0 == kEpiSwiGLU ? 2 : 1;
  __shared__ i32x4_t red[WAVES * NB * NBL * 2 * kWave];
  const int block = blockIdx.x;
  if (block < blocks0)
    rows_block<NBL, WAVES, EPI0>(a, block, red);
  else
    rows_block<NBL, WAVES, EPI1>(b, block - blocks0, red);
}

int64_t rows_blocks(const I8GemmArgs& a, int cols) {
  const int64_t tiles = a.tiles ? a.max_tiles : (static_cast<int64_t>(a.dense_rows) + kI8RowsBM - 1) / kI8RowsBM;
  return tiles * ((a.N + cols - 1) / cols);
}

template <int NBL, int WAVES, int EPI0, int EPI1>
hipError_t run_rows(const I8GemmArgs& a, const I8GemmArgs* b, hipStream_t stream) {
  const int64_t first = rows_blocks(a, 16 * NBL), work = first + (b ? rows_blocks(*b, 16 * NBL) : 0);
  if (work <= 0) return hipSuccess;
  if (work > 0x7fffffff) return hipErrorInvalidValue;
  gemm_i8_rows_kernel<NBL, WAVES, EPI0, EPI1>
      <<<static_cast<unsigned>(work), WAVES * kWave, 0, stream>>>(a, b ? *b : a, static_cast<int>(first));
  return hipGetLastError();
}

// Columns per workgroup and waves per workgroup.  A CU streams some 40 GB/s, so
// while there are at most a CU's worth of 16-column blocks the finest split is
// the fastest, with the K axis over eight waves (1 x 2048 x 7168: 8.8 us, 12.1
// with four waves, 13.8 with 32 columns); past that wider blocks read the
// activations less often (64 x 7168 x 2048: 11.4 us with 64 columns, 15.3 with
// 16).  SwiGLU blocks hold gate and up columns and stay at 16 (the layer of
// 7168 x 2048 and 256 experts at one token: 114 us, 121 with 32; at 64 tokens
// 1.70 ms and 1.68); four waves do there once the blocks fill the chip (122 us
// with eight).
template <int EPI0, int EPI1>
hipError_t pick_rows(const I8GemmArgs& a, const I8GemmArgs* b, hipStream_t stream) {
  const int64_t blocks = rows_blocks(a, 16) + (b ? rows_blocks(*b, 16) : 0);
  if (blocks <= 256) return run_rows<1, 8, EPI0, EPI1>(a, b, stream);
  if constexpr (EPI0 == kEpiSwiGLU) {
    return run_rows<1, 4, EPI0, EPI1>(a, b, stream);
  } else {
    if (blocks <= 512) return run_rows<2, 4, EPI0, EPI1>(a, b, stream);
    return run_rows<4, 4, EPI0, EPI1>(a, b, stream);
  }
}

hipError_t check_i8(const I8GemmArgs& a, int epilogue) {
  if (a.K <= 0 || a.K % kStage || a.K > 65536 || a.N <= 0 || a.a_rows <= 0) return hipErrorInvalidValue;
  if (a.a_rows * a.K >= (int64_t(1) << 31) || static_cast<int64_t>(a.N) * a.K >= (int64_t(1) << 31))
    return hipErrorInvalidValue;
  if (a.b_plane != 0 && a.b_plane != a.N) return hipErrorInvalidValue;
  if (a.tiles && !a.tile_count) return hipErrorInvalidValue;
  for (const void* p : {static_cast<const void*>(a.A), static_cast<const void*>(a.B0),
                        static_cast<const void*>(epilogue == kEpiSwiGLU ? a.B1 : a.B0), static_cast<const void*>(a.C)})
    if (!p || reinterpret_cast<uintptr_t>(p) % 16) return hipErrorInvalidValue;
  return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_i8(const I8GemmArgs& a, int epilogue, hipStream_t stream) {
  const hipError_t bad = check_i8(a, epilogue);
  if (bad != hipSuccess) return bad;
  if (a.tile_rows != kI8RowsBM) return launch_gemm_i8_tiles(a, epilogue, stream);
  switch (epilogue) {
    case kEpiSwiGLU:
      return pick_rows<kEpiSwiGLU, kEpiSwiGLU>(a, nullptr, stream);
    case kEpiBF16:
      return pick_rows<kEpiBF16, kEpiBF16>(a, nullptr, stream);
    case kEpiF32:
      return pick_rows<kEpiF32, kEpiF32>(a, nullptr, stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm_i8_pair(const I8GemmArgs& a, int epi_a, const I8GemmArgs& b, int epi_b, hipStream_t stream) {
  for (const auto& [x, e] : {std::pair<const I8GemmArgs&, int>(a, epi_a), std::pair<const I8GemmArgs&, int>(b, epi_b)}) {
    const hipError_t bad = check_i8(x, e);
    if (bad != hipSuccess) return bad;
    if (x.tile_rows != kI8RowsBM) return hipErrorInvalidValue;
  }
  if (epi_a == kEpiSwiGLU && epi_b == kEpiSwiGLU) return pick_rows<kEpiSwiGLU, kEpiSwiGLU>(a, &b, stream);
  if (epi_a == kEpiBF16 && epi_b == kEpiF32) return pick_rows<kEpiBF16, kEpiF32>(a, &b, stream);
  return hipErrorInvalidValue;
}

}  // namespace moe
