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

#include "common.h"
#include "i8.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStage = 128;  // bytes of K per stage

// Where a product's activation fragments come from: quantised rows in memory,
// or rows that the workgroup quantised into LDS itself.
template <int RB>
struct GlobalRows {
  const int8_t* p[RB];  // this lane's row and K offset
  __device__ __forceinline__ i32x4_t operator()(int rb, int st, int s) const {
    return *reinterpret_cast<const i32x4_t*>(p[rb] + static_cast<int64_t>(st) * kStage + s * 64);
  }
};
struct LdsRows {
  const char* p;
  __device__ __forceinline__ i32x4_t operator()(int, int st, int s) const {
    return *reinterpret_cast<const i32x4_t*>(p + st * kStage + s * 64);
  }
};

// The sums of this wave's K stages: NBL blocks of 16 columns (SwiGLU: of gate
// and of up) by RB blocks of 16 rows.
template <int NB, int NBL, int RB, int WAVES, typename Rows>
__device__ __forceinline__ void rows_sums(const I8GemmArgs& a, int e, int n0, const Rows& rows, int wave, int lane,
                                          i32x4_t (&acc)[NB][NBL][RB]) {
  const int r16 = lane & 15, kq = lane >> 4;
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
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int b = 0; b < NBL; ++b)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) acc[h][b][rb] = i32x4_t{};

  // (several stages' loads in flight per wave measured no faster: the other
  // waves of the CU cover them)
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
      for (int s = 0; s < 2; ++s) av[rb][s] = rows(rb, st, s);
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
}

// The waves' sums meet in LDS; each wave finishes some of the (column block,
// row block) pairs.  scale(rb): the scale of this lane's row.
template <int NB, int NBL, int RB, int WAVES, int EPI, typename Scale>
__device__ __forceinline__ void rows_finish(const I8GemmArgs& a, int e, int64_t p0, int nrows, int n0, i32x4_t* red,
                                            int wave, int lane, const i32x4_t (&acc)[NB][NBL][RB],
                                            const Scale& scale) {
  const int r16 = lane & 15, kq = lane >> 4;
  constexpr int BLK = NB * NBL * RB;
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int b = 0; b < NBL; ++b)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) red[(wave * BLK + (h * NBL + b) * RB + rb) * kWave + lane] = acc[h][b][rb];
  __syncthreads();
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
    const float sa = scale(rb);
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

template <int NBL, int RB, int WAVES, int EPI>
__device__ __forceinline__ void rows_item(const I8GemmArgs& a, int e, int64_t p0, int nrows, int n0, i32x4_t* red) {
  constexpr int NB = EPI == kEpiSwiGLU ? 2 : 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  int64_t arow[RB];
  GlobalRows<RB> rows;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = rb * 16 + (lane & 15);
    arow[rb] = i8_a_row(a, p0 + (row < nrows ? row : nrows - 1));
    rows.p[rb] = a.A + arow[rb] * a.K + (lane >> 4) * 16;
  }
  i32x4_t acc[NB][NBL][RB];
  rows_sums<NB, NBL, RB, WAVES>(a, e, n0, rows, wave, lane, acc);
  rows_finish<NB, NBL, RB, WAVES, EPI>(a, e, p0, nrows, n0, red, wave, lane, acc,
                                       [&](int rb) { return a.As[arow[rb]]; });
}

// Block `block` of a product in blocks of COLS columns: its expert, rows and
// first column; false if there is none (past the last tile).
template <int COLS>
__device__ __forceinline__ bool find_block(const I8GemmArgs& a, int block, int& e, int64_t& p0, int& nrows, int& n0) {
  const int n_blocks = (a.N + COLS - 1) / COLS;
  const int ti = block / n_blocks;
  n0 = block % n_blocks * COLS;
  if (a.tiles) {
    if (ti >= *a.tile_count) return false;
    const int4 t = a.tiles[ti];
    e = t.x & 1023;
    p0 = t.y;
    nrows = t.z;
  } else {
    e = 0;
    p0 = static_cast<int64_t>(ti) * kI8RowsBM;
    nrows = static_cast<int>(min(static_cast<int64_t>(kI8RowsBM), a.dense_rows - p0));
  }
  return true;
}

template <int NBL, int WAVES, int EPI>
__device__ __forceinline__ void rows_block(const I8GemmArgs& a, int block, i32x4_t* red) {
  int e, nrows, n0;
  int64_t p0;
  if (!find_block<16 * NBL>(a, block, e, p0, nrows, n0)) return;
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

// ---- a dense product of up to three rows that quantises them itself: every
// workgroup reads the rows x [.][K] (out of L2) and keeps their quotients in LDS,
// which saves a launch (1 x 2048 x 7168: 9.8 us in a graph against 13.2, called
// from Python 10.1 against 13.6; three rows 12.9 against 13.2 and 10.6 against
// 13.6; four rows 14.4 against 13.5).  In a layer, where the next launch waits on
// the GPU, it gains nothing.  a: as for the other products, without A and As.
// (LDS: the rows beside the partial sums, within the 64 KB of a plain launch.) ----
constexpr int kFusedRows = 3, kFusedLds = 40 * 1024;

template <int WAVES, int EPI, bool VEC, typename T>
__global__ __launch_bounds__(WAVES* kWave) void linear_i8_rows_kernel(const I8GemmArgs a, const T* __restrict__ x,
                                                                      int K) {
  extern __shared__ __attribute__((aligned(16))) char xq[];
  __shared__ i32x4_t red[WAVES * kWave];
  __shared__ uint32_t part[kFusedRows][WAVES];
  const int n0 = blockIdx.x * 16, nrows = a.dense_rows;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int chunks = a.K / kI8Chunk;
  const int stride = a.K + 16;  // rows at one K position fall on distinct banks
  for (int m = 0; m < nrows; ++m) {
    const T* __restrict__ row = x + static_cast<int64_t>(m) * K;
    uint32_t bits = 0;
    for (int c = tid; c < chunks; c += WAVES * kWave) {
      float v[kI8Chunk];
      i8_load_chunk<VEC>(row, c, K, v);
      bits = i8_max_bits(v, bits);
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const uint32_t o = __shfl_xor(bits, d);
      bits = o > bits ? o : bits;
    }
    if (lane == 0) part[m][wave] = bits;
  }
  __syncthreads();
  auto row_bits = [&](int m) {
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) bits = part[m][w] > bits ? part[m][w] : bits;
    return bits;
  };
  for (int m = 0; m < nrows; ++m) {
    const T* __restrict__ row = x + static_cast<int64_t>(m) * K;
    const I8RowScale quant(row_bits(m));
    for (int c = tid; c < chunks; c += WAVES * kWave) {
      float v[kI8Chunk];
      i8_load_chunk<VEC>(row, c, K, v);
      *reinterpret_cast<uint2*>(xq + m * stride + c * kI8Chunk) = quant(v);
    }
  }
  __syncthreads();
  const int row = (lane & 15) < nrows ? lane & 15 : nrows - 1;
  const LdsRows rows{xq + row * stride + (lane >> 4) * 16};
  i32x4_t acc[1][1][1];
  rows_sums<1, 1, 1, WAVES>(a, 0, n0, rows, wave, lane, acc);
  rows_finish<1, 1, 1, WAVES, EPI>(a, 0, 0, nrows, n0, red, wave, lane, acc,
                                   [&](int) { return I8RowScale(row_bits(row)).scale; });
}

template <int EPI, typename T>
hipError_t run_linear(const I8GemmArgs& a, const void* x, int64_t K, hipStream_t stream) {
  constexpr int kWaves = 8;
  const T* src = static_cast<const T*>(x);
  const bool vec = K % (16 / sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const dim3 grid((a.N + 15) / 16), block(kWaves * kWave);
  const size_t lds = static_cast<size_t>(a.dense_rows) * (a.K + 16);
  if (vec)
    linear_i8_rows_kernel<kWaves, EPI, true, T><<<grid, block, lds, stream>>>(a, src, static_cast<int>(K));
  else
    linear_i8_rows_kernel<kWaves, EPI, false, T><<<grid, block, lds, stream>>>(a, src, static_cast<int>(K));
  return hipGetLastError();
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
// the fastest, with the K axis over eight waves (the product alone of
// 1 x 2048 x 7168, as moe_matmul_int8 runs it: 8.4 us, 12.1 with four waves, 13.8
// with 32 columns); past that wider blocks read the
// activations less often (64 x 7168 x 2048: 11.1 us with 64 columns, 15.3 with
// 16).  SwiGLU blocks hold gate and up columns and stay at 16 (the layer of
// 7168 x 2048 and 256 experts at one token: 96 us, 103 with 32; at 64 tokens
// 1.63 ms and 1.64); four waves do there once the blocks fill the chip (99 us
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

bool linear_i8_fused(int64_t M, int64_t K) { return M <= kFusedRows && M * (K + 16) <= kFusedLds; }

hipError_t launch_linear_i8_fused(const I8GemmArgs& a, const void* x, bool x_f32, int64_t K, int epilogue,
                                  hipStream_t stream) {
  if (!x || K > a.K || K <= a.K - kStage || a.K % kStage || !linear_i8_fused(a.dense_rows, a.K))
    return hipErrorInvalidValue;
  if (epilogue == kEpiBF16)
    return x_f32 ? run_linear<kEpiBF16, float>(a, x, K, stream) : run_linear<kEpiBF16, uint16_t>(a, x, K, stream);
  if (epilogue == kEpiF32)
    return x_f32 ? run_linear<kEpiF32, float>(a, x, K, stream) : run_linear<kEpiF32, uint16_t>(a, x, K, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_i8_pair(const I8GemmArgs& a, int epi_a, const I8GemmArgs& b, int epi_b, hipStream_t stream) {
  const hipError_t bad_a = check_i8(a, epi_a), bad_b = check_i8(b, epi_b);
  if (bad_a != hipSuccess) return bad_a;
  if (bad_b != hipSuccess) return bad_b;
  if (a.tile_rows != kI8RowsBM || b.tile_rows != kI8RowsBM) return hipErrorInvalidValue;
  if (epi_a == kEpiSwiGLU && epi_b == kEpiSwiGLU) return pick_rows<kEpiSwiGLU, kEpiSwiGLU>(a, &b, stream);
  if (epi_a == kEpiBF16 && epi_b == kEpiF32) return pick_rows<kEpiBF16, kEpiF32>(a, &b, stream);
  return hipErrorInvalidValue;
}

}  // namespace moe
