// Products in 8-bit integers on gfx950, for many rows: C[r, n] = sa[r] sb[n]
// sum_k A[r, k] B[n, k], over the experts' tile lists or dense, in the pipeline
// of the MXFP8 kernels: 256 x BN tiles, 8 waves, K stages of 128 bytes per row
// in two LDS rings fed by direct buffer->LDS loads (activation rows one stage
// ahead, weight rows two), one barrier per stage.
//
// v_mfma_i32_32x32x32_i8 multiplies a 32x32 block of A by one of B in int32;
// lane l supplies row l % 32, 16 bytes of K chosen by l / 32.  Which bytes does
// not matter as long as A and B agree, and integer sums do not depend on their
// order.  A sum of 65536 products stays below 2^30.
//
// The scales are applied once, to the int32 sums: a row's from LDS, a column's
// from a register.  Epilogues, staged through LDS so that rows leave in 16-byte
// stores: SwiGLU in fp32 (h is quantised when its whole row is known), bf16
// scattered to the rows' routes, and fp32 in 128-row bands.

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBM = kI8BM;
constexpr int kRB = 128;           // bytes (K elements) of one stage row
constexpr int kNSA = 2, kNSB = 3;  // ring slots: activation rows, weight rows
constexpr int kWM = 4, kWN = 2;    // waves along rows and columns, two per SIMD
constexpr int kNW = kWM * kWN;

struct I8Src {
  __amdgpu_buffer_rsrc_t a, b0, b1;
};

// Row of the tile held by 32-row block fm of a wave in row group wm.
__device__ __forceinline__ int tile_row(int wm, int fm) { return (fm * kWM + wm) * 32; }

// The K loop of one workgroup; FML of the wave's FM row blocks hold tile rows.
template <int BN, int NB, int FML, int FM, int FN, int AI, int BI>
__device__ __forceinline__ void k_loop_i8(char* smem, const I8Src& src, const uint32_t (&a_off)[AI],
                                          const uint32_t (&b_off)[BI], int b_stage, int nk, int a_rows, int tid,
                                          int wm, int wn, i32x16_t (&acc)[NB][FM][FN]) {
  constexpr int BROWS = NB * BN, WTN = BN / kWN;
  constexpr int ASLOT = kBM * kRB, BSLOT = BROWS * kRB;
  constexpr int ROWS_PER_LD = 1024 / kRB;
  static_assert(AI * ROWS_PER_LD * kNW == kBM && BI * ROWS_PER_LD * kNW == BROWS, "loads per wave per stage");
  static_assert(BI < 16, "vmcnt range");
  char* const sa0 = smem;
  char* const sb0 = smem + kNSA * ASLOT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int frag_row = lane & 31, frag_h = lane >> 5;

  // a stage past the last loads the last one again, into a free slot, so
  // that every step issues the same number of loads
  auto issue_a = [&](int kt) __attribute__((always_inline)) {
    const int kc = kt < nk ? kt : nk - 1;
    char* sa = sa0 + (kt % kNSA) * ASLOT;
#pragma unroll
    for (int j = 0; j < AI; ++j)
      dma16(src.a, sa + (wave * AI + j) * 1024, (wave * AI + j) * ROWS_PER_LD < a_rows ? a_off[j] : a_off[0],
            kc * kRB);
  };
  auto issue_b = [&](int kt) __attribute__((always_inline)) {
    const int kc = kt < nk ? kt : nk - 1;
    char* sb = sb0 + (kt % kNSB) * BSLOT;
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      const int g = wave * BI + j;
      dma16((NB == 2 && g * ROWS_PER_LD >= BN) ? src.b1 : src.b0, sb + g * 1024, b_off[j], kc * b_stage);
    }
  };

  struct Frags {
    i32x4_t a[FML > 0 ? FML : 1][2];
    i32x4_t b[NB][FN][2];
  };
  // LDS offsets of this lane's fragment halves per step: the swizzle term is
  // the same for all fragment rows of a lane (they differ by multiples of 32)
  static_assert((BN / 2) % 8 == 0, "fragment rows share the swizzle term");
  uint32_t abase[2][2], bbase[2][2];
#pragma unroll
  for (int step = 0; step < 2; ++step)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = step * 4 + frag_h + 2 * j;
      abase[step][j] = swz<kRB>(tile_row(wm, 0) + frag_row, c);
      bbase[step][j] = swz<kRB>(wn * WTN + frag_row, c);
    }
  auto read_frags = [&](int kt, int step, Frags& f) __attribute__((always_inline)) {
    const char* sa = sa0 + (kt % kNSA) * ASLOT;
    const char* sb = sb0 + (kt % kNSB) * BSLOT;
    constexpr int kFragA = kWM * 32 * kRB;  // bytes between a lane's A fragment rows
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int fm = 0; fm < FML; ++fm)
        f.a[fm][j] = *reinterpret_cast<const i32x4_t*>(sa + abase[step][j] + fm * kFragA);
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
          f.b[h][fn][j] = *reinterpret_cast<const i32x4_t*>(sb + bbase[step][j] + (h * BN + fn * 32) * kRB);
    }
  };
  auto mfmas = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int fm = 0; fm < FML; ++fm)
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int fn = 0; fn < FN; ++fn)
            acc[h][fm][fn] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[fm][j], f.b[h][fn][j], acc[h][fm][fn], 0, 0, 0);
  };
  constexpr int NMF = 2 * FML * NB * FN;
  constexpr int NRD = 2 * (FML + NB * FN);
  // fragment reads spread under the MFMAs; in step 0 also the A loads
  auto interleave = [&](bool loads) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NMF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < NRD) __builtin_amdgcn_sched_group_barrier(0x100, NMF < NRD ? 2 : 1, 0);
      if (loads && i < AI) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };

  issue_a(0);
  issue_b(0);
  issue_b(1);
  asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(BI, 15)) : "memory");  // A(0), B(0) landed
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags f[2];
  if constexpr (FML > 0) read_frags(0, 0, f[0]);
  for (int kt = 0; kt < nk; ++kt) {
    issue_a(kt + 1);
    if constexpr (FML > 0) {
      read_frags(kt, 1, f[1]);
      mfmas(f[0]);
      interleave(true);
    }
    issue_b(kt + 2);
    // A(kt+1) and B(kt+1) have landed (B(kt+2) may still be in flight) and
    // this wave's reads of stage kt are done
    asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(BI, 0)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (FML > 0) {
      // past the last stage: a slot whose data is never used
      read_frags(kt + 1, 0, f[0]);
      mfmas(f[1]);
      interleave(false);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may still target LDS when the workgroup ends
}

// One work item (row tile, N block): its K loop and its epilogue.  The
// workgroup's LDS is free on entry and on return.
template <int BN, int EPI>
__device__ __forceinline__ void gemm_i8_item(const I8GemmArgs& args, int w, int n_blocks, int dense_tiles, char* smem,
                                             int wave0) {
  constexpr int NB = (EPI == kEpiSwiGLU) ? 2 : 1;
  constexpr int BROWS = NB * BN;
  constexpr int WTN = BN / kWN;
  constexpr int FM = kBM / kWM / 32, FN = WTN / 32;
  constexpr int ROWS_PER_LD = 1024 / kRB;
  constexpr int AI = kBM / (kNW * ROWS_PER_LD), BI = BROWS / (kNW * ROWS_PER_LD);
  constexpr int LDS_BYTES = kNSA * kBM * kRB + kNSB * BROWS * kRB;

  constexpr bool kItemLoop = EPI == kEpiBF16;  // resident workgroups walk several items
  const int tid = kItemLoop ? item_thread_index(wave0) : static_cast<int>(threadIdx.x);
  const int lane = tid & (kWave - 1), wave = kItemLoop ? wave0 : __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / kWN, wn = wave % kWN;

  int e = 0, nb, lt, nrows;
  int64_t p0;
  if (args.tiles) {
    const int4 g = load_uniform(args.tiles + w / n_blocks);
    const int nt = g.x >> 10, first = g.w;
    grouped_item(w - first * n_blocks, nt, n_blocks, nb, lt);
    const int4 t = load_uniform(args.tiles + first + lt);
    e = t.x & 1023;
    p0 = t.y;
    nrows = t.z;
  } else {  // rows 0 .. dense_rows - 1 in tiles of equal height, a multiple of 32
    grouped_item(w, dense_tiles, n_blocks, nb, lt);
    const int h = ((args.dense_rows + dense_tiles - 1) / dense_tiles + 31) / 32 * 32;
    p0 = static_cast<int64_t>(lt) * h;
    nrows = args.dense_rows - static_cast<int>(p0) < h ? args.dense_rows - static_cast<int>(p0) : h;
    if (nrows <= 0) return;  // rounding the height up may leave the last tiles empty
  }
  const int n0 = nb * BN;
  const int K = args.K;

  // the scale of tile row tid, kept through the K loop
  const float my_scale = tid < kBM ? args.As[i8_a_row(args, p0 + (tid < nrows ? tid : nrows - 1))] : 0.f;
  // ---- byte offsets of the 16-byte chunks this lane fetches ----
  constexpr int CH = kRB / 16;
  uint32_t a_off[AI];
#pragma unroll
  for (int j = 0; j < AI; ++j) {
    const int row = ROWS_PER_LD * (wave * AI + j) + lane / CH;
    const int c = (lane % CH) ^ ((row / (256 / kRB)) & (CH - 1));
    a_off[j] = static_cast<uint32_t>(i8_a_row(args, p0 + (row < nrows ? row : nrows - 1)) * K + c * 16);
  }
  const bool b_tiled = args.b_plane > 0;
  const int b_stage = b_tiled ? static_cast<int>(args.b_plane * kRB) : kRB;
  uint32_t b_off[BI];
#pragma unroll
  for (int j = 0; j < BI; ++j) {
    const int row = ROWS_PER_LD * (wave * BI + j) + lane / CH;
    const int c = (lane % CH) ^ ((row / (256 / kRB)) & (CH - 1));
    const int half = row / BN;
    int n = n0 + (row - half * BN);
    n = n < args.N ? n : args.N - 1;
    b_off[j] = static_cast<uint32_t>(b_tiled ? n * kRB + c * 16 : n * K + c * 16);
  }
  constexpr int kRsrcWord3 = 0x00020000;
  I8Src src;
  src.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(args.A), 0, static_cast<int>(args.a_rows * K),
                                            kRsrcWord3);
  const int b_bytes = args.N * K;
  src.b0 = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(args.B0 + static_cast<int64_t>(e) * b_bytes), 0,
                                             b_bytes, kRsrcWord3);
  if constexpr (NB == 2)
    src.b1 = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(args.B1 + static_cast<int64_t>(e) * b_bytes), 0,
                                               b_bytes, kRsrcWord3);
  else
    src.b1 = src.b0;
  i32x16_t acc[NB][FM][FN];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) acc[h][fm][fn] = i32x16_t{};

  // 32-row blocks of this wave that hold tile rows (wave-uniform)
  int fm_live = ((nrows + 31) / 32 - wm + kWM - 1) / kWM;
  fm_live = fm_live < 0 ? 0 : (fm_live > FM ? FM : fm_live);
  const int nk = K / kRB;
  static_assert(FM == 2, "cases below");
  switch (fm_live) {
    case 0:
      k_loop_i8<BN, NB, 0, FM, FN, AI, BI>(smem, src, a_off, b_off, b_stage, nk, nrows, tid, wm, wn, acc);
      break;
    case 1:
      k_loop_i8<BN, NB, 1, FM, FN, AI, BI>(smem, src, a_off, b_off, b_stage, nk, nrows, tid, wm, wn, acc);
      break;
    default:
      k_loop_i8<BN, NB, 2, FM, FN, AI, BI>(smem, src, a_off, b_off, b_stage, nk, nrows, tid, wm, wn, acc);
      break;
  }

  // ---- epilogue: scales, then rows leave through LDS in 16-byte pieces ----
  // The MFMA layout gives lane l column l % 32 of rows 8*(r/4) + 4*(l/32) +
  // r%4 of each 32 x 32 block.
  float sb[NB][FN];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      int n = n0 + wn * WTN + fn * 32 + (lane & 31);
      n = n < args.N ? n : args.N - 1;
      sb[h][fn] = (h ? args.Bs1 : args.Bs0)[static_cast<int64_t>(e) * args.N + n];
    }
  __syncthreads();  // every wave is done with the K loop's LDS
  constexpr int kScaleAt = LDS_BYTES - kBM * 4;  // row scales, past every staged tile
  float* row_s = reinterpret_cast<float*>(smem + kScaleAt);
  if (tid < kBM) row_s[tid] = my_scale;
  __syncthreads();
  auto value = [&](int h, int fm, int fn, int r, float s) {
    return static_cast<float>(acc[h][fm][fn][r]) * s * sb[h][fn];
  };
  if constexpr (EPI == kEpiSwiGLU) {
    constexpr int VS = BN * 4 + 16;  // fp32 row stride of the staged tile
    static_assert(kBM * VS <= kScaleAt, "staged tile fits");
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      if (fm >= fm_live) continue;  // wave-uniform
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int row0 = tile_row(wm, fm) + r4 * 8 + (lane >> 5) * 4;
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row_s + row0);
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float*>(smem + (row0 + i) * VS + (wn * WTN + fn * 32 + (lane & 31)) * 4) =
                silu_mul(value(0, fm, fn, r4 * 4 + i, s[i]), value(NB - 1, fm, fn, r4 * 4 + i, s[i]));
      }
    }
    __syncthreads();
    constexpr int CPR = BN * 4 / 16;
    for (int idx = tid; idx < nrows * CPR; idx += 64 * kNW) {
      const int row = idx / CPR, ch = idx - row * CPR;
      const int col = n0 + ch * 4;
      const int64_t crow = i8_c_row(args, p0 + row);
      if (col >= args.N || crow < 0) continue;  // N % 128 == 0: a chunk is all in or out
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(args.C) + crow * args.ldc + col) =
          *reinterpret_cast<const f32x4_t*>(smem + row * VS + ch * 16);
    }
  } else if constexpr (EPI == kEpiF32) {
    // one 128-row band per 32-row block index fm
    constexpr int CS = BN * 4 + 16;
    constexpr int BAND = kWM * 32;
    static_assert(BAND * CS <= kScaleAt, "staged band fits");
    constexpr int CPR = BN * 4 / 16;
    const bool whole = args.N % 4 == 0 && args.ldc % 4 == 0;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      if (fm * BAND >= nrows) break;  // workgroup-uniform
      if (fm > 0) __syncthreads();    // the previous band's copy-out is done with the LDS
      if (fm < fm_live) {             // wave-uniform
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int row_b = wm * 32 + r4 * 8 + (lane >> 5) * 4;
          const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row_s + fm * BAND + row_b);
#pragma unroll
          for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float*>(smem + (row_b + i) * CS + (wn * WTN + fn * 32 + (lane & 31)) * 4) =
                  value(0, fm, fn, r4 * 4 + i, s[i]);
        }
      }
      __syncthreads();
      const int band_rows = min(BAND, nrows - fm * BAND);
      for (int idx = tid; idx < band_rows * CPR; idx += 64 * kNW) {
        const int row = idx / CPR, ch = idx - row * CPR;
        const int col = n0 + ch * 4;
        const int64_t crow = i8_c_row(args, p0 + fm * BAND + row);
        if (col >= args.N || crow < 0) continue;
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(smem + row * CS + ch * 16);
        float* c = static_cast<float*>(args.C) + crow * args.ldc + col;
        if (whole)
          *reinterpret_cast<f32x4_t*>(c) = v;
        else
          for (int i = 0; i < 4 && col + i < args.N; ++i) c[i] = v[i];
      }
    }
  } else {
    constexpr int CS = BN * 2 + 16;  // bf16 row stride of the staged tile
    static_assert(kBM * CS <= kScaleAt, "staged tile fits");
    constexpr int CPR = BN * 2 / 16;
    // In pass `it`, wave w stores tile rows it * RSTEP + w * RPI + lane / CPR.
    // A row table's entries are read once, before any store, and passed on by
    // a cross-lane read (a table load among the stores would wait for them).
    constexpr int RPI = 64 / CPR, RSTEP = RPI * kNW;
    static_assert(64 % CPR == 0 && kBM <= 64 * kNW, "copy-out mapping");
    int row_entry = -1;
    {
      const int r = (lane / RPI) * RSTEP + wave * RPI + lane % RPI;
      if (r < nrows) row_entry = static_cast<int>(i8_c_row(args, p0 + r));
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      if (fm >= fm_live) continue;  // wave-uniform
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int row0 = tile_row(wm, fm) + r4 * 8 + (lane >> 5) * 4;
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row_s + row0);
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint16_t*>(smem + (row0 + i) * CS + (wn * WTN + fn * 32 + (lane & 31)) * 2) =
                f32_to_bf16(value(0, fm, fn, r4 * 4 + i, s[i]));
      }
    }
    __syncthreads();
    const bool whole = args.N % 8 == 0 && args.ldc % 8 == 0;
    for (int it = 0; it * RSTEP < nrows; ++it) {
      const int row = it * RSTEP + wave * RPI + lane / CPR, ch = lane % CPR;
      const int crow = __shfl(row_entry, it * RPI + lane / CPR);
      const int col = n0 + ch * 8;
      if (row >= nrows || col >= args.N || crow < 0) continue;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + row * CS + ch * 16);
      uint16_t* c = static_cast<uint16_t*>(args.C) + static_cast<int64_t>(crow) * args.ldc + col;
      if (whole)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(c));
      else
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < args.N) c[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)));
    }
  }
}

// Work items are cut into 8 contiguous runs, one per XCD, as in the MXFP8
// kernels: workgroup b takes item b / 8 of the run of XCD b mod 8, and the
// bf16 epilogue's resident workgroups walk their run side by side, so that one
// item's output stores drain under the next one's first loads.
template <int BN, int EPI>
__global__ __launch_bounds__(64 * kNW) void gemm_i8_kernel(const I8GemmArgs args, int dense_tiles) {
  constexpr int NB = (EPI == kEpiSwiGLU) ? 2 : 1;
  __shared__ __attribute__((aligned(1024))) char smem[kNSA * kBM * kRB + kNSB * NB * BN * kRB];
  const int n_blocks = (args.N + BN - 1) / BN;
  const int xcd = static_cast<int>(blockIdx.x) % kXcds;
  int run0, len;
  if (args.tiles) {  // positions in 1/kTileRunFrac of a tile
    run0 = static_cast<int>(static_cast<int64_t>(__builtin_amdgcn_readfirstlane(args.tile_runs[xcd])) * n_blocks /
                            kTileRunFrac);
    len = static_cast<int>(static_cast<int64_t>(__builtin_amdgcn_readfirstlane(args.tile_runs[xcd + 1])) * n_blocks /
                           kTileRunFrac) -
          run0;
  } else {
    const int W = dense_tiles * n_blocks, chunk = (W + kXcds - 1) / kXcds;
    run0 = xcd * chunk;
    len = W - run0 < chunk ? W - run0 : chunk;
  }
  const int first = static_cast<int>(blockIdx.x) / kXcds;
  const int per_xcd = static_cast<int>(gridDim.x) / kXcds;  // the grid is a multiple of kXcds
  const int wave0 = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  if constexpr (EPI != kEpiBF16) {
    if (first < len) gemm_i8_item<BN, EPI>(args, run0 + first, n_blocks, dense_tiles, smem, wave0);
  } else {
    for (int local = first; local < len; local += per_xcd) {
      if (local > first) __syncthreads();  // the previous item's copy-out has read the LDS
      gemm_i8_item<BN, EPI>(args, __builtin_amdgcn_readfirstlane(run0 + local), n_blocks, dense_tiles, smem, wave0);
    }
  }
}

template <int BN, int EPI>
hipError_t run_i8(const I8GemmArgs& a, hipStream_t stream) {
  const int64_t n_blocks = (a.N + BN - 1) / BN;
  const int64_t dense_tiles = a.tiles ? 0 : (static_cast<int64_t>(a.dense_rows) + kBM - 1) / kBM;
  const int64_t work = (a.tiles ? a.max_tiles : dense_tiles) * n_blocks;
  if (work <= 0) return hipSuccess;
  if (work > 0x7ffffff0) return hipErrorInvalidValue;
  auto kernel = gemm_i8_kernel<BN, EPI>;
  // with room for balanced runs of up to tile_run_cap tiles on every XCD
  int64_t cap = a.tiles ? int64_t(kXcds) * tile_run_cap(a.max_tiles) * n_blocks : work;
  if (EPI == kEpiBF16) {
    static std::atomic<int64_t> resident_cache{0};
    int64_t resident = resident_cache.load(std::memory_order_relaxed);
    if (resident <= 0) {
      resident = resident_workgroups(reinterpret_cast<const void*>(kernel), 64 * kNW);
      if (resident <= 0) return hipErrorInvalidValue;
      resident_cache.store(resident, std::memory_order_relaxed);
    }
    cap = std::min(work, resident);
  }
  const int64_t grid = (cap + kXcds - 1) / kXcds * kXcds;
  kernel<<<static_cast<unsigned>(grid), 64 * kNW, 0, stream>>>(a, static_cast<int>(dense_tiles));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8_tiles(const I8GemmArgs& a, int epilogue, hipStream_t stream) {
  if (a.tiles && !a.tile_runs) return hipErrorInvalidValue;
  switch (epilogue) {
    case kEpiSwiGLU:
      if (a.N % 4 || a.ldc % 4) return hipErrorInvalidValue;
      return run_i8<128, kEpiSwiGLU>(a, stream);
    case kEpiBF16:
      return run_i8<256, kEpiBF16>(a, stream);
    case kEpiF32:
      return run_i8<256, kEpiF32>(a, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace moe
