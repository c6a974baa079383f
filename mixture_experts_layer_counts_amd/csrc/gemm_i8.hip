// Products in 8-bit integers on gfx950, for many rows: C[r, n] = sa[r] sb[n]
// sum_k A[r, k] B[n, k], over the experts' tile lists or dense, in the pipeline
// of the bf16 kernels: K stages of 128 bytes per row in two LDS rings fed by
// direct buffer->LDS loads (activation rows one stage ahead, weight rows two
// where LDS holds a third slot), one barrier per stage.  The bytes per stage and
// the matrix instructions' cycles are those of the bf16 kernels, at twice the
// products.
//
// What bounds them is the load path: a CU streams rows into LDS at about 42
// GB/s however deep its rings are (five stages ahead measured no faster than
// two), so few rows want many small tiles on many CUs and many rows want the
// fewest bytes per product, the 256- and 320-row tiles.
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

constexpr int kRB = 128;  // bytes (K elements) of one stage row

// LDS ring slots: activation rows and weight rows.  A ring of n slots loads its
// rows n - 1 stages ahead.
constexpr int ring_bytes(int bm, int brows, int nsa, int nsb) { return (nsa * bm + nsb * brows) * kRB; }

struct I8Src {
  __amdgpu_buffer_rsrc_t a, b0, b1;
};

// Row of the tile held by 32-row block fm of a wave in row group wm: blocks
// are dealt to the row groups in turn, so a partly filled tile keeps every
// wave busy.
template <int WM>
__device__ __forceinline__ int tile_row(int wm, int fm) {
  return (fm * WM + wm) * 32;
}

// The K loop of one workgroup, the bf16 kernels' protocol: a slot is refilled
// right after the barrier that ends its stage's reads, the fragments of the
// next 32-wide sub-step are read under the current MFMAs, and one barrier per
// stage waits for the next stage's rows.  FML of the wave's FM row blocks hold
// tile rows.
template <int BM, int BN, int WM, int WN, int NSA, int NSB, int NB, int FML, int FM, int FN, int AI, int BI>
__device__ __forceinline__ void k_loop_i8(char* smem, const I8Src& src, const uint32_t (&a_off)[AI],
                                          const uint32_t (&b_off)[BI], int b_stage, int nk, int a_rows, int tid,
                                          int wm, int wn, i32x16_t (&acc)[NB][FM][FN]) {
  constexpr int BROWS = NB * BN, WTN = BN / WN;
  static_assert(NSA >= 2 && NSB >= NSA, "ring depths");
  constexpr int ASLOT = BM * kRB, BSLOT = BROWS * kRB;
  constexpr int KS = 4;  // 32-wide sub-steps per stage
  constexpr int ROWS_PER_LD = 1024 / kRB;
  static_assert(AI * ROWS_PER_LD * WM * WN == BM && BI * ROWS_PER_LD * WM * WN == BROWS, "loads per wave per stage");
  char* const sa0 = smem;
  char* const sb0 = smem + NSA * ASLOT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int frag_row = lane & 31, frag_c = lane >> 5;

  // a stage past the last (in the prologue of a short K) loads the last one
  // again, into a free slot, so that the prologue issues the same number of
  // loads; row groups past the tile reload the first one for the same reason
  auto issue_a = [&](int kt) __attribute__((always_inline)) {
    const int ko = (kt < nk ? kt : nk - 1) * kRB;
    char* sa = sa0 + (kt % NSA) * ASLOT;
#pragma unroll
    for (int j = 0; j < AI; ++j)
      dma16(src.a, sa + (wave * AI + j) * 1024, (wave * AI + j) * ROWS_PER_LD < a_rows ? a_off[j] : a_off[0], ko);
  };
  auto issue_b = [&](int kt) __attribute__((always_inline)) {
    const int ko = (kt < nk ? kt : nk - 1) * b_stage;
    char* sb = sb0 + (kt % NSB) * BSLOT;
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      const int g = wave * BI + j;
      dma16((NB == 2 && g * ROWS_PER_LD >= BN) ? src.b1 : src.b0, sb + g * 1024, b_off[j], ko);
    }
  };
  using frag_a_t = i32x4_t[FML > 0 ? FML : 1];
  using frag_b_t = i32x4_t[NB][FN];
  auto read_frags = [&](int kt, int step, frag_a_t& af, frag_b_t& bfr) __attribute__((always_inline)) {
    const char* sa = sa0 + (kt % NSA) * ASLOT;
    const char* sb = sb0 + (kt % NSB) * BSLOT;
    const int c = step * 2 + frag_c;
#pragma unroll
    for (int fm = 0; fm < FML; ++fm)
      af[fm] = *reinterpret_cast<const i32x4_t*>(sa + swz<kRB>(tile_row<WM>(wm, fm) + frag_row, c));
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        bfr[h][fn] = *reinterpret_cast<const i32x4_t*>(sb + swz<kRB>(h * BN + wn * WTN + fn * 32 + frag_row, c));
  };
  auto mfmas = [&](const frag_a_t& af, const frag_b_t& bfr) __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FML; ++fm)
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
          acc[h][fm][fn] = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[fm], bfr[h][fn], acc[h][fm][fn], 0, 0, 0);
  };
  constexpr int NMF = FML * NB * FN;
  constexpr int NRD = FML + NB * FN;
  // one fragment read under each MFMA; after the barrier also the stage's loads
  auto interleave = [&](bool loads) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NMF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < NRD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (loads && i < AI + BI) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };

  // Loads that may still be in flight once A(s) and B(s) have landed are those
  // issued after A(s): B(s - NSA + NSB) at the same barrier (unless NSB == NSA,
  // when that is B(s)), and all of the NSA - 1 (prologue) or NSA - 2 (loop)
  // later barriers.
  constexpr int VM_AFTER = NSB > NSA ? BI : 0;
  constexpr int VM_FIRST = VM_AFTER + (NSA - 1) * (AI + BI);
  constexpr int VM_STAGE = VM_AFTER + (NSA - 2) * (AI + BI);
  static_assert(VM_FIRST < 64, "vmcnt range");
#pragma unroll
  for (int v = -NSB; v < 0; ++v) {
    if (v + NSA >= 0) issue_a(v + NSA);
    issue_b(v + NSB);
  }
  asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(VM_FIRST, 15)) : "memory");  // A(0), B(0) landed
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  frag_a_t af[2];
  frag_b_t bf[2];
  if constexpr (FML > 0) read_frags(0, 0, af[0], bf[0]);
  auto step = [&](int kt, auto loads) __attribute__((always_inline)) {
    constexpr bool kLoads = decltype(loads)::value;
    if constexpr (FML > 0) {
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) {
        read_frags(kt, ks + 1, af[(ks + 1) & 1], bf[(ks + 1) & 1]);
        mfmas(af[ks & 1], bf[ks & 1]);
        interleave(false);
      }
    }
    // A(kt+1) and B(kt+1) have landed and this wave's reads of stage kt are
    // done, before any wave refills a slot (in the tail by draining the counter)
    if constexpr (kLoads)
      asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(VM_STAGE, 0)) : "memory");
    else
      asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(0, 0)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (kLoads) {
      issue_a(kt + NSA);
      issue_b(kt + NSB);
    } else if constexpr (NSB > NSA) {
      if (kt + NSA < nk) issue_a(kt + NSA);  // a stage still to come (uniform branch)
    }
    if constexpr (FML > 0) {
      // past the last stage this reads a slot whose data is not used
      read_frags(kt + 1, 0, af[0], bf[0]);
      mfmas(af[1], bf[1]);
      interleave(kLoads);
    }
  };
  int kt = 0;
  for (; kt < nk - NSB; ++kt) step(kt, std::true_type{});
  for (; kt < nk; ++kt) step(kt, std::false_type{});
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may still target LDS when the workgroup ends
}

// One work item (row tile, N block): its K loop and its epilogue.  The
// workgroup's LDS is free on entry and on return.
template <int BM, int BN, int WM, int WN, int NSA, int NSB, int EPI>
__device__ __forceinline__ void gemm_i8_item(const I8GemmArgs& args, int w, int n_blocks, int dense_tiles, char* smem,
                                             int wave0) {
  constexpr int NB = (EPI == kEpiSwiGLU) ? 2 : 1;
  constexpr int BROWS = NB * BN;
  constexpr int WTN = BN / WN, NW = WM * WN;
  constexpr int FM = BM / WM / 32, FN = WTN / 32;
  constexpr int ROWS_PER_LD = 1024 / kRB;
  constexpr int AI = BM / (NW * ROWS_PER_LD), BI = BROWS / (NW * ROWS_PER_LD);
  static_assert(FM >= 1 && FM <= 5 && FN >= 1, "tile shape");

  constexpr bool kItemLoop = EPI == kEpiBF16;  // resident workgroups walk several items
  const int tid = kItemLoop ? item_thread_index(wave0) : static_cast<int>(threadIdx.x);
  const int lane = tid & (kWave - 1), wave = kItemLoop ? wave0 : __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;

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
  static_assert(BM <= 64 * NW, "one row scale per thread");
  const float my_scale = tid < BM ? args.As[i8_a_row(args, p0 + (tid < nrows ? tid : nrows - 1))] : 0.f;
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
  int fm_live = ((nrows + 31) / 32 - wm + WM - 1) / WM;
  fm_live = fm_live < 0 ? 0 : (fm_live > FM ? FM : fm_live);
  const int nk = K / kRB;
  switch (fm_live) {
#define MOE_CASE(n)                                                                                                \
  case n:                                                                                                          \
    if constexpr (n <= FM)                                                                                         \
      k_loop_i8<BM, BN, WM, WN, NSA, NSB, NB, n, FM, FN, AI, BI>(smem, src, a_off, b_off, b_stage, nk, nrows, tid,   \
                                                                 wm, wn, acc);                                     \
    break;
    MOE_CASE(0)
    MOE_CASE(1)
    MOE_CASE(2)
    MOE_CASE(3)
    MOE_CASE(4)
    MOE_CASE(5)
#undef MOE_CASE
    default:
      break;
  }

  // ---- epilogue: scales, then rows leave through LDS in 16-byte pieces ----
  // The MFMA layout gives lane l column l % 32 of rows 8*(r/4) + 4*(l/32) +
  // r%4 of each 32 x 32 block.  The tile (or a band of it) is written to LDS
  // row by row, then copied out by all threads.
  constexpr int ESZ = EPI == kEpiBF16 ? 2 : 4;
  constexpr int CS = BN * ESZ + 16;                  // LDS row stride (padded against bank conflicts)
  constexpr int SCALE_AT = ring_bytes(BM, BROWS, NSA, NSB) - BM * 4;  // row scales, past the staged band
  constexpr int FMP_FIT = SCALE_AT / CS / (WM * 32);
  constexpr int FMP = FMP_FIT < FM ? FMP_FIT : FM;   // 32-row blocks per row group and band
  constexpr int NBANDS = (FM + FMP - 1) / FMP;
  static_assert(FMP >= 1, "epilogue bands");
  constexpr int BAND = FMP * WM * 32;
  constexpr int CPR = BN * ESZ / 16, EPC = 16 / ESZ;  // chunks per row, elements per chunk
  // In pass `it` of a band, wave w stores rows it * RSTEP + w * RPI + lane /
  // CPR.  Each row's output row is found once, before any store, and passed
  // on by a cross-lane read (a table load among the stores waits for them).
  constexpr int RPI = 64 / CPR, RSTEP = RPI * NW;
  static_assert(64 % CPR == 0 && BAND % RSTEP == 0, "copy-out mapping");
  int row_entry = -1;
  {
    const int r = (lane / RPI) * RSTEP + wave * RPI + lane % RPI;
    if (r < nrows) row_entry = static_cast<int>(i8_c_row(args, p0 + r));
  }
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
  float* row_s = reinterpret_cast<float*>(smem + SCALE_AT);
  if (tid < BM) row_s[tid] = my_scale;
  __syncthreads();
  const bool whole = args.N % EPC == 0 && args.ldc % EPC == 0;
#pragma unroll
  for (int band = 0; band < NBANDS; ++band) {
    if (band > 0 && band * BAND >= nrows) break;  // workgroup-uniform
#pragma unroll
    for (int fm = band * FMP; fm < (band + 1) * FMP && fm < FM; ++fm) {
      if (fm >= fm_live) continue;  // wave-uniform
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int row0 = tile_row<WM>(wm, fm) + r4 * 8 + (lane >> 5) * 4;
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row_s + row0);
        char* to = smem + (row0 - band * BAND) * CS;
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
          const int col_l = wn * WTN + fn * 32 + (lane & 31);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = static_cast<float>(acc[0][fm][fn][r4 * 4 + i]) * s[i] * sb[0][fn];
            if constexpr (EPI == kEpiSwiGLU)
              v = silu_mul(v, static_cast<float>(acc[NB - 1][fm][fn][r4 * 4 + i]) * s[i] * sb[NB - 1][fn]);
            if constexpr (ESZ == 4)
              *reinterpret_cast<float*>(to + i * CS + col_l * 4) = v;
            else
              *reinterpret_cast<uint16_t*>(to + i * CS + col_l * 2) = f32_to_bf16(v);
          }
        }
      }
    }
    __syncthreads();
    const int band_rows = min(BAND, nrows - band * BAND);
    for (int it = 0; it * RSTEP < band_rows; ++it) {
      const int row_b = it * RSTEP + wave * RPI + lane / CPR, ch = lane % CPR;
      const int crow = __shfl(row_entry, (band * BAND / RSTEP + it) * RPI + lane / CPR);
      const int col = n0 + ch * EPC;
      if (row_b >= band_rows || col >= args.N || crow < 0) continue;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + row_b * CS + ch * 16);
      char* dst = static_cast<char*>(args.C) + (static_cast<int64_t>(crow) * args.ldc + col) * ESZ;
      if (whole) {
        // bf16 rows are next read long after they leave the caches
        if constexpr (ESZ == 2)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(dst));
        else
          *reinterpret_cast<u32x4_t*>(dst) = v;
      } else {
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          if (col + i >= args.N) continue;
          if constexpr (ESZ == 4)
            reinterpret_cast<uint32_t*>(dst)[i] = v[i];
          else
            reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)));
        }
      }
    }
    if (band + 1 < NBANDS) __syncthreads();  // the next band reuses the LDS
  }
}

// Work items are cut into 8 contiguous runs, one per XCD, as in the bf16 and
// MXFP8 kernels: workgroup b takes item b / 8 of the run of XCD b mod 8, and
// the bf16 epilogue's resident workgroups walk their run side by side, so that
// one item's output stores drain under the next one's first loads.
template <int BM, int BN, int WM, int WN, int NSA, int NSB, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_kernel(const I8GemmArgs args, int dense_tiles) {
  constexpr int NB = (EPI == kEpiSwiGLU) ? 2 : 1;
  __shared__ __attribute__((aligned(1024))) char smem[ring_bytes(BM, NB * BN, NSA, NSB)];
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
    if (first < len) gemm_i8_item<BM, BN, WM, WN, NSA, NSB, EPI>(args, run0 + first, n_blocks, dense_tiles, smem, wave0);
  } else {
    for (int local = first; local < len; local += per_xcd) {
      if (local > first) __syncthreads();  // the previous item's copy-out has read the LDS
      gemm_i8_item<BM, BN, WM, WN, NSA, NSB, EPI>(args, __builtin_amdgcn_readfirstlane(run0 + local), n_blocks, dense_tiles,
                                        smem, wave0);
    }
  }
}

template <int BM, int BN, int WM, int WN, int NSA, int NSB, int EPI>
hipError_t run_i8(const I8GemmArgs& a, hipStream_t stream) {
  const int64_t n_blocks = (a.N + BN - 1) / BN;
  const int64_t dense_tiles = a.tiles ? 0 : (static_cast<int64_t>(a.dense_rows) + BM - 1) / BM;
  const int64_t work = (a.tiles ? a.max_tiles : dense_tiles) * n_blocks;
  if (work <= 0) return hipSuccess;
  if (work > 0x7ffffff0) return hipErrorInvalidValue;
  auto kernel = gemm_i8_kernel<BM, BN, WM, WN, NSA, NSB, EPI>;
  // with room for balanced runs of up to tile_run_cap tiles on every XCD
  int64_t cap = a.tiles ? int64_t(kXcds) * tile_run_cap(a.max_tiles) * n_blocks : work;
  if (EPI == kEpiBF16) {
    static std::atomic<int64_t> resident_cache{0};
    int64_t resident = resident_cache.load(std::memory_order_relaxed);
    if (resident <= 0) {
      resident = resident_workgroups(reinterpret_cast<const void*>(kernel), 64 * WM * WN);
      if (resident <= 0) return hipErrorInvalidValue;
      resident_cache.store(resident, std::memory_order_relaxed);
    }
    cap = std::min(work, resident);
  }
  const int64_t grid = (cap + kXcds - 1) / kXcds * kXcds;
  kernel<<<static_cast<unsigned>(grid), 64 * WM * WN, 0, stream>>>(a, static_cast<int>(dense_tiles));
  return hipGetLastError();
}

// 320- and 256-row tiles: 8 waves, two per SIMD, 64 x 128 or 160 x 64 outputs
// a wave.  128- and 64-row tiles: fewer outputs a workgroup, two workgroups or
// more per CU.
template <int EPI>
hipError_t run_height(const I8GemmArgs& a, hipStream_t stream) {
  constexpr int kHalf = EPI == kEpiSwiGLU ? 2 : 1;  // SwiGLU: gate and up share the columns of a tile
  switch (a.tile_rows) {
    case 320:
      return run_i8<320, 256 / kHalf, 2, 4, 2, 2, EPI>(a, stream);
    case 256:
      return run_i8<256, 256 / kHalf, 4, 2, 2, 3, EPI>(a, stream);
    case 128:
      return run_i8<128, 128 / kHalf, 4, 2, 2, 3, EPI>(a, stream);
    case 64:
      // dense tiles half as wide while they still get a CU each: a CU's load
      // path is the bound, and more CUs take part (777 x 1001 x 1536: 10.2 us
      // against 11.8; 512 x 2048 x 7168: 26.9 against 31.2)
      if constexpr (EPI != kEpiSwiGLU)
        if (!a.tiles && ((a.dense_rows + 63) / 64) * ((a.N + 63) / 64) <= device_compute_units())
          return run_i8<64, 64, 2, 2, 2, 3, EPI>(a, stream);
      return run_i8<64, 128 / kHalf, 2, 2, 2, 3, EPI>(a, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace

// Heights for `rows` rows spread over `groups` weight matrices of N rows.
//
// Routed, measured for whole layers (D x I, experts): up to 4 rows an expert
// the few-rows kernel (7168 x 2048, 256 experts, 64 tokens: 1.68 ms against
// 1.66 with 64-row tiles; 4 tokens: 0.30 against 0.34), up to 48 rows 64-row
// tiles (512 tokens: 2.04 ms against 2.07 with 128 and 2.41 with the few-rows
// kernel).  From 192 rows on 320-row tiles, whose waves read the fewest bytes
// per product, where their items make two rounds over the chip (8192 tokens:
// 4.23 ms against 4.68 with 256 and 5.18 with 128; 1024 x 1024, 32 experts, 512
// rows each: 187 us against 206 and 196); between, 256-row tiles if their items
// make five rounds (2048 tokens: 2.40 ms against 2.47 with 128 and 2.63 with
// 320), else 128-row tiles, which fill the last round better (2048 x 768, 128
// experts, 128 rows each: 307 us against 332 with 256; 1024 x 1024, 32 experts,
// 256 rows each: 134 us against 145 with 320).
//
// Dense: the few-rows kernel while its workgroups fit the chip at once (256 x
// 2048 x 7168: 24 us against 32 with 64-row tiles), else the least rounds times
// the measured cost of a round (us per 128-byte stage: 64-row tiles 0.94 with
// two workgroups on every CU and 0.57 with one, 128-row tiles 1.49 and 0.80,
// 256-row 1.85, 320-row 2.2).
int i8_tile_rows(int64_t rows, int64_t groups, int64_t N) {
  const int64_t known = device_compute_units(), cus = known > 0 ? known : 256;
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (groups > 1) {
    if (rows <= 4 * groups) return kI8RowsBM;
    if (rows <= 48 * groups) return 64;
    const auto items = [&](int bm) { return groups * ceil_div(rows, bm * groups) * ceil_div(N, 128); };
    if (rows >= 192 * groups) return items(320) >= 2 * cus ? 320 : 128;
    return items(256) >= 5 * cus ? 256 : 128;
  }
  if (ceil_div(rows, kI8RowsBM) * ceil_div(N, 64) <= cus) return kI8RowsBM;
  int best = 0;
  double least = 0.0;
  auto consider = [&](int bm, int bn, int per_cu, double one, double full) {
    const int64_t items = ceil_div(rows, bm) * ceil_div(N, bn);
    const double cost = items <= cus ? one : static_cast<double>(ceil_div(items, per_cu * cus)) * full;
    if (!best || cost < least) {
      best = bm;
      least = cost;
    }
  };
  consider(64, 128, 2, 0.57, 0.94);
  consider(128, 128, 2, 0.80, 1.49);
  consider(256, 256, 1, 1.85, 1.85);
  consider(320, 256, 1, 2.2, 2.2);
  return best;
}

hipError_t launch_gemm_i8_tiles(const I8GemmArgs& a, int epilogue, hipStream_t stream) {
  if (a.tiles && !a.tile_runs) return hipErrorInvalidValue;
  switch (epilogue) {
    case kEpiSwiGLU:
      return run_height<kEpiSwiGLU>(a, stream);
    case kEpiBF16:
      return run_height<kEpiBF16>(a, stream);
    case kEpiF32:
      return run_height<kEpiF32>(a, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace moe
