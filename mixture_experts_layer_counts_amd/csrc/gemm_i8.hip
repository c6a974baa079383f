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
// The scales are applied once, to the int32 sums.  Epilogues: SwiGLU in fp32 (h
// is quantised when its whole row is known), bf16 scattered to the rows'
// routes, and fp32.
//
// A workgroup's next item begins under its epilogue: the first loads are issued
// before the stores, and the next K loop's first waits count the stores behind
// them.  In the bf16 kernels these drain under that loop's first stages, which
// took the down product of the 7168 x 2048 layer at 8192 tokens from 1.36 to
// 1.30 ms and an 8192 x 7168 x 2048 product from 140 to 134 us; the one
// workgroup on a CU otherwise wrote 160 KB with no load in flight.  In the fp32
// and SwiGLU kernels the loads are only issued early: before each 8-row piece
// the compiler waits for every memory operation (it takes the LDS that the
// direct loads write for what the piece reads of row_out), so the loads have
// landed and the stores have drained before the K loop begins.
//
// The 320-row kernels spill 8 to 11 vector registers (36 to 48 bytes of scratch
// a lane); the others spill none.

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

// Row of the tile held by 32-row block fm of a wave in row group wm: blocks
// are dealt to the row groups in turn, so a partly filled tile keeps every
// wave busy.
template <int WM>
__device__ __forceinline__ int tile_row(int wm, int fm) {
  return (fm * WM + wm) * 32;
}

// One item's operands as this lane fetches them.
template <int AI, int BI>
struct I8Stream {
  __amdgpu_buffer_rsrc_t a, b0, b1;
  uint32_t a_off[AI], b_off[BI];  // byte offsets of the 16-byte chunks of stage 0
  int b_stage;                    // bytes from one stage of a weight row to the next
  int nk, a_rows;
};

// The loads of stage kt into its ring slots (lane l's 16 bytes land at base +
// 16 l).  A stage past the last (in the prologue of a short K) loads the last
// one again, into a free slot, so that the prologue issues the same number of
// loads; row groups past the tile reload the first one for the same reason.
template <int BM, int NSA, int AI, int BI>
__device__ __forceinline__ void issue_a(char* smem, const I8Stream<AI, BI>& s, int wave, int kt) {
  constexpr int ROWS_PER_LD = 1024 / kRB;
  const int ko = (kt < s.nk ? kt : s.nk - 1) * kRB;
  char* sa = smem + (kt % NSA) * (BM * kRB);
#pragma unroll
  for (int j = 0; j < AI; ++j)
    dma16(s.a, sa + (wave * AI + j) * 1024, (wave * AI + j) * ROWS_PER_LD < s.a_rows ? s.a_off[j] : s.a_off[0], ko);
}
template <int BM, int BN, int NB, int NSA, int NSB, int AI, int BI>
__device__ __forceinline__ void issue_b(char* smem, const I8Stream<AI, BI>& s, int wave, int kt) {
  constexpr int ROWS_PER_LD = 1024 / kRB;
  const int ko = (kt < s.nk ? kt : s.nk - 1) * s.b_stage;
  char* sb = smem + NSA * BM * kRB + (kt % NSB) * (NB * BN * kRB);
#pragma unroll
  for (int j = 0; j < BI; ++j) {
    const int g = wave * BI + j;
    dma16((NB == 2 && g * ROWS_PER_LD >= BN) ? s.b1 : s.b0, sb + g * 1024, s.b_off[j], ko);
  }
}

// Wait until at most N vector memory operations are outstanding, plus what a
// previous epilogue's `stores` (issued after every load waited for) may be:
// rounded down to one of a few counts.
template <int N, int FULL>
__device__ __forceinline__ void wait_behind(int stores) {
  constexpr int kFull = N + FULL < 63 ? N + FULL : 63, kHalf = N + FULL / 2 < 63 ? N + FULL / 2 : 63;
  if (stores >= FULL)
    asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(kFull, 0)) : "memory");
  else if (stores >= FULL / 2)
    asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(kHalf, 0)) : "memory");
  else
    asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(N, 0)) : "memory");
}

// The K loop of one workgroup, the bf16 kernels' protocol: a slot is refilled
// right after the barrier that ends its stage's reads, the fragments of the
// next 32-wide sub-step are read under the current MFMAs, and one barrier per
// stage waits for the next stage's rows.  The first stages' loads are in flight
// on entry, behind them `stores` stores of the previous item; the ring is free
// on return.  FML of the wave's FM row blocks hold tile rows.
template <int BM, int BN, int WM, int WN, int NSA, int NSB, int NB, int FML, int FM, int FN, int STORES, int AI, int BI>
__device__ __forceinline__ void k_loop_i8(char* smem, const I8Stream<AI, BI>& src, int stores, int wave, int lane,
                                          int wm, int wn, i32x16_t (&acc)[NB][FM][FN]) {
  constexpr int BROWS = NB * BN, WTN = BN / WN;
  static_assert(NSA >= 2 && NSB >= NSA, "ring depths");
  constexpr int ASLOT = BM * kRB, BSLOT = BROWS * kRB;
  constexpr int KS = 4;  // 32-wide sub-steps per stage
  char* const sa0 = smem;
  char* const sb0 = smem + NSA * ASLOT;
  const int frag_row = lane & 31, frag_c = lane >> 5;
  const int nk = src.nk;

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
  // A(0), B(0) and the tables in LDS have landed
  wait_behind<VM_FIRST, STORES>(stores);
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
    // done, before any wave refills a slot (in the tail by draining the counter;
    // the stages of the prologue landed before the stores behind them)
    if constexpr (kLoads) {
      if (kt == 0)
        wait_behind<VM_STAGE, STORES>(stores);
      else
        asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(VM_STAGE, 0)) : "memory");
    } else {
      asm volatile("s_waitcnt %0" ::"n"(waitcnt_imm(0, 0)) : "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (kLoads) {
      issue_a<BM, NSA>(smem, src, wave, kt + NSA);
      issue_b<BM, BN, NB, NSA, NSB>(smem, src, wave, kt + NSB);
    } else if constexpr (NSB > NSA) {
      if (kt + NSA < nk) issue_a<BM, NSA>(smem, src, wave, kt + NSA);  // a stage still to come (uniform branch)
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
}

// Who walks which item of a tile list.  The items are cut into 8 contiguous runs,
// one per XCD (neighbours share operands in its L2).  Tiles of about equal rows
// give equal runs, walked in fixed strides: runs balanced by cost there differ by
// a few items, and one that is two items longer than a whole number of rounds
// costs the chip a round (2048 x 768, 128 experts, 4096 tokens: 438 us against
// 404; 7168 x 2048, 256 experts, 4096 tokens: 2.82 ms against 2.68).  Under skewed
// routing the runs balance cost, and the items past the first round are handed
// out as the workgroups get to them: from the XCD's own queue, and when that run
// is used up from the longest rest of another's (Zipf(1.2) routes, 7168 x 2048,
// 256 experts: 4.65 -> 4.38 ms at 8192 tokens and 1.66 -> 1.56 at 2048; 4096 x
// 1408, 96 experts: 1.61 -> 1.52 at 8192).  A draw is made an item ahead, so its
// trip to memory is hidden; drawn when needed, small layers took 10 us more.
__device__ __forceinline__ int draw(int32_t* queue, int xcd) {
  return __hip_atomic_fetch_add(queue + xcd * kQueueStride, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Item at which the run of XCD j (at most kXcds: the end) starts, balanced by
// the tiles' cost.
__device__ __forceinline__ int run_start(const int32_t* __restrict__ runs, int n_blocks, int j) {
  return static_cast<int>(static_cast<int64_t>(runs[j]) * n_blocks / kTileRunFrac);
}

// An item of another XCD's run, or -1 if all are handed out.  Queues only grow,
// so a draw that fails shows its run to be used up: at most 8 passes.
__device__ __forceinline__ int steal(int32_t* queue, const int32_t* __restrict__ runs, int n_blocks, int per_xcd) {
  const int lane = lane_id(), j = lane < kXcds ? lane : 0;
  const int first = run_start(runs, n_blocks, j), len = run_start(runs, n_blocks, j + 1) - first;
  for (;;) {
    const int left =
        len - per_xcd - __hip_atomic_load(queue + j * kQueueStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    int best = left > 0 ? left * kXcds + j : -1;
#pragma unroll
    for (int d = 1; d < kXcds; d *= 2) best = max(best, __shfl_xor(best, d));
    best = __builtin_amdgcn_readfirstlane(best);
    if (best < 0) return -1;
    const int from = best % kXcds;
    int drawn = 0;
    if (lane == 0) drawn = draw(queue, from);
    drawn = __builtin_amdgcn_readfirstlane(drawn);
    if (drawn < __builtin_amdgcn_readlane(len, from) - per_xcd)
      return __builtin_amdgcn_readlane(first, from) + per_xcd + drawn;
  }
}

// What the epilogue needs of an item beside its sums: the scales of its rows
// and columns and the output rows, kept in LDS past the rings, twice (the next
// item's are filled in before this one's epilogue).
template <int BM, int BROWS>
struct I8Tables {
  float row_scale[BM];
  int row_out[BM];  // output row, or -1
  float col_scale[BROWS];
};

// Resident workgroups walk items.  An item's first loads are issued before the
// previous item's epilogue, which needs nothing of the rings: fp32 rows go
// straight from the registers (32 lanes hold 128 consecutive bytes), bf16 rows
// through 8-row pieces that each wave stages for itself.
template <int BM, int BN, int WM, int WN, int NSA, int NSB, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_kernel(const I8GemmArgs args, int dense_tiles) {
  constexpr int NB = (EPI == kEpiSwiGLU) ? 2 : 1;
  constexpr int BROWS = NB * BN;
  constexpr int WTN = BN / WN, NW = WM * WN;
  constexpr int FM = BM / WM / 32, FN = WTN / 32;
  constexpr int ROWS_PER_LD = 1024 / kRB;
  constexpr int AI = BM / (NW * ROWS_PER_LD), BI = BROWS / (NW * ROWS_PER_LD);
  static_assert(FM >= 1 && FM <= 5 && FN >= 1, "tile shape");
  static_assert(AI * ROWS_PER_LD * NW == BM && BI * ROWS_PER_LD * NW == BROWS, "loads per wave per stage");
  static_assert(BM <= 64 * NW && BROWS <= 64 * NW, "one table entry per thread");
  // bf16 pieces: 8 rows of the wave's WTN columns, padded against bank conflicts
  constexpr int PS = WTN * 2 + 16, PIECE = EPI == kEpiBF16 ? 8 * PS : 0;
  constexpr int CPR = WTN * 2 / 16;                // 16-byte chunks per bf16 row
  constexpr int PIECE_STORES = EPI == kEpiBF16 ? (8 * CPR + 63) / 64 : 4 * FN;  // stores per 8-row piece
  constexpr int STORES = FM * 4 * PIECE_STORES;    // of a whole tile
  constexpr int RING = ring_bytes(BM, BROWS, NSA, NSB);
  using Tables = I8Tables<BM, BROWS>;
  // the next item goes into the padding behind the last piece's last row
  constexpr int NEXT = RING + 2 * sizeof(Tables) + (PIECE ? NW * PIECE - 16 : 0);
  __shared__ __attribute__((aligned(1024))) char smem[NEXT + 16];
  Tables* const tables = reinterpret_cast<Tables*>(smem + RING);
  int* const next_s = reinterpret_cast<int*>(smem + NEXT);

  const int n_blocks = (args.N + BN - 1) / BN;
  const int xcd = static_cast<int>(blockIdx.x) % kXcds;
  // the run of XCD b mod 8, where workgroup b starts with item b / 8.  Walked in
  // strides of the XCD's workgroups, or with `queued` drawn, when the runs
  // balanced by cost start further than half a round or a sixteenth of a run from
  // equal ones.
  const int per_xcd = static_cast<int>(gridDim.x) / kXcds;  // the grid is a multiple of kXcds
  bool queued = false;
  int run0, len;
  if (args.tiles) {
    const int lane = lane_id(), j = lane < kXcds ? lane : kXcds;
    const int start = run_start(args.tile_runs, n_blocks, j);
    const int items = __builtin_amdgcn_readlane(start, kXcds), share = (items + kXcds - 1) / kXcds;
    const int equal = j * share < items ? j * share : items;
    queued = __any(abs(start - equal) > max(per_xcd / 2, share / 16));
    run0 = __builtin_amdgcn_readlane(queued ? start : equal, xcd);
    len = __builtin_amdgcn_readlane(queued ? start : equal, xcd + 1) - run0;
  } else {
    const int W = dense_tiles * n_blocks, chunk = (W + kXcds - 1) / kXcds;
    run0 = xcd * chunk;
    len = W - run0 < chunk ? W - run0 : chunk;
  }
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int wm = wave / WN, wn = wave % WN;
  int local = static_cast<int>(blockIdx.x) / kXcds;
  // wave 0 draws, the others read it from LDS: an item, or -1
  auto publish = [&](int drawn) __attribute__((always_inline)) {  // drawn: from its own queue
    if (wave == 0) {
      const int ticket = per_xcd + __builtin_amdgcn_readfirstlane(drawn);
      *next_s = ticket < len ? run0 + ticket : steal(args.queue, args.tile_runs, n_blocks, per_xcd);
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*next_s);
  };
  int item = run0 + local, drawn = 0;
  if (local >= len) {
    if (!queued) return;
    item = publish(len);
    if (item < 0) return;
  }

  I8Stream<AI, BI> src;
  src.nk = args.K / kRB;
  src.b_stage = args.b_plane ? static_cast<int>(args.b_plane * kRB) : kRB;
  constexpr int kRsrcWord3 = 0x00020000;
  src.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(args.A), 0, static_cast<int>(args.a_rows * args.K),
                                            kRsrcWord3);

  // Item `w`: its place, its tables into buffer `buf`, its addresses, and the
  // loads of its first stages.
  int nrows, n0;
  auto begin = [&](int w, int buf) __attribute__((always_inline)) {
    const int tid = item_thread_index(wave), lane = tid & (kWave - 1);
    const int K = args.K;
    int e = 0, nb, lt;
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
      const int left = args.dense_rows - static_cast<int>(p0);
      nrows = left < h ? left : h;  // at least 1: (dense_tiles - 1) h < dense_rows
    }
    n0 = nb * BN;
    // ---- byte offsets of the 16-byte chunks this lane fetches; rows past the
    // tile are clamped onto its last row and rows past N onto row N - 1: their
    // products only reach outputs that are dropped ----
    constexpr int CH = kRB / 16;
#pragma unroll
    for (int j = 0; j < AI; ++j) {
      const int row = ROWS_PER_LD * (wave * AI + j) + lane / CH;
      const int c = (lane % CH) ^ ((row / (256 / kRB)) & (CH - 1));
      src.a_off[j] = static_cast<uint32_t>(i8_a_row(args, p0 + (row < nrows ? row : nrows - 1)) * K + c * 16);
    }
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      const int row = ROWS_PER_LD * (wave * BI + j) + lane / CH;
      const int c = (lane % CH) ^ ((row / (256 / kRB)) & (CH - 1));
      const int half = row / BN;
      int n = n0 + (row - half * BN);
      n = n < args.N ? n : args.N - 1;
      src.b_off[j] = static_cast<uint32_t>(args.b_plane ? n * kRB + c * 16 : n * K + c * 16);
    }
    src.a_rows = nrows;
    const int b_bytes = args.N * K;
    src.b0 = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(args.B0 + static_cast<int64_t>(e) * b_bytes), 0,
                                               b_bytes, kRsrcWord3);
    src.b1 = NB == 2 ? __builtin_amdgcn_make_buffer_rsrc(
                           const_cast<int8_t*>(args.B1 + static_cast<int64_t>(e) * b_bytes), 0, b_bytes, kRsrcWord3)
                     : src.b0;
    // the tables: read before the stage loads, so that these stay in flight
    float rs = 0.f, cs = 0.f;
    int ro = -1;
    if (tid < BM) {
      rs = args.As[i8_a_row(args, p0 + (tid < nrows ? tid : nrows - 1))];
      if (tid < nrows) ro = static_cast<int>(i8_c_row(args, p0 + tid));
    }
    if (tid < BROWS) {
      const int half = tid / BN;
      int n = n0 + tid - half * BN;
      n = n < args.N ? n : args.N - 1;
      cs = (half ? args.Bs1 : args.Bs0)[static_cast<int64_t>(e) * args.N + n];
    }
#pragma unroll
    for (int v = -NSB; v < 0; ++v) {
      if (v + NSA >= 0) issue_a<BM, NSA>(smem, src, wave, v + NSA);
      issue_b<BM, BN, NB, NSA, NSB>(smem, src, wave, v + NSB);
    }
    if (tid < BM) {
      tables[buf].row_scale[tid] = rs;
      tables[buf].row_out[tid] = ro;
    }
    if (tid < BROWS) tables[buf].col_scale[tid] = cs;
  };

  // (the draw for the item after this one is on its way ahead of the loads)
  if (queued && threadIdx.x == 0) drawn = draw(args.queue, xcd);
  begin(item, 0);
  int stores = 0;  // issued by the last epilogue, at least
  for (int turn = 0;; ++turn) {
    // 32-row blocks of this wave that hold tile rows (wave-uniform)
    int fm_live = ((nrows + 31) / 32 - wm + WM - 1) / WM;
    fm_live = fm_live < 0 ? 0 : (fm_live > FM ? FM : fm_live);
    i32x16_t acc[NB][FM][FN];
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) acc[h][fm][fn] = i32x16_t{};
    {
      const int lane = item_thread_index(wave) & (kWave - 1);
      switch (fm_live) {
#define MOE_CASE(n)                                                                                                \
  case n:                                                                                                          \
    if constexpr (n <= FM)                                                                                         \
      k_loop_i8<BM, BN, WM, WN, NSA, NSB, NB, n, FM, FN, STORES, AI, BI>(smem, src, stores, wave, lane, wm, wn, acc); \
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
    }
    const int col0 = n0 + wn * WTN, buf = turn & 1, rows = nrows;
    bool more;
    if (queued) {
      item = publish(drawn);
      more = item >= 0;
      if (more && threadIdx.x == 0) drawn = draw(args.queue, xcd);
    } else {
      local += per_xcd;
      more = local < len;
      item = __builtin_amdgcn_readfirstlane(run0 + local);
    }
    if (more) begin(item, buf ^ 1);

    // ---- epilogue.  The MFMA layout gives lane l column l % 32 of rows 8*(r/4)
    // + 4*(l/32) + r%4 of each 32 x 32 block. ----
    const int lane = item_thread_index(wave) & (kWave - 1);
    const Tables& t = tables[buf];
    const bool whole = EPI != kEpiBF16 || (args.N % 8 == 0 && args.ldc % 8 == 0);
    // A store that no lane has a row for (past the tile's last one, or with a
    // table's row out of range) is branched round, so each is counted where it is
    // issued: the next item's waits may let this many operations be outstanding
    // behind its loads, and one too many would pass before a load has landed.
    stores = 0;
    float sb[NB][FN];
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) sb[h][fn] = t.col_scale[h * BN + wn * WTN + fn * 32 + (lane & 31)];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      if (fm >= fm_live) continue;  // wave-uniform
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int row0 = tile_row<WM>(wm, fm) + r4 * 8;
        if (row0 >= rows) continue;  // wave-uniform
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(&t.row_scale[row0 + (lane >> 5) * 4]);
        if constexpr (EPI == kEpiBF16) {
          char* piece = smem + RING + 2 * sizeof(Tables) + wave * PIECE;
#pragma unroll
          for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint16_t*>(piece + ((lane >> 5) * 4 + i) * PS + (fn * 32 + (lane & 31)) * 2) =
                  f32_to_bf16(static_cast<float>(acc[0][fm][fn][r4 * 4 + i]) * s[i] * sb[0][fn]);
          // the wave's LDS instructions run in order; the compiler must keep them so
          asm volatile("" ::: "memory");
#pragma unroll
          for (int it = 0; it < PIECE_STORES; ++it) {
            const int q = it * 64 + lane, row = q / CPR % 8, ch = q % CPR;
            const int col = col0 + ch * 8, out = t.row_out[row0 + row];
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(piece + row * PS + ch * 16);
            const bool live = q < 8 * CPR && out >= 0 && col < args.N;
            stores += __ballot(live) ? 1 : 0;
            if (!live) continue;
            uint16_t* c = static_cast<uint16_t*>(args.C) + static_cast<int64_t>(out) * args.ldc + col;
            if (whole) {
              // next read long after they leave the caches
              __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(c));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (col + i < args.N) c[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2)));
            }
          }
          asm volatile("" ::: "memory");
        } else {
          const int4 out = *reinterpret_cast<const int4*>(&t.row_out[row0 + (lane >> 5) * 4]);
          const int outs[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool live = outs[i] >= 0;
            stores += __ballot(live) ? FN : 0;
            if (!live) continue;
            float* c = static_cast<float*>(args.C) + static_cast<int64_t>(outs[i]) * args.ldc + col0 + (lane & 31);
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) {
              float v = static_cast<float>(acc[0][fm][fn][r4 * 4 + i]) * s[i] * sb[0][fn];
              if constexpr (EPI == kEpiSwiGLU)
                v = silu_mul(v, static_cast<float>(acc[NB - 1][fm][fn][r4 * 4 + i]) * s[i] * sb[NB - 1][fn]);
              if (col0 + fn * 32 + (lane & 31) < args.N) c[fn * 32] = v;
            }
          }
        }
      }
    }
    if (!more) break;
    if (!whole || col0 + WTN > args.N) stores = 0;  // other stores than those counted
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may still target LDS when the workgroup ends
}

template <int BM, int BN, int WM, int WN, int NSA, int NSB, int EPI>
hipError_t run_i8(const I8GemmArgs& a, hipStream_t stream) {
  const int64_t n_blocks = (a.N + BN - 1) / BN;
  const int64_t dense_tiles = a.tiles ? 0 : (static_cast<int64_t>(a.dense_rows) + BM - 1) / BM;
  const int64_t work = (a.tiles ? a.max_tiles : dense_tiles) * n_blocks;
  if (work <= 0) return hipSuccess;
  if (work > 0x7ffffff0) return hipErrorInvalidValue;
  auto kernel = gemm_i8_kernel<BM, BN, WM, WN, NSA, NSB, EPI>;
  static std::atomic<int64_t> resident_cache{0};
  int64_t resident = resident_cache.load(std::memory_order_relaxed);
  if (resident <= 0) {
    resident = resident_workgroups(reinterpret_cast<const void*>(kernel), 64 * WM * WN);
    if (resident <= 0) return hipErrorInvalidValue;
    resident_cache.store(resident, std::memory_order_relaxed);
  }
  const int64_t cap = std::min(work, resident);
  const int64_t grid = (cap + kXcds - 1) / kXcds * kXcds;
  kernel<<<static_cast<unsigned>(grid), 64 * WM * WN, 0, stream>>>(a, static_cast<int>(dense_tiles));
  return hipGetLastError();
}

// 192- to 320-row tiles: 8 waves, two per SIMD, one workgroup on a CU; three
// slots of weight rows where LDS holds them beside the tables (256-row tiles
// lose 4% of a routed layer with two).  128- and 64-row tiles: fewer outputs a
// workgroup, two workgroups on a CU.  256 rows serve dense products only.
template <int EPI>
hipError_t run_height(const I8GemmArgs& a, hipStream_t stream) {
  constexpr int kHalf = EPI == kEpiSwiGLU ? 2 : 1;  // SwiGLU: gate and up share the columns of a tile
  switch (a.tile_rows) {
    case 320:
      return run_i8<320, 256 / kHalf, 2, 4, 2, 2, EPI>(a, stream);
    case 256:
      return run_i8<256, 256 / kHalf, 4, 2, 2, 2, EPI>(a, stream);
    case 192:
      return run_i8<192, 256 / kHalf, 2, 4, 2, 3, EPI>(a, stream);
    case 128:
      return run_i8<128, 128 / kHalf, 4, 2, 2, 2, EPI>(a, stream);
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

// Heights for `rows` rows spread over `groups` weight matrices of N rows (pair: N
// of gate and N of up).
//
// Routed, measured for whole layers: up to 4 rows an expert the few-rows kernel
// (7168 x 2048, 256 experts, 4 tokens: 0.27 ms against 0.34 with 64-row tiles).
// Where 192-row items make five rounds over the chip, the weights' stream is
// the bound and a third slot of it is what counts: 192 rows (7168 x 2048, 256
// experts, 512 tokens: 1.98 ms against 2.07 with 64 and 2.24 with 320; 4096
// tokens: 2.68 against 3.25 with 128 and 2.93 with 320), from 96 rows an expert on
// with three rounds too (2048 x 768, 128 experts, 128 rows each: 288 us against
// 300 with 128; 64 rows each 240 against 231).  320 rows from 192 an expert on,
// where segments would often need two (7168 x 2048, 8192 tokens: 4.10 ms against
// 5.12 with 192), given three rounds (2048 x 768, 256 rows each: 405 us against
// 430 with 192).  With fewer rounds small tiles fill the last one better: 64
// rows up to 48 an expert, then 128 (1024 x 1024, 32 experts, 375 rows each: 155
// us against 164 with 320 and 177 with 192).
//
// Dense: the few-rows kernel while its workgroups fit the chip at once (256 x
// 2048 x 7168: 24.7 us against 26.2 with 64-row tiles), else the least rounds
// times the measured cost of a round (us per 128-byte stage: 64-row tiles 0.85
// with two workgroups on every CU and 0.56 with one, 128-row tiles 1.35 and
// 0.87, 256-row 1.95, 320-row 2.4).
int i8_tile_rows(int64_t rows, int64_t groups, int64_t N, bool pair) {
  const int64_t known = device_compute_units(), cus = known > 0 ? known : 256;
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (groups > 1) {
    if (rows <= 4 * groups) return kI8RowsBM;
    const auto items = [&](int bm) { return groups * ceil_div(rows, bm * groups) * ceil_div(N, 128); };
    if (rows >= 192 * groups) return items(320) >= 3 * cus ? 320 : 128;
    if (items(192) >= (rows >= 96 * groups ? 3 : 5) * cus) return 192;
    return rows <= 48 * groups ? 64 : 128;
  }
  if (ceil_div(rows, kI8RowsBM) * ceil_div(N, 64) <= cus) return kI8RowsBM;
  // a tile of SwiGLU holds gate and up side by side (counted as N columns, a 7168
  // x 2048 shared expert and a small routed one at 4096 tokens took 445 us for 418)
  const int64_t cols = pair ? 2 * N : N;
  int best = 0;
  double least = 0.0;
  auto consider = [&](int bm, int bn, int per_cu, double one, double full) {
    const int64_t items = ceil_div(rows, bm) * ceil_div(cols, bn);
    const double cost = items <= cus ? one : static_cast<double>(ceil_div(items, per_cu * cus)) * full;
    if (!best || cost < least) {
      best = bm;
      least = cost;
    }
  };
  consider(64, 128, 2, 0.56, 0.85);
  consider(128, 128, 2, 0.87, 1.35);
  consider(256, 256, 1, 1.95, 1.95);
  consider(320, 256, 1, 2.4, 2.4);
  return best;
}

hipError_t launch_gemm_i8_tiles(const I8GemmArgs& a, int epilogue, hipStream_t stream) {
  if (a.tiles && (!a.tile_runs || !a.queue)) return hipErrorInvalidValue;
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
