// The whole layer for a few tokens, in one launch, on gfx950 (moe_few in
// include/moe.h): router projection, choice and gates, shared and routed
// experts, combine.
//
// With a token or some tens of them the bytes of the chosen experts' weights are
// the time, and the steps of the layer are short: what costs is the chip
// standing still between launches, and weights that are not yet asked for.  So
// the work is cut into items in one order,
//
//   router rows | x in MXFP8 | choice of 4 tokens and, behind the last, the list
//   of experts (by the choice's own item where there is one only) |
//   shared up/gate | routed up/gate, expert by expert | (h in MXFP8) |
//   shared down | routed down, expert by expert | combine
//
// and workgroups draw the next item (or few) from a counter until none is left.
// An item waits, if it must, only for items that come before it in that order.
// Those were drawn earlier, by workgroups that run, that do their items in order
// and wait for still earlier ones only, so every wait ends however few
// workgroups are resident and whatever else the GPU runs.  By the time an item
// is drawn what it waits for is mostly done: the shared expert's up/gate runs
// while the tokens are routed, and an expert's down projection comes one pass
// over the experts after its up/gate.
//
// An item of a product is 16 M weight rows (of up/gate: 8 M gate rows and the
// 8 M up rows of the same columns, so that SwiGLU needs no other item) by all
// tokens of one expert, M = 1 to 4 by the rule at run_few: four waves share out K in stages of 128 bytes, weights and tokens
// go straight from memory to the matrix core (v_mfma_f32_16x16x32_bf16, or
// v_mfma_scale_f32_16x16x128_f8f6f4) with the weights as row operand, and the
// waves' sums meet in LDS in a fixed order.  The first stages of the next item's
// weights are asked for before an item's sums meet.
//
// Roundings: sums are fp32.  In bf16 h is kept as two bf16 terms (17 bits of
// it; the second product costs nothing beside the weights' stream), in MXFP8 it
// is quantised as the layer defines.  (The matrix core sums products of 8-bit
// values less exactly than others: 128 random products of E4M3 come out 1.5e-5 of
// their sum's RMS off, 2.5e-4 of the largest product at most, by
// v_mfma_scale_f32_16x16x128 and v_mfma_f32_16x16x32 alike.  So one value of h in
// 600 falls on the other side of a border between two values of E4M3, here as in
// moe_forward.)  Every expert's output stays fp32 until the combine,
// acc = fma(g_s, y_s, acc) over the slots, then + shared.
//
// Between workgroups: results that others read are stored past the caches
// (agent-scope stores), have arrived (vector memory completes in order, and a
// later load's data was waited for, or s_waitcnt) before the workgroup counts
// them, and are read past the caches (agent-scope loads) by who has seen the
// count.  Fences took 50 us an item with 512 workgroups at it (a release writes
// an XCD's whole cache back); an atomic on one address takes 11.5 ns, one after
// the other, which is what bounds the number of items.  The last workgroup to
// leave clears the counters for the next call.
//
// Measured (bf16, top 8, weights read once, from x to out): 7168 x 2048 and 256
// experts, one token, 797 MB in 192 us (4.2 TB/s; 384 experts in MXFP8 457 MB in 144
// us); eight tokens 5.2 GB in 740 to 780 us (6.6 to 7.0 TB/s); 2048 x 768 and 128
// experts, one token, 86 MB in 65 us and 64 tokens, 1.2 GB in 292 us (4.1 TB/s; in
// MXFP8 0.62 GB in 223 us).  With many tokens the bound
// is memory.  With one it is the phases' chain: about 20 us until the list is
// there, 30 us for a workgroup's first item of a kind (cold code, cold memory) and
// 7 to 17 for a later one.  Two workgroups of a compute unit: three or four take
// 248 to 284 us where two take 195, their counters' traffic growing with them.

#include <algorithm>

#include "common.h"
#include "gemm_common.h"
#include "kernels.h"
#include "mx.h"
#include "route_scores.h"

namespace moe {

namespace {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kPerCu = 2;     // workgroups of a compute unit
constexpr int kStageB = 128;  // bytes of a row per K stage
constexpr int kRouterRows = 32;  // of an item
constexpr int kCombCols = 64;    // of a combine item, at least
constexpr int kErrPipeline = 0x8;     // MOE_DEVERR_PIPELINE
constexpr int kFewSpinCap = 1 << 20;  // polls of about 0.5 us each

// Words of the control block, apart by a cache line.  Its place in the workspace
// and that of every word in it are the same for all shapes: calls of several
// shapes may share a workspace, and what they leave cleared stays where the next
// one looks.
constexpr int kTicket = 0, kExit = 64, kRouted = 128, kChosen = 192, kState = 256, kCounts = 320;
// The state word: kReady from the initialisation on, until a call gives up.  A call
// that finds anything else (bytes never initialised, counters and flags that a call
// which gave up left behind) reports it and does nothing.
constexpr uint32_t kReady = 0x6d6f6531u;
constexpr int kMaxExperts = 1024, kMaxWidth = 65536;
__host__ __device__ constexpr int up_count_at(int a) { return kCounts + a; }  // a: place among the active experts; E: shared
__host__ __device__ constexpr int down_count_at(int block) { return kCounts + kMaxExperts + 1 + block; }  // block: of combine

// "The list is there", a word for every workgroup: hundreds that poll one word
// hold up the counters beside it.  Each clears its own.
constexpr int kFewGrid = 256 * kPerCu, kFlagStride = 32;
constexpr int kFlags = (down_count_at(kMaxWidth / kCombCols) + kFlagStride - 1) / kFlagStride * kFlagStride;
static_assert(kFlags + kFewGrid * kFlagStride == kFewCtlInts, "the block's size");

// A draw, as it is used at most: no item of a call lies past it (1024 experts, 65536
// columns by 8), and its batches of at most 64 items stay below 2^31.  So an item is
// never in front of the first one, whatever the workspace holds.
constexpr uint32_t kMaxDraw = 1u << 24;

// The list of active experts in the workspace: their number, ids, first
// positions and the routes by position (expert by expert, then by route).
__host__ __device__ inline int list_ids(int) { return 1; }
__host__ __device__ inline int list_starts(int E) { return 1 + E; }
__host__ __device__ inline int list_order(int E) { return 1 + E + E + 1; }

// ---- memory that other workgroups write or read ----
__device__ __forceinline__ void put32(void* p, uint32_t v) {
  __hip_atomic_store(static_cast<uint32_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put64(void* p, uint32_t lo, uint32_t hi) {
  __hip_atomic_store(static_cast<uint64_t*>(p), static_cast<uint64_t>(hi) << 32 | lo, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_f4(float* p, f32x4_t v) {
  put64(p, __float_as_uint(v[0]), __float_as_uint(v[1]));
  put64(p + 2, __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint32_t get32(const void* p) {
  return __hip_atomic_load(static_cast<const uint32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t get_f4(const float* p) {
  const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
  const uint64_t lo = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t hi = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return f32x4_t{__uint_as_float(static_cast<uint32_t>(lo)), __uint_as_float(static_cast<uint32_t>(lo >> 32)),
                 __uint_as_float(static_cast<uint32_t>(hi)), __uint_as_float(static_cast<uint32_t>(hi >> 32))};
}
// Cache policy of buffer loads past the caches (sc1, as agent-scope loads).
constexpr int kCoherent = 16;

__device__ __forceinline__ int scalar_of(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct FewShared {
  int next[2];  // by the item's parity
  int flag, n_active, ready;
  int wave_sum[kWaves];
  uint16_t id[1024];    // active expert -> expert
  uint16_t start[1025];  // its first position
  uint8_t token[1024];  // position -> token
  uint16_t place[1024];  // route -> position
  // the waves' sums, of 16-token items in halves by the item's parity; also the
  // choice's values (2048 doubles and floats) and the list's counts
  f32x4_t red[2][kWaves * 4 * kWave];
};
static_assert(sizeof(FewShared::red) >= 12 * 2048 && sizeof(FewShared::red) >= 3 * 4096, "scratch");

// This workgroup's stores have arrived; then *ctr += 1.
__device__ __forceinline__ void signal(int* ctr) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's
  __syncthreads();                                   // and every wave's
  if (threadIdx.x == 0) __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Wait for ctl[at] >= target.  It ends without a time limit (see above); the
// limit is for counters that something else wrote to, and stops the launch.
__device__ __forceinline__ bool wait_for(FewShared& sh, int* ctl, int at, int target, int* err) {
  if (threadIdx.x == 0) {
    int ok = 1;
    for (int spins = 0; static_cast<int>(get32(ctl + at)) < target; ++spins) {
      if ((spins & 63) == 63 && (spins > kFewSpinCap || get32(ctl + kState) != kReady)) {
        put32(ctl + kState, 0);
        raise_error(err, kErrPipeline);
        ok = 0;
        break;
      }
      __builtin_amdgcn_s_sleep(16);
    }
    sh.flag = ok;
  }
  __syncthreads();
  const bool ok = scalar_of(sh.flag) != 0;
  __syncthreads();  // the flag has been read
  return ok;
}
// The first of the experts e, e + 1, ... (64 of them at most, below A) whose
// count has not come to `need`.
__device__ __forceinline__ int complete_from(FewShared& sh, const int* ctl, int e, int A, int need) {
  if (threadIdx.x < kWave) {
    const int i = e + static_cast<int>(threadIdx.x);
    const uint64_t open = __ballot(i < A && static_cast<int>(get32(ctl + up_count_at(i))) < need);
    if (threadIdx.x == 0) sh.flag = open ? e + __builtin_ctzll(open) : min(e + kWave, A);
  }
  __syncthreads();
  const int to = scalar_of(sh.flag);
  __syncthreads();
  return to;
}

// ---- products ----
// The tokens an expert has in this call.
struct Part {
  int expert;       // index of its matrices (0 for the shared expert)
  int rows, first;  // tokens, and the first row of h and y
  int place;        // among the active experts; E: shared
  bool shared;
};
__device__ __forceinline__ Part listed_part(const FewArgs& a, const FewShared& sh, int e) {
  const int first = scalar_of(sh.start[e]), end = scalar_of(sh.start[e + 1]);
  return Part{scalar_of(sh.id[e]), min(end - first, a.T), first, e, false};
}

// A buffer resource, certainly in scalar registers: a load whose resource the
// compiler holds in vector registers takes a loop over the lanes' values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t source(const void* p, int64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint64_t uniform = static_cast<uint64_t>(static_cast<uint32_t>(scalar_of(static_cast<int>(at >> 32)))) << 32 |
                           static_cast<uint32_t>(scalar_of(static_cast<int>(at)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform), 0, scalar_of(static_cast<int>(bytes)),
                                           0x00020000);
}

// The weights of an item: M blocks of 16 rows, this lane's row of each.
template <int M>
struct WeightSource {
  const char* w[M];
  const uint32_t* s[M];  // MXFP8: scale words
  int stage_b, s_stage;  // bytes, words
};
template <int M, bool MX>
struct WeightStage {
  u32x4_t w[M][2];
  uint32_t s[M];
  __device__ __forceinline__ void load(const WeightSource<M>& o, int st) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const u32x4_t* const p = reinterpret_cast<const u32x4_t*>(o.w[m] + static_cast<int64_t>(st) * o.stage_b);
      w[m][0] = p[0];
      w[m][1] = p[4];
      if constexpr (MX) s[m] = o.s[m][static_cast<int64_t>(st) * o.s_stage];
    }
  }
};
// The tokens of an item: NB blocks of 16 columns, SPLIT terms.
template <int NB>
struct TokenSource {
  __amdgpu_buffer_rsrc_t b, s;
  uint32_t at[NB], s_at[NB];
  int term_b;
};
template <int NB, int SPLIT, bool MX, bool COHERENT>
struct TokenStage {
  u32x4_t b[NB][SPLIT][2];
  uint32_t s[NB];
  __device__ __forceinline__ void load(const TokenSource<NB>& o, int st, int nb) {
    constexpr int kPolicy = COHERENT ? kCoherent : 0;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (NB > 1 && n >= nb) continue;
#pragma unroll
      for (int t = 0; t < SPLIT; ++t) {
        const int at = st * kStageB + t * o.term_b;
        b[n][t][0] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(o.b, o.at[n], at, kPolicy));
        b[n][t][1] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(o.b, o.at[n] + 64, at, kPolicy));
      }
      if constexpr (MX) s[n] = __builtin_amdgcn_raw_buffer_load_b32(o.s, o.s_at[n], st * 4, kPolicy);
    }
  }
};
template <int M, int NB, int SPLIT, bool MX, bool COHERENT>
__device__ __forceinline__ void multiply(const WeightStage<M, MX>& w, const TokenStage<NB, SPLIT, MX, COHERENT>& x,
                                         f32x4_t (&acc)[M][NB], int nb, int kq) {
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    if (NB > 1 && n >= nb) continue;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if constexpr (MX) {
        const i32x8_t wv = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(w.w[m][0], w.w[m][1], 0, 1, 2, 3, 4, 5, 6, 7));
        const i32x8_t xv = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(x.b[n][0][0], x.b[n][0][1], 0, 1, 2, 3, 4, 5, 6, 7));
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, acc[m][n], 0, 0, 0,
                                                                     static_cast<int>(w.s[m] >> (8 * kq)), 0,
                                                                     static_cast<int>(x.s[n] >> (8 * kq)));
      } else {
#pragma unroll
        for (int t = 0; t < SPLIT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w.w[m][h]),
                                                                __builtin_bit_cast(bf16x8_t, x.b[n][t][h]), acc[m][n],
                                                                0, 0, 0);
      }
    }
  }
}

// A wave's stages of an item of `stages` from `first` on: the waves take them in turn.
struct Stages {
  int n, s0, last;
  __device__ __forceinline__ Stages(int first, int stages) {
    const int wave = scalar_of(static_cast<int>(threadIdx.x) / kWave);
    n = stages > wave ? (stages - wave + kWaves - 1) / kWaves : 0;
    s0 = first + wave;
    last = first + stages - 1;
  }
  __device__ __forceinline__ int operator()(int i) const { return min(s0 + kWaves * i, last); }
};

// The first stages of an item's weights.
template <int M, bool MX, int PF>
__device__ __forceinline__ void first_stages(WeightStage<M, MX> (&f)[PF], const WeightSource<M>& w, const Stages& at) {
#pragma unroll
  for (int p = 0; p < PF; ++p) f[p].load(w, at(p));
}

// The sums of an item into LDS; the first stages of its weights are in flight
// already.  (Every bound here is scalar: a matrix instruction does not heed the
// lane mask, it must be jumped over.)
template <int NB, int SPLIT, bool COHERENT, int M, bool MX, int PF>
__device__ __forceinline__ void item_sums(FewShared& sh, WeightStage<M, MX> (&f)[PF], const WeightSource<M>& w,
                                          const TokenSource<NB>& x, const Stages& at, int nb, int parity) {
  const int lane = lane_id(), kq = lane >> 4;
  const int wave = scalar_of(static_cast<int>(threadIdx.x) / kWave);
  f32x4_t acc[M][NB];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int n = at.n;
  if constexpr (NB == 1) {
    TokenStage<1, SPLIT, MX, COHERENT> g[PF];
    // (no branch round a load and a first group of its own: the compiler counts
    // the loads in flight and would wait for all of them where paths with
    // different counts meet)
#pragma unroll
    for (int p = 0; p < PF; ++p) g[p].load(x, at(p), 1);
    auto group = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        multiply(f[p], g[p], acc, 1, kq);
        f[p].load(w, at(i + p + PF));
        g[p].load(x, at(i + p + PF), 1);
      }
    };
    int i = 0;
    if (n >= 2 * PF) {
      group(0);
      for (i = PF; i + 2 * PF <= n; i += PF) group(i);
    }
    for (; i < n; i += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        if (i + p < n) multiply(f[p], g[p], acc, 1, kq);
        if (i + p + PF < n) {
          f[p].load(w, at(i + p + PF));
          g[p].load(x, at(i + p + PF), 1);
        }
      }
    }
  } else {  // more than 16 tokens: their stages come from the caches as they are needed
    for (int i = 0; i < n; i += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        if (i + p < n) {
          TokenStage<NB, SPLIT, MX, COHERENT> g;
          g.load(x, at(i + p), nb);
          multiply(f[p], g, acc, nb, kq);
        }
        if (i + p + PF < n) f[p].load(w, at(i + p + PF));
      }
    }
  }
  f32x4_t* const red = NB == 1 ? sh.red[parity] : sh.red[0];
  if (NB > 1) __syncthreads();  // the item before has read its sums
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (NB == 1 || b < nb) red[((m * NB + b) * kWaves + wave) * kWave + lane] = acc[m][b];
}
// Sum over the waves, in their order, of one lane's four values of a block.
template <int NB>
__device__ __forceinline__ f32x4_t wave_total(const FewShared& sh, int parity, int block, int lane) {
  const f32x4_t* const red = (NB == 1 ? sh.red[parity] : sh.red[0]) + block * kWaves * kWave + lane;
  f32x4_t v = red[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += red[w * kWave];
  return v;
}

// Where an expert's h is: fp32 (MXFP8: before it is quantised), or two planes of
// bf16.  The routed experts' rows and the shared expert's have a region each.
struct HRows {
  char* base;
  int64_t first, plane;  // the part's first element; elements of a plane
  uint8_t* q;
  uint32_t* s;
};
__device__ __forceinline__ HRows h_rows(const FewArgs& a, const Part& p) {
  const int64_t routed = static_cast<int64_t>(a.T) * a.k * a.I, begin = p.shared ? routed : 0;
  return HRows{static_cast<char*>(a.h) + 4 * begin, p.shared ? 0 : static_cast<int64_t>(p.first) * a.I,
               p.shared ? static_cast<int64_t>(a.T) * a.Is : routed, a.hq + begin, a.hs + begin / 128};
}

// ---- the choice of a token's experts, by one wave ----
// As route_scored_kernel forms it with a wave per token (the same sums in the
// same order): lane j holds experts 4 (64 q + j) .. + 3, here in LDS, c_s and
// l_s [1024], so that this seldom run part does not set the kernel's registers.
// The logits are given, or the sums of the router's K parts in their order.
__device__ __forceinline__ void choose(const FewArgs& a, int token, double* c_s, float* l_s) {
  const int lane = lane_id(), E = a.E, k = a.k;
  const RouterArgs& r = a.router;
  float* const row = a.logits + static_cast<int64_t>(token) * E;
  const int quads = (E + 4 * kWave - 1) / (4 * kWave);
  auto settle = [] {  // the wave's LDS writes, before any lane reads them
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  bool bad = false;
  float m = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < quads; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (kWave * q + lane) + i, at = min(e, E - 1);
      float v;
      if (a.w_router) {
        const float* part = a.parts + static_cast<int64_t>(token) * E + at;
        float p[kFewParts];
#pragma unroll
        for (int j = 0; j < kFewParts; ++j)
          p[j] = j < a.n_parts ? __uint_as_float(get32(part + static_cast<int64_t>(j) * a.T * E)) : 0.f;
        v = p[0];
#pragma unroll
        for (int j = 1; j < kFewParts; ++j) v += j < a.n_parts ? p[j] : 0.f;
        if (e < E) row[e] = v;
      } else {
        v = row[at];
      }
      const float b = a.bias ? a.bias[at] : 0.f;
      bad |= e < E && (!__builtin_isfinite(v) || !__builtin_isfinite(b));
      v = e < E ? clean_logit(v) : -INFINITY;
      l_s[e] = v;
      m = fmaxf(m, v);
    }
  }
  if (bad) raise_error(a.err, kErrNonFinite);
  m = lanes_max<kWave>(m);
  const bool by_logit = !a.bias && (r.kept_groups == r.groups || !r.top2 || r.group_size == 1);
  const bool sums = !r.sigmoid && !(by_logit && r.renorm);  // softmax scores themselves
  double inv = 1.0;
  if (sums) {
    double sum = 0.0;
#pragma unroll 1
    for (int q = 0; q < quads; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * (kWave * q + lane) + i;
        const double z = exp_below(l_s[e], m);
        c_s[e] = z;
        sum += z;
      }
    }
    sum = lanes_sum<kWave>(sum);
    inv = sum > 0.0 ? recip64(sum) : 0.0;
  }
#pragma unroll 1
  for (int q = 0; q < quads; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (kWave * q + lane) + i;
      const float l = l_s[e];
      const double b = a.bias && e < E ? static_cast<double>(a.bias[e]) : 0.0;
      const double v = by_logit ? static_cast<double>(l) : r.sigmoid ? sigmoid64(l) + b : c_s[e] * inv + b;
      c_s[e] = e < E ? (v > kLast ? (v < -kLast ? v : -kLast) : kLast) : -INFINITY;
    }
  }
  uint64_t kept = ~uint64_t(0);
  int per = 1;
  if (r.kept_groups < r.groups) {
    settle();
    // a group by `per` neighbouring lanes
    while (2 * per * r.groups <= kWave) per *= 2;
    const int group = lane / per;
    double best = -INFINITY, next = -INFINITY;
    if (group < r.groups)
      for (int e = lane % per; e < r.group_size; e += per) {
        const double v = c_s[group * r.group_size + e];
        next = max64(next, min64(best, v));
        best = max64(best, v);
      }
    for (int d = 1; d < per; d *= 2) {
      const double ob = __shfl_xor(best, d), on = __shfl_xor(next, d);
      next = max64(min64(best, ob), max64(next, on));
      best = max64(best, ob);
    }
    const double v = r.top2 && r.group_size > 1 ? best + next : best;
    int better = 0;
    for (int o = 0; o < r.groups; ++o) {
      const double u = __shfl(v, o * per);
      better += u > v || (u == v && o < group);
    }
    kept = __ballot(group < r.groups && better < r.kept_groups);
    settle();  // every lane has read
  }
  // candidates, and this lane's largest
  double best = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < quads; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (kWave * q + lane) + i;
      const double v = c_s[e];
      const bool in = (kept >> (((__umul24(static_cast<uint32_t>(e), r.group_magic) >> 20) * per) & 63)) & 1;
      const double key = in && v > -INFINITY ? candidate(v, e) : -INFINITY;
      c_s[e] = key;
      best = max64(best, key);
    }
  }
  double mine = -INFINITY;
  for (int s = 0; s < k; ++s) {
    const double top = lanes_best64<kWave>(best);
    mine = lane == s ? top : mine;
    if (best == top) {  // a candidate is one expert's alone: this lane's next
      best = -INFINITY;
      for (int q = 0; q < quads; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double v = c_s[4 * (kWave * q + lane) + i];
          best = v < top ? max64(best, v) : best;
        }
      }
    }
  }
  const int id = lane < k ? min(candidate_id(mine), E - 1) : 0;
  const float my_l = lane < k ? l_s[id] : -INFINITY;
  double w;
  if (r.renorm) {
    w = chosen_score(r.sigmoid, my_l, lanes_max<kWave>(my_l));
    const double W = lanes_sum<kWave>(w);
    w = W > 0.0 ? w / W : 0.0;
  } else {
    w = r.sigmoid ? sigmoid64(my_l) : exp_below(my_l, m) * inv;
  }
  if (lane < k) {
    const int64_t at = static_cast<int64_t>(token) * k + lane;
    put32(a.idx + at, static_cast<uint32_t>(id));
    put32(a.gate + at, __float_as_uint(static_cast<float>(w * r.scale)));
  }
}

// ---- the list of active experts, by one workgroup, from every token's choice ----
__device__ __forceinline__ void build_list(const FewArgs& a, FewShared& sh) {
  const int tid = static_cast<int>(threadIdx.x), lane = lane_id(), wave = tid / kWave;
  const int n = a.T * a.k, E = a.E;
  int* const count = reinterpret_cast<int*>(sh.red);       // [1024]
  int* const begin = count + 1024;                         // [1024]
  int* const expert = begin + 1024;                        // [1024] of a route
  for (int e = tid; e < 1024; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int j = tid; j < n; j += kThreads) {
    const int e = min(max(static_cast<int>(get32(a.idx + j)), 0), E - 1);
    expert[j] = e;
    atomicAdd(&count[e], 1);
  }
  __syncthreads();
  // (active experts, routes) before this thread's kOwn experts, in one word
  constexpr int kOwn = 1024 / kThreads;
  int c[kOwn], mine = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    c[i] = count[kOwn * tid + i];
    mine += c[i] + (c[i] > 0 ? 65536 : 0);
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int o = __shfl_up(upto, d);
    upto += lane >= d ? o : 0;
  }
  if (lane == kWave - 1) sh.wave_sum[wave] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < wave; ++w) before += sh.wave_sum[w];
  int at = before & 0xffff, place = before >> 16;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    begin[kOwn * tid + i] = at;
    if (c[i] > 0) {
      put32(a.list + list_ids(E) + place, kOwn * tid + i);
      put32(a.list + list_starts(E) + place, at);
      ++place;
    }
    at += c[i];
  }
  if (tid == kThreads - 1) {
    put32(a.list, place);
    put32(a.list + list_starts(E) + place, n);
  }
  __syncthreads();
  if (wave > 0) return;
  // one wave, 64 routes at a time in their order: lanes of one expert find each
  // other bit by bit of its id
  for (int j0 = 0; j0 < n; j0 += kWave) {
    const int j = j0 + lane;
    const int e = j < n ? expert[j] : -1;
    uint64_t same = __ballot(j < n);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
      const uint64_t set = __ballot((e >> bit) & 1);
      same &= (e >> bit) & 1 ? set : ~set;
    }
    if (j < n) {
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const int p = begin[e] + rank;
      put32(a.list + list_order(E) + p, j);
      if (rank == __popcll(same) - 1) begin[e] = p + 1;  // the last of them, behind every lane's read
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

// The list into LDS.  Bounds are kept whatever the workspace holds.
__device__ __forceinline__ void load_list(const FewArgs& a, FewShared& sh) {
  const int tid = static_cast<int>(threadIdx.x), n = a.T * a.k, E = a.E;
  const int A = min(max(static_cast<int>(get32(a.list)), 0), min(n, E));
  if (tid == 0) sh.n_active = A;
  for (int i = tid; i < A; i += kThreads) {
    sh.id[i] = static_cast<uint16_t>(min(max(static_cast<int>(get32(a.list + list_ids(E) + i)), 0), E - 1));
    sh.start[i] = static_cast<uint16_t>(min(max(static_cast<int>(get32(a.list + list_starts(E) + i)), 0), n - 1));
  }
  if (tid == 0) sh.start[A] = static_cast<uint16_t>(n);
  for (int p = tid; p < n; p += kThreads) {
    const int j = min(max(static_cast<int>(get32(a.list + list_order(E) + p)), 0), n - 1);
    sh.token[p] = static_cast<uint8_t>(j / a.k);
    sh.place[j] = static_cast<uint16_t>(p);
  }
  __syncthreads();
}

// 128 fp32 values in MXFP8, and x: 128 values of a token a thread.
__device__ __forceinline__ void quantize_group(const float* v, uint8_t* q, uint32_t* s) {
  uint32_t word = 0;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    float w[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4_t u = get_f4(v + 32 * b + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = u[j];
    }
    u32x4_t lo, hi;
    word |= static_cast<uint32_t>(quantize32_f32(w, lo, hi)) << (8 * b);
    put64(q + 32 * b, lo[0], lo[1]);
    put64(q + 32 * b + 8, lo[2], lo[3]);
    put64(q + 32 * b + 16, hi[0], hi[1]);
    put64(q + 32 * b + 24, hi[2], hi[3]);
  }
  put32(s, word);
}
__device__ __forceinline__ void quantize_x(const FewArgs& a, int group) {
  if (group >= a.T * (a.D / 128)) return;
  uint32_t word = 0;
  uint8_t* q = a.xq + static_cast<int64_t>(group) * 128;
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.x + static_cast<int64_t>(group) * 128);
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    float w[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4_t u = src[4 * b + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        w[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
    u32x4_t lo, hi;
    word |= static_cast<uint32_t>(quantize32_f32(w, lo, hi)) << (8 * b);
    put64(q + 32 * b, lo[0], lo[1]);
    put64(q + 32 * b + 8, lo[2], lo[3]);
    put64(q + 32 * b + 16, hi[0], hi[1]);
    put64(q + 32 * b + 24, hi[2], hi[3]);
  }
  put32(a.xs + group, word);
}

// ---- items ----
// The weights of an up/gate item (8 columns a block: rows 0 .. 7 of the block are
// gate's, 8 .. 15 up's) or a down item (16 columns a block).
template <bool UP, bool MX, int M>
__device__ __forceinline__ WeightSource<M> weights_of(const FewArgs& a, const Part& p, int n0) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  const bool tiled = !p.shared && a.routed.tiled, of_up = r16 >= 8;
  const int I = p.shared ? a.Is : a.I, N = UP ? I : a.D, K = UP ? a.D : I;
  const int row_bytes = MX ? K : 2 * K, row_b = tiled ? kStageB : row_bytes;
  const void* const down = p.shared ? a.shared.down : a.routed.down;
  const void* const gate = p.shared ? a.shared.gate : a.routed.gate;
  const void* const up = p.shared ? a.shared.up : a.routed.up;
  const char* const base = static_cast<const char*>(UP ? (of_up ? up : gate) : down) +
                           static_cast<int64_t>(p.expert) * N * row_bytes + kq * 16;
  const int row0 = UP ? n0 + (r16 & 7) : n0 + r16;
  WeightSource<M> o;
  o.stage_b = tiled ? N * kStageB : kStageB;
#pragma unroll
  for (int m = 0; m < M; ++m) o.w[m] = base + static_cast<int64_t>(row0 + (UP ? 8 : 16) * m) * row_b;
  if constexpr (MX) {
    const uint8_t* const s_down = p.shared ? a.shared.s_down : a.routed.s_down;
    const uint8_t* const s_gate = p.shared ? a.shared.s_gate : a.routed.s_gate;
    const uint8_t* const s_up = p.shared ? a.shared.s_up : a.routed.s_up;
    const uint32_t* const s_base = reinterpret_cast<const uint32_t*>(UP ? (of_up ? s_up : s_gate) : s_down) +
                                   static_cast<int64_t>(p.expert) * N * (K / 128);
    o.s_stage = N;
#pragma unroll
    for (int m = 0; m < M; ++m) o.s[m] = s_base + row0 + (UP ? 8 : 16) * m;
  }
  return o;
}

// x rows of an expert's tokens (the shared one's: of every token).
template <int NB, bool MX>
__device__ __forceinline__ TokenSource<NB> tokens_of(const FewArgs& a, const FewShared& sh, const Part& p) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  TokenSource<NB> o;
  const int row_b = MX ? a.D : 2 * a.D;
  o.b = source(MX ? static_cast<const void*>(a.xq) : a.x, static_cast<int64_t>(a.T) * row_b);
  if constexpr (MX) o.s = source(a.xs, static_cast<int64_t>(a.T) * (a.D / 32));
  o.term_b = 0;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int c = min(16 * n + r16, p.rows - 1);
    const int t = p.shared ? c : sh.token[p.first + c];
    o.at[n] = static_cast<uint32_t>(t) * row_b + kq * 16;
    o.s_at[n] = static_cast<uint32_t>(t) * (a.D / 32);
  }
  return o;
}
// h rows of an expert's tokens.
template <int NB, bool MX>
__device__ __forceinline__ TokenSource<NB> hidden_of(const FewArgs& a, const Part& p) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  const HRows hr = h_rows(a, p);
  const int I = p.shared ? a.Is : a.I;
  TokenSource<NB> o;
  if constexpr (MX) {
    o.b = source(hr.q + hr.first, static_cast<int64_t>(p.rows) * I);
    o.s = source(hr.s + hr.first / 128, static_cast<int64_t>(p.rows) * (I / 32));
    o.term_b = 0;
  } else {
    o.b = source(hr.base + 2 * hr.first, 2 * (hr.plane + static_cast<int64_t>(p.rows) * I));
    o.term_b = scalar_of(static_cast<int>(2 * hr.plane));
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int c = min(16 * n + r16, p.rows - 1);
    o.at[n] = static_cast<uint32_t>(c) * (MX ? I : 2 * I) + kq * 16;
    o.s_at[n] = static_cast<uint32_t>(c) * (I / 32);
  }
  return o;
}

// Logits of experts 32 item / n_parts .. + 31, one K part of them.
template <int NB>
__device__ __forceinline__ void router_item(const FewArgs& a, FewShared& sh, int item) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  const int block = item / a.n_parts, part = item - block * a.n_parts, n0 = block * kRouterRows;
  WeightSource<2> w;
#pragma unroll
  for (int m = 0; m < 2; ++m)
    w.w[m] = reinterpret_cast<const char*>(a.w_router) +
             static_cast<int64_t>(min(n0 + 16 * m + r16, a.E - 1)) * a.D * 2 + kq * 16;
  w.stage_b = kStageB;
  const int all = a.D / 64, first = part * all / a.n_parts;
  const Stages at(first, (part + 1) * all / a.n_parts - first);
  const int nb = (a.T + 15) / 16;
  WeightStage<2, false> f[4];
  first_stages(f, w, at);
  item_sums<NB, 1, false>(sh, f, w, tokens_of<NB, false>(a, sh, Part{0, a.T, 0, a.E, true}), at, nb, 0);
  __syncthreads();
  float* const plane = a.parts + static_cast<int64_t>(part) * a.T * a.E;
  for (int q = threadIdx.x; q < 2 * nb * kWave; q += kThreads) {
    const int l = q & (kWave - 1), m = (q / kWave) & 1, n = q / kWave / 2;
    const int t = 16 * n + (l & 15), e0 = n0 + 16 * m + 4 * (l >> 4);
    if (t >= a.T) continue;
    const f32x4_t v = wave_total<NB>(sh, 0, m * NB + n, l);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < a.E) put32(plane + static_cast<int64_t>(t) * a.E + e0 + i, __float_as_uint(v[i]));
  }
}
// h of an up/gate item from its sums.
template <int M, int NB, bool MX>
__device__ __forceinline__ void finish_up(const FewArgs& a, const FewShared& sh, const Part& p, int n0, int parity) {
  const HRows hr = h_rows(a, p);
  const int I = p.shared ? a.Is : a.I, nb = (p.rows + 15) / 16;
  // lanes 0 .. 31 of a block hold gate, 32 .. 63 up
  for (int q = threadIdx.x; q < M * nb * 32; q += kThreads) {
    const int l = q & 31, m = (q >> 5) % M, n = (q >> 5) / M;
    const int c = 16 * n + (l & 15), col = n0 + 8 * m + 4 * (l >> 4);
    if (c >= p.rows) continue;
    const f32x4_t g = wave_total<NB>(sh, parity, m * NB + n, l), u = wave_total<NB>(sh, parity, m * NB + n, l + 32);
    f32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu_mul(g[i], u[i]);
    const int64_t at = hr.first + static_cast<int64_t>(c) * I + col;
    if constexpr (MX) {
      put_f4(reinterpret_cast<float*>(hr.base) + at, h);
    } else {
      // h = hi + lo, each to nearest (hi cut off where it would round past the largest float)
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t near = f32_to_bf16(h[i]);
        const bool finite = __builtin_isfinite(h[i]);
        hi[i] = finite && (near & 0x7fffu) == 0x7f80u ? __float_as_uint(h[i]) >> 16 : near;
        lo[i] = finite ? f32_to_bf16(h[i] - bf16_to_f32(static_cast<uint16_t>(hi[i]))) : 0u;
      }
      uint16_t* const p16 = reinterpret_cast<uint16_t*>(hr.base) + at;
      put64(p16, hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      put64(p16 + hr.plane, lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    }
  }
}
// y of a down item.
template <int M, int NB>
__device__ __forceinline__ void finish_down(const FewArgs& a, const FewShared& sh, const Part& p, int n0, int parity) {
  const int nb = (p.rows + 15) / 16;
  for (int q = threadIdx.x; q < M * nb * kWave; q += kThreads) {
    const int l = q & (kWave - 1), m = (q / kWave) % M, n = q / kWave / M;
    const int c = 16 * n + (l & 15), col = n0 + 16 * m + 4 * (l >> 4);
    if (c >= p.rows) continue;
    put_f4(a.y + static_cast<int64_t>(p.first + c) * a.D + col, wave_total<NB>(sh, parity, m * NB + n, l));
  }
}

// Output columns n0 .. n0 + cols - 1 of every token.
__device__ __forceinline__ void combine(const FewArgs& a, const FewShared& sh, int n0, int cols) {
  const int D = a.D, k = a.k, quads = cols / 4;
  for (int q = threadIdx.x; q < a.T * quads; q += kThreads) {
    const int t = q / quads, col = n0 + 4 * (q - t * quads);
    const f32x4_t shared = get_f4(a.y + static_cast<int64_t>(a.T * k + t) * D + col);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s0 = 0; s0 < k; s0 += 8) {  // the loads of eight slots side by side
      f32x4_t y[8];
      float g[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int route = t * k + min(s0 + s, k - 1);
        g[s] = __uint_as_float(get32(a.gate + route));
        y[s] = get_f4(a.y + static_cast<int64_t>(sh.place[route]) * D + col);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(g[s], y[s][i], acc[i]);
        }
    }
    acc += shared;
    const int64_t at = static_cast<int64_t>(t) * D + col;
    *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    if (a.out32) *reinterpret_cast<f32x4_t*>(a.out32 + at) = acc;
  }
}

// h of one expert in MXFP8.
__device__ __forceinline__ void quantize_h(const FewArgs& a, const Part& p) {
  const HRows hr = h_rows(a, p);
  const int I = p.shared ? a.Is : a.I;
  for (int g = threadIdx.x; g < p.rows * (I / 128); g += kThreads) {
    const int64_t at = hr.first + static_cast<int64_t>(g) * 128;
    quantize_group(reinterpret_cast<const float*>(hr.base) + at, hr.q + at, hr.s + at / 128);
  }
}

// The kernel's arguments, read anew: held over the loops they would take more
// scalar registers than there are.
__device__ __forceinline__ FewArgs arguments() {
#ifdef __HIP_DEVICE_COMPILE__
  typedef const __attribute__((address_space(4))) FewArgs* Ptr;
  Ptr p = (Ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
#else
  return FewArgs{};  // the host's pass over device code
#endif
}

// A workgroup's way through the items.  Those before the routed experts' are
// drawn one by one, up/gate and what follows it in batches of their own.
struct Walk {
  int t;         // this item, or past `b_up` the draw itself while there is no list
  int left;      // items of its batch from it on
  int parity;    // of the number of items so far
  int drawn;     // thread 0: the next draw, once asked for
  int* pending;  // the count that the last product's stores are to be added to
  int b_up, b_after, b_end;  // first routed up/gate item, first item past them, end; the last two from the list on
};
__device__ __forceinline__ int draw(const FewArgs& a) {
  return __hip_atomic_fetch_add(a.ctl + kTicket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Ask for what comes after this item, while it runs.
__device__ __forceinline__ void ask(const FewArgs& a, Walk& w) {
  w.parity ^= 1;
  if (w.left == 1 && threadIdx.x == 0) w.drawn = draw(a);
}
// The item of a draw.
__device__ __forceinline__ void resolve(const FewArgs& a, Walk& w, int v) {
  v = static_cast<int>(min(static_cast<uint32_t>(v), kMaxDraw));
  w.t = v;
  w.left = 1;
  if (v < w.b_up || w.b_after == 0) return;
  const int draws = (w.b_after - w.b_up + a.up_batch - 1) / a.up_batch;
  const bool up = v < w.b_up + draws;
  const int base = up ? w.b_up : w.b_after, batch = up ? a.up_batch : a.down_batch;
  w.t = base + (v - (up ? w.b_up : w.b_up + draws)) * batch;
  w.left = min(batch, (up ? w.b_after : w.b_end) - w.t);  // (past the end: any number)
}
// Thread 0, before a barrier.
__device__ __forceinline__ void tell(FewShared& sh, const Walk& w) {
  if (threadIdx.x == 0) sh.next[w.parity] = w.drawn;
}
// Behind that barrier: the next item.
__device__ __forceinline__ void advance(const FewArgs& a, const FewShared& sh, Walk& w) {
  if (w.left > 1) {
    --w.left;
    ++w.t;
  } else {
    resolve(a, w, scalar_of(sh.next[w.parity]));
  }
}
__device__ __forceinline__ void flush(Walk& w) {
  if (w.pending) signal(w.pending);
  w.pending = nullptr;
}

// The items of one kind of product, of the shared expert or of the routed ones,
// from this one to `end`; they begin at `begin`.  False if the launch was stopped.
// need: what the count of what they read comes to before they may begin.
template <bool UP, bool MX, bool WIDE, int M, int DEPTH>
__device__ __forceinline__ bool products(FewShared& sh, Walk& walk, bool shared, int begin, int end,
                                         int need, int A) {
  const FewArgs first_args = arguments();
  constexpr int NBW = WIDE ? 4 : 1, kCols = (UP ? 8 : 16) * M, SPLIT = UP || MX ? 1 : 2;
  constexpr bool kCoh = !UP || MX;  // h, and x in MXFP8, are other workgroups' stores
  const int I = shared ? first_args.Is : first_args.I, per = (UP ? I : first_args.D) / kCols, K = UP ? first_args.D : I;
  const Stages at(0, MX ? K / 128 : K / 64);
  int complete = 0;  // active experts whose h is complete, as far as this workgroup has seen
  Part p{0, first_args.T, UP ? 0 : first_args.T * first_args.k, first_args.E, true};
  int n0 = 0;
  auto locate = [&](const FewArgs& a, int t) __attribute__((always_inline)) {
    const int e = shared ? 0 : (t - begin) / per;
    n0 = (t - begin - e * per) * kCols;
    if (!shared) p = listed_part(a, sh, e);
  };
  locate(first_args, walk.t);
  WeightStage<M, MX> f[DEPTH / M];
  WeightSource<M> w = weights_of<UP, MX, M>(first_args, p, n0);
  first_stages(f, w, at);
  if (shared && (!UP || MX)) {
    flush(walk);
    if (!wait_for(sh, first_args.ctl, UP ? kRouted : up_count_at(first_args.E), need, first_args.err)) return false;
  }
  for (;;) {
    const FewArgs a = arguments();
    ask(a, walk);
    if (!UP && !shared && p.place >= complete) {
      flush(walk);
      complete = complete_from(sh, a.ctl, p.place, A, need);
      if (complete == p.place) {
        if (!wait_for(sh, a.ctl, up_count_at(p.place), need, a.err)) return false;
        complete = p.place + 1;
      }
    }
    const int nb = scalar_of((p.rows + 15) / 16);
    const bool narrow = !WIDE || nb <= 1;
    if (narrow) {
      // (0 only where something else wrote to the list: no index from it then)
      if (nb > 0) item_sums<1, SPLIT, kCoh>(sh, f, w, UP ? tokens_of<1, MX>(a, sh, p) : hidden_of<1, MX>(a, p), at, nb, walk.parity);
    } else {
      item_sums<NBW, SPLIT, kCoh>(sh, f, w, UP ? tokens_of<NBW, MX>(a, sh, p) : hidden_of<NBW, MX>(a, p), at, nb, walk.parity);
    }
    // The waves meet: their sums are in LDS, and the stores of the product
    // before have arrived.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    tell(sh, walk);
    __syncthreads();
    if (walk.pending && threadIdx.x == 0)
      __hip_atomic_fetch_add(walk.pending, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const Part done = p;
    const int done_n0 = n0, parity = walk.parity;
    advance(a, sh, walk);
    const bool more = walk.t < end;
    if (more) {
      locate(a, walk.t);
      w = weights_of<UP, MX, M>(a, p, n0);
      first_stages(f, w, at);
    }
    if (UP) {
      if (narrow)
        finish_up<M, 1, MX>(a, sh, done, done_n0, parity);
      else
        finish_up<M, NBW, MX>(a, sh, done, done_n0, parity);
    } else {
      if (narrow)
        finish_down<M, 1>(a, sh, done, done_n0, parity);
      else
        finish_down<M, NBW>(a, sh, done, done_n0, parity);
    }
    if (!narrow) __syncthreads();  // its sums take both halves
    walk.pending = a.ctl + (UP ? up_count_at(done.place) : down_count_at(done_n0 / a.comb_cols));
    if (!more) return true;
  }
}

// The workgroup's way; false if the launch was stopped.
template <bool WIDE, bool MXR, bool MXS, int UM, int DM>
__device__ __forceinline__ bool walk_items(const FewArgs& a, FewShared& sh) {
  constexpr int NBW = WIDE ? 4 : 1;
  constexpr bool MXW = MXR || MXS;
  constexpr int kUpCols = 8 * UM, kDownCols = 16 * DM;
  // Blocks of 16 rows by a stage that a wave has in flight: four, and of items of four
  // blocks eight, two stages.  Eight for all items of up to 16 tokens gain nothing
  // (2048 x 768, one token: 66.8 us either way; 1472 x 320, 13 tokens: 108, four 102),
  // and for items of one block cost registers (7168 x 2048, one token: 190 us, four
  // 189; in MXFP8 158, four 144).
  constexpr int kDepth = 4, kDownDepth = DM == 4 ? 8 : kDepth;
  const int tid = static_cast<int>(threadIdx.x);
  // where the items of a kind begin
  const int b_quant = a.w_router ? (a.E + kRouterRows - 1) / kRouterRows * a.n_parts : 0;
  const int b_choose = b_quant + (MXW ? (a.T * (a.D / 128) + kThreads - 1) / kThreads : 0);
  const int n_choose = (a.T + kWaves - 1) / kWaves;  // (a single one builds the list itself)
  const int b_build = b_choose + n_choose, b_up_s = b_build + (n_choose > 1 ? 1 : 0);
  const int b_up = b_up_s + a.Is / kUpCols;

  Walk walk{0, 1, 0, 0, nullptr, b_up, 0, 0};
  if (tid == 0) {
    walk.drawn = draw(a);
    sh.ready = get32(a.ctl + kState) == kReady;  // (both in flight together)
  }
  tell(sh, walk);
  __syncthreads();
  if (!scalar_of(sh.ready)) {
    if (tid == 0) raise_error(a.err, kErrPipeline);
    return false;
  }
  advance(a, sh, walk);
  while (walk.t < b_up_s) {
    ask(a, walk);
    if (walk.t < b_quant) {
      router_item<NBW>(a, sh, walk.t);
      signal(a.ctl + kRouted);
    } else if (walk.t < b_choose) {
      quantize_x(a, (walk.t - b_quant) * kThreads + tid);
      signal(a.ctl + kRouted);
    } else if (walk.t < b_build) {
      if (!wait_for(sh, a.ctl, kRouted, b_choose, a.err)) return false;
      const int wave = scalar_of(tid / kWave), token = (walk.t - b_choose) * kWaves + wave;  // a wave a token
      // (two waves at a time where a token's values take more of LDS)
      const int size = a.E <= 512 ? 512 : 1024, slots = 2048 / size;
      double* const c_s = reinterpret_cast<double*>(sh.red) + wave % slots * size;
      float* const l_s = reinterpret_cast<float*>(sh.red) + 4096 + wave % slots * size;
      for (int turn = 0; turn < kWaves / slots; ++turn) {
        if (wave / slots == turn && token < a.T) choose(a, token, c_s, l_s);
        __syncthreads();
      }
      if (n_choose > 1) {
        signal(a.ctl + kChosen);
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
      }
    }
    if (walk.t == b_up_s - 1) {
      if (n_choose > 1 && !wait_for(sh, a.ctl, kChosen, n_choose, a.err)) return false;
      build_list(a, sh);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      for (int i = tid; i < static_cast<int>(gridDim.x); i += kThreads) put32(a.flags + i * kFlagStride, 1);
    }
    tell(sh, walk);
    __syncthreads();
    advance(a, sh, walk);
  }
  // (one loop for the shared and the routed experts' products: the same code, which
  // is cold when a launch begins)
  int A = 0, b_quant_h = 0, b_down_s = 0, b_down = 0, b_combine = 0;
#pragma unroll 1
  for (int routed = 0; routed < 2; ++routed) {
    if (routed) {
      flush(walk);
      int* const flag = a.flags + blockIdx.x * kFlagStride;
      if (!wait_for(sh, a.ctl, static_cast<int>(flag - a.ctl), 1, a.err)) return false;
      if (tid == 0) put32(flag, 0);
      load_list(a, sh);
      A = scalar_of(sh.n_active);
      b_quant_h = b_up + A * (a.I / kUpCols);
      b_down_s = b_quant_h + (MXS ? 1 : 0) + (MXR ? A : 0);
      b_down = b_down_s + a.D / kDownCols;
      b_combine = b_down + A * (a.D / kDownCols);
      walk.b_after = b_quant_h;
      walk.b_end = b_combine + a.D / a.comb_cols;
      resolve(a, walk, walk.t);
    }
    const int begin = routed ? b_up : b_up_s, end = routed ? b_quant_h : b_up;
    if (walk.t >= end) continue;
    if (MXR == MXS || routed) {
      if (!products<true, MXR, WIDE, UM, kDepth>(sh, walk, !routed, begin, end, b_choose, A)) return false;
    } else {
      if (!products<true, MXS, WIDE, UM, kDepth>(sh, walk, !routed, begin, end, b_choose, A)) return false;
    }
  }
  const int need_s = a.Is / kUpCols, need_r = a.I / kUpCols;
  if constexpr (MXW) {
    while (walk.t < b_down_s) {
      flush(walk);
      ask(a, walk);
      const int e = walk.t - b_quant_h - (MXS ? 1 : 0);
      const Part p = e < 0 ? Part{0, a.T, 0, a.E, true} : listed_part(a, sh, e);
      if (!wait_for(sh, a.ctl, up_count_at(p.place), e < 0 ? need_s : need_r, a.err)) return false;
      quantize_h(a, p);
      signal(a.ctl + up_count_at(p.place));
      tell(sh, walk);
      __syncthreads();
      advance(a, sh, walk);
    }
  }
#pragma unroll 1
  for (int routed = 0; routed < 2; ++routed) {
    const int begin = routed ? b_down : b_down_s, end = routed ? b_combine : b_down;
    if (walk.t >= end) continue;
    if (MXR == MXS || routed) {
      if (!products<false, MXR, WIDE, DM, kDownDepth>(sh, walk, !routed, begin, end, (routed ? need_r : need_s) + (MXR ? 1 : 0), A))
        return false;
    } else {
      if (!products<false, MXS, WIDE, DM, kDownDepth>(sh, walk, !routed, begin, end, need_s + (MXS ? 1 : 0), A)) return false;
    }
  }
  flush(walk);
  while (walk.t < walk.b_end) {
    ask(a, walk);
    const int block = walk.t - b_combine;
    if (!wait_for(sh, a.ctl, down_count_at(block), (A + 1) * (a.comb_cols / kDownCols), a.err)) return false;
    combine(a, sh, block * a.comb_cols, a.comb_cols);
    tell(sh, walk);
    __syncthreads();
    advance(a, sh, walk);
  }
  return true;
}

// WIDE: more than 16 tokens.  MXR, MXS: routed and shared experts in MXFP8.  UM, DM:
// blocks of 16 rows of an up/gate and of a down item.
template <bool WIDE, bool MXR, bool MXS, int UM, int DM>
__global__ __launch_bounds__(kThreads, kPerCu) void few_kernel(const FewArgs a) {
  __shared__ FewShared sh;
  walk_items<WIDE, MXR, MXS, UM, DM>(a, sh);
  // the last workgroup to leave clears the counters (the state stays as it is)
  const int tid = static_cast<int>(threadIdx.x);
  __syncthreads();
  if (tid == 0) sh.flag = __hip_atomic_fetch_add(a.ctl + kExit, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (sh.flag == static_cast<int>(gridDim.x) - 1) {
    const int counts = kCounts + a.E + 1, n = counts + a.D / a.comb_cols;
    for (int i = tid; i < n; i += kThreads)
      if (i != kState) put32(a.ctl + (i < counts ? i : down_count_at(i - counts)), 0);
  }
}

template <bool WIDE, bool MXR, bool MXS>
hipError_t run_few(const FewArgs& a, int grid, hipStream_t stream) {
  FewArgs b = a;
  const int64_t experts = std::min<int64_t>(a.E, static_cast<int64_t>(a.T) * a.k) + 1;
  const int e_bytes = MXR ? 1 : 2;
  const int64_t up = experts * (a.I / 16), down = experts * (a.D / 32);
  const bool fine = !WIDE && up >= grid && up + down < 8 * grid;
  const bool long_down = !fine && !WIDE && down > grid && down <= 2 * grid;
  // Rows of an item.  `fine`, 16 of up/gate: short items where a workgroup has some
  // but not many, so that the rounds end evenly (7168 x 2048, one token: 195 us; 32
  // rows 212).  With many, or with less than a round of them, 32 (2048 x 768, one
  // token: 66.5; 16 rows 69.5).  More than 16 tokens are read again for every item,
  // so that twice the items cost more (4096 x 1024, 8 experts: 17 tokens 100 us, 16
  // rows 115 to 123; 64 tokens 139, 16 rows 171; the same in MXFP8 97 and 121, 136
  // and 171; 2048 x 1024, 16 experts, 17 tokens, the one that lost: 110, 16 rows 105).
  // `long_down`, 64 of down: where 32 would make between one round and two, 64 makes
  // one (2048 x 768, one token: 66.5; 32 rows 73.6).  Not with more than 16 tokens,
  // whose sums take the registers.
  // Items of a draw: bytes enough for the draws not to be the limit, while every workgroup has several
  auto batch = [&](int64_t items, int64_t bytes) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(65536 / bytes, items / (4 * grid))));
  };
  const int um = fine ? 1 : 2, dm = long_down ? 4 : 2;
  b.up_batch = batch(experts * (a.I / (8 * um)), static_cast<int64_t>(16) * um * a.D * e_bytes);
  b.down_batch = batch(experts * (a.D / (16 * dm)), static_cast<int64_t>(16) * dm * a.I * e_bytes);
  if constexpr (!WIDE) {
    if (fine || long_down) {
      if (fine)
        few_kernel<false, MXR, MXS, 1, 2><<<grid, kThreads, 0, stream>>>(b);
      else
        few_kernel<false, MXR, MXS, 2, 4><<<grid, kThreads, 0, stream>>>(b);
      return hipGetLastError();
    }
  }
  few_kernel<WIDE, MXR, MXS, 2, 2><<<grid, kThreads, 0, stream>>>(b);
  return hipGetLastError();
}

}  // namespace

__global__ void few_init_kernel(int* err, int32_t* ctl) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < kFewCtlInts) ctl[i] = i == kState ? static_cast<int32_t>(kReady) : 0;
  if (i == 0) *err = 0;
}
hipError_t launch_few_init(int* err, int32_t* ctl, hipStream_t stream) {
  few_init_kernel<<<(kFewCtlInts + kThreads - 1) / kThreads, kThreads, 0, stream>>>(err, ctl);
  return hipGetLastError();
}

int few_list_ints(int E, int routes) { return list_order(E) + routes; }

hipError_t launch_few(const FewArgs& args, bool mx_routed, bool mx_shared, hipStream_t stream) {
  FewArgs a = args;
  if (a.T < 1 || a.T > kFewTokens || a.k < 1 || a.k > 16 || a.E < a.k || a.E > kMaxExperts || a.D % 64 || a.I % 64 ||
      a.Is % 64 || a.D > kMaxWidth || a.router.groups > kMaxGroups || a.E % a.router.groups)
    return hipErrorInvalidValue;
  if ((mx_routed || mx_shared) && a.D % 128) return hipErrorInvalidValue;
  if ((mx_routed && a.I % 128) || (mx_shared && a.Is % 128)) return hipErrorInvalidValue;
  a.router.group_size = a.E / a.router.groups;
  a.router.group_magic = (1u << 20) / static_cast<uint32_t>(a.router.group_size) + 1;  // exact for e < 1024
  a.flags = a.ctl + kFlags;
  const int64_t cus = device_compute_units();
  const int grid = static_cast<int>(std::min<int64_t>(kFewGrid, kPerCu * (cus > 0 ? cus : 256)));
  // K parts of a router row: 16 stages of 64 values or so
  a.n_parts = std::min(kFewParts, std::max(1, a.D / 1024));
  // combine: fewer columns an item the more tokens there are, a divisor of D
  a.comb_cols = a.T <= 8 && a.D % 256 == 0 ? 256 : a.T <= 16 && a.D % 128 == 0 ? 128 : 64;
  const bool wide = a.T > 16;
#define MOE_FEW(R, S) return wide ? run_few<true, R, S>(a, grid, stream) : run_few<false, R, S>(a, grid, stream)
  if (mx_routed && mx_shared) MOE_FEW(true, true);
  if (mx_routed) MOE_FEW(true, false);
  if (mx_shared) MOE_FEW(false, true);
  MOE_FEW(false, false);
#undef MOE_FEW
}

}  // namespace moe
