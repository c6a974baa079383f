// The whole layer for a few tokens, in one launch, on gfx950 (moe_few in
// include/moe.h): router projection, choice and gates, shared and routed
// experts, combine.
//
// With a token or some tens of them the bytes of the chosen experts' weights are
// the time, and the steps of the layer are short: what costs is the chip
// standing still between launches, and weights that are not yet asked for.  So
// the work is cut into items in one order,
//
//   router rows | x in MXFP8 | choice of 8 tokens | shared up/gate |
//   routed up/gate, expert by expert | shared down | routed down, expert by expert
//
// and workgroups take the next item from a ticket counter until none is left.
// An item waits, if it must, only for items that come before it in that order.
// Those were taken earlier, by workgroups that run and that wait for still
// earlier ones only, so every wait ends however few workgroups are resident and
// whatever else the GPU runs.  By the time an item is taken what it waits for
// is mostly done: the shared expert's up/gate runs while the tokens are routed,
// and an expert's down projection comes one pass over the experts after its
// up/gate.
//
// An item is 16 (or 32) weight rows by all tokens of one expert: four waves
// share out K in stages of 128 bytes, weights and tokens go straight from
// memory to the matrix core (v_mfma_f32_16x16x32_bf16, or
// v_mfma_scale_f32_16x16x128_f8f6f4) with the weights as row operand, and the
// waves' sums meet in LDS in a fixed order.  An up/gate block holds 8 gate and
// the 8 up rows of the same columns, so that SwiGLU needs no other item.
//
// Roundings: sums are fp32.  In bf16 h is kept as two bf16 terms (16 bits of
// it; the second product costs nothing beside the weights' stream), in MXFP8 it
// is quantised as the layer defines.  Every expert's output stays fp32 until the
// combine, acc = fma(g_s, y_s, acc) over the slots, then + shared.
//
// Between workgroups: results that others read are stored write-through
// (agent-scope stores) and counted; a reader sees the count, then
// invalidates its caches (an acquire).  The last workgroup to leave clears the
// counters for the next call.

#include "common.h"
#include "gemm_common.h"
#include "kernels.h"
#include "mx.h"
#include "route_scores.h"

namespace moe {

namespace {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kPerCu = 2;  // workgroups of a compute unit
constexpr int kStageB = 128;  // bytes of a row per K stage
constexpr int kErrPipeline = 0x8;  // MOE_DEVERR_PIPELINE
constexpr int kFewSpinCap = 1 << 23;  // polls of about 0.1 us each

// Words of the control block, apart by a cache line.
constexpr int kTicket = 0, kExit = 32, kRouted = 64, kChosen = 96, kList = 128, kAbort = 160, kCounts = 192;
__host__ __device__ inline int up_count_at(int a) { return kCounts + a; }  // a: place among the active experts; E: shared
__host__ __device__ inline int down_count_at(int E, int block) { return kCounts + E + 1 + block; }

// The list of active experts in the workspace: their number, ids, first
// positions and the routes by position (expert by expert, then by route).
__host__ __device__ inline int list_ids(int) { return 1; }
__host__ __device__ inline int list_starts(int E) { return 1 + E; }
__host__ __device__ inline int list_order(int E) { return 1 + E + E + 1; }

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

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

struct FewShared {
  int next, flag, n_active;
  int total;  // scratch of the list's scan
  int wave_sum[kWaves];
  uint16_t id[1024];      // active expert -> expert
  uint16_t start[1025];   // its first position
  uint8_t token[1024];    // position -> token
  uint16_t place[1024];   // route -> position
  // the waves' sums; also the choice's values (kWaves x 1024 doubles) and the list's counts
  f32x4_t red[kWaves * 8 * kWave];
};
static_assert(sizeof(FewShared::red) >= sizeof(double) * kWaves * 1024 && sizeof(FewShared::red) >= 3 * 4096, "scratch");

// This workgroup's stores have reached memory; then *ctr += 1.  Returns the
// count before it, on every thread.
__device__ __forceinline__ int signal(FewShared& sh, int* ctr) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have completed
  __syncthreads();                                   // and every wave's
  if (threadIdx.x == 0) sh.flag = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(sh.flag);
}
__device__ __forceinline__ void acquire() {
  if (threadIdx.x == 0) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  __syncthreads();
}
// Wait for *ctr >= target.  It ends without a time limit (see above); the limit
// is for a workspace that was never initialised, and stops the whole launch.
__device__ __forceinline__ bool wait_for(FewShared& sh, int* ctl, int at, int target, int* err) {
  if (threadIdx.x == 0) {
    int ok = 1;
    for (int spins = 0;; ++spins) {
      if (__hip_atomic_load(ctl + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= target) break;
      if ((spins & 63) == 63 &&
          (spins > kFewSpinCap || __hip_atomic_load(ctl + kAbort, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))) {
        __hip_atomic_store(ctl + kAbort, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        raise_error(err, kErrPipeline);
        ok = 0;
        break;
      }
      __builtin_amdgcn_s_sleep(2);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    sh.flag = ok;
  }
  __syncthreads();
  const bool ok = __builtin_amdgcn_readfirstlane(sh.flag) != 0;
  __syncthreads();  // the flag has been read
  return ok;
}

// ---- sums of one item ----
// The operand rows of this lane: weights (MB blocks of 16 rows), tokens (NB
// blocks of 16 columns, SPLIT terms b_term bytes apart).
template <int MB, int NB>
struct Operands {
  const char* a[MB];
  int64_t a_stage;  // bytes from a stage to the next
  const char* b[NB];
  int64_t b_term;
  // MXFP8: the scale words (4 blocks of 32 per stage)
  const uint32_t* as[MB];
  int64_t as_stage;  // words
  const uint32_t* bs[NB];
};

template <int MB, int NB, int SPLIT, bool MX>
struct Stage {
  u32x4_t a[MB][2], b[NB][SPLIT][2];
  uint32_t as[MB], bs[NB];

  __device__ __forceinline__ void load(const Operands<MB, NB>& o, int st, int nb) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(o.a[m] + st * o.a_stage);
      a[m][0] = __builtin_nontemporal_load(p);
      a[m][1] = __builtin_nontemporal_load(p + 4);
      if constexpr (MX) as[m] = o.as[m][st * o.as_stage];
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (NB > 1 && n >= nb) continue;
#pragma unroll
      for (int s = 0; s < SPLIT; ++s) {
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(o.b[n] + s * o.b_term + static_cast<int64_t>(st) * kStageB);
        b[n][s][0] = p[0];
        b[n][s][1] = p[4];
      }
      if constexpr (MX) bs[n] = o.bs[n][st];
    }
  }
  __device__ __forceinline__ void multiply(f32x4_t (&acc)[MB][NB], int nb, int kq) const {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (NB > 1 && n >= nb) continue;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if constexpr (MX) {
          const i32x8_t av = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(a[m][0], a[m][1], 0, 1, 2, 3, 4, 5, 6, 7));
          const i32x8_t bv =
              __builtin_bit_cast(i32x8_t, __builtin_shufflevector(b[n][0][0], b[n][0][1], 0, 1, 2, 3, 4, 5, 6, 7));
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              av, bv, acc[m][n], 0, 0, 0, static_cast<int>(as[m] >> (8 * kq)), 0, static_cast<int>(bs[n] >> (8 * kq)));
        } else {
#pragma unroll
          for (int s = 0; s < SPLIT; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[m][h]),
                                                                  __builtin_bit_cast(bf16x8_t, b[n][s][h]),
                                                                  acc[m][n], 0, 0, 0);
        }
      }
    }
  }
};

// Waves take the stages in turn; PF of them are in flight.
template <int MB, int NB, int SPLIT, bool MX, int PF>
__device__ __forceinline__ void item_sums(FewShared& sh, const Operands<MB, NB>& o, int stages, int nb) {
  const int lane = lane_id(), kq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  f32x4_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // (scalar, as every bound here: a matrix instruction does not heed the lane mask, so it must be jumped over)
  const int n = __builtin_amdgcn_readfirstlane(stages > wave ? (stages - wave + kWaves - 1) / kWaves : 0);
  Stage<MB, NB, SPLIT, MX> f[PF];
  auto at = [&](int i) { return wave + kWaves * i; };
#pragma unroll
  for (int p = 0; p < PF; ++p)
    if (p < n) f[p].load(o, at(p), nb);
  int i = 0;
  for (; i + 2 * PF <= n; i += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      f[p].multiply(acc, nb, kq);
      f[p].load(o, at(i + p + PF), nb);
    }
  }
  for (; i < n; i += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      if (i + p < n) f[p].multiply(acc, nb, kq);
      if (i + p + PF < n) f[p].load(o, at(i + p + PF), nb);
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (NB == 1 || b < nb) sh.red[((m * NB + b) * kWaves + wave) * kWave + lane] = acc[m][b];
  __syncthreads();
}
// Sum over the waves, in their order, of one lane's four values of a block.
__device__ __forceinline__ f32x4_t wave_total(const FewShared& sh, int block, int lane) {
  f32x4_t v = sh.red[block * kWaves * kWave + lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += sh.red[(block * kWaves + w) * kWave + lane];
  return v;
}

__device__ __forceinline__ int scalar_of(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One expert's part in an item: its weights' place and its tokens.
struct Part {
  int64_t expert;  // index of its matrices
  int rows;        // tokens
  int first;       // first row of h and y
  bool shared;
};

// Where a part's h is: fp32 (MXFP8: before it is quantised), or two planes of
// bf16.  The routed experts' rows and the shared expert's have a region each.
struct HRows {
  char* base;
  int64_t first, plane;  // the part's first element; elements of a plane
  uint8_t* q;
  uint32_t* s;
};
__device__ __forceinline__ HRows h_rows(const FewArgs& a, const Part& p) {
  const int64_t routed = static_cast<int64_t>(a.T) * a.k * a.I;
  if (p.shared)
    return HRows{static_cast<char*>(a.h) + 4 * routed, 0, static_cast<int64_t>(a.T) * a.Is, a.hq + routed, a.hs + routed / 128};
  return HRows{static_cast<char*>(a.h), static_cast<int64_t>(p.first) * a.I, routed, a.hq, a.hs};
}

__device__ __forceinline__ Part listed_part(const FewArgs& a, const FewShared& sh, int e) {
  const int first = scalar_of(sh.start[e]), end = scalar_of(sh.start[e + 1]);
  return Part{scalar_of(sh.id[e]), min(end - first, a.T), first, false};
}

// ---- the choice of a token's experts, by one wave ----
// As route_scored_kernel forms it with a wave per token (the same sums in the
// same order): lane j holds experts 4 (64 q + j) .. + 3, here in LDS, c_s
// [1024], so that this seldom run part does not set the kernel's registers.
__device__ __forceinline__ void choose(const FewArgs& a, int token, double* c_s) {
  const int lane = lane_id(), E = a.E, k = a.k;
  const RouterArgs& r = a.router;
  const float* row = a.logits + static_cast<int64_t>(token) * E;
  const int quads = (E + 4 * kWave - 1) / (4 * kWave);
  auto logit = [&](int e) { return e < E ? clean_logit(row[e]) : -INFINITY; };
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
      const int e = 4 * (kWave * q + lane) + i;
      bad |= e < E && (!__builtin_isfinite(row[e]) || (a.bias && !__builtin_isfinite(a.bias[e])));
      m = fmaxf(m, logit(e));
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
        const double z = exp_below(logit(e), m);
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
      const float l = logit(e);
      const double b = a.bias && e < E ? static_cast<double>(a.bias[e]) : 0.0;
      const double v = by_logit ? static_cast<double>(l) : r.sigmoid ? sigmoid64(l) + b : c_s[e] * inv + b;
      c_s[e] = e < E ? (v > kLast ? (v < -kLast ? v : -kLast) : kLast) : -INFINITY;
    }
  }
  uint64_t kept = ~uint64_t(0);
  if (r.kept_groups < r.groups) {
    settle();
    double best = -INFINITY, next = -INFINITY;
    if (lane < r.groups)
      for (int e = 0; e < r.group_size; ++e) {
        const double v = c_s[lane * r.group_size + e];
        next = max64(next, min64(best, v));
        best = max64(best, v);
      }
    const double v = r.top2 && r.group_size > 1 ? best + next : best;
    int better = 0;
    for (int o = 0; o < r.groups; ++o) {
      const double u = __shfl(v, o);
      better += u > v || (u == v && o < lane);
    }
    kept = __ballot(lane < r.groups && better < r.kept_groups);
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
      const bool in = (kept >> ((__umul24(static_cast<uint32_t>(e), r.group_magic) >> 20) & 63)) & 1;
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
  const float my_l = lane < k ? clean_logit(row[id]) : -INFINITY;
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
    const int e = min(max(a.idx[j], 0), E - 1);
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
  for (int j = tid; j < n; j += kThreads) {
    const int e = expert[j];
    int p = begin[e];
    for (int o = 0; o < j; ++o) p += expert[o] == e;
    put32(a.list + list_order(E) + p, j);
  }
}

// The list into LDS.  Bounds are kept whatever the workspace holds.
__device__ __forceinline__ void load_list(const FewArgs& a, FewShared& sh) {
  const int tid = static_cast<int>(threadIdx.x), n = a.T * a.k, E = a.E;
  const int A = min(max(a.list[0], 0), min(n, E));
  if (tid == 0) sh.n_active = A;
  for (int i = tid; i < A; i += kThreads) {
    sh.id[i] = static_cast<uint16_t>(min(max(a.list[list_ids(E) + i], 0), E - 1));
    sh.start[i] = static_cast<uint16_t>(min(max(a.list[list_starts(E) + i], 0), n - 1));
  }
  if (tid == 0) sh.start[A] = static_cast<uint16_t>(n);
  for (int p = tid; p < n; p += kThreads) {
    const int j = min(max(a.list[list_order(E) + p], 0), n - 1);
    sh.token[p] = static_cast<uint8_t>(j / a.k);
    sh.place[j] = static_cast<uint16_t>(p);
  }
  __syncthreads();
}

// x in MXFP8: 128 values of a token a thread.
__device__ __forceinline__ void quantize_group(const float* v, uint8_t* q, uint32_t* s) {
  uint32_t word = 0;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    float w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = v[32 * b + i];
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
template <int NB>
__device__ __forceinline__ void router_item(const FewArgs& a, FewShared& sh, int item) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  Operands<1, NB> o{};
  const int e = min(16 * item + r16, a.E - 1);
  o.a[0] = reinterpret_cast<const char*>(a.w_router) + static_cast<int64_t>(e) * a.D * 2 + kq * 16;
  o.a_stage = kStageB;
  const int nb = (a.T + 15) / 16;
#pragma unroll
  for (int n = 0; n < NB; ++n)
    o.b[n] = reinterpret_cast<const char*>(a.x) + static_cast<int64_t>(min(16 * n + r16, a.T - 1)) * a.D * 2 + kq * 16;
  item_sums<1, NB, 1, false, NB == 1 ? 8 : 1>(sh, o, a.D / 64, nb);
  for (int q = threadIdx.x; q < nb * kWave; q += kThreads) {
    const int n = q / kWave, l = q & (kWave - 1);
    const int t = 16 * n + (l & 15), e0 = 16 * item + 4 * (l >> 4);
    if (t >= a.T) continue;
    const f32x4_t v = wave_total(sh, n, l);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < a.E) put32(a.logits + static_cast<int64_t>(t) * a.E + e0 + i, __float_as_uint(v[i]));
  }
}

// h columns n0 .. n0 + 8 MB - 1 of one expert: block m holds gate rows (its
// rows 0 .. 7) and up rows (8 .. 15) of 8 of them.
template <int MB, int NB, bool MX>
__device__ __forceinline__ void up_item(const FewArgs& a, const FewWeights& w, FewShared& sh, const Part& p, int n0,
                                        int N) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  const int64_t K = a.D, row_bytes = MX ? K : 2 * K;
  const int64_t row_b = w.tiled ? kStageB : row_bytes;
  const int64_t matrix = p.expert * N * row_bytes;
  Operands<MB, NB> o{};
  o.a_stage = w.tiled ? static_cast<int64_t>(N) * kStageB : kStageB;
  const char* const base = static_cast<const char*>(r16 < 8 ? w.gate : w.up) + matrix + kq * 16;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int row = n0 + 8 * m + (r16 & 7);
    o.a[m] = base + row * row_b;
    if constexpr (MX) {
      o.as[m] = reinterpret_cast<const uint32_t*>(r16 < 8 ? w.s_gate : w.s_up) + p.expert * (K / 128) * N + row;
      o.as_stage = N;
    }
  }
  const int nb = (p.rows + 15) / 16;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int c = min(16 * n + r16, p.rows - 1);
    const int t = p.shared ? c : sh.token[p.first + c];
    if constexpr (MX) {
      o.b[n] = reinterpret_cast<const char*>(a.xq) + t * K + kq * 16;
      o.bs[n] = a.xs + static_cast<int64_t>(t) * (K / 128);
    } else {
      o.b[n] = reinterpret_cast<const char*>(a.x) + t * K * 2 + kq * 16;
    }
  }
  item_sums<MB, NB, 1, MX, NB == 1 ? 8 / MB : 1>(sh, o, static_cast<int>(row_bytes / kStageB), nb);
  // lanes 0 .. 31 of a block hold gate, 32 .. 63 up
  for (int q = threadIdx.x; q < MB * nb * 32; q += kThreads) {
    const int l = q & 31, m = (q >> 5) % MB, n = (q >> 5) / MB;
    const int c = 16 * n + (l & 15), col = n0 + 8 * m + 4 * (l >> 4);
    if (c >= p.rows) continue;
    const f32x4_t g = wave_total(sh, m * NB + n, l), u = wave_total(sh, m * NB + n, l + 32);
    f32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu_mul(g[i], u[i]);
    const HRows hr = h_rows(a, p);
    const int64_t at = static_cast<int64_t>(c) * N + col;
    if constexpr (MX) {
      put_f4(reinterpret_cast<float*>(hr.base) + hr.first + at, h);
    } else {
      // h = hi + lo: the upper 8 bits cut off, the rest rounded
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u32 = __float_as_uint(h[i]) & 0xffff0000u;
        const bool finite = __builtin_isfinite(h[i]);
        hi[i] = finite ? u32 >> 16 : f32_to_bf16(h[i]);
        lo[i] = finite ? f32_to_bf16(h[i] - __uint_as_float(u32)) : 0u;
      }
      uint16_t* const p16 = reinterpret_cast<uint16_t*>(hr.base) + hr.first + at;
      put64(p16, hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      put64(p16 + hr.plane, lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    }
  }
}

// Output columns n0 .. n0 + 16 MB - 1 of one expert.
template <int MB, int NB, bool MX>
__device__ __forceinline__ void down_item(const FewArgs& a, const FewWeights& w, FewShared& sh, const Part& p, int n0,
                                          int K) {
  const int lane = lane_id(), r16 = lane & 15, kq = lane >> 4;
  const int N = a.D;
  const int64_t row_bytes = MX ? K : 2 * static_cast<int64_t>(K);
  const int64_t row_b = w.tiled ? kStageB : row_bytes;
  Operands<MB, NB> o{};
  o.a_stage = w.tiled ? static_cast<int64_t>(N) * kStageB : kStageB;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int row = n0 + 16 * m + r16;
    o.a[m] = static_cast<const char*>(w.down) + p.expert * N * row_bytes + row * row_b + kq * 16;
    if constexpr (MX) {
      o.as[m] = reinterpret_cast<const uint32_t*>(w.s_down) + p.expert * (K / 128) * N + row;
      o.as_stage = N;
    }
  }
  const int nb = (p.rows + 15) / 16;
  const HRows hr = h_rows(a, p);
  o.b_term = 2 * hr.plane;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int64_t at = hr.first + static_cast<int64_t>(min(16 * n + r16, p.rows - 1)) * K;
    if constexpr (MX) {
      o.b[n] = reinterpret_cast<const char*>(hr.q) + at + kq * 16;
      o.bs[n] = hr.s + at / 128;
    } else {
      o.b[n] = hr.base + 2 * at + kq * 16;
    }
  }
  item_sums<MB, NB, MX ? 1 : 2, MX, NB == 1 ? 8 / MB : 1>(sh, o, static_cast<int>(row_bytes / kStageB), nb);
  const int y0 = p.shared ? a.T * a.k : p.first;
  for (int q = threadIdx.x; q < MB * nb * kWave; q += kThreads) {
    const int l = q & (kWave - 1), m = (q / kWave) % MB, n = (q / kWave) / MB;
    const int c = 16 * n + (l & 15), col = n0 + 16 * m + 4 * (l >> 4);
    if (c >= p.rows) continue;
    put_f4(a.y + static_cast<int64_t>(y0 + c) * N + col, wave_total(sh, m * NB + n, l));
  }
}

// Output columns n0 .. n0 + COLS - 1 of every token, once every expert's are there.
template <int COLS>
__device__ __forceinline__ void combine_block(const FewArgs& a, const FewShared& sh, int n0) {
  const int D = a.D, k = a.k;
  for (int q = threadIdx.x; q < a.T * (COLS / 4); q += kThreads) {
    const int t = q / (COLS / 4), col = n0 + 4 * (q % (COLS / 4));
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < k; ++s) {
      const float g = a.gate[t * k + s];
      const f32x4_t y = *reinterpret_cast<const f32x4_t*>(a.y + static_cast<int64_t>(sh.place[t * k + s]) * D + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(g, y[i], acc[i]);
    }
    acc += *reinterpret_cast<const f32x4_t*>(a.y + static_cast<int64_t>(a.T * k + t) * D + col);
    const int64_t at = static_cast<int64_t>(t) * D + col;
    *reinterpret_cast<u32x2_t*>(a.out + at) = u32x2_t{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
    if (a.out32) *reinterpret_cast<f32x4_t*>(a.out32 + at) = acc;
  }
}

// h of one expert in MXFP8, by the workgroup that finished its up/gate.
__device__ __forceinline__ void quantize_h(const FewArgs& a, const Part& p, int K) {
  const HRows hr = h_rows(a, p);
  for (int g = threadIdx.x; g < p.rows * (K / 128); g += kThreads) {
    const int64_t at = hr.first + static_cast<int64_t>(g) * 128;
    quantize_group(reinterpret_cast<const float*>(hr.base) + at, hr.q + at, hr.s + at / 128);
  }
}

// WIDE: more than 16 tokens.  MXR, MXS: routed and shared experts in MXFP8.
template <bool WIDE, bool MXR, bool MXS, int MBU, int MBD>
__global__ __launch_bounds__(kThreads, kPerCu * kWaves / 4) void few_kernel(const FewArgs a) {
  constexpr int NBW = WIDE ? 4 : 1;
  constexpr int UC = 8 * MBU, DC = 16 * MBD;  // columns of an up/gate and of a down item
  __shared__ FewShared sh;
  const int tid = static_cast<int>(threadIdx.x);
  int* const ctl = a.ctl;
  const int n_router = a.w_router ? (a.E + 15) / 16 : 0;
  const int n_quant = MXR || MXS ? (a.T * (a.D / 128) + kThreads - 1) / kThreads : 0;
  const int n_choose = (a.T + kWaves - 1) / kWaves;
  const int up_r = a.I / UC, up_s = a.Is / UC, down_n = a.D / DC;
  const int b_quant = n_router, b_choose = b_quant + n_quant, b_up_s = b_choose + n_choose, b_up = b_up_s + up_s;
  int b_down_s = 0, b_down = 0, b_end = 0;
  bool listed = false;

  if (tid == 0) sh.next = __hip_atomic_fetch_add(ctl + kTicket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  for (;;) {
    const int t = __builtin_amdgcn_readfirstlane(sh.next);
    if (t >= b_up && !listed) {
      if (!wait_for(sh, ctl, kList, 1, a.err)) break;
      load_list(a, sh);
      const int A = __builtin_amdgcn_readfirstlane(sh.n_active);
      b_down_s = b_up + A * up_r;
      b_down = b_down_s + down_n;
      b_end = b_down + A * down_n;
      listed = true;
    }
    if (t >= b_up && t >= b_end) break;
    // the next ticket comes while this item runs
    int next = 0;
    if (tid == 0) next = __hip_atomic_fetch_add(ctl + kTicket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

    if (t < b_choose) {
      if (t < b_quant)
        router_item<NBW>(a, sh, t);
      else
        quantize_x(a, (t - b_quant) * kThreads + tid);
      signal(sh, ctl + kRouted);
    } else if (t < b_up_s) {
      if (!wait_for(sh, ctl, kRouted, n_router + n_quant, a.err)) break;
      // a wave a token
      const int first = (t - b_choose) * kWaves, wave = tid / kWave;
      if (first + wave < a.T) choose(a, first + wave, reinterpret_cast<double*>(sh.red) + wave * 1024);
      if (signal(sh, ctl + kChosen) == n_choose - 1) {
        acquire();
        build_list(a, sh);
        signal(sh, ctl + kList);
      }
    } else if (t < b_down_s || t < b_up) {  // up/gate
      Part p;
      int item, a_count;
      if (t < b_up) {
        p = Part{0, a.T, 0, true};
        item = t - b_up_s;
        a_count = a.E;
        // x in MXFP8 is complete once its items are
        if (MXS && !wait_for(sh, ctl, kRouted, n_router + n_quant, a.err)) break;
      } else {
        const int e = (t - b_up) / up_r;
        item = (t - b_up) - e * up_r;
        p = listed_part(a, sh, e);
        a_count = e;
      }
      if (p.rows > 0) {
        const int n0 = item * UC;
        if (p.shared) {
          up_item<MBU, NBW, MXS>(a, a.shared, sh, p, n0, a.Is);
        } else if (!WIDE || p.rows <= 16) {
          up_item<MBU, 1, MXR>(a, a.routed, sh, p, n0, a.I);
        } else {
          up_item<MBU, NBW, MXR>(a, a.routed, sh, p, n0, a.I);
        }
      }
      const int n_items = p.shared ? up_s : up_r;
      if (signal(sh, ctl + up_count_at(a_count)) == n_items - 1 && (p.shared ? MXS : MXR)) {
        acquire();
        quantize_h(a, p, p.shared ? a.Is : a.I);
        signal(sh, ctl + up_count_at(a_count));
      }
    } else {  // down
      Part p;
      int item, a_count;
      if (t < b_down) {
        p = Part{0, a.T, a.T * a.k, true};
        item = t - b_down_s;
        a_count = a.E;
      } else {
        const int e = (t - b_down) / down_n;
        item = (t - b_down) - e * down_n;
        p = listed_part(a, sh, e);
        a_count = e;
      }
      const int need = p.shared ? up_s + (MXS ? 1 : 0) : up_r + (MXR ? 1 : 0);
      if (!wait_for(sh, ctl, up_count_at(a_count), need, a.err)) break;
      const int n0 = item * DC;
      if (p.rows > 0) {
        if (p.shared) {
          down_item<MBD, NBW, MXS>(a, a.shared, sh, p, n0, a.Is);
        } else if (!WIDE || p.rows <= 16) {
          down_item<MBD, 1, MXR>(a, a.routed, sh, p, n0, a.I);
        } else {
          down_item<MBD, NBW, MXR>(a, a.routed, sh, p, n0, a.I);
        }
      }
      if (signal(sh, ctl + down_count_at(a.E, item)) == sh.n_active) {  // every active expert, and the shared one
        acquire();
        combine_block<DC>(a, sh, n0);
      }
    }
    __syncthreads();
    if (tid == 0) sh.next = next;
    __syncthreads();
  }

  // the last workgroup to leave clears the counters
  __syncthreads();
  if (tid == 0) sh.flag = __hip_atomic_fetch_add(ctl + kExit, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (sh.flag == static_cast<int>(gridDim.x) - 1) {
    const int n = down_count_at(a.E, a.D / 16);
    for (int i = tid; i < n; i += kThreads)
      __hip_atomic_store(ctl + i, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

template <bool WIDE, bool MXR, bool MXS>
hipError_t run_few(const FewArgs& a, int grid, hipStream_t stream) {
  few_kernel<WIDE, MXR, MXS, 1, WIDE ? 1 : 2><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int few_ctl_ints(int E, int D) { return down_count_at(E, D / 16); }
int few_list_ints(int E, int routes) { return list_order(E) + routes; }

hipError_t launch_few(const FewArgs& args, bool mx_routed, bool mx_shared, hipStream_t stream) {
  FewArgs a = args;
  if (a.T < 1 || a.T > kFewTokens || a.k < 1 || a.k > 16 || a.E < a.k || a.E > 1024 || a.D % 64 || a.I % 64 ||
      a.Is % 64 || a.router.groups > kMaxGroups || a.E % a.router.groups)
    return hipErrorInvalidValue;
  if ((mx_routed || mx_shared) && a.D % 128) return hipErrorInvalidValue;
  if ((mx_routed && a.I % 128) || (mx_shared && a.Is % 128)) return hipErrorInvalidValue;
  a.router.group_size = a.E / a.router.groups;
  a.router.group_magic = (1u << 20) / static_cast<uint32_t>(a.router.group_size) + 1;  // exact for e < 1024
  const int64_t cus = device_compute_units();
  const int grid = static_cast<int>(kPerCu * (cus > 0 ? cus : 256));
  const bool wide = a.T > 16;
#define MOE_FEW(R, S) return wide ? run_few<true, R, S>(a, grid, stream) : run_few<false, R, S>(a, grid, stream)
  if (mx_routed && mx_shared) MOE_FEW(true, true);
  if (mx_routed) MOE_FEW(true, false);
  if (mx_shared) MOE_FEW(false, true);
  MOE_FEW(false, false);
#undef MOE_FEW
}

}  // namespace moe
