// The norms, gate, dropout and residual sum around a layer, on gfx950
// (moe_block_norm and moe_block_norm_backward in include/moe.h):
//
//   z = x + scale gate drop(N(y) w_post),  h = N(z) w_pre,  N(v) = v / sqrt(mean v^2 + eps)
//
// One pass over the rows: a row stays in the registers of the threads that read
// it (8 or 16 values each, one to sixteen waves a row) between its sums and its
// results.  In the forward the parameters stay there too, and the next row's
// values are asked for before this row's sums: it runs at the rate of a copy
// (8192 x 7168, x fp32: 162 us, 4.3 TB/s; above 8192 columns, where 19 to 53 registers
// of a thread spill, 3.0: 4096 x 16384 in bf16 182 us).  In the backward vector
// arithmetic (one operation for every value of 8192 x 7168 takes 1.5 us) comes
// close to the memory's time; Philox's products alone are some 35 operations a
// value.  It needs no statistics from the forward: it reads z and y whole anyway,
// and forms their sums beside its own.  With a = w_pre dh:
//
//   dz' = dz + r_z (a - z r_z^2 mean(a z)),   r = 1 / sqrt(mean v^2 + eps)
//   dn = scale drop'(dz'),  dgate = sum_rows dn N(y) w_post,  b = dn gate w_post
//   dy = r_y (b - y r_y^2 mean(b y)),  dw_post = sum_rows dn gate y r_y,  dw_pre = sum_rows dh z r_z
//
// in two reductions (sum z^2, sum a z, sum y^2; then sum b y).  Column sums are
// kept in registers over a run of consecutive rows and met by a second kernel in
// the runs' order, so results repeat bit for bit.
//
// The dropout mask is never stored: element (t, d) is kept if word d % 4 of
// Philox-4x32 of ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011), at the counter (d / 4, t, offset) under
// the key (seed), is at least p 2^32; both passes form the words anew.
//
// Sums, statistics and column sums are fp32; h and z are rounded once each, and
// h is formed from z before it is rounded.

#include <algorithm>

#include "common.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

namespace {

// A 16-byte piece at any alignment of its elements, of rows that are also written
// by single elements.
struct __attribute__((packed, aligned(2), may_alias)) Piece {
  uint32_t w[4];
};

// 8 values of a row as they are stored: bf16 (F32 false) or fp32.
template <bool F32>
struct Raw {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};
// Values d .. d + 7 of a row.
template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* row, int d) {
  const char* const p = static_cast<const char*>(row) + static_cast<int64_t>(d) * (F32 ? 4 : 2);
  Raw<F32> r;
#pragma unroll
  for (int q = 0; q < (F32 ? 2 : 1); ++q) {
    const Piece v = *reinterpret_cast<const Piece*>(p + 16 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[4 * q + i] = v.w[i];
  }
  return r;
}
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
template <bool F32>
__device__ __forceinline__ void store8(void* row, int d, const float (&v)[8]) {
  char* const p = static_cast<char*>(row) + static_cast<int64_t>(d) * (F32 ? 4 : 2);
#pragma unroll
  for (int q = 0; q < (F32 ? 2 : 1); ++q) {
    Piece o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32)
        o.w[i] = __float_as_uint(v[4 * q + i]);
      else  // the hardware's rounding to nearest even
        o.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[2 * i], v[2 * i + 1]}, bf16x2_t));
    }
    *reinterpret_cast<Piece*>(p + 16 * q) = o;
  }
}
// A parameter's values d .. d + 7, plus `offset`; 1 where there is none.
__device__ __forceinline__ void parameter(const void* p, int64_t row, int D, int d, bool f32, float offset,
                                          float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.f;
  if (!p) return;
  if (f32) {
    const Raw<true> r = load8<true>(static_cast<const float*>(p) + row * D, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i) + offset;
  } else {
    const Raw<false> r = load8<false>(static_cast<const uint16_t*>(p) + row * D, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i) + offset;
  }
}

// A thread's chunk of 8 columns.  The last chunk of a row ends with the row and
// so begins inside the one before, if D is no multiple of 8 (TAIL): its first
// `skip` values are that one's in the sums (both write them, the same bits).
// Chunks past the row are not `there`: they read its last one's values.
struct Chunk {
  int d, skip;
  bool there;
  __device__ __forceinline__ Chunk() {}
  __device__ __forceinline__ Chunk(int first, int D) {
    there = first < D;
    d = first < D - 8 ? first : D - 8;
    skip = there ? first - d : 8;
  }
};
// sum of f(i) over a chunk's own values
template <bool TAIL, typename F>
__device__ __forceinline__ float own_sum(const Chunk& c, const F& f) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = f(i);
    s += !TAIL || i >= c.skip ? v : 0.f;
  }
  return TAIL || c.there ? s : 0.f;
}

// Philox-4x32-10.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint64_t offset, uint64_t seed, uint32_t (&out)[4]) {
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  out[0] = c0;
  out[1] = c1;
  out[2] = c2;
  out[3] = c3;
}
// Which of the values d .. d + 7 of row t are kept.
template <bool TAIL>
__device__ __forceinline__ void kept(const NormArgs& a, const uint64_t (&rng)[2], int64_t t, int d, bool (&keep)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) keep[i] = true;
  if (!a.drop) return;
  if constexpr (TAIL) {
    uint32_t bits = 0;
    const int quads = d & 3 ? 3 : 2;
#pragma unroll 1
    for (int q = 0; q < quads; ++q) {
      uint32_t w[4];
      philox(static_cast<uint32_t>(d / 4 + q), static_cast<uint32_t>(t), rng[1], rng[0], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) bits |= (w[i] >= a.threshold ? 1u : 0u) << (4 * q + i);
    }
    bits >>= d & 3;
#pragma unroll
    for (int i = 0; i < 8; ++i) keep[i] = (bits >> i) & 1;
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t w[4];
      philox(static_cast<uint32_t>(d / 4 + q), static_cast<uint32_t>(t), rng[1], rng[0], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) keep[4 * q + i] = w[i] >= a.threshold;
    }
  }
}

// Sums over the threads of a row, a wave or a whole workgroup, the same on all of
// them; `part`: one buffer for each of two reductions in a row.
constexpr int kMaxWaves = 16;
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float (*part)[kMaxWaves][4], int& turn) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], d);
  if (lanes == kWave) return;
  float (*const p)[4] = part[turn];
  turn ^= 1;
  if (lane_id() == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) p[threadIdx.x / kWave][n] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.f;
  for (int w = 0; w < lanes / kWave; ++w) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += p[w][n];
  }
}

// CH chunks of 8 values a thread; rows are dealt in turn to teams of a.lanes
// threads, a wave each or a whole workgroup.
template <bool XF, bool YF, int CH, bool TAIL>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
  __shared__ float part[2][kMaxWaves][4];
  int turn = 0;
  const int D = a.D, lanes = a.lanes, teams = static_cast<int>(blockDim.x) / lanes;
  const int team = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team;
  if (t >= a.T) return;  // (a team that meets at barriers is its workgroup)
  Chunk d[CH];
  float wq[CH][8], wp[CH][8], g[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    d[c] = Chunk((c * lanes + lane) * 8, D);
    parameter(a.post, 0, D, d[c].d, a.w_f32, a.offset, wq[c]);
    parameter(a.pre, 0, D, d[c].d, a.w_f32, a.offset, wp[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[c][i] = 1.f;
  }
  const float inv_d = 1.f / static_cast<float>(D);
  uint64_t rng[2] = {0, 0};
  if (a.drop) {
    rng[0] = a.rng[0];
    rng[1] = a.rng[1];
  }
  auto row_of = [&](const void* p, int64_t row, bool f32) { return static_cast<const char*>(p) + row * D * (f32 ? 4 : 2); };
  Raw<XF> xr[CH];
  Raw<YF> yr[CH];
  auto ask = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      xr[c] = load8<XF>(row_of(a.x, row, XF), d[c].d);
      if (a.y) yr[c] = load8<YF>(row_of(a.y, row, YF), d[c].d);
    }
  };
  ask(t);
  int64_t group = -1;
  for (; t < a.T; t += step) {
    if (a.gate && t / a.group != group) {
      group = t / a.group;
#pragma unroll
      for (int c = 0; c < CH; ++c) parameter(a.gate, group, D, d[c].d, a.w_f32, 0.f, g[c]);
    }
    float z[CH][8], n[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[c][i] = xr[c].at(i);
        n[c][i] = a.y ? yr[c].at(i) : 0.f;
      }
    if (t + step < a.T) ask(t + step);
    if (a.y) {
      float r = 1.f;
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) s[0] += own_sum<TAIL>(d[c], [&](int i) { return n[c][i] * n[c][i]; });
        row_sums(s, lanes, part, turn);
        r = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        bool keep[8];
        kept<TAIL>(a, rng, t, d[c].d, keep);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = n[c][i] * r * wq[c][i] * g[c][i];
          // (a dropped value adds nothing, whatever it was; with w_post it is part of r)
          z[c][i] = keep[i] ? fmaf(v, a.factor, z[c][i]) : z[c][i];
        }
      }
    }
    if (a.z) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (d[c].there) store8<XF>(static_cast<char*>(a.z) + t * D * (XF ? 4 : 2), d[c].d, z[c]);
    }
    if (a.pre) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c) s[0] += own_sum<TAIL>(d[c], [&](int i) { return z[c][i] * z[c][i]; });
      row_sums(s, lanes, part, turn);
      const float r = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = z[c][i] * r * wp[c][i];
        if (d[c].there) store8<false>(static_cast<char*>(a.h) + t * D * 2, d[c].d, h);
      }
    }
  }
}

// Teams take runs of a.run consecutive rows.  Their column sums go to
// a.parts: [runs][D] each of w_pre's and w_post's, and of the gate's groups that
// begin or end in another run [runs][2][D]: slot 0 for a group that the run
// begins with, slot 1 for one that goes on behind it.  Gate and w_post share
// their sum over the rows of a group, S = sum_t dn y r_y: dgate = w_post S, and
// the group adds gate S to dw_post.
//
// A row is one chain of loads, two reductions and stores, and a compute unit's
// registers hold one row of 7168 with sixteen waves: nothing is read ahead, and the
// parameters are read again from the caches for every row, so that little spills: 2
// to 12 registers a thread up to D = 8192, 8 in this case (8192 x 7168 in bf16, dh
// fp32, with dropout: 257 to 266 us in all; 405 with eight waves of 16 values a thread
// that kept parameters and the next row in registers).  Above 8192, with two chunks a
// thread, 71 to 112 spill: 4096 x 16384 takes 456 us, 2.1 TB/s, where 8192 x 8192
// reaches 3.5 (269 us).
template <bool XF, bool YF, bool HF, int CH, bool TAIL>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const NormArgs a) {
  __shared__ float part[2][kMaxWaves][4];
  int turn = 0;
  const int D = a.D, lanes = a.lanes, teams = static_cast<int>(blockDim.x) / lanes;
  const int team = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * teams + team;
  const int64_t begin = id * a.run, end = begin + a.run < a.T ? begin + a.run : a.T;
  if (begin >= a.T) return;  // (a team that meets at barriers is its workgroup)
  Chunk d[CH];
  float dpre[CH][8], S[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    d[c] = Chunk((c * lanes + lane) * 8, D);
#pragma unroll
    for (int i = 0; i < 8; ++i) dpre[c][i] = S[c][i] = 0.f;
  }
  const float inv_d = 1.f / static_cast<float>(D);
  uint64_t rng[2] = {0, 0};
  if (a.drop) {
    rng[0] = a.rng[0];
    rng[1] = a.rng[1];
  }
  auto row_of = [&](const void* p, int64_t row, bool f32) { return static_cast<const char*>(p) + row * D * (f32 ? 4 : 2); };
  // the group's sums of its rows `from` .. `to` - 1
  bool first_group = true;
  auto end_group = [&](int64_t group, int64_t from, int64_t to) {
    const bool whole = from == group * a.group && to == (group + 1) * a.group;
    float* const gate_dst = whole ? a.dgate + group * D : a.parts + (2 * a.runs + 2 * id + (from != begin)) * D;
    float* const post_dst = a.parts + (a.runs + id) * D;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float v[8], w[8];
      if (a.gate) {
        parameter(a.post, 0, D, d[c].d, a.w_f32, a.offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = S[c][i] * w[i];
        if (d[c].there) store8<true>(gate_dst, d[c].d, v);
      }
      if (a.post) {
        parameter(a.gate, group, D, d[c].d, a.w_f32, 0.f, w);
        if (first_group) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0.f;
        } else {
          const Raw<true> r = load8<true>(post_dst, d[c].d);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = r.at(i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(S[c][i], w[i], v[i]);
        if (TAIL && d[c].there && d[c].skip > 0) {  // the chunk before adds to the values that both have
#pragma unroll
          for (int i = 1; i < 8; ++i)
            if (i >= d[c].skip) post_dst[d[c].d + i] = v[i];
        } else if (d[c].there) {
          store8<true>(post_dst, d[c].d, v);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) S[c][i] = 0.f;
    }
    first_group = false;
  };
  int64_t group = a.gate ? begin / a.group : 0, group_from = begin;
  for (int64_t t = begin; t < end; ++t) {
    if (a.gate && t / a.group != group) {
      end_group(group, group_from, t);
      group = t / a.group;
      group_from = t;
    }
    Raw<XF> z[CH];
    Raw<YF> y[CH];
    float dz[CH][8], b[CH][8];
    float s[3] = {0.f, 0.f, 0.f};  // sum z^2, sum (w_pre dh) z, sum y^2
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[c][i] = b[c][i] = 0.f;
      if (a.dz) {
        const Raw<XF> r = load8<XF>(row_of(a.dz, t, XF), d[c].d);
#pragma unroll
        for (int i = 0; i < 8; ++i) dz[c][i] = r.at(i);
      }
      if (a.pre) {
        z[c] = load8<XF>(row_of(a.x, t, XF), d[c].d);
        const Raw<HF> r = load8<HF>(row_of(a.dh, t, HF), d[c].d);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] = r.at(i);
      }
      if (a.post || a.gate) {
        y[c] = load8<YF>(row_of(a.y, t, YF), d[c].d);
      } else {
#pragma unroll
        for (uint32_t& w : y[c].w) w = 0;  // dy does not depend on y
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.pre) {
        float w[8];
        parameter(a.pre, 0, D, d[c].d, a.w_f32, a.offset, w);
        s[0] += own_sum<TAIL>(d[c], [&](int i) { return z[c].at(i) * z[c].at(i); });
        s[1] += own_sum<TAIL>(d[c], [&](int i) { return b[c][i] * w[i] * z[c].at(i); });
      }
      if (a.post) s[2] += own_sum<TAIL>(d[c], [&](int i) { return y[c].at(i) * y[c].at(i); });
    }
    row_sums(s, lanes, part, turn);
    const float ry = a.post ? 1.f / sqrtf(fmaf(s[2], inv_d, a.eps)) : 1.f;
    if (a.pre) {
      const float rz = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps)), m = s[1] * inv_d * rz * rz;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float w[8];
        parameter(a.pre, 0, D, d[c].d, a.w_f32, a.offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dpre[c][i] = fmaf(b[c][i], z[c].at(i) * rz, dpre[c][i]);
          dz[c][i] = fmaf(rz, fmaf(-z[c].at(i), m, b[c][i] * w[i]), dz[c][i]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (d[c].there) store8<XF>(static_cast<char*>(a.dx) + t * D * (XF ? 4 : 2), d[c].d, dz[c]);
    if (!a.y) continue;
    float s2[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      bool keep[8];
      kept<TAIL>(a, rng, t, d[c].d, keep);
      float w[8], g[8];
      parameter(a.post, 0, D, d[c].d, a.w_f32, a.offset, w);
      parameter(a.gate, group, D, d[c].d, a.w_f32, 0.f, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float dn = dz[c][i] * a.factor, n = y[c].at(i) * ry;
        // (a dropped value has no part in these sums, whatever it is; in its row's
        // statistics, ry and m, it has, as the formulas say)
        S[c][i] = keep[i] ? fmaf(dn, n, S[c][i]) : S[c][i];
        b[c][i] = keep[i] ? dn * g[i] * w[i] : 0.f;
      }
      s2[0] += own_sum<TAIL>(d[c], [&](int i) { return b[c][i] * y[c].at(i); });
    }
    if (a.post) {
      row_sums(s2, lanes, part, turn);
      const float m = s2[0] * inv_d * ry * ry;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] = ry * fmaf(-y[c].at(i), m, b[c][i]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (d[c].there) store8<YF>(static_cast<char*>(a.dy) + t * D * (YF ? 4 : 2), d[c].d, b[c]);
  }
  end_group(group, group_from, end);
  if (a.pre) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (d[c].there) store8<true>(a.parts + id * D, d[c].d, dpre[c]);
  }
}

// The runs' column sums, in their order: 64 columns a block, the runs in 16
// consecutive parts.  blockIdx.y: 0 w_pre, 1 w_post, 2 + g the gate's row g.
// A few trips to memory bound it: with one load in flight a thread 10.5 and 9.5 us
// (777 x 1001, 8192 x 7168), with eight 7.1 and 7.8.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const NormArgs a) {
  __shared__ float sum[16][64];
  const int col = blockIdx.x * 64 + (static_cast<int>(threadIdx.x) & 63), slice = static_cast<int>(threadIdx.x) / 64;
  for (int64_t what = blockIdx.y; what < 2 + a.groups; what += gridDim.y) {
    if (what == 0 ? !a.pre : what == 1 ? !a.post : !a.gate) continue;
    float* dst;
    const float* src;
    int64_t n, first_step = 1, step = 1;  // rows of D: the first, how far to the second, and so on
    if (what < 2) {
      dst = what == 0 ? a.dpre : a.dpost;
      src = a.parts + what * a.runs * a.D;
      n = a.runs;
    } else {
      const int64_t g = what - 2, from = g * a.group, to = from + a.group;
      dst = a.dgate + g * a.D;
      const int64_t r0 = a.group ? from / a.run : 0, r1 = a.group ? (to - 1) / a.run : 0;
      if (a.group && r0 == r1) continue;  // its run has written it
      n = a.group ? r1 - r0 + 1 : 0;
      const int64_t slot = from == r0 * a.run ? 0 : 1;
      src = a.parts + (2 * a.runs + 2 * r0 + slot) * a.D;
      first_step = 2 - slot;
      step = 2;
    }
    const int64_t per = (n + 15) / 16, lo = slice * per, hi = lo + per < n ? lo + per : n;
    float s = 0.f;
    if (col < a.D) {
      for (int64_t i0 = lo; i0 < hi; i0 += 8) {  // the loads of eight runs side by side
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t i = i0 + j < hi ? i0 + j : hi - 1;
          v[j] = src[(i == 0 ? 0 : first_step + (i - 1) * step) * a.D + col];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j < hi) s += v[j];
      }
    }
    sum[slice][threadIdx.x & 63] = s;
    __syncthreads();
    if (slice == 0 && col < a.D) {
      for (int w = 1; w < 16; ++w) s += sum[w][threadIdx.x & 63];
      dst[col] = s;
    }
    __syncthreads();
  }
}

// Threads of a row, and of a workgroup.
int lanes_of(int D) {
  int lanes = 64;
  while (lanes < 64 * kMaxWaves && lanes * 8 < D) lanes *= 2;
  return lanes;
}
int block_of(int lanes) { return lanes == 64 ? 256 : lanes; }

int64_t compute_units() {
  const int64_t cus = device_compute_units();
  return cus > 0 ? cus : 256;
}

// The kernel for D: its chunks a thread (1 or 2), and whether its last one overlaps.
template <template <int, bool> class Run>
hipError_t by_width(const NormArgs& a, int grid, int block, hipStream_t stream) {
  const int chunks = (a.D + a.lanes * 8 - 1) / (a.lanes * 8);
  const bool tail = a.D % 8 != 0;
  if (chunks == 1 && !tail) return Run<1, false>::run(a, grid, block, stream);
  if (chunks == 1) return Run<1, true>::run(a, grid, block, stream);
  return Run<2, true>::run(a, grid, block, stream);
}

template <bool XF, bool YF>
struct Forward {
  template <int CH, bool TAIL>
  struct Run {
    static hipError_t run(const NormArgs& a, int grid, int block, hipStream_t stream) {
      norm_kernel<XF, YF, CH, TAIL><<<grid, block, 0, stream>>>(a);
      return hipGetLastError();
    }
  };
};
template <bool XF, bool YF, bool HF>
struct Backward {
  template <int CH, bool TAIL>
  struct Run {
    static hipError_t run(const NormArgs& a, int grid, int block, hipStream_t stream) {
      norm_backward_kernel<XF, YF, HF, CH, TAIL><<<grid, block, 0, stream>>>(a);
      return hipGetLastError();
    }
  };
};

}  // namespace

// Runs of the backward: as many as fill the chip, each of some rows where there
// are many (their column sums are written and read again).
NormRuns norm_runs(int64_t T, int D) {
  const int lanes = lanes_of(D), teams = block_of(lanes) / lanes;
  const int64_t want = kNormWaves * kWave / lanes;
  const int64_t runs = std::max<int64_t>(1, std::min<int64_t>(want, (T + 1) / 2));
  NormRuns r;
  r.run = std::max<int64_t>(1, (T + runs - 1) / runs);
  r.runs = (T + r.run - 1) / r.run;
  r.blocks = (r.runs + teams - 1) / teams;
  return r;
}

hipError_t launch_norm(const NormArgs& args, bool xf, bool yf, hipStream_t stream) {
  NormArgs a = args;
  if (a.T <= 0) return hipSuccess;
  if (a.D < 8 || a.D > kNormWidth) return hipErrorInvalidValue;
  a.lanes = lanes_of(a.D);
  const int block = block_of(a.lanes), teams = block / a.lanes;
  const int grid = static_cast<int>(std::min<int64_t>((a.T + teams - 1) / teams, compute_units() * (2048 / block)));
  if (xf) return yf ? by_width<Forward<true, true>::Run>(a, grid, block, stream)
                    : by_width<Forward<true, false>::Run>(a, grid, block, stream);
  return yf ? by_width<Forward<false, true>::Run>(a, grid, block, stream)
            : by_width<Forward<false, false>::Run>(a, grid, block, stream);
}

hipError_t launch_norm_backward(const NormArgs& args, bool xf, bool yf, bool hf, hipStream_t stream) {
  NormArgs a = args;
  if (a.D < 8 || a.D > kNormWidth || a.T < 0) return hipErrorInvalidValue;
  const NormRuns r = norm_runs(a.T, a.D);
  a.lanes = lanes_of(a.D);
  a.run = r.run;
  a.runs = r.runs;
  if (a.T > 0) {
    const int block = block_of(a.lanes), grid = static_cast<int>(r.blocks);
    hipError_t e;
#define MOE_RUN(X, Y, H) e = by_width<Backward<X, Y, H>::Run>(a, grid, block, stream)
    switch ((xf ? 4 : 0) | (yf ? 2 : 0) | (hf ? 1 : 0)) {
      case 0: MOE_RUN(false, false, false); break;
      case 1: MOE_RUN(false, false, true); break;
      case 2: MOE_RUN(false, true, false); break;
      case 3: MOE_RUN(false, true, true); break;
      case 4: MOE_RUN(true, false, false); break;
      case 5: MOE_RUN(true, false, true); break;
      case 6: MOE_RUN(true, true, false); break;
      default: MOE_RUN(true, true, true); break;
    }
#undef MOE_RUN
    if (e != hipSuccess) return e;
  }
  if (!a.pre && !a.post && !a.gate) return hipSuccess;
  const dim3 grid((a.D + 63) / 64, static_cast<unsigned>(std::min<int64_t>(2 + a.groups, 1024)));
  norm_columns_kernel<<<grid, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
