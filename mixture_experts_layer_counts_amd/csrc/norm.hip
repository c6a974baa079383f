// The norms, gate, dropout and residual sum around a layer, on gfx950
// (moe_block_norm and moe_block_norm_backward in include/moe.h):
//
//   z = x + scale gate drop(N(y) w_post),  h = N(z) w_pre,  N(v) = v / sqrt(mean v^2 + eps)
//
// Memory is the time: one pass over the rows.  A row stays in the registers of
// the threads that read it (8 or 16 values each, a wave to sixteen waves a row)
// between its sums and its results, and the next row's values are asked for
// before this row's sums.  The parameters stay in registers over the rows of a
// thread.  The backward needs no statistics from the forward: it reads z and y
// whole anyway, and forms their sums beside its own.  With a = w_pre dh:
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

// A 16-byte piece at any alignment of its elements.
struct __attribute__((packed, aligned(2))) Piece {
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
template <bool F32>
__device__ __forceinline__ void store8(void* row, int d, const float (&v)[8]) {
  char* const p = static_cast<char*>(row) + static_cast<int64_t>(d) * (F32 ? 4 : 2);
#pragma unroll
  for (int q = 0; q < (F32 ? 2 : 1); ++q) {
    Piece o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o.w[i] = F32 ? __float_as_uint(v[4 * q + i]) : pack_bf16x2(v[(2 * i) & 7], v[(2 * i + 1) & 7]);
    *reinterpret_cast<Piece*>(p + 16 * q) = o;
  }
}

// A thread's chunk of 8 columns.  The last chunk of a row ends with the row and
// so begins inside the one before, if D is no multiple of 8: its first `skip`
// values are that one's in the sums (both write them, the same bits).  Chunks
// past the row take no part (`there`), and read and write its last one's values.
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
// Which of the values d .. d + 7 of row t are kept, a bit each.
__device__ __forceinline__ uint32_t kept(const NormArgs& a, const uint64_t (&rng)[2], int64_t t, int d) {
  if (!a.drop) return 0xff;
  uint32_t bits = 0;
  const int quads = d & 3 ? 3 : 2;
#pragma unroll 1
  for (int q = 0; q < quads; ++q) {
    uint32_t w[4];
    philox(static_cast<uint32_t>(d / 4 + q), static_cast<uint32_t>(t), rng[1], rng[0], w);
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= (w[i] >= a.threshold ? 1u : 0u) << (4 * q + i);
  }
  return bits >> (d & 3);
}

// Sums over the `lanes` threads of a row (a power of two from 64 on), the same
// on all of them; `part`: one buffer for each of two reductions in a row.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float (*part)[16][4], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) v[n] += __shfl_xor(v[n], d);
  if (lanes == kWave) return;
  float (*const p)[4] = part[turn];
  turn ^= 1;
  const int wave = static_cast<int>(threadIdx.x) / kWave, first = wave / (lanes / kWave) * (lanes / kWave);
  if (lane_id() == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) p[wave][n] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.f;
  for (int w = 0; w < lanes / kWave; ++w) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += p[first + w][n];
  }
}

// A parameter's values with the weights' offset; 1 where there is none.
template <bool WF>
__device__ __forceinline__ float weight(bool there, const Raw<WF>& w, int i, float offset) {
  return there ? w.at(i) + offset : 1.f;
}

// CH chunks of 8 values a thread; rows are dealt to teams of a.lanes threads in turn.
template <bool XF, bool YF, bool WF, int CH>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
  __shared__ float part[2][16][4];
  int turn = 0;
  const int D = a.D, lanes = a.lanes, teams = static_cast<int>(blockDim.x) / lanes;
  const int team = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  Chunk d[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) d[c] = Chunk((c * lanes + lane) * 8, D);
  const float inv_d = 1.f / static_cast<float>(D);
  uint64_t rng[2] = {0, 0};
  if (a.drop) {
    rng[0] = a.rng[0];
    rng[1] = a.rng[1];
  }
  Raw<WF> wq[CH], wp[CH], g[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (a.post) wq[c] = load8<WF>(a.post, d[c].d);
    if (a.pre) wp[c] = load8<WF>(a.pre, d[c].d);
  }
  const char* const x = static_cast<const char*>(a.x);
  const char* const y = static_cast<const char*>(a.y);
  auto at = [&](int64_t t, bool f32) { return t * D * (f32 ? 4 : 2); };
  Raw<XF> xr[CH];
  Raw<YF> yr[CH];
  int64_t t = static_cast<int64_t>(blockIdx.x) * teams + team, group = -1;
  // every team of a block takes as many turns: they meet at the barriers
  int64_t turns = (a.T - static_cast<int64_t>(blockIdx.x) * teams + step - 1) / step;
  auto ask = [&](int64_t row) {
    const int64_t r = row < a.T ? row : a.T - 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      xr[c] = load8<XF>(x + at(r, XF), d[c].d);
      if (a.y) yr[c] = load8<YF>(y + at(r, YF), d[c].d);
    }
  };
  ask(t);
  for (; turns > 0; --turns, t += step) {
    const bool live = t < a.T;
    const int64_t row = live ? t : a.T - 1;
    if (a.gate && row / a.group != group) {
      group = row / a.group;
#pragma unroll
      for (int c = 0; c < CH; ++c) g[c] = load8<WF>(static_cast<const char*>(a.gate) + at(group, WF), d[c].d);
    }
    float z[CH][8], n[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[c][i] = xr[c].at(i);
        n[c][i] = a.y ? yr[c].at(i) : 0.f;
      }
    if (turns > 1) ask(t + step);
    if (a.y) {
      float r = 1.f;
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = i >= d[c].skip ? fmaf(n[c][i], n[c][i], s[0]) : s[0];
        row_sums(s, lanes, part, turn);
        r = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t keep = kept(a, rng, row, d[c].d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v = a.post ? n[c][i] * r * weight<WF>(true, wq[c], i, a.offset) : n[c][i];
          if (a.gate) v *= g[c].at(i);
          // (a dropped value adds nothing, whatever it was)
          z[c][i] = (keep >> i) & 1 ? fmaf(v, a.factor, z[c][i]) : z[c][i];
        }
      }
    }
    if (live && a.z) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (d[c].there) store8<XF>(static_cast<char*>(a.z) + at(row, XF), d[c].d, z[c]);
    }
    if (a.pre) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = i >= d[c].skip ? fmaf(z[c][i], z[c][i], s[0]) : s[0];
      row_sums(s, lanes, part, turn);
      const float r = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
      if (live) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = z[c][i] * r * weight<WF>(true, wp[c], i, a.offset);
          if (d[c].there) store8<false>(static_cast<char*>(a.h) + at(row, false), d[c].d, h);
        }
      }
    }
  }
}

// Teams take runs of a.run consecutive rows.  Their column sums go to
// a.parts: [runs][D] each of w_pre's and w_post's, and of the gate's groups that
// begin or end in another run [runs][2][D]: slot 0 for a group that the run
// begins with, slot 1 for one that goes on behind it.
template <bool XF, bool YF, bool WF, bool HF, int CH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const NormArgs a) {
  __shared__ float part[2][16][4];
  int turn = 0;
  const int D = a.D, lanes = a.lanes, teams = static_cast<int>(blockDim.x) / lanes;
  const int team = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * teams + team;
  Chunk d[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) d[c] = Chunk((c * lanes + lane) * 8, D);
  const float inv_d = 1.f / static_cast<float>(D);
  uint64_t rng[2] = {0, 0};
  if (a.drop) {
    rng[0] = a.rng[0];
    rng[1] = a.rng[1];
  }
  Raw<WF> wq[CH], wp[CH], g[CH];
  float dpre[CH][8], dpost[CH][8], dgate[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (a.post) wq[c] = load8<WF>(a.post, d[c].d);
    if (a.pre) wp[c] = load8<WF>(a.pre, d[c].d);
#pragma unroll
    for (int i = 0; i < 8; ++i) dpre[c][i] = dpost[c][i] = dgate[c][i] = 0.f;
  }
  auto at = [&](int64_t t, bool f32) { return t * D * (f32 ? 4 : 2); };
  const int64_t begin = id * a.run, end = begin + a.run < a.T ? begin + a.run : a.T;
  Raw<XF> zr[CH], dzr[CH];
  Raw<YF> yr[CH];
  Raw<HF> dhr[CH];
  auto ask = [&](int64_t t) {
    const int64_t r = t < a.T ? t : a.T - 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.pre) {
        zr[c] = load8<XF>(static_cast<const char*>(a.x) + at(r, XF), d[c].d);
        dhr[c] = load8<HF>(static_cast<const char*>(a.dh) + at(r, HF), d[c].d);
      }
      if (a.dz) dzr[c] = load8<XF>(static_cast<const char*>(a.dz) + at(r, XF), d[c].d);
      if (a.y) yr[c] = load8<YF>(static_cast<const char*>(a.y) + at(r, YF), d[c].d);
    }
  };
  auto put = [&](float* dst, float (&v)[CH][8]) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (d[c].there) store8<true>(dst, d[c].d, v[c]);
  };
  // the gate's sums of rows `from` .. `to` - 1 of group gr
  auto put_gate = [&](int64_t gr, int64_t from, int64_t to) {
    const bool whole = from == gr * a.group && to == (gr + 1) * a.group;
    float* const dst = whole ? a.dgate + gr * D : a.parts + (2 * a.runs + 2 * id + (from != begin)) * D;
    put(dst, dgate);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) dgate[c][i] = 0.f;
  };
  int64_t group = -1, group_from = begin;
  ask(begin);
  // (every team of the block takes a.run turns: they meet at the barriers)
  for (int64_t t = begin; t < begin + a.run; ++t) {
    const bool live = t < end;
    const int64_t row = live ? t : a.T - 1;
    if (a.gate && live && row / a.group != group) {
      if (group >= 0) put_gate(group, group_from, t);
      group = row / a.group;
      group_from = t;
#pragma unroll
      for (int c = 0; c < CH; ++c) g[c] = load8<WF>(static_cast<const char*>(a.gate) + at(group, WF), d[c].d);
    }
    // z and y stay as they are stored: their values are formed where they are used
    Raw<XF> z[CH];
    Raw<YF> y[CH];
    float dz[CH][8], b[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      z[c] = zr[c];
      y[c] = yr[c];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[c][i] = a.pre ? dhr[c].at(i) : 0.f;
        dz[c][i] = a.dz ? dzr[c].at(i) : 0.f;
      }
    }
    if (t + 1 < begin + a.run) ask(t + 1);
    float s[3] = {0.f, 0.f, 0.f};  // sum z^2, sum (w_pre dh) z, sum y^2
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < d[c].skip) continue;
        if (a.pre) {
          s[0] = fmaf(z[c].at(i), z[c].at(i), s[0]);
          s[1] = fmaf(b[c][i] * weight<WF>(true, wp[c], i, a.offset), z[c].at(i), s[1]);
        }
        if (a.post) s[2] = fmaf(y[c].at(i), y[c].at(i), s[2]);
      }
    row_sums(s, lanes, part, turn);
    const float ry = a.post ? 1.f / sqrtf(fmaf(s[2], inv_d, a.eps)) : 1.f;
    if (a.pre) {
      const float rz = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps)), m = s[1] * inv_d * rz * rz;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) dpre[c][i] = fmaf(b[c][i], z[c].at(i) * rz, dpre[c][i]);
          dz[c][i] = fmaf(rz, fmaf(-z[c].at(i), m, b[c][i] * weight<WF>(true, wp[c], i, a.offset)), dz[c][i]);
        }
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (d[c].there) store8<XF>(static_cast<char*>(a.dx) + at(row, XF), d[c].d, dz[c]);
    }
    if (!a.y) continue;
    float s2[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t keep = kept(a, rng, row, d[c].d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float dn = (keep >> i) & 1 ? dz[c][i] * a.factor : 0.f;
        const float w = weight<WF>(a.post, wq[c], i, a.offset), gv = a.gate ? g[c].at(i) : 1.f, n = y[c].at(i) * ry;
        // (a dropped value has no part in the sums, whatever it is)
        if (live && (keep >> i) & 1) {
          dgate[c][i] = fmaf(dn, n * w, dgate[c][i]);
          dpost[c][i] = fmaf(dn * gv, n, dpost[c][i]);
        }
        b[c][i] = dn * gv * w;
        s2[0] = i >= d[c].skip ? fmaf(b[c][i], y[c].at(i), s2[0]) : s2[0];
      }
    }
    if (a.post) {
      row_sums(s2, lanes, part, turn);
      const float m = s2[0] * inv_d * ry * ry;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] = ry * fmaf(-y[c].at(i), m, b[c][i]);
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (d[c].there) store8<YF>(static_cast<char*>(a.dy) + at(row, YF), d[c].d, b[c]);
    }
  }
  if (begin >= a.T) return;
  if (a.pre) put(a.parts + id * D, dpre);
  if (a.post) put(a.parts + (a.runs + id) * D, dpost);
  if (a.gate) put_gate(group, group_from, end);
}

// The runs' column sums, in their order: 64 columns a block, the runs in 16
// consecutive parts.  blockIdx.y: 0 w_pre, 1 w_post, 2 + g the gate's row g.
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
      for (int64_t i = lo; i < hi; ++i) s += src[(i == 0 ? 0 : first_step + (i - 1) * step) * a.D + col];
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

// Threads of a row, and of a block.
int lanes_of(int D) {
  int lanes = 64;
  while (lanes < 1024 && lanes * 8 < D) lanes *= 2;
  return lanes;
}
int block_of(int lanes) { return std::max(256, lanes); }

int64_t compute_units() {
  const int64_t cus = device_compute_units();
  return cus > 0 ? cus : 256;
}

}  // namespace

// Runs of the backward: as many as fill the chip once, of eight rows at least.
NormRuns norm_runs(int64_t T, int D) {
  const int lanes = lanes_of(D), teams = block_of(lanes) / lanes;
  const int64_t want = kNormWaves * kWave / lanes;
  const int64_t runs = std::max<int64_t>(1, std::min<int64_t>(want, (T + 7) / 8));
  NormRuns r;
  r.run = std::max<int64_t>(1, (T + runs - 1) / runs);
  r.runs = (T + r.run - 1) / r.run;
  r.blocks = (r.runs + teams - 1) / teams;
  return r;
}

#define MOE_TYPES(RUN)                                                      \
  do {                                                                      \
    const int key = (xf ? 4 : 0) | (yf ? 2 : 0) | (wf ? 1 : 0);             \
    switch (key) {                                                          \
      case 0: RUN(false, false, false); break;                              \
      case 1: RUN(false, false, true); break;                               \
      case 2: RUN(false, true, false); break;                               \
      case 3: RUN(false, true, true); break;                                \
      case 4: RUN(true, false, false); break;                               \
      case 5: RUN(true, false, true); break;                                \
      case 6: RUN(true, true, false); break;                                \
      default: RUN(true, true, true); break;                                \
    }                                                                       \
  } while (0)

hipError_t launch_norm(const NormArgs& args, bool xf, bool yf, bool wf, hipStream_t stream) {
  NormArgs a = args;
  if (a.T <= 0) return hipSuccess;
  if (a.D < 8 || a.D > kNormWidth) return hipErrorInvalidValue;
  a.lanes = lanes_of(a.D);
  const int block = block_of(a.lanes), teams = block / a.lanes;
  const int grid = static_cast<int>(std::min<int64_t>((a.T + teams - 1) / teams, compute_units() * (2048 / block)));
#define MOE_RUN(X, Y, W)                                                              \
  (a.lanes * 8 >= a.D ? norm_kernel<X, Y, W, 1> : norm_kernel<X, Y, W, 2>)<<<grid, block, 0, stream>>>(a)
  MOE_TYPES(MOE_RUN);
#undef MOE_RUN
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& args, bool xf, bool yf, bool wf, bool hf, hipStream_t stream) {
  NormArgs a = args;
  if (a.D < 8 || a.D > kNormWidth || a.T < 0) return hipErrorInvalidValue;
  const NormRuns r = norm_runs(a.T, a.D);
  a.lanes = lanes_of(a.D);
  a.run = r.run;
  a.runs = r.runs;
  if (a.T > 0) {
    const int block = block_of(a.lanes), grid = static_cast<int>(r.blocks);
#define MOE_RUN(X, Y, W)                                                                                        \
  (hf ? (a.lanes * 8 >= a.D ? norm_backward_kernel<X, Y, W, true, 1> : norm_backward_kernel<X, Y, W, true, 2>)  \
      : (a.lanes * 8 >= a.D ? norm_backward_kernel<X, Y, W, false, 1> : norm_backward_kernel<X, Y, W, false, 2>)) \
      <<<grid, block, 0, stream>>>(a)
    MOE_TYPES(MOE_RUN);
#undef MOE_RUN
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.pre && !a.post && !a.gate) return hipSuccess;
  const dim3 grid((a.D + 63) / 64, static_cast<unsigned>(std::min<int64_t>(2 + a.groups, 1024)));
  norm_columns_kernel<<<grid, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
