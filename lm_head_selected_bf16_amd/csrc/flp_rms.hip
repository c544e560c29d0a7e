// The norms around a model's block, root mean square ones, forward and backward:
//
//   p = y              or  y rstd(y) post_weight          (y: the block's output)
//   r = x + scale gate p                                  (x: the residual stream)
//   n = r rstd(r) weight                                  (what the next block reads)
//
// with rstd(v) = 1 / sqrt(sum_d v_d^2 / D + eps); without y, r = x.  The backward takes the
// gradients of r and n:
//
//   gw  = grad_n weight,   d_r = grad_r + rstd (gw - rhat mean_d(gw rhat)),   rhat = r rstd
//   d_x = d_r,  d_weight = sum_i grad_n rhat,  d_gate = sum scale d_r p  over a gate's rows
//   g   = scale gate d_r post_weight,  d_y = rstd_y (g - yhat mean_d(g yhat)),  yhat = y rstd_y
//   d_post_weight = sum_i scale gate d_r yhat
//
// All arithmetic is fp32 and every output is rounded once: n comes from r before its
// rounding, and the backward makes that r again from x and y instead of reading the rounded
// one.
//
// Bound by memory: the forward reads x and y and writes r and n, the backward reads both
// gradients, x and y and writes d_x and d_y; every row is read once and held in registers.
// Measured, 16384 x 2688 bf16 with both norms and a gate: forward 70 us (5.0 TB/s), backward 119
// (4.4 TB/s: its 194 registers leave room for one workgroup per compute unit, and the 256 slabs
// give it no more) and the fold 6, a gate for each row 103, 176 and 5; 4097 x 1345 fp16 with fp32
// parameters and 17 gates 20, 27 and 8.  Wider rows of the same 134 MB a tensor, forward and backward:
// 4096 bf16 93 and 183 us, fp32 103 and 165; 8192 bf16 104 and 175, fp32 112 and 172; 16384 bf16 106
// and 193 (28 bytes of a thread spilled); 4096 rows of 16384 fp32 (268 MB) 203 and 488, 3.3 TB/s (212
// bytes spilled).
//
// A row's sums run in an order fixed by D and the type alone, so r, n, d_x, d_y and the
// statistics of a row are bitwise the same whatever the other rows are.  The sums over rows
// run in slabs: within a slab each of its teams adds every k-th row in ascending order, the
// teams are joined in order, and over the slabs thirty-two sums of every 32nd slab are
// joined by a fixed tree.  N, D, the number of gates and the type fix the order: no atomics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "flp_launch.h"
#include "flp_row.h"

namespace flp {
namespace {

// A row belongs to a team of one wave, of four or of eight, in the backward of two too (by_width_*
// below).
constexpr int kThreads = 512;
// Workgroups of a forward launch: two for each compute unit, in turn (16384 x 2688 bf16 with y: 256 of them 74 us,
// 512 and 768 74 to 76, 1024 78, 2048 82; 16384 x 512 fp32: 23.4, 22.5, 22.6, 23.9, 28.3).
constexpr int64_t kFwdGroups = 512;

// Sum over the team, the same bits in every thread.  A team of several waves meets in LDS
// (`red`: a float per wave of the workgroup, another slot for each call of a row, and other
// ones for the next row).
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float* red) {
  x = wave_sum(x);
  if constexpr (TEAM == 64) return x;
  constexpr int kWaves = TEAM / 64;
  const int wave = threadIdx.x >> 6, first = wave & ~(kWaves - 1);
  if ((threadIdx.x & 63) == 0) red[wave] = x;
  __syncthreads();
  if constexpr (kWaves == 2) return red[first] + red[first + 1];
  float s = (red[first] + red[first + 1]) + (red[first + 2] + red[first + 3]);
  if constexpr (kWaves == 8)
    s += (red[first + 4] + red[first + 5]) + (red[first + 6] + red[first + 7]);
  return s;
}

// Whether a sum of squares says nothing, or little, of the row: it left fp32's middle range, and
// at the low end eps does not cover that.
__device__ __forceinline__ bool off_range(float s, float eps) {
  return !(s < 0x1p120f) || (s < 0x1p-60f && eps < 0x1p-30f);
}

// 1 / sqrt(mean of squares + eps) of a team's row, from the thread's part of the sum of squares.
// each(f) calls f with every value of the thread.  Rows whose squares leave fp32 (values above
// 1e18, or below 1e-9 with next to no eps) are summed again in units of a power of two near their
// largest value, a rare turn that all teams of the workgroup take together, since it has barriers.
template <int TEAM, class Each>
__device__ __forceinline__ float rstd_of(float part, float inv, float eps, float (*red)[8],
                                         Each each) {
  const float s = team_sum<TEAM>(part, red[0]);
  const bool mine = off_range(s, eps);
  bool any = mine;
  if constexpr (TEAM == 256)  // both teams' sums stand in LDS
    any = off_range((red[0][0] + red[0][1]) + (red[0][2] + red[0][3]), eps) ||
          off_range((red[0][4] + red[0][5]) + (red[0][6] + red[0][7]), eps);
  const float rstd = 1.0f / sqrtf(s * inv + eps);
  if (!any) return rstd;
  float top = sqrtf(eps);
  each([&](float v) { top = fmaxf(top, fabsf(v)); });
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
  if constexpr (TEAM > 64) {
    const int wave = threadIdx.x >> 6, first = wave & ~(TEAM / 64 - 1);
    if ((threadIdx.x & 63) == 0) red[1][wave] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TEAM / 64; ++k) top = fmaxf(top, red[1][first + k]);
  }
  // the inverse of its power of two, or the normal value nearest to that; 1 for a row of zeros,
  // infinities or NaN
  const int e = int(__float_as_uint(top) >> 23);
  const float c = top == 0.f || e == 255
                      ? 1.0f : __uint_as_float(uint32_t(max(min(254 - e, 253), 1)) << 23);
  float q = 0.f;
  each([&](float v) { q = fmaf(v * c, v * c, q); });
  q = team_sum<TEAM>(q, red[2]);
  return mine ? c / sqrtf(q * inv + eps * c * c) : rstd;
}

// The gate row of a row of x.
__device__ __forceinline__ int64_t gate_of(int64_t row, int64_t rows_per_gate, int64_t N) {
  if (N <= 0xFFFFFFFFll) return int64_t(uint32_t(row) / uint32_t(rows_per_gate));
  return row / rows_per_gate;
}

// The factors of a row as fp32 in LDS, in two planes (the chunks' first and second four
// elements) so that a wave's 16-byte reads are contiguous: lds[0, 2 plane) holds weight (1
// where it is absent), the next two planes scale gate post_weight, without the gate where
// gate is null.
template <class T>
__device__ __forceinline__ void stage_factors(f32x4* lds, int plane, const void* weight,
                                              const void* post_weight, const void* gate,
                                              float scale, bool branch, bool wide, int64_t D) {
  for (int c = threadIdx.x; c < plane; c += kThreads) {
    const int64_t d = int64_t(c) * kChunk, n = D - d;
    float w[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) w[e] = 1.0f;
    if (weight != nullptr) load_params<T>(weight, wide, d, n, w);
    lds[c] = f32x4{w[0], w[1], w[2], w[3]};
    lds[plane + c] = f32x4{w[4], w[5], w[6], w[7]};
    if (!branch) continue;
    float f[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) f[e] = scale;
    if (post_weight != nullptr) {
      load_params<T>(post_weight, wide, d, n, w);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] *= w[e];
    }
    if (gate != nullptr) {  // last, as where a row's gate is read with it: the same bits
      load_params<T>(gate, wide, d, n, w);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] *= w[e];
    }
    lds[2 * plane + c] = f32x4{f[0], f[1], f[2], f[3]};
    lds[3 * plane + c] = f32x4{f[4], f[5], f[6], f[7]};
  }
}

// Y: there is a block's output.  GATES: every row has a gate row that is read with it (else
// the one gate row, if any, is among the factors in LDS).
//
// The workgroups stay and take rows in turn, the next rows in flight.
template <class T, int TEAM, int NCH, bool Y, bool GATES>
__global__ __launch_bounds__(kThreads) void k_rms_fwd(RmsFwdArgs p) {
  constexpr int kTeams = kThreads / TEAM;
  extern __shared__ f32x4 lds[];
  __shared__ float red[2][6][8];
  const int t = threadIdx.x % TEAM;
  const int64_t D = p.D, step = int64_t(gridDim.x) * kTeams;
  const int plane = int((D + kChunk - 1) / kChunk);
  const float inv = 1.0f / float(D);
  const T* x = static_cast<const T*>(p.x);
  const T* y = static_cast<const T*>(p.y);
  int64_t row = int64_t(blockIdx.x) * kTeams + threadIdx.x / TEAM;
  int turn = 0;
  struct Rows {
    Row<T, TEAM, NCH> x, y;
  };
  auto load = [&](Rows& to, int64_t r) {
    to.x.load(x + r * D, D, t, r < p.N);
    if constexpr (Y) to.y.load(y + r * D, D, t, r < p.N);
  };
  auto work = [&](Rows& cur, Rows& nxt) {
    const bool live = row < p.N;
    load(nxt, row + step);
    float rstd_y = 1.0f;
    if (Y && p.post) {  // uniform over the launch
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          const float v = to_f32(T(cur.y.c[k].v[e]));
          q = fmaf(v, v, q);
        }
        s += q;
      }
      rstd_y = rstd_of<TEAM>(s, inv, p.eps, red[turn], [&](auto f) {
#pragma unroll
        for (int k = 0; k < NCH; ++k)
#pragma unroll
          for (int e = 0; e < kChunk; ++e) f(to_f32(T(cur.y.c[k].v[e])));
      });
    }
    float r[NCH][kChunk];
    float s = 0.f;
    const int64_t gate_row = GATES ? gate_of(live ? row : 0, p.rows_per_gate, p.N) * D : 0;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      __builtin_amdgcn_sched_barrier(0);  // one chunk's factors at a time in registers
#pragma unroll
      for (int e = 0; e < kChunk; ++e) r[k][e] = to_f32(T(cur.x.c[k].v[e]));
      if (c >= plane) continue;
      if constexpr (Y) {
        const f32x4 f0 = lds[2 * plane + c], f1 = lds[3 * plane + c];
        float g[kChunk];
        if constexpr (GATES)
          load_params<T>(p.gate, p.wide, gate_row + int64_t(c) * kChunk, D - int64_t(c) * kChunk,
                         g);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          float f = e < 4 ? f0[e & 3] : f1[e & 3];
          if constexpr (GATES) f *= g[e];
          r[k][e] = fmaf(to_f32(T(cur.y.c[k].v[e])) * rstd_y, f, r[k][e]);
        }
      }
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) q = fmaf(r[k][e], r[k][e], q);
      s += q;
    }
    const float rstd = rstd_of<TEAM>(s, inv, p.eps, red[turn] + 3, [&](auto f) {
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int e = 0; e < kChunk; ++e) f(r[k][e]);
    });
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      __builtin_amdgcn_sched_barrier(0);
      if (c >= plane) continue;
      const f32x4 w0 = lds[c], w1 = lds[plane + c];
      const int64_t n = live ? D - int64_t(c) * kChunk : 0, at = row * D + int64_t(c) * kChunk;
      Chunk<T> o;
      if constexpr (Y) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) o.v[e] = T(r[k][e]);
        o.store(static_cast<T*>(p.out_r) + at, n);
      }
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        o.v[e] = T(r[k][e] * rstd * (e < 4 ? w0[e & 3] : w1[e & 3]));
      o.store(static_cast<T*>(p.out_n) + at, n);
    }
    if (t == 0 && live) {
      if (p.rstd != nullptr) p.rstd[row] = rstd;
      if (Y && p.post_rstd != nullptr) p.post_rstd[row] = rstd_y;
    }
    row += step;
    turn ^= 1;
  };
  Rows a, b;
  load(a, row);
  stage_factors<T>(lds, plane, p.weight, p.post_weight, GATES ? nullptr : p.gate, p.scale, Y,
                   p.wide, D);
  __syncthreads();
  // Every team of the workgroup makes every step (they share barriers): r0 is its first.
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < p.N; r0 += 2 * step) {
    work(a, b);
    if (r0 + step < p.N) work(b, a);
  }
}

// d_x, d_y, gates of their own (GATES), and the slab's partial sums: part[slab][0] of
// grad_n rhat, part[slab][1] of d_r yhat (times the rows' gates with GATES), from which the
// fold makes d_weight, d_post_weight and d_gate.  Every thread owns the same columns in
// every row of its slab, so the sums stay in its registers and the rows are read once.
template <class T, int TEAM, int NCH, bool Y, bool GATES>
__global__ __launch_bounds__(kThreads) void k_rms_bwd(RmsBwdArgs p) {
  constexpr int kTeams = kThreads / TEAM;
  extern __shared__ f32x4 lds[];
  __shared__ float red[2][2][8];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t D = p.D;
  const int plane = int((D + kChunk - 1) / kChunk);
  const float inv = 1.0f / float(D);
  // slabs lie within the rows of one gate
  const int64_t of = blockIdx.x / p.slabs_per_gate, in = blockIdx.x % p.slabs_per_gate;
  const int64_t r0 = of * p.rows_per_gate + in * p.slab_rows;
  const int64_t r1 = min(r0 + p.slab_rows, (of + 1) * p.rows_per_gate);
  float aw[NCH][kChunk], as[NCH][kChunk];
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int e = 0; e < kChunk; ++e) aw[k][e] = as[k][e] = 0.f;
  int turn = 0;
  int64_t row = r0 + team;
  Row<T, TEAM, NCH> cx, cy, cr, cn;
  float rstd, rstd_y;
  auto load = [&](int64_t r) {  // all but y
    const bool live = r < r1;
    cx.load(static_cast<const T*>(p.x) + r * D, D, t, live);
    cn.load(static_cast<const T*>(p.grad_n) + r * D, D, t, live && p.grad_n != nullptr);
    cr.load(static_cast<const T*>(p.grad_r) + r * D, D, t, live && p.grad_r != nullptr);
    rstd = live ? p.rstd[r] : 0.f;
  };
  auto load_y = [&](int64_t r) {
    const bool live = r < r1;
    if constexpr (Y) cy.load(static_cast<const T*>(p.y) + r * D, D, t, live);
    rstd_y = !live ? 0.f : Y && p.post ? p.post_rstd[r] : 1.f;
  };
  load(row);
  load_y(row);
  const int64_t gate_bytes = (p.wide ? 4 : int64_t(sizeof(T))) * D;
  const void* gate = p.gate == nullptr || GATES
                         ? nullptr
                         : static_cast<const char*>(p.gate) + of * gate_bytes;
  stage_factors<T>(lds, plane, p.weight, p.post_weight, gate, p.scale, Y, p.wide, D);
  __syncthreads();
  for (int64_t first = r0; first < r1; first += kTeams) {
    const bool live = row < r1;
    // r (a chunk of it) and, with GATES, the gates of the row
    auto remake = [&](int k, int c, float (&f)[kChunk], float (&g)[kChunk], float (&r)[kChunk],
                      float (&yh)[kChunk]) {
      if constexpr (Y) {
        const f32x4 f0 = lds[2 * plane + c], f1 = lds[3 * plane + c];
        if constexpr (GATES) {
          load_params<T>(p.gate, p.wide, row * D + int64_t(c) * kChunk,
                         live ? D - int64_t(c) * kChunk : 0, g);
        }
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          f[e] = e < 4 ? f0[e & 3] : f1[e & 3];
          yh[e] = to_f32(T(cy.c[k].v[e])) * rstd_y;
          r[e] = fmaf(yh[e], GATES ? f[e] * g[e] : f[e], to_f32(T(cx.c[k].v[e])));
        }
      } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) r[e] = to_f32(T(cx.c[k].v[e]));
      }
    };
    float m2 = 0.f;
    if (p.grad_n != nullptr) {  // uniform over the launch
      float s2 = 0.f;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int c = k * TEAM + t;
        __builtin_amdgcn_sched_barrier(0);
        if (c >= plane) continue;  // past the row: zeros, and no factors
        float f[kChunk], g[kChunk], r[kChunk], yh[kChunk];
        remake(k, c, f, g, r, yh);
        const f32x4 w0 = lds[c], w1 = lds[plane + c];
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          const float gn = to_f32(T(cn.c[k].v[e])), rh = r[e] * rstd;
          aw[k][e] = fmaf(gn, rh, aw[k][e]);
          q = fmaf(gn * (e < 4 ? w0[e & 3] : w1[e & 3]), rh, q);
        }
        s2 += q;
      }
      m2 = team_sum<TEAM>(s2, red[turn][0]) * inv;
    }
    float dr[NCH][kChunk];
    float s3 = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      __builtin_amdgcn_sched_barrier(0);
      if (c >= plane) continue;
      float f[kChunk], g[kChunk], r[kChunk], yh[kChunk];
      remake(k, c, f, g, r, yh);
      const f32x4 w0 = lds[c], w1 = lds[plane + c];
      const int64_t n = live ? D - int64_t(c) * kChunk : 0, at = row * D + int64_t(c) * kChunk;
      Chunk<T> o;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) dr[k][e] = to_f32(T(cr.c[k].v[e]));
      if (p.grad_n != nullptr) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          const float gw = to_f32(T(cn.c[k].v[e])) * (e < 4 ? w0[e & 3] : w1[e & 3]);
          dr[k][e] = fmaf(rstd, fmaf(-(r[e] * rstd), m2, gw), dr[k][e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kChunk; ++e) o.v[e] = T(dr[k][e]);
      if (p.d_x != nullptr) o.store(static_cast<T*>(p.d_x) + at, n);
      if constexpr (Y) {
        float q = 0.f;
        if constexpr (GATES) {
          if (p.d_gate != nullptr) {
            float d[kChunk];
#pragma unroll
            for (int e = 0; e < kChunk; ++e) d[e] = dr[k][e] * f[e] * yh[e];
            if (p.wide || sizeof(T) == 4) {
              Chunk<float> ow;
#pragma unroll
              for (int e = 0; e < kChunk; ++e) ow.v[e] = d[e];
              ow.store(static_cast<float*>(p.d_gate) + at, n);
            } else {
#pragma unroll
              for (int e = 0; e < kChunk; ++e) o.v[e] = T(d[e]);
              o.store(static_cast<T*>(p.d_gate) + at, n);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          as[k][e] = fmaf(GATES ? dr[k][e] * g[e] : dr[k][e], yh[e], as[k][e]);
          dr[k][e] *= GATES ? f[e] * g[e] : f[e];
          q = fmaf(dr[k][e], yh[e], q);
        }
        s3 += q;
      }
    }
    load(row + kTeams);  // y's registers are the only ones still needed
    if (Y && p.d_y != nullptr) {
      float m3 = 0.f;
      if (p.post) m3 = team_sum<TEAM>(s3, red[turn][1]) * inv;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int c = k * TEAM + t;
        if (c >= plane) continue;
        const int64_t n = live ? D - int64_t(c) * kChunk : 0;
        Chunk<T> o;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          const float yh = to_f32(T(cy.c[k].v[e])) * rstd_y;
          o.v[e] = T(p.post ? rstd_y * fmaf(-yh, m3, dr[k][e]) : dr[k][e]);
        }
        o.store(static_cast<T*>(p.d_y) + row * D + int64_t(c) * kChunk, n);
      }
    }
    row += kTeams;
    turn ^= 1;
    load_y(row);
  }
  if (p.part == nullptr) return;
  // The teams' sums side by side in LDS, added in their order.
  float* out = p.part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
  for (int which = 0; which < (Y ? 2 : 1); ++which) {
    f32x4* mine = lds + team * 2 * plane;
    __syncthreads();  // what stands there has been read
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      if (c >= plane) continue;
      const float(&a)[kChunk] = which == 0 ? aw[k] : as[k];
      mine[c] = f32x4{a[0], a[1], a[2], a[3]};
      mine[plane + c] = f32x4{a[4], a[5], a[6], a[7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < plane; c += kThreads) {
      f32x4 v0 = lds[c], v1 = lds[plane + c];
#pragma unroll
      for (int j = 1; j < kTeams; ++j) {
        v0 += lds[j * 2 * plane + c];
        v1 += lds[j * 2 * plane + plane + c];
      }
      Chunk<float> o;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) o.v[e] = e < 4 ? v0[e & 3] : v1[e & 3];
      o.store(out + which * D + int64_t(c) * kChunk, D - int64_t(c) * kChunk);
    }
  }
}

// The sums over rows from the slab partials: what = 0 d_weight, 1 d_post_weight (and with one
// gate row, d_gate, which has the same sums), 2 + k row k of d_gate.  32 columns per workgroup,
// thirty-two threads per column each adding every 32nd slab in ascending order (eight loads in
// flight), then the thirty-two by a fixed tree.
constexpr int kFoldCols = 32, kFoldWays = 32;
template <class T>
__global__ __launch_bounds__(kFoldCols * kFoldWays) void k_rms_fold(RmsBwdArgs p, int64_t blocks,
                                                                    int64_t per) {
  __shared__ float s[kFoldWays][kFoldCols + 1];
  const int c = threadIdx.x % kFoldCols, q = threadIdx.x / kFoldCols;
  const bool one_gate = p.gate_rows == 1 && !p.gates;
  auto param = [&](const void* base, int64_t i) {
    return p.wide || sizeof(T) == 4 ? static_cast<const float*>(base)[i]
                                    : to_f32(static_cast<const T*>(base)[i]);
  };
  auto put = [&](void* out, int64_t at, float v) {
    if (out == nullptr) return;
    if (p.wide || sizeof(T) == 4)
      static_cast<float*>(out)[at] = v;
    else
      static_cast<T*>(out)[at] = T(v);
  };
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t what = b / per, d = (b % per) * kFoldCols + c;
    void* const out = what == 0 ? p.d_weight : what == 1 ? p.d_post_weight : p.d_gate;
    if (out == nullptr && !(what == 1 && one_gate && p.d_gate != nullptr)) continue;  // all of it
    const int64_t lo = what < 2 ? 0 : (what - 2) * p.slabs_per_gate;
    const int64_t hi = what < 2 ? p.slabs : lo + p.slabs_per_gate;
    // d_post_weight: each gate's sums times the gate (with a gate per row they hold it already)
    const bool gated = what == 1 && p.gate != nullptr && !p.gates && !one_gate;
    float a = 0.f;
    if (d < p.D) {
      const float* src = p.part + (what == 0 ? 0 : p.D) + d;
      for (int64_t k = lo + q; k < hi; k += 8 * kFoldWays) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t slab = k + kFoldWays * u;
          v[u] = slab < hi ? src[slab * 2 * p.D] : 0.f;
          if (gated && slab < hi) v[u] *= param(p.gate, int64_t(uint32_t(slab) / uint32_t(p.slabs_per_gate)) * p.D + d);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) a += v[u];
      }
    }
    __syncthreads();  // the values of the turn before have been read
    s[q][c] = a;
#pragma unroll
    for (int h = kFoldWays / 2; h >= 1; h >>= 1) {
      __syncthreads();
      if (q < h) s[q][c] += s[q + h][c];
    }
    if (q == 0 && d < p.D) {
      float v = s[0][c];
      if (what > 0) v *= p.scale;
      const float to_gate = p.post_weight != nullptr && p.d_gate != nullptr && what > 0
                                ? v * param(p.post_weight, d) : v;
      if (what == 1 && one_gate) {
        put(p.d_gate, d, to_gate);
        if (p.gate != nullptr) v *= param(p.gate, d);
      }
      if (what < 2)
        put(out, d, v);
      else
        put(out, (what - 2) * p.D + d, to_gate);
    }
  }
}

// f(TEAM, NCH) for the smallest instance that holds a row.  Forward: one wave holds up to six
// chunks per thread of a 16-bit row (three of an fp32 one), four and eight waves up to four.
template <class T, class F>
void by_width_fwd(int64_t D, F f) {
  using std::integral_constant;
  const int64_t chunks = (D + kChunk - 1) / kChunk;
  constexpr integral_constant<int, 64> w1{};
  constexpr integral_constant<int, 256> w4{};
  constexpr integral_constant<int, 512> w8{};
  if (chunks <= 64) return f(w1, integral_constant<int, 1>{});
  if (chunks <= 128) return f(w1, integral_constant<int, 2>{});
  if constexpr (sizeof(T) == 2) {
    if (chunks <= 256) return f(w1, integral_constant<int, 4>{});
    if (chunks <= 384) return f(w1, integral_constant<int, 6>{});
  } else {
    if (chunks <= 192) return f(w1, integral_constant<int, 3>{});
    if (chunks <= 256) return f(w4, integral_constant<int, 1>{});
  }
  if (chunks <= 512) return f(w4, integral_constant<int, 2>{});
  if (chunks <= 1024) return f(w4, integral_constant<int, 4>{});
  return f(w8, integral_constant<int, 4>{});
}

// Backward: four rows' chunks and two sums for each, so one wave holds up to four chunks per
// thread of a 16-bit row (six spill), three of an fp32 one, and two waves three.  (16384 x 2688
// bf16: one wave with six 139 us, two with three 127; 4097 x 1345 fp16: four waves 36, one 28.)
template <class T, class F>
void by_width_bwd(int64_t D, F f) {
  using std::integral_constant;
  const int64_t chunks = (D + kChunk - 1) / kChunk;
  constexpr integral_constant<int, 64> w1{};
  constexpr integral_constant<int, 128> w2{};
  constexpr integral_constant<int, 256> w4{};
  constexpr integral_constant<int, 512> w8{};
  if (chunks <= 64) return f(w1, integral_constant<int, 1>{});
  if (chunks <= 128) return f(w1, integral_constant<int, 2>{});
  if (chunks <= 192) return f(w1, integral_constant<int, 3>{});
  if (chunks <= 256)
    return f(integral_constant<int, sizeof(T) == 2 ? 64 : 128>{},
             integral_constant<int, sizeof(T) == 2 ? 4 : 2>{});
  if (chunks <= 384) return f(w2, integral_constant<int, 3>{});
  if (chunks <= 512) return f(w4, integral_constant<int, 2>{});
  if (chunks <= 1024) return f(w8, integral_constant<int, 2>{});
  return f(w8, integral_constant<int, 4>{});
}

// f(there is y, a gate row per row read with it).
template <class F>
void by_parts(bool y, bool gates, F f) {
  if (!y) return f(std::false_type{}, std::false_type{});
  if (!gates) return f(std::true_type{}, std::false_type{});
  return f(std::true_type{}, std::true_type{});
}

constexpr size_t lds_bytes(int64_t D, int planes) {
  return size_t((D + kChunk - 1) / kChunk) * kChunk * 4 * planes;
}

template <class T>
hipError_t rms_fwd(const RmsFwdArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  by_width_fwd<T>(a.D, [&](auto team, auto nch) {
    by_parts(a.y != nullptr, a.gates, [&](auto has_y, auto gates) {
      constexpr int kTeam = decltype(team)::value, kNch = decltype(nch)::value;
      constexpr bool kY = decltype(has_y)::value, kGates = decltype(gates)::value;
      constexpr int64_t kTeams = kThreads / kTeam;
      constexpr int kPlanes = kY ? 2 : 1;
      static std::atomic<int> ready[kMaxDevices];
      e = prepare(k_rms_fwd<T, kTeam, kNch, kY, kGates>,
                  lds_bytes(int64_t(kTeam) * kNch * kChunk, kPlanes), ready);
      if (e != hipSuccess) return;
      const int64_t grid = std::min<int64_t>((a.N + kTeams - 1) / kTeams, kFwdGroups);
      hipLaunchKernelGGL((k_rms_fwd<T, kTeam, kNch, kY, kGates>), dim3(unsigned(grid)),
                         dim3(kThreads), lds_bytes(a.D, kPlanes), s, a);
    });
  });
  return e != hipSuccess ? e : hipGetLastError();
}

template <class T>
hipError_t rms_bwd(const RmsBwdArgs& a, hipStream_t s) {
  if (a.slabs > 0) {
    hipError_t e = hipSuccess;
    by_width_bwd<T>(a.D, [&](auto team, auto nch) {
      by_parts(a.y != nullptr, a.gates, [&](auto has_y, auto gates) {
        constexpr int kTeam = decltype(team)::value, kNch = decltype(nch)::value;
        constexpr bool kY = decltype(has_y)::value, kGates = decltype(gates)::value;
        // the factors, then a sum per team
        constexpr int kPlanes = std::max(kY ? 2 : 1, kThreads / kTeam);
        static std::atomic<int> ready[kMaxDevices];
        e = prepare(k_rms_bwd<T, kTeam, kNch, kY, kGates>,
                    lds_bytes(int64_t(kTeam) * kNch * kChunk, kPlanes), ready);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL((k_rms_bwd<T, kTeam, kNch, kY, kGates>), dim3(unsigned(a.slabs)),
                           dim3(kThreads), lds_bytes(a.D, kPlanes), s, a);
      });
    });
    if (e != hipSuccess) return e;
  }
  const bool gate_sums = a.d_gate != nullptr && !a.gates;
  if (a.d_weight == nullptr && a.d_post_weight == nullptr && !gate_sums) return hipGetLastError();
  RmsBwdArgs b = a;
  if (!gate_sums) b.d_gate = nullptr;
  if (a.slabs == 0) b.gate = b.post_weight = nullptr;  // no rows: zeros, whatever they hold
  const int64_t per = (a.D + kFoldCols - 1) / kFoldCols, blocks = per * (2 + (gate_sums && a.gate_rows > 1 ? a.gate_rows : 0));
  hipLaunchKernelGGL(k_rms_fold<T>, dim3(unsigned(std::min<int64_t>(blocks, 1 << 16))),
                     dim3(kFoldCols * kFoldWays), 0, s, b, blocks, per);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_forward(flp_dtype x, flp_dtype w, const RmsFwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_RMS_NORM, s);
  RmsFwdArgs b = a;
  b.wide = w == FLP_F32;
  if (x == FLP_F32) return rms_fwd<float>(b, s);
  return x == FLP_BF16 ? rms_fwd<__bf16>(b, s) : rms_fwd<_Float16>(b, s);
}

hipError_t launch_rms_backward(flp_dtype x, flp_dtype w, const RmsBwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_RMS_NORM, s);
  RmsBwdArgs b = a;
  b.wide = w == FLP_F32;
  if (x == FLP_F32) return rms_bwd<float>(b, s);
  return x == FLP_BF16 ? rms_bwd<__bf16>(b, s) : rms_bwd<_Float16>(b, s);
}

}  // namespace flp
