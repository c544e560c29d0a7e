// Layer norm over the last dimension, forward and backward.
//
//   mean_i = sum_d x_id / D,  rstd_i = 1 / sqrt(sum_d (x_id - mean_i)^2 / D + eps)
//   xhat   = (x - mean) rstd,  out = xhat w + b
//   d_x    = rstd (g - mean_d(g) - xhat mean_d(g xhat)),  g = grad w
//   d_w    = sum_i grad xhat,  d_b = sum_i grad
//
// All arithmetic is fp32; out, d_x, d_w and d_b are rounded once.  The variance comes from
// centred values, so a large common offset of a row does not cancel, and the mean is
// corrected by theirs (Centre): a sum of D values over D is off by some of its last
// places, which a row far from zero with little spread would show.
//
// Bound by memory: the forward reads x and writes out, the backward reads grad and x and
// writes d_x.
//
// A row's sums run in an order fixed by D alone, so out, mean, rstd and d_x of a
// row are bitwise the same whatever the other rows are.  d_w and d_b add rows in
// slabs cut by N alone.  Within a slab, each of its k teams or waves (k by D and the type:
// 8 or 2 teams, 4 waves for wide rows) adds every k-th row in ascending order, and the k
// sums are joined in a fixed order; over the slabs, sixteen sums of every sixteenth slab are
// joined by a fixed tree.  N, D and the type fix the order: no atomics, the same bits on
// every run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "flp_launch.h"
#include "flp_row.h"

namespace flp {
namespace {

// Mean and rstd of a row from a first mean m and the means u of x - m and q of (x - m)^2:
// x - m is exact where the offset is large, so m + u is the mean up to half a step, and a
// constant row has exactly its value as mean and no variance.
struct Centre {
  float mean, rstd;
  __device__ __forceinline__ Centre(float m, float u, float q, float eps) : mean(m + u) {
    const float d = fmaf(-u, u, q);
    const float var = d >= 0.f ? d : d < 0.f ? 0.f : q;  // neither: u^2 and q passed fp32
    rstd = 1.0f / sqrtf(var + eps);
  }
};

// ---- rows held in registers (up to kTeamMax elements) ------------------------------------------------
//
// A team of TEAM threads (one wave, or four) owns a row; thread t holds the chunks of
// eight elements t, t + TEAM, ... (at most NCH).  A row is read from memory once, with
// 16-byte loads that all stay in flight, and both its sums run over the registers.

// Sum over the team, the same bits in every thread.  A team of four waves meets in LDS
// (`red`: a float per wave of the workgroup, another slot on every call in turn).
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float* red) {
  x = wave_sum(x);
  if constexpr (TEAM == 64) return x;
  const int wave = threadIdx.x >> 6, first = wave & ~3;
  if ((threadIdx.x & 63) == 0) red[wave] = x;
  __syncthreads();
  return (red[first] + red[first + 1]) + (red[first + 2] + red[first + 3]);
}

// Two sums over a team of four waves, behind one barrier.
__device__ __forceinline__ void team_sum2(float& x, float& y, float (&red)[3][8]) {
  x = wave_sum(x);
  y = wave_sum(y);
  const int wave = threadIdx.x >> 6, first = wave & ~3;
  if ((threadIdx.x & 63) == 0) {
    red[1][wave] = x;
    red[2][wave] = y;
  }
  __syncthreads();
  x = (red[1][first] + red[1][first + 1]) + (red[1][first + 2] + red[1][first + 3]);
  y = (red[2][first] + red[2][first + 1]) + (red[2][first + 2] + red[2][first + 3]);
}

constexpr int kTeamThreads = 512;
// Workgroups of a forward launch: two per compute unit (256 and 1024 measured the same).
constexpr int64_t kFwdGroups = 512;

// A [D] parameter in LDS as fp32, in two planes (the chunks' first and second four
// elements) so that a wave's 16-byte reads are contiguous; `value` where it is absent.
template <class T>
__device__ __forceinline__ void stage_param(f32x4* lds, const void* base, bool wide, int64_t D,
                                            float value) {
  const int plane = int((D + kChunk - 1) / kChunk);
  for (int c = threadIdx.x; c < plane; c += kTeamThreads) {
    float w[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) w[e] = value;
    if (base != nullptr) load_params<T>(base, wide, int64_t(c) * kChunk, D - int64_t(c) * kChunk, w);
    lds[c] = f32x4{w[0], w[1], w[2], w[3]};
    lds[plane + c] = f32x4{w[4], w[5], w[6], w[7]};
  }
}

// The workgroups stay and take rows in turn: the parameters are staged in LDS once, and
// the next row is in flight while the current one is worked on.  16384 x 2688 bf16 on
// MI355X: 38 us for 176 MB (4.6 TB/s; one row per wave and launch took 46, with the
// parameters read from the caches).
template <class T, int TEAM, int NCH>
__global__ __launch_bounds__(kTeamThreads) void k_norm_fwd_row(NormFwdArgs p) {
  constexpr int kTeams = kTeamThreads / TEAM;
  extern __shared__ f32x4 lds[];
  __shared__ float red[2][3][8];
  const int t = threadIdx.x % TEAM;
  const int64_t D = p.D, step = int64_t(gridDim.x) * kTeams;
  const int plane = int((D + kChunk - 1) / kChunk);
  const float inv = 1.0f / float(D);
  const T* x = static_cast<const T*>(p.x);
  int64_t row = int64_t(blockIdx.x) * kTeams + threadIdx.x / TEAM;
  int turn = 0;
  auto work = [&](Row<T, TEAM, NCH>& cur, Row<T, TEAM, NCH>& nxt) {
    const bool live = row < p.N;
    nxt.load(x + (row + step) * D, D, t, row + step < p.N);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) q += to_f32(T(cur.c[k].v[e]));
      s += q;
    }
    const float m = team_sum<TEAM>(s, red[turn][0]) * inv;
    // the thread's part of the sums q of the centred values' squares and u of the values
    float q = 0.f, u = 0.f;
    auto centred = [&](auto squares, auto values) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int64_t n = D - int64_t(k * TEAM + t) * kChunk;
        float cq = 0.f, cu = 0.f;
        auto add = [&](float v) {
          if constexpr (decltype(squares)::value) cq = fmaf(v, v, cq);
          if constexpr (decltype(values)::value) cu += v;
        };
        if (n >= kChunk) {
#pragma unroll
          for (int e = 0; e < kChunk; ++e) add(to_f32(T(cur.c[k].v[e])) - m);
        } else if (n > 0) {
#pragma unroll
          for (int e = 0; e < kChunk; ++e) add(e < n ? to_f32(T(cur.c[k].v[e])) - m : 0.f);
        }
        q += cq;
        u += cu;
      }
    };
    // One wave corrects its mean only where that is four times the spread or more: below, a
    // sum's relative rounding moves xhat by at most five times itself (the size above takes
    // 36.7 us, 37.7 with all rows corrected, 35.5 with none).  A team of four waves always
    // does, behind the barrier of the squares (4096 x 8192 bf16 27.2 us, 26.5 without the
    // correction; behind a barrier of its own 34).
    if constexpr (TEAM == 64) {
      centred(std::true_type{}, std::false_type{});
      q = wave_sum(q) * inv;
      if (!(m * m < 16.0f * q)) {
        centred(std::false_type{}, std::true_type{});
        u = wave_sum(u) * inv;
      }
    } else {
      centred(std::true_type{}, std::true_type{});
      team_sum2(u, q, red[turn]);
      u *= inv;
      q *= inv;
    }
    const Centre at(m, u, q, p.eps);
    const float mean = at.mean, rstd = at.rstd;
    T* out = static_cast<T*>(p.out) + row * D;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      __builtin_amdgcn_sched_barrier(0);  // one chunk's parameters at a time in registers
      if (c >= plane) continue;
      const f32x4 w0 = lds[c], w1 = lds[plane + c];
      const f32x4 b0 = lds[2 * plane + c], b1 = lds[3 * plane + c];
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        cur.c[k].v[e] = T(fmaf((to_f32(T(cur.c[k].v[e])) - mean) * rstd,
                               e < 4 ? w0[e & 3] : w1[e & 3], e < 4 ? b0[e & 3] : b1[e & 3]));
      cur.c[k].store(out + int64_t(c) * kChunk, live ? D - int64_t(c) * kChunk : 0);
    }
    if (t == 0 && live) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    row += step;
    turn ^= 1;
  };
  Row<T, TEAM, NCH> a, b;
  a.load(x + row * D, D, t, row < p.N);
  stage_param<T>(lds, p.weight, p.wide, D, 1.0f);
  stage_param<T>(lds + 2 * plane, p.bias, p.wide, D, 0.0f);
  __syncthreads();
  // Every team of the workgroup makes every step (they share barriers): r0 is its first.
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < p.N; r0 += 2 * step) {
    work(a, b);
    if (r0 + step < p.N) work(b, a);
  }
}

// d_x, and the slab's partial d_w and d_b.  Every thread owns the same columns in every
// row of its slab, so the parameter sums stay in its registers and the rows are read
// once.  16384 x 2688 bf16 on MI355X: 57 us for 264 MB (4.7 TB/s; a large copy reaches
// 4.9).  Loading the next row ahead as the forward does spills (72 us against 64 at the
// time); teams in workgroups of 256 threads took 70.
template <class T, int TEAM, int NCH>
__global__ __launch_bounds__(kTeamThreads) void k_norm_bwd_row(NormBwdArgs p) {
  constexpr int kTeams = kTeamThreads / TEAM;
  extern __shared__ f32x4 lds[];
  __shared__ float red[2][2][8];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t D = p.D;
  const int plane = int((D + kChunk - 1) / kChunk);
  const float inv = 1.0f / float(D);
  const int64_t r1 = min(p.N, (int64_t(blockIdx.x) + 1) * p.slab_rows);
  const T* x = static_cast<const T*>(p.x);
  const T* g = static_cast<const T*>(p.grad);
  int64_t row = int64_t(blockIdx.x) * p.slab_rows + team;
  float aw[NCH][kChunk], ab[NCH][kChunk];
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int e = 0; e < kChunk; ++e) aw[k][e] = ab[k][e] = 0.f;
  int turn = 0;
  Row<T, TEAM, NCH> cx, cg;
  float mean, rstd;
  auto load = [&] {
    const bool live = row < r1;
    cx.load(x + row * D, D, t, live);
    cg.load(g + row * D, D, t, live);
    mean = live ? p.mean[row] : 0.f;
    rstd = live ? p.rstd[row] : 0.f;
  };
  load();
  stage_param<T>(lds, p.weight, p.wide, D, 1.0f);
  __syncthreads();
  for (int64_t r0 = int64_t(blockIdx.x) * p.slab_rows; r0 < r1; r0 += kTeams) {
    const bool live = row < r1;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      __builtin_amdgcn_sched_barrier(0);
      if (c >= plane) continue;  // past the row: zeros, and no weight
      const f32x4 w0 = lds[c], w1 = lds[plane + c];
      float q1 = 0.f, q2 = 0.f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        const float gr = to_f32(T(cg.c[k].v[e]));
        const float xh = (to_f32(T(cx.c[k].v[e])) - mean) * rstd;
        const float gw = gr * (e < 4 ? w0[e & 3] : w1[e & 3]);
        q1 += gw;
        q2 = fmaf(gw, xh, q2);
        aw[k][e] = fmaf(gr, xh, aw[k][e]);
        ab[k][e] += gr;
      }
      s1 += q1;
      s2 += q2;
    }
    if (p.d_x != nullptr) {  // uniform over the launch
      const float m1 = team_sum<TEAM>(s1, red[turn][0]) * inv;
      const float m2 = team_sum<TEAM>(s2, red[turn][1]) * inv;
      // d_x = rstd (gw - m1 - (x - mean) rstd m2): no factor rstd^2, which passes fp32 for
      // rows that rstd itself, and d_x, can still take (a spread of 2^-65 with eps = 0)
      const float a = -(rstd * m2);
      T* dx = static_cast<T*>(p.d_x) + row * D;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int c = k * TEAM + t;
        __builtin_amdgcn_sched_barrier(0);
        if (c >= plane) continue;
        const f32x4 w0 = lds[c], w1 = lds[plane + c];
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          const float xc = to_f32(T(cx.c[k].v[e])) - mean;
          const float gw = to_f32(T(cg.c[k].v[e])) * (e < 4 ? w0[e & 3] : w1[e & 3]);
          cx.c[k].v[e] = T(rstd * fmaf(xc, a, gw - m1));
        }
        cx.c[k].store(dx + int64_t(c) * kChunk, live ? D - int64_t(c) * kChunk : 0);
      }
    }
    row += kTeams;
    turn ^= 1;
    load();
  }
  if (p.part == nullptr) return;
  // The teams' sums side by side in LDS, added in their order: first those of d_w, then
  // those of d_b (team after team through one copy: 64 us instead of 57 in all).
  float* out = p.part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    f32x4* mine = lds + team * 2 * plane;
    __syncthreads();  // what stands there has been read
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int c = k * TEAM + t;
      if (c >= plane) continue;
      const float(&a)[kChunk] = which == 0 ? aw[k] : ab[k];
      mine[c] = f32x4{a[0], a[1], a[2], a[3]};
      mine[plane + c] = f32x4{a[4], a[5], a[6], a[7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < plane; c += kTeamThreads) {
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

// ---- wider rows ----------------------------------------------------------------------------------

constexpr int kRowThreads = 256;

// Sum of v over the workgroup, the same bits in every thread: xor butterfly inside
// each wave, then the four waves in order.  `red` holds one float per wave.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  __syncthreads();  // the previous call's values have been read
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// One workgroup per row: the row is read three times (mean, variance, output); only the
// first read reaches HBM.
template <class T, class W>
__global__ __launch_bounds__(kRowThreads) void k_norm_fwd(NormFwdArgs p) {
  __shared__ float red[4];
  const W* w = static_cast<const W*>(p.weight);
  const W* b = static_cast<const W*>(p.bias);
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.D;
    T* out = static_cast<T*>(p.out) + row * p.D;
    float s = 0.f;
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) s += to_f32(x[d]);
    const float m = block_sum(s, red) / float(p.D);
    float u = 0.f, q = 0.f;
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) {
      const float c = to_f32(x[d]) - m;
      u += c;
      q = fmaf(c, c, q);
    }
    u = block_sum(u, red) / float(p.D);
    const Centre at(m, u, block_sum(q, red) / float(p.D), p.eps);
    const float mean = at.mean, rstd = at.rstd;
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) {
      float y = (to_f32(x[d]) - mean) * rstd;
      if (w != nullptr) y *= to_f32(w[d]);
      if (b != nullptr) y += to_f32(b[d]);
      out[d] = T(y);
    }
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
  }
}

template <class T, class W>
__global__ __launch_bounds__(kRowThreads) void k_norm_dx(NormBwdArgs p) {
  __shared__ float red[4];
  const W* w = static_cast<const W*>(p.weight);
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.D;
    const T* g = static_cast<const T*>(p.grad) + row * p.D;
    T* dx = static_cast<T*>(p.d_x) + row * p.D;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) {
      const float gw = to_f32(g[d]) * (w != nullptr ? to_f32(w[d]) : 1.0f);
      s1 += gw;
      s2 = fmaf(gw, (to_f32(x[d]) - mean) * rstd, s2);
    }
    const float m1 = block_sum(s1, red) / float(p.D);
    const float m2 = block_sum(s2, red) / float(p.D);
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) {
      const float gw = to_f32(g[d]) * (w != nullptr ? to_f32(w[d]) : 1.0f);
      const float xhat = (to_f32(x[d]) - mean) * rstd;
      dx[d] = T(rstd * (gw - m1 - xhat * m2));
    }
  }
}

// Slab partials of d_w and d_b: part[slab][0][D] and part[slab][1][D].  64 columns
// per workgroup; each of its four waves adds every fourth row of the slab, then
// the waves are added in order.
template <class T>
__global__ __launch_bounds__(256) void k_norm_params(NormBwdArgs p) {
  __shared__ float sw[4][64], sb[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t d = int64_t(blockIdx.x) * 64 + lane;
  const int64_t r1 = min(p.N, (int64_t(blockIdx.y) + 1) * p.slab_rows);
  float aw = 0.f, ab = 0.f;
  if (d < p.D) {
    for (int64_t r = int64_t(blockIdx.y) * p.slab_rows + wave; r < r1; r += 4) {
      const float g = to_f32(static_cast<const T*>(p.grad)[r * p.D + d]);
      const float x = to_f32(static_cast<const T*>(p.x)[r * p.D + d]);
      aw = fmaf(g, (x - p.mean[r]) * p.rstd[r], aw);
      ab += g;
    }
  }
  sw[wave][lane] = aw;
  sb[wave][lane] = ab;
  __syncthreads();
  if (wave == 0 && d < p.D) {
    float* out = p.part + int64_t(blockIdx.y) * 2 * p.D + d;
    out[0] = (sw[0][lane] + sw[1][lane]) + (sw[2][lane] + sw[3][lane]);
    out[p.D] = (sb[0][lane] + sb[1][lane]) + (sb[2][lane] + sb[3][lane]);
  }
}

// d_w (blockIdx.y = 0) and d_b (1) from the slab partials: 16 columns per workgroup,
// sixteen threads per column each adding every sixteenth slab in ascending order (eight
// loads in flight), then the sixteen by a fixed tree.
template <class W>
__global__ __launch_bounds__(256) void k_norm_fold(NormBwdArgs p) {
  __shared__ float s[16][17];
  W* out = static_cast<W*>(blockIdx.y == 0 ? p.d_weight : p.d_bias);
  if (out == nullptr) return;
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t d = int64_t(blockIdx.x) * 16 + c;
  float a = 0.f;
  if (d < p.D) {
    const float* src = p.part + int64_t(blockIdx.y) * p.D + d;
    for (int64_t k = q; k < p.slabs; k += 128) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = k + 16 * u < p.slabs ? src[(k + 16 * u) * 2 * p.D] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
  }
  s[q][c] = a;
#pragma unroll
  for (int h = 8; h >= 1; h >>= 1) {
    __syncthreads();
    if (q < h) s[q][c] += s[q + h][c];
  }
  if (q == 0 && d < p.D) out[d] = W(s[0][c]);
}

// Rows beyond this many workgroups are taken in turn (a launch holds fewer than 2^32
// threads).
unsigned row_grid(int64_t N) { return unsigned(std::min<int64_t>(N, 1 << 20)); }

// A thread holds up to 8 chunks of a 16-bit row or 6 of an fp32 one (a seventh spills in
// the backward).  Rows that fit one wave that way belong to one wave, which needs no
// barrier; wider ones to four; beyond that the looping kernels take them.
template <class T>
constexpr int kMaxChunks = sizeof(T) == 2 ? 8 : 6;
template <class T>
constexpr int64_t kTeamMax = int64_t(256) * kMaxChunks<T> * kChunk;

// f(TEAM, NCH) for the smallest instance that holds a row.
template <class T, class F>
void by_width(int64_t D, F f) {
  using std::integral_constant;
  const int64_t chunks = (D + kChunk - 1) / kChunk;
  if (chunks <= 64 * kMaxChunks<T>) {
    const int64_t k = (chunks + 63) / 64;
    constexpr integral_constant<int, 64> w{};
    if (k <= 1) return f(w, integral_constant<int, 1>{});
    if (k <= 2) return f(w, integral_constant<int, 2>{});
    if (k <= 4) return f(w, integral_constant<int, 4>{});
    if (k <= 6) return f(w, integral_constant<int, 6>{});
    if constexpr (kMaxChunks<T> > 6) return f(w, integral_constant<int, 8>{});
  }
  const int64_t k = (chunks + 255) / 256;
  constexpr integral_constant<int, 256> w{};
  if (sizeof(T) == 4 && k <= 2) return f(w, integral_constant<int, sizeof(T) == 4 ? 2 : 4>{});
  if (k <= 4) return f(w, integral_constant<int, 4>{});
  if (k <= 6) return f(w, integral_constant<int, 6>{});
  if constexpr (kMaxChunks<T> > 6) return f(w, integral_constant<int, 8>{});
}

template <class T, class W>
hipError_t norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  if (a.D > kTeamMax<T>) {
    hipLaunchKernelGGL((k_norm_fwd<T, W>), dim3(row_grid(a.N)), dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
  }
  hipError_t e = hipSuccess;
  by_width<T>(a.D, [&](auto team, auto nch) {
    constexpr int kTeam = decltype(team)::value, kNch = decltype(nch)::value;
    constexpr int64_t kTeams = kTeamThreads / kTeam;
    static std::atomic<int> ready[kMaxDevices];
    e = prepare(k_norm_fwd_row<T, kTeam, kNch>, 2 * kTeam * kNch * kChunk * 4, ready);
    if (e != hipSuccess) return;
    const int64_t grid = std::min<int64_t>((a.N + kTeams - 1) / kTeams, kFwdGroups);
    const size_t lds = size_t((a.D + kChunk - 1) / kChunk) * kChunk * 2 * 4;
    hipLaunchKernelGGL((k_norm_fwd_row<T, kTeam, kNch>), dim3(unsigned(grid)), dim3(kTeamThreads),
                       lds, s, a);
  });
  return e != hipSuccess ? e : hipGetLastError();
}

template <class T, class W>
hipError_t norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  const bool params = a.d_weight != nullptr || a.d_bias != nullptr;
  if (a.D > kTeamMax<T>) {
    if (a.d_x != nullptr)
      hipLaunchKernelGGL((k_norm_dx<T, W>), dim3(row_grid(a.N)), dim3(kRowThreads), 0, s, a);
    if (params && a.slabs > 0)
      hipLaunchKernelGGL(k_norm_params<T>, dim3(unsigned((a.D + 63) / 64), unsigned(a.slabs)),
                         dim3(256), 0, s, a);
  } else if (a.slabs > 0) {
    hipError_t e = hipSuccess;
    by_width<T>(a.D, [&](auto team, auto nch) {
      constexpr int kTeam = decltype(team)::value, kNch = decltype(nch)::value;
      static std::atomic<int> ready[kMaxDevices];
      e = prepare(k_norm_bwd_row<T, kTeam, kNch>, kTeamThreads * kNch * kChunk * 4, ready);
      if (e != hipSuccess) return;
      // the weights, then a sum per team
      const size_t lds = size_t((a.D + kChunk - 1) / kChunk) * kChunk * 4 * (kTeamThreads / kTeam);
      hipLaunchKernelGGL((k_norm_bwd_row<T, kTeam, kNch>), dim3(unsigned(a.slabs)),
                         dim3(kTeamThreads), lds, s, a);
    });
    if (e != hipSuccess) return e;
  }
  if (params)
    hipLaunchKernelGGL(k_norm_fold<W>, dim3(unsigned((a.D + 15) / 16), 2), dim3(256), 0, s, a);
  return hipGetLastError();
}

// f(element type, parameter type): the parameters have the rows' type or fp32.
template <class F>
hipError_t by_types(flp_dtype x, flp_dtype w, F f) {
  if (x == FLP_F32) return f(float{}, float{});
  if (x == FLP_BF16) return w == FLP_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
  return w == FLP_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
}

}  // namespace

hipError_t launch_layer_norm_forward(flp_dtype x, flp_dtype w, const NormFwdArgs& a,
                                     hipStream_t s) {
  ProfScope ps(FLP_K_LAYER_NORM, s);
  NormFwdArgs b = a;
  b.wide = w == FLP_F32;
  return by_types(x, w, [&](auto t, auto u) { return norm_fwd<decltype(t), decltype(u)>(b, s); });
}

hipError_t launch_layer_norm_backward(flp_dtype x, flp_dtype w, const NormBwdArgs& a,
                                      hipStream_t s) {
  ProfScope ps(FLP_K_LAYER_NORM, s);
  NormBwdArgs b = a;
  b.wide = w == FLP_F32;
  if (a.d_weight == nullptr && a.d_bias == nullptr) b.part = nullptr;
  return by_types(x, w, [&](auto t, auto u) { return norm_bwd<decltype(t), decltype(u)>(b, s); });
}

}  // namespace flp
