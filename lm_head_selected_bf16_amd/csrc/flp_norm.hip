// Layer norm over the last dimension, forward and backward.
//
//   mean_i = sum_d x_id / D,  rstd_i = 1 / sqrt(sum_d (x_id - mean_i)^2 / D + eps)
//   xhat   = (x - mean) rstd,  out = xhat w + b
//   d_x    = rstd (g - mean_d(g) - xhat mean_d(g xhat)),  g = grad w
//   d_w    = sum_i grad xhat,  d_b = sum_i grad
//
// All arithmetic is fp32 (the variance from the centred values, so a large common
// offset of a row does not cancel); out, d_x, d_w and d_b are rounded once.
//
// A row's sums run in an order fixed by D alone, so out, mean, rstd and d_x of a
// row are bitwise the same whatever the other rows are.  d_w and d_b add rows in
// fixed slabs (cut by N alone), each slab in ascending order, then the slabs in
// ascending order: no atomics, the same bits on every run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "flp_launch.h"

namespace flp {
namespace {

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return float(v);
}

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

// One workgroup per row, any D: the row is read three times (mean, variance,
// output); only the first read reaches HBM.
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
    const float mean = block_sum(s, red) / float(p.D);
    float q = 0.f;
    for (int64_t d = threadIdx.x; d < p.D; d += kRowThreads) {
      const float c = to_f32(x[d]) - mean;
      q = fmaf(c, c, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, red) / float(p.D) + p.eps);
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

// d_w (blockIdx.y = 0) and d_b (1) from the slab partials: 32 columns per
// workgroup, eight threads per column each adding every eighth slab in ascending
// order, then the eight in order.
template <class W>
__global__ __launch_bounds__(256) void k_norm_fold(NormBwdArgs p) {
  __shared__ float s[8][32];
  W* out = static_cast<W*>(blockIdx.y == 0 ? p.d_weight : p.d_bias);
  if (out == nullptr) return;
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t d = int64_t(blockIdx.x) * 32 + c;
  float a = 0.f;
  if (d < p.D)
    for (int64_t k = q; k < p.slabs; k += 8) a += p.part[(k * 2 + blockIdx.y) * p.D + d];
  s[q][c] = a;
  __syncthreads();
  if (q == 0 && d < p.D)
    out[d] = W(((s[0][c] + s[1][c]) + (s[2][c] + s[3][c])) +
               ((s[4][c] + s[5][c]) + (s[6][c] + s[7][c])));
}

// Rows beyond this many workgroups are taken in turn (a launch holds fewer than 2^32
// threads).
unsigned row_grid(int64_t N) { return unsigned(std::min<int64_t>(N, 1 << 20)); }

template <class T, class W>
hipError_t norm_fwd(const NormFwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_fwd<T, W>), dim3(row_grid(a.N)), dim3(kRowThreads), 0, s, a);
  return hipGetLastError();
}

template <class T, class W>
hipError_t norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.d_x != nullptr)
    hipLaunchKernelGGL((k_norm_dx<T, W>), dim3(row_grid(a.N)), dim3(kRowThreads), 0, s, a);
  if (a.d_weight != nullptr || a.d_bias != nullptr) {
    if (a.slabs > 0)
      hipLaunchKernelGGL(k_norm_params<T>, dim3(unsigned((a.D + 63) / 64), unsigned(a.slabs)),
                         dim3(256), 0, s, a);
    hipLaunchKernelGGL(k_norm_fold<W>, dim3(unsigned((a.D + 31) / 32), 2), dim3(256), 0, s, a);
  }
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
  return by_types(x, w, [&](auto t, auto u) { return norm_fwd<decltype(t), decltype(u)>(a, s); });
}

hipError_t launch_layer_norm_backward(flp_dtype x, flp_dtype w, const NormBwdArgs& a,
                                      hipStream_t s) {
  ProfScope ps(FLP_K_LAYER_NORM, s);
  return by_types(x, w, [&](auto t, auto u) { return norm_bwd<decltype(t), decltype(u)>(a, s); });
}

}  // namespace flp
