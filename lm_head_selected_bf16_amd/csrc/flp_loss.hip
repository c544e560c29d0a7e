// Row kernels of the linear cross entropy: what stands between the logit tiles and their
// merge (flp_kernels.hip) and the caller.  The reduced loss is a sum over the rows, and
//
//   dz_iv  = g_i ((1 + 2 c lse_i) p_iv - (1 - s) [v = t_i] - s / V)
//
// with the label smoothing s and the z-loss factor c; g_i is the upstream gradient of
// the row's loss, over the number of counted rows for a mean.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "flp_chunk.h"
#include "flp_launch.h"

namespace flp {
namespace {

__device__ __forceinline__ bool counted(const void* t, int t64, int64_t i, int64_t V) {
  const int64_t v = t64 ? static_cast<const int64_t*>(t)[i]
                        : int64_t(static_cast<const int32_t*>(t)[i]);
  return v >= 0 && v < V;
}

constexpr int kSumThreads = 1024;

// Sum over the workgroup by a fixed tree, the same bits in every thread.
template <class T>
__device__ __forceinline__ T sum_all(T v, T* red) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[threadIdx.x & 15];
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// 1 / the number of counted rows (1 if there are none), in every thread.
__device__ __forceinline__ float inverse_count(int64_t N, int64_t V, const void* targets, int t64,
                                               int64_t* red) {
  int64_t n = 0;
  for (int64_t i = threadIdx.x; i < N; i += kSumThreads) n += counted(targets, t64, i, V) ? 1 : 0;
  n = sum_all(n, red);
  return 1.0f / float(n > 0 ? n : 1);
}

__global__ __launch_bounds__(kSumThreads) void k_loss_count(int64_t N, int64_t V,
                                                            const void* targets, int t64,
                                                            float* inv) {
  __shared__ int64_t red[16];
  const float v = inverse_count(N, V, targets, t64, red);
  if (threadIdx.x == 0) *inv = v;
}

// The reduced loss, by one workgroup: a batch has few rows next to what its logits cost.
__global__ __launch_bounds__(kSumThreads) void k_loss_sum(LossSumArgs p) {
  __shared__ float fred[16];
  __shared__ int64_t ired[16];
  float s = 0.f;
  int64_t n = 0;
  for (int64_t i = threadIdx.x; i < p.N; i += kSumThreads) {
    s += p.rows[i];
    n += counted(p.targets, p.t64, i, p.V) ? 1 : 0;
  }
  s = sum_all(s, fred);
  n = sum_all(n, ired);
  if (threadIdx.x == 0)
    *p.loss = p.mean ? s / float(n > 0 ? n : 1) : s;
}

// Per-row factors of dz, by one workgroup (it counts the rows of a mean, and finds the
// largest factor for fp16, whose dz would otherwise underflow: a mean over 16384 rows has
// entries p / 16384, most of them below the 6e-8 that fp16 can hold).  The scaling is a
// power of two, so it changes no other rounding.
__global__ __launch_bounds__(kSumThreads) void k_loss_grad(LossGradArgs p) {
  __shared__ int64_t ired[16];
  __shared__ float fred[16];
  const float s = p.smoothing, zl = p.z_loss;
  float inv = 1.0f;
  if (p.reduction == FLP_REDUCE_MEAN)
    inv = p.inv != nullptr ? *p.inv : inverse_count(p.N, p.V, p.targets, p.t64, ired);
  float up = 0.f;
  if (p.reduction != FLP_REDUCE_NONE) up = (p.grad_out != nullptr ? p.grad_out[0] : 1.0f) * inv;
  const float sv = s / float(p.V);
  float big = 0.f;
  for (int64_t i = threadIdx.x; i < p.N; i += kSumThreads) {
    const bool in = counted(p.targets, p.t64, i, p.V);
    const float g = !in ? 0.f : p.reduction == FLP_REDUCE_NONE ? p.grad_out[i] : up;
    const float c = in ? g * fmaf(2.0f * zl, p.lse[i], 1.0f) : 0.f;
    p.softmax[i] = c;
    p.onehot[i] = -g * (1.0f - s);
    p.uniform[i] = -g * sv;
    big = fmaxf(big, fmaxf(fabsf(c), fabsf(g)));
  }
  float up2 = 1.0f, down = 1.0f;
  if (p.rescale) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) big = fmaxf(big, __shfl_xor(big, off));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) fred[threadIdx.x >> 6] = big;
    __syncthreads();
    big = fred[threadIdx.x & 15];
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) big = fmaxf(big, __shfl_xor(big, off));
    if (big > 0.f && big <= 3e38f) {
      int e = 10 - ilogbf(big);
      e = e > 120 ? 120 : e < -120 ? -120 : e;
      up2 = ldexpf(1.0f, e);
      down = ldexpf(1.0f, -e);
    }
    for (int64_t i = threadIdx.x; i < p.N; i += kSumThreads) {  // each thread's own entries
      p.softmax[i] *= up2;
      p.onehot[i] *= up2;
      p.uniform[i] *= up2;
    }
  }
  if (threadIdx.x == 0) *p.unscale = down;
}

// A chunk of eight elements per thread and step.  An upstream gradient of 1 (the usual
// case: loss.backward()) ends the launch after one load per thread.
template <class T>
__global__ __launch_bounds__(256) void k_scale(int64_t n, T* x, const float* factor) {
  const float f = *factor;
  if (f == 1.0f) return;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b * kChunk < n; b += step) {
    Chunk<T> c;
    c.load(x + b * kChunk, n - b * kChunk);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) c.v[k] = T(float(T(c.v[k])) * f);
    c.store(x + b * kChunk, n - b * kChunk);
  }
}

}  // namespace

hipError_t launch_loss_count(int64_t N, int64_t V, const void* targets, bool t64, float* inv,
                             hipStream_t s) {
  ProfScope ps(FLP_K_LOSS, s);
  hipLaunchKernelGGL(k_loss_count, dim3(1), dim3(kSumThreads), 0, s, N, V, targets, t64 ? 1 : 0,
                     inv);
  return hipGetLastError();
}

hipError_t launch_scale(flp_dtype x_dtype, int64_t n, void* x, const float* factor,
                        hipStream_t s) {
  ProfScope ps(FLP_K_LOSS, s);
  const dim3 grid(unsigned(std::min<int64_t>((n + 2047) / 2048, 4096)));
  if (x_dtype == FLP_BF16)
    hipLaunchKernelGGL(k_scale<__bf16>, grid, dim3(256), 0, s, n, static_cast<__bf16*>(x), factor);
  else if (x_dtype == FLP_F16)
    hipLaunchKernelGGL(k_scale<_Float16>, grid, dim3(256), 0, s, n, static_cast<_Float16*>(x),
                       factor);
  else
    hipLaunchKernelGGL(k_scale<float>, grid, dim3(256), 0, s, n, static_cast<float*>(x), factor);
  return hipGetLastError();
}

hipError_t launch_loss_sum(const LossSumArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_LOSS, s);
  hipLaunchKernelGGL(k_loss_sum, dim3(1), dim3(kSumThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_LOSS, s);
  hipLaunchKernelGGL(k_loss_grad, dim3(1), dim3(kSumThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace flp
