// Dropout whose mask is recomputed, never stored.
//
//   out_e = keep_e ? x_e / (1 - q) : 0,   keep_e = (u_e >= 65536 q),  q = round(65536 p) / 65536
//
// u_e is the 16-bit piece e % 8 of the 128 bits that the ten-round 4 x 32 counter-based
// generator of Salmon, Moraes, Dror and Shaw ("Parallel random numbers: as easy as
// 1, 2, 3", 2011) gives for the key rng[0] and the counter (e / 8, rng[1]): the forward
// and the backward call with the same two numbers draw the same mask, and calls with
// another rng[1] draw independent ones.
//
// 16 bits per element: one generator call (20 products of 32 x 32 bits, each of a
// quarter of the rate of an addition) serves eight elements, one 16-byte chunk of a
// 16-bit row.  p is thereby rounded to a multiple of 2^-16; the scale uses the rounded
// value, so the expectation of out is exactly x.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "flp_chunk.h"
#include "flp_launch.h"

namespace flp {
namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words random_words(uint64_t block, uint64_t seed, uint64_t offset) {
  uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32);
  uint32_t c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c1 = uint32_t(b);
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// A chunk of eight elements per thread (two, four and eight at once measured slower).  A
// launch holds fewer than 2^32 threads, so very long inputs take several steps.  Bound by
// memory: 16384 x 2688 bf16 on MI355X take 32 us for 176 MB (5.5 TB/s; element by element
// it took 82).
template <class T>
__global__ __launch_bounds__(256) void k_dropout(int64_t n, const T* __restrict__ x,
                                                 const uint64_t* __restrict__ rng, uint32_t drop,
                                                 float scale, T* __restrict__ out) {
  const uint64_t seed = rng[0], offset = rng[1];
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b * kChunk < n; b += step) {
    Chunk<T> c;
    c.load(x + b * kChunk, n - b * kChunk);
    const Words r = random_words(uint64_t(b), seed, offset);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      const uint32_t bits = (k & 1) ? r.w[k >> 1] >> 16 : r.w[k >> 1] & 0xFFFFu;
      c.v[k] = bits >= drop ? T(float(T(c.v[k])) * scale) : T(0.0f);
    }
    c.store(out + b * kChunk, n - b * kChunk);
  }
}

}  // namespace

hipError_t launch_dropout(flp_dtype x_dtype, int64_t n, const void* x, const uint64_t* rng,
                          uint32_t drop, float scale, void* out, hipStream_t s) {
  ProfScope ps(FLP_K_DROPOUT, s);
  const dim3 grid(unsigned(std::min<int64_t>((n + 2047) / 2048, 1 << 22)));
  if (x_dtype == FLP_BF16)
    hipLaunchKernelGGL(k_dropout<__bf16>, grid, dim3(256), 0, s, n, static_cast<const __bf16*>(x),
                       rng, drop, scale, static_cast<__bf16*>(out));
  else if (x_dtype == FLP_F16)
    hipLaunchKernelGGL(k_dropout<_Float16>, grid, dim3(256), 0, s, n,
                       static_cast<const _Float16*>(x), rng, drop, scale,
                       static_cast<_Float16*>(out));
  else
    hipLaunchKernelGGL(k_dropout<float>, grid, dim3(256), 0, s, n, static_cast<const float*>(x),
                       rng, drop, scale, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace flp
