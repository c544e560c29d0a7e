// Chunks of eight elements in registers, moved with 16-byte loads and stores that need no
// alignment beyond the element's (the memory path takes them at full width); a partial
// chunk goes element by element, so nothing outside a tensor is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flp {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 loose __attribute__((aligned(2)));

constexpr int kChunk = 8;

template <class T>
struct Chunk {
  static constexpr int kWords = kChunk * int(sizeof(T)) / 16;
  typedef T vec __attribute__((ext_vector_type(kChunk)));
  union {
    u32x4 w[kWords];
    vec v;
  };

  // n valid elements of the chunk at p (zeros past them); n <= 0 loads nothing.
  __device__ __forceinline__ void load(const T* p, int64_t n) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = u32x4{0u, 0u, 0u, 0u};
    if (n >= kChunk) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = reinterpret_cast<const loose*>(p)[k];
    } else if (n > 0) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (k < n) v[k] = p[k];
    }
  }
  __device__ __forceinline__ void store(T* p, int64_t n) const {
    if (n >= kChunk) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) reinterpret_cast<loose*>(p)[k] = w[k];
    } else if (n > 0) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (k < n) p[k] = v[k];
    }
  }
};

}  // namespace flp
