// Rows held in registers by a team of threads, for the norms: thread t of a team of TEAM holds
// the chunks of eight elements t, t + TEAM, ... of its row.
#pragma once

#include <type_traits>

#include "flp_chunk.h"

namespace flp {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return float(v);
}

// Eight parameters as fp32 (`wide`: they are stored as fp32, else in T).
template <class T>
__device__ __forceinline__ void load_params(const void* base, bool wide, int64_t d, int64_t n,
                                            float (&x)[kChunk]) {
  if (sizeof(T) == 4 || wide) {
    Chunk<float> c;
    c.load(static_cast<const float*>(base) + d, n);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) x[k] = c.v[k];
  } else {
    Chunk<T> c;
    c.load(static_cast<const T*>(base) + d, n);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) x[k] = to_f32(T(c.v[k]));
  }
}

// Sum over the wave, the same bits in every lane: quad permutations, the mirrors of 8
// and 16 lanes (each then meets the other half's value), and the 16- and 32-lane swaps,
// all of them VALU moves.
__device__ __forceinline__ float wave_sum(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x += dpp(x, std::integral_constant<int, 0xB1>{});
  x += dpp(x, std::integral_constant<int, 0x4E>{});
  x += dpp(x, std::integral_constant<int, 0x141>{});
  x += dpp(x, std::integral_constant<int, 0x140>{});
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A row's chunks of one thread.
template <class T, int TEAM, int NCH>
struct Row {
  Chunk<T> c[NCH];
  __device__ __forceinline__ void load(const T* row, int64_t D, int t, bool live) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int64_t d = int64_t(k * TEAM + t) * kChunk;
      c[k].load(row + d, live ? D - d : 0);
    }
  }
};

}  // namespace flp
