// One AdamW step over many tensors.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,   g = grad * grad_scale
//   p = p (1 - lr wd) - lr / (1 - b1^t)  m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// All arithmetic is fp32; p is rounded once to its type, or kept whole in an fp32 master
// copy beside it.  m and v are held in fp32, or in 8 bits: each block of 256 elements has
// a scale (its largest magnitude over 448), and an element is the e4m3 code of its ratio to
// the scale (relative rounding error 2^-4, range 2^-18 within a block).  What is held of v
// is its root: its range halves that way, and the update divides by the root.  A positive
// root never rounds to 0: a coordinate whose m survives would otherwise be divided by eps.
//
// Half a step of e4m3 is 3 to 6 % of the value, while one step of the optimizer moves the root by
// (1 - b2) / 2 of itself, 0.05 % at b2 = 0.999: rounded to nearest it would stand still.  So codes
// are rounded up or down by a threshold that runs over time evenly through all of the step between
// two codes (multiples of an irrational number, plus an offset of the element's own, a function of
// step and index alone): what a code holds is right on average, and a drift far below half a step
// arrives.  The roots' distribution around fp32's, gradients of fixed spread, and of a spread that
// fell to a tenth (5 %, median, 95 % of the elements after six windows of b2 and more):
//   b2 = 0.95    nearest 0.91 1.06 1.22, 0.90 1.03 1.25    dithered 0.85 1.00 1.16, 0.87 0.99 1.17
//   b2 = 0.98    nearest 1.14 1.57 1.96, 5.8  11.6 16.7    dithered 0.81 1.00 1.21, 0.84 0.98 1.22
//   b2 = 0.999   nearest 0.81 1.15 1.52, 6.4  9.0  13.2    dithered 0.77 1.00 1.25, 0.79 0.95 1.23
// To nearest where b1 <= 0.9 and b2 <= 0.95: there the gradients' own spread moves a root by more
// than half a step between two codes, an m without gradients decays by more than one down to five
// times the least code, and each code is within half a step of its value.  From there on 0.9 of a code
// rounds to the same code, and the element would move at a constant rate for good (0.2 lr a step beside
// others of unit gradients): an m below five least codes whose gradient adds less than half of one is
// rounded by its threshold here too, until it is 0.
//
// Bound by memory: one pass over grad, p, m, v and the master copies.  Measured: 347 M bf16
// elements with master copies and 32-bit states 1812 us, 5.36 TB/s; 584 M with 8-bit states and
// none, rounded to nearest, 1032 to 1071 us, 5.45 to 5.65 TB/s (a large copy reaches 5.1).  2^28
// bf16 elements, 8-bit states: to nearest 495 us, dithered 538 (485 and 580 with the step's number on
// the device, for which each workgroup computes its corrections); with master copies 807 and 802.
//
// The tensors of one mix of types go in launches of up to kAdamTensors; a launch's table of
// tensors is its argument, so a captured call needs no memory of its own.  The elements are
// cut into tiles of 2048 that never span two tensors.
// Every element's result is a function of its own block alone: no atomics, the same bits
// on every run and in every grouping of the tensors.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "flp_chunk.h"
#include "flp_launch.h"

namespace flp {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kThreads * kChunk;
constexpr float kTop = 448.0f;            // the largest e4m3 value
constexpr float kLeast = 0x1p-9f;         // the smallest positive one
constexpr float kFaint = 5.0f * kLeast;   // 0.9 of up to five least codes is rounded to the same again
constexpr float kBlockFloor = 0x1p-100f;  // a block's largest magnitude counts as at least this

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 loose8 __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight codes: n valid elements at p (zeros past them).
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t n) {
  if (n >= kChunk) return *reinterpret_cast<const loose8*>(p);
  u32x2 w = {0u, 0u};
#pragma unroll
  for (int k = 0; k < kChunk; ++k)
    if (k < n) w[k >> 2] |= uint32_t(p[k]) << (8 * (k & 3));
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t n, u32x2 w) {
  if (n >= kChunk) {
    *reinterpret_cast<loose8*>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < kChunk; ++k)
    if (k < n) p[k] = uint8_t(w[k >> 2] >> (8 * (k & 3)));
}

__device__ __forceinline__ void decode(u32x2 w, float scale, float (&x)[kChunk]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[h]), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[h]), true);
    x[4 * h] = lo.x * scale;
    x[4 * h + 1] = lo.y * scale;
    x[4 * h + 2] = hi.x * scale;
    x[4 * h + 3] = hi.y * scale;
  }
}

// The largest over the 32 lanes that hold a block, the same in each: quad permutations, the
// mirrors of 8 and 16 lanes, and the 16-lane swap.
__device__ __forceinline__ float block_max(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}));
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}));
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// How the states are held: fp32, or codes rounded to nearest or by the threshold of the step.
enum Held { kWide, kNearest, kDithered };

// The odd integers nearest to 2^32 times (sqrt(5) - 1) / 2, sqrt(1 / 2) and sqrt(3) / 2: multiples of
// these, modulo 2^32, fill the range evenly.
constexpr uint32_t kGolden = 0x9E3779B9u, kRoot2 = 0xB504F333u, kRoot3 = 0xDDB3D743u;

// Thresholds of a chunk (its element e has kRoot3 e more).
__device__ __forceinline__ uint32_t chunk_offset(int64_t chunk) {
  uint32_t h = (uint32_t(chunk) * kGolden) ^ (uint32_t(uint64_t(chunk) >> 32) * kRoot3);
  h ^= h >> 16;
  h *= kRoot2;
  return h ^ (h >> 15);
}

// q on the grid of e4m3, away from 0 where what it is past a grid point, as a part of the step to
// the next, is at least 1 - u / 2^32 (in 20 bits: fp32's mantissa has 20 more than e4m3's).
__device__ __forceinline__ float to_grid(float q, uint32_t u) {
  const float a = fminf(fabsf(q), kTop);
  const float base = a < 0x1p-6f ? 0x1p-6f : 0.f;  // below 2^-6 the grid's step is that of 2^-6
  const uint32_t b = (__float_as_uint(a + base) + (u >> 12)) & 0xFFF00000u;
  return q == q ? copysignf(__uint_as_float(b) - base, q) : q;
}

// Codes of x and the block's scale.  The ratio is at most 448 (1 + 2^-22), which rounds to 448.  The
// scale of a block with an infinite element is NaN, and so is then all that it holds.
// FADE: to nearest, but for small x that `added` (what its gradient added, or more where it was 0
// before) does not keep from 0.
template <bool DIVISOR, bool DITHER, bool FADE>
__device__ __forceinline__ u32x2 encode(const float (&x)[kChunk], float& scale, uint32_t u,
                                        const float (&added)[kChunk]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kChunk; ++k) top = fmaxf(top, fabsf(x[k]));
  top = fmaxf(block_max(top), kBlockFloor);
  scale = top < __builtin_inff() ? top * (1.0f / kTop) : __builtin_nanf("");
  const float inv = (1.0f / top) * kTop;
  float q[kChunk];
  bool fades = false;
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    q[k] = x[k] * inv;
    if (FADE) fades |= fabsf(q[k]) < kFaint && fabsf(added[k]) * inv < 0.5f * kLeast;
    if (DITHER) q[k] = to_grid(q[k], u + uint32_t(k) * kRoot3);
    if (DIVISOR) q[k] = x[k] > 0.f && q[k] < kLeast ? kLeast : q[k];  // NaN stays
  }
  if (FADE && __builtin_amdgcn_ballot_w64(fades) != 0) {  // of few waves
#pragma unroll
    for (int k = 0; k < kChunk; ++k)
      if (fabsf(q[k]) < kFaint && fabsf(added[k]) * inv < 0.5f * kLeast)
        q[k] = to_grid(q[k], u + uint32_t(k) * kRoot3);
  }
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    w[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true));
  }
  return w;
}

// The roots of v.  Where all of a wave's lie in the middle of fp32's range, an approximation and
// one step of Newton's iteration: correctly rounded but for a case in some ten million, at half of
// what the library's root costs, which takes the others (zeros, infinities).
__device__ __forceinline__ void roots_of(const float (&v)[kChunk], float (&root)[kChunk]) {
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int e = 1; e < kChunk; ++e) {
    lo = fminf(lo, v[e]);
    hi = fmaxf(hi, v[e]);
  }
  if (__builtin_amdgcn_ballot_w64(!(lo > 0x1p-100f && hi < 0x1p100f)) != 0) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) root[e] = sqrtf(v[e]);
    return;
  }
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    const float y = __builtin_amdgcn_rsqf(v[e]);
    const float r = v[e] * y;
    root[e] = fmaf(fmaf(-r, r, v[e]), 0.5f * y, r);
  }
}

// P, G: element types of the parameters and gradients.
//
// m and v are rounded after every product and sum, as the formula in fp32 tensors does it: codes
// rounded to nearest then agree with it bit for bit, where a fused product would move some of them
// across a rounding border.
template <class P, class G, Held HELD, bool MASTER>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamArgs a) {
  constexpr bool kEight = HELD != kWide;
  // 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t) in 64 bits: fp32 loses the early steps of b2 near 1
  double lr = a.lr, c1 = a.c1, c2 = a.c2;
  uint32_t step_now = a.step;
  if (a.lr_on_device != nullptr) lr = *a.lr_on_device;
  if (a.step_on_device != nullptr) {
    __shared__ double corrections[2];
    const int64_t step = max(*a.step_on_device, int64_t(1));
    const double t = double(step);
    step_now = uint32_t(step);
    if (threadIdx.x < 64) {  // one wave: these take some hundred instructions
      corrections[0] = -1.0 / expm1(t * a.log_b1);
      corrections[1] = 1.0 / sqrt(-expm1(t * a.log_b2));
    }
    __syncthreads();
    c1 = corrections[0];
    c2 = corrections[1];
  }
  const float rate = float(lr * c1), root_scale = float(c2);
  const float grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const int lane8 = int(threadIdx.x) * kChunk;
  // Lane k knows tensor k's first tile: a ballot finds a tile's tensor (a walk through the table
  // costs a load's latency for each tensor).
  const int lane = threadIdx.x & 63;
  const int64_t first_of = lane < a.count ? a.t[lane].first : INT64_MAX;
  AdamTensor t;
  float keep = 1.0f;
  int k = -1;

  // The tile's elements from `first` on; FULL: all of them exist.
  auto work = [&](int64_t first, auto whole) {
    constexpr bool kFull = decltype(whole)::value;
    const int64_t at = first + lane8;
    const int64_t n = kFull ? int64_t(kChunk) : t.n - at;
    float p[kChunk], m[kChunk], v[kChunk], root[kChunk], added[kChunk];
    Chunk<G> g;
    Chunk<float> w, x;
    Chunk<P> c;
    g.load(static_cast<const G*>(t.grad) + at, n);
    if constexpr (MASTER)
      w.load(t.master + at, n);
    else
      c.load(static_cast<const P*>(t.param) + at, n);
    if constexpr (kEight) {
      const int64_t block = at / kAdamBlock;
      const u32x2 cm = load_codes(static_cast<const uint8_t*>(t.m) + at, n);
      const u32x2 cv = load_codes(static_cast<const uint8_t*>(t.v) + at, n);
      decode(cm, n > 0 ? t.m_scale[block] : 0.f, m);
      decode(cv, n > 0 ? t.v_scale[block] : 0.f, v);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[e] *= v[e];
    } else {
      x.load(static_cast<const float*>(t.m) + at, n);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m[e] = x.v[e];
      x.load(static_cast<const float*>(t.v) + at, n);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[e] = x.v[e];
    }
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      if constexpr (MASTER)
        p[e] = w.v[e];
      else
        p[e] = float(P(c.v[e]));
      const float ge = float(G(g.v[e])) * grad_scale;
      added[e] = m[e] != 0.f ? a.one_b1 * ge : __builtin_inff();
      m[e] = a.b1 * m[e] + a.one_b1 * ge;
      v[e] = a.b2 * v[e] + a.one_b2 * (ge * ge);
    }
    roots_of(v, root);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const float by = __builtin_amdgcn_rcpf(fmaf(root[e], root_scale, a.eps));
      p[e] = fmaf(-rate, m[e] * by, p[e] * keep);
    }
    if constexpr (MASTER) {
      // What is rounded is the master copy as stored: the compiler would make one instruction of
      // the last sum and its rounding to fp16, which rounds the unrounded sum.
#pragma unroll
      for (int e = 0; e < kChunk; ++e) asm volatile("" : "+v"(p[e]));
#pragma unroll
      for (int e = 0; e < kChunk; ++e) w.v[e] = p[e];
      w.store(t.master + at, n);
    }
#pragma unroll
    for (int e = 0; e < kChunk; ++e) c.v[e] = P(p[e]);
    c.store(static_cast<P*>(t.param) + at, n);
    if constexpr (kEight) {
      // past the tensor's end everything is 0, which changes no block's scale
      float sm, sv;
      constexpr bool kDither = HELD == kDithered;
      const uint32_t u = chunk_offset(at / kChunk);
      const u32x2 cm = encode<false, kDither, !kDither>(m, sm, u + step_now * kGolden, added);
      const u32x2 cv = encode<true, kDither, false>(
          root, sv, ((u << 16) | (u >> 16)) + step_now * kRoot2, added);
      store_codes(static_cast<uint8_t*>(t.m) + at, n, cm);
      store_codes(static_cast<uint8_t*>(t.v) + at, n, cv);
      if ((threadIdx.x & (kAdamBlock / kChunk - 1)) == 0 && n > 0) {
        t.m_scale[at / kAdamBlock] = sm;
        t.v_scale[at / kAdamBlock] = sv;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) x.v[e] = m[e];
      x.store(static_cast<float*>(t.m) + at, n);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) x.v[e] = v[e];
      x.store(static_cast<float*>(t.v) + at, n);
    }
  };
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int now = __popcll(__builtin_amdgcn_ballot_w64(tile >= first_of)) - 1;
    if (now != k) {
      k = now;
      t = a.t[k];
      keep = float(1.0 - lr * double(t.decay));
    }
    const int64_t first = (tile - t.first) * kTile;
    if (t.n - first >= kTile)
      work(first, std::true_type{});
    else
      work(first, std::false_type{});
  }
}

// f(parameter type, gradient type): gradients have the parameters' type or fp32.
template <class F>
void by_types(flp_dtype p, flp_dtype g, F f) {
  if (p == FLP_F32) return f(float{}, float{});
  if (p == FLP_BF16) return g == FLP_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
  return g == FLP_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
}

}  // namespace

hipError_t launch_adamw(flp_dtype p, flp_dtype g, bool eight, bool master, AdamArgs& a,
                        hipStream_t s) {
  ProfScope ps(FLP_K_ADAMW, s);
  int64_t tiles = 0;
  for (int k = 0; k < a.count; ++k) {
    a.t[k].first = tiles;
    tiles += (a.t[k].n + kTile - 1) / kTile;
  }
  a.tiles = tiles;
  // A workgroup per tile (a launch holds fewer than 2^32 threads).  Workgroups that stay and take
  // tiles in turn read and write further apart: 2^28 bf16 elements with 2048 of them and with one
  // for each tile: 32-bit states 1190 and 1093 us, with master copies 1507 and 1391; 8-bit ones 613
  // and 484, 889 and 807.  Up to 2^22 elements there is no difference.
  const dim3 grid(unsigned(std::min<int64_t>(tiles, int64_t(1) << 23)));
  by_types(p, g, [&](auto x, auto y) {
    using P = decltype(x);
    using G = decltype(y);
    auto run = [&](auto held) {
      constexpr Held kHeld = decltype(held)::value;
      if (master)
        hipLaunchKernelGGL((k_adamw<P, G, kHeld, true>), grid, dim3(kThreads), 0, s, a);
      else
        hipLaunchKernelGGL((k_adamw<P, G, kHeld, false>), grid, dim3(kThreads), 0, s, a);
    };
    if (!eight)
      run(std::integral_constant<Held, kWide>{});
    else if (a.dither)
      run(std::integral_constant<Held, kDithered>{});
    else
      run(std::integral_constant<Held, kNearest>{});
  });
  return hipGetLastError();
}

}  // namespace flp
