// The gated projection of a feed-forward block, forward and backward:
//
//   z = x Wg^T,  u = x Wu^T,  out = act(z) u
//   dz = grad u act'(z),  du = grad act(z)
//   d_x = dz Wg + du Wu,  d_Wg = dz^T x,  d_Wu = du^T x
//
// Forward: one pass of the MFMA engine whose B operand interleaves the two weights, so that
// a lane holds z and u of the same elements and the epilogue needs nothing else.  For the
// backward it keeps a = act(z) and b = u act'(z), so that no third product is needed:
// dz = grad b, du = grad a.  Beside 16-bit types they are kept in 24 bits (fp32 without its
// last 8): kept in 16, their roundings make the gradients' error 3.1e-3 where the rounding of
// dz, du and the result alone gives 2.4e-3.
//
// Backward: dz and du side by side, rounded to the element type that the matrix instructions
// take, and two products, d_x = [dz | du] [Wg; Wu] and [d_Wg; d_Wu] = [dz | du]^T x.  The
// 16-bit ones read every operand as it lies and turn it on the way from LDS to the registers
// (flp_tr.h); the fp32 ones take transposed copies, which cost little beside their products.
//
// Bound by the matrix instructions for many rows, by reading the weights for few.  Measured: 16384 x
// 2688 x 7168 bf16 silu forward 1042 to 1110 us by the box (1210 to 1140 TFLOP/s with act and 0.94 GB of
// stores; a library product of the size alone 920), dz 269 (1.41 GB, 5.2 TB/s), d_x 933 to 970
// (1350 to 1300 TFLOP/s), both weights' 1036 to 1095 (1220 to 1150); one row of 2688 x 7168 12.4 us
// (6.2 TB/s, part of it from the Infinity Cache).  fp32, 4096 x 1344 x 3584: forward 645 us
// (122 TFLOP/s; a library product 154), operands 133, d_x 835 (94), weights' 719 (110).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "flp_chunk.h"
#include "flp_engine.h"
#include "flp_gemm.h"
#include "flp_launch.h"
#include "flp_tr.h"

namespace flp {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + exp(-v)); no cancellation on either side.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

// The factor f(z) of act(z) = z f(z): the logistic function (silu), the normal distribution's
// (gelu), or the logistic one of its odd cubic approximation (gelu_tanh: 0.5 (1 + tanh v) is
// the logistic function of 2 v).
//
// gelu: with x = |z| / sqrt(2) and t = 1 / (1 + 0.4 x), 0.5 erfc(x) exp(x^2) is t times a polynomial
// of t to 1.3e-7 of its value for every x (a weighted least-squares fit of degree 8), and the
// exponential is the one that the slope needs: 20 instructions, where the library's erfc alone
// takes some 60.  The exponentials' arguments are rounded fp32 products, so that a factor's relative
// error grows with its exponent: z^2 roundings on gelu's far side (1e-5 of a factor of 1e-38 at
// z = -13), |v| of them in the logistic function of v < 0; on the scale of z both stay at a few 1e-7.
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
constexpr float kTail[9] = {0.112837933f, 0.112834759f, 0.103921957f, 0.084266752f, 0.0707311779f, -0.00283535989f, 0.084579125f, -0.0914728194f, 0.0251365416f};
// f(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void act_of(float z, float& f, float& slope) {
  if constexpr (ACT == FLP_ACT_GELU) {
    const float q = fast_exp2(-0.5f * kLog2e * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.4f * 0.70710678118654752f, 1.0f));
    float p = kTail[8];
#pragma unroll
    for (int k = 7; k >= 0; --k) p = fmaf(p, t, kTail[k]);
    const float tail = p * t * q;
    f = z < 0.f ? tail : 1.0f - tail;
    slope = fmaf(z * 0.39894228040143268f, q, f);
  } else if constexpr (ACT == FLP_ACT_GELU_TANH) {
    const float zz = fminf(z * z, 0x1p120f);  // finite: f (1 - f) = 0 meets it in the slope
    f = sigmoid(kTanhA * z * fmaf(kTanhB, zz, 1.0f));
    slope = fmaf(z * f * (1.0f - f), kTanhA * fmaf(3.0f * kTanhB, zz, 1.0f), f);
  } else {
    f = sigmoid(z);
    slope = f * fmaf(z, 1.0f - f, 1.0f);
  }
}

// What the forward keeps of four consecutive columns of a row: a and b, 12 bytes each (the upper
// halves of their fp32 values, then the next bytes) or, in fp32, 16.  A block of 16 x 16 elements
// is one MFMA tile in the order of its lanes, so that every store is one contiguous piece: 16
// bytes of each lane (row i % 16, columns 4 (lane / 16)), then the rest of each.  (In rows, a
// lane's 24 bytes after the other's, the forward of 16384 x 2688 x 7168 took 1100 us, now 1042.)
template <class E>
struct Kept {
  static constexpr int kRest = E::kSize == 2 ? 8 : 16;  // bytes of a lane's second piece
  static constexpr int kBlock = 64 * (16 + kRest);
  static __device__ __forceinline__ int64_t block(int64_t row, int64_t col, int64_t ld) {
    return ((row >> 4) * (ld >> 4) + (col >> 4)) * kBlock;
  }
  static __device__ __forceinline__ int lane(int64_t row, int64_t col) {
    return int((col >> 2) & 3) * 16 + int(row & 15);
  }
  struct Packed {
    uint32_t h0, h1, lo;
  };
  // Four values to 24 bits, to nearest: half a step is added and the rest cut off.  Infinities
  // stay, and so do NaN, whose last bits are zeros (they come from 16-bit operands or are the
  // instructions' own).
  __device__ __forceinline__ static Packed pack(const f32x4_t& v) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(v[e]) + 0x80u;
    return {__builtin_amdgcn_perm(b[1], b[0], 0x07060302u),
            __builtin_amdgcn_perm(b[3], b[2], 0x07060302u),
            __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0501u) |
                __builtin_amdgcn_perm(b[3], b[2], 0x05010C0Cu)};
  }
  __device__ __forceinline__ static void store(char* block, int lane, const f32x4_t& a,
                                               const f32x4_t& b) {
    u32x4* const first = reinterpret_cast<u32x4*>(block) + lane;
    if constexpr (E::kSize == 2) {
      const Packed u = pack(a), v = pack(b);
      *first = u32x4{u.h0, u.h1, v.h0, v.h1};
      reinterpret_cast<u32x2*>(block + 1024)[lane] = u32x2{u.lo, v.lo};
    } else {
      *reinterpret_cast<f32x4_t*>(first) = a;
      reinterpret_cast<f32x4_t*>(block + 1024)[lane] = b;
    }
  }
  __device__ __forceinline__ static void unpack(uint32_t h0, uint32_t h1, uint32_t lo, float* v) {
    v[0] = __uint_as_float((h0 << 16) | ((lo << 8) & 0xFF00u));
    v[1] = __uint_as_float((h0 & 0xFFFF0000u) | (lo & 0xFF00u));
    v[2] = __uint_as_float((h1 << 16) | ((lo >> 8) & 0xFF00u));
    v[3] = __uint_as_float((h1 & 0xFFFF0000u) | ((lo >> 16) & 0xFF00u));
  }
  // Four columns: a and b.
  __device__ __forceinline__ static void load4(const char* block, int lane, float* a, float* b) {
    const u32x4 w = reinterpret_cast<const u32x4*>(block)[lane];
    if constexpr (E::kSize == 2) {
      const u32x2 l = reinterpret_cast<const u32x2*>(block + 1024)[lane];
      unpack(w.x, w.y, l.x, a);
      unpack(w.z, w.w, l.y, b);
    } else {
      const u32x4 v = reinterpret_cast<const u32x4*>(block + 1024)[lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __uint_as_float(w[e]);
        b[e] = __uint_as_float(v[e]);
      }
    }
  }
};

// The B operand of a forward tile of BN rows, CW for each column of waves: of a wave's rows the
// first half are rows of Wg, the second the same rows of Wu.
template <int BN, int NW, int CW>
struct PairTile {
  using Plain = DTile<BN, NW>;
  static constexpr int kHalf = CW / 2;
  static_assert(kHalf % 8 == 0, "an instruction loads eight rows of one weight");
  const char* up;  // first row of the tile in Wu (the base that issue gets is Wg's)
  int q, c0, c1;
  int64_t ld, ks, rows_valid;
  bool full;

  __device__ __forceinline__ void init(int64_t ld_, int64_t ks_, int64_t rows_valid_, int lane,
                                       const char* up_) {
    up = up_;
    ld = ld_;
    ks = ks_;
    rows_valid = rows_valid_;
    full = rows_valid_ >= BN / 2;
    q = lane >> 3;
    c0 = (lane & 7) ^ (q >> 1);
    c1 = c0 ^ 4;
  }
  __device__ __forceinline__ void issue(const char* base, int stage, bool half, u32x4* lds,
                                        int wave) const {
    const int64_t at = int64_t(stage) * ks;
#pragma unroll
    for (int j = 0; j < Plain::kPer; ++j) {
      const int inst = wave * Plain::kPer + j;
      if (Plain::kInsts % NW == 0 || inst < Plain::kInsts) {
        const int first = inst * 8, in = first % CW;
        const char* sb = (in < kHalf ? base : up) + at;
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void*)sb, (short)0, 0x7FFFFFFF, 0x00020000);
        int c = (inst & 1) ? c1 : c0;
        c = half ? (c & 3) : c;
        int64_t r = first / CW * kHalf + in % kHalf + q;
        if (!full) r = r < rows_valid ? r : rows_valid - 1;
        const uint32_t off = uint32_t(r * ld) + uint32_t(c * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(lds + inst * 64), 16, int(off), 0, 0, 0);
      }
    }
  }
};

// Four consecutive values to an address that only fits the element, n of them valid.
template <class E>
__device__ __forceinline__ void store_loose4(void* base, int64_t idx, const f32x4_t& v, int64_t n) {
  if constexpr (E::kSize == 2) {
    typedef u32x2 loose2 __attribute__((aligned(2)));
    uint16_t* p = static_cast<uint16_t*>(base) + idx;
    if (n >= 4) {
      *reinterpret_cast<loose2*>(p) = u32x2{pack2<E>(v.x, v.y), pack2<E>(v.z, v.w)};
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < n) p[r] = uint16_t(bits16<E>(v[r]));
    }
  } else {
    typedef f32x4_t loose4 __attribute__((aligned(4)));
    float* p = static_cast<float*>(base) + idx;
    if (n >= 4) {
      *reinterpret_cast<loose4*>(p) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < n) p[r] = v[r];
    }
  }
}

template <class E, int BM, int BN, int WM, int WN, int NS, bool ODD, int ACT>
__global__ __launch_bounds__(64 * WM * WN) void k_gated_fwd(GatedFwdArgs p) {
  using Eng = Engine<E, BM, BN, WM, WN, NS>;
  constexpr int RW = Eng::RW, CW = Eng::CW, WMB = Eng::WMB, WNB = Eng::WNB, kHalf = CW / 2;
  static_assert(WNB % 2 == 0, "a wave holds z and u of the same columns");
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  constexpr int kCols = BN / 2;
  const int nbm = int((p.N + BM - 1) / BM), nbn = int((p.F + kCols - 1) / kCols);
  int tm, tn;
  tile_of(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t row0 = int64_t(tm) * BM, col0 = int64_t(tn) * kCols;
  const int64_t kbytes = p.D * E::kSize;
  f32x4_t acc[WMB][WNB];
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < WNB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Eng::template walk<ODD, PairTile<BN, Eng::NW, CW>>(
      acc, static_cast<const char*>(p.x) + row0 * kbytes, kbytes, 128, p.N - row0,
      static_cast<const char*>(p.w_gate) + col0 * kbytes, kbytes, 128, p.F - col0, kbytes, smem,
      static_cast<const char*>(p.w_up) + col0 * kbytes);
#pragma unroll
  for (int mb = 0; mb < WMB; ++mb) {
    const int64_t row = row0 + wm * RW + mb * 16 + i;
    if (row >= p.N) continue;
#pragma unroll
    for (int nb = 0; nb < WNB / 2; ++nb) {
      const int64_t col = col0 + wn * kHalf + nb * 16 + 4 * g;
      if (col >= p.F) continue;
      const f32x4_t z = acc[mb][nb], u = acc[mb][nb + WNB / 2];
      f32x4_t a, b;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float f, slope;
        act_of<ACT>(z[r], f, slope);
        a[r] = z[r] * f;
        b[r] = u[r] * slope;
      }
      if (p.saved != nullptr)
        Kept<E>::store(static_cast<char*>(p.saved) + Kept<E>::block(row, col, p.ld_saved), lane, a,
                       b);
      store_loose4<E>(p.out, row * p.F + col, a * u, p.F - col);
    }
  }
}

// ---- dz and du, for both products -------------------------------------------------------------

template <class E>
struct Elem;
template <>
struct Elem<BF16> {
  using T = __bf16;
};
template <>
struct Elem<F16> {
  using T = _Float16;
};
template <>
struct Elem<F32> {
  using T = float;
};

// What the lanes of a wave wrote to LDS is there for its other lanes behind this.  The hardware keeps
// a wave's LDS accesses in order, so it costs no instruction; the fences keep the compiler to it.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// fp16 holds normal values from 2^-14 to 2^16 only.  Where the largest finite dz or du of a call leaves
// [1, 2^15), all of them are multiplied by the power of two that takes it to about 2^10, and the
// products' fp32 sums by its inverse: gradients of 1e-6, whose dz would keep 5 of their 11 bits,
// then lose none, and ones above 65504 stay finite.  Within those limits nothing is changed.  The
// largest is known when dz has been made: a second launch makes it again with its factor, or ends at
// once, as ordinary gradients let it (5 us at 1000 x 3587, where looking for the largest first took
// 10; 12 at 16384 x 7168).
//
// The factor's exponent, from the largest values of `parts` workgroups; all threads call it.
__device__ __forceinline__ int fp16_exponent(const float* top, int parts) {
  __shared__ float tops[4];
  float m = 0.f;
  for (int k = threadIdx.x; k < parts; k += 256) m = fmaxf(m, top[k]);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  if (m == 0.f || (m >= 1.0f && m < 0x1p15f)) return 0;
  return min(10 + 127 - int(__float_as_uint(m) >> 23), 120);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// 16-bit types: [dz | du] as rows.  A wave takes 16 rows x 64 columns: the gradient as whole
// lines, through LDS into the lanes of the kept blocks, and dz and du back through LDS into whole
// lines (straight from the lanes, 32 bytes of a row at a time, 361 us for 16384 x 7168; 280 with
// lines both ways).  Columns past F are zeros.
enum DzPass {
  kOnly,   // bf16
  kFirst,  // fp16: without a factor, and their largest finite magnitudes, one for each workgroup
  kAgain,  // fp16: with the factor, if there is one; behind the magnitudes, its inverse
};
template <class E, DzPass PASS>
__global__ __launch_bounds__(256) void k_gated_dz(GatedDzArgs p) {
  using T = typename Elem<E>::T;
  constexpr int kPitch = 72;  // elements of a row in LDS: 16 bytes more than its 64
  __shared__ __attribute__((aligned(16))) uint16_t tiles[4][2][16 * kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t* const one = tiles[wave][0];
  uint16_t* const two = tiles[wave][1];
  const int i = lane & 15, g = lane >> 4;  // of the kept blocks
  const int lr = lane >> 3, lc = (lane & 7) * 8;  // of the lines: rows lr and lr + 8
  float factor = 1.0f, top = 0.f;
  if constexpr (PASS == kAgain) {
    const int e = fp16_exponent(p.top, p.parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.top[p.parts] = power_of_two(-e);
    if (e == 0) return;
    factor = power_of_two(e);
  }
  auto tile = [&](int64_t row0, int64_t col0) {
    Chunk<T> gr[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t row = row0 + lr + 8 * q;
      gr[q].load(static_cast<const T*>(p.grad) + row * p.F + col0 + lc,
                 row < p.N ? p.F - (col0 + lc) : 0);
    }
    float a[4][4], b[4][4];
    const char* const block = static_cast<const char*>(p.saved) + Kept<E>::block(row0, col0, p.ld_saved);
#pragma unroll
    for (int k = 0; k < 4; ++k) Kept<E>::load4(block + k * Kept<E>::kBlock, lane, a[k], b[k]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<u32x4*>(one + (lr + 8 * q) * kPitch + lc) = gr[q].w[0];
    wave_exchange();  // the lines have been written by all lanes
    u32x2 dz[4], du[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      typedef T vec __attribute__((ext_vector_type(4)));
      const int at = i * kPitch + k * 16 + 4 * g;
      const vec gv = *reinterpret_cast<const vec*>(one + at);
      // what was kept past the rows' and columns' ends was not written: no product of it
      const int64_t n = row0 + i < p.N ? p.F - (col0 + k * 16 + 4 * g) : 0;
      float z[4], u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gf = float(T(gv[e]));
        z[e] = e < n ? gf * b[k][e] : 0.f;
        u[e] = e < n ? gf * a[k][e] : 0.f;
        if constexpr (PASS == kAgain) z[e] *= factor, u[e] *= factor;
        if constexpr (PASS == kFirst) {
          const float x = fabsf(z[e]), y = fabsf(u[e]);
          top = fmaxf(top, fmaxf(x < __builtin_inff() ? x : 0.f, y < __builtin_inff() ? y : 0.f));
        }
      }
      dz[k] = u32x2{pack2<E>(z[0], z[1]), pack2<E>(z[2], z[3])};
      du[k] = u32x2{pack2<E>(u[0], u[1]), pack2<E>(u[2], u[3])};
    }
    wave_exchange();  // the gradient has been read
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = i * kPitch + k * 16 + 4 * g;
      *reinterpret_cast<u32x2*>(one + at) = dz[k];
      *reinterpret_cast<u32x2*>(two + at) = du[k];
    }
    wave_exchange();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t row = row0 + lr + 8 * q;
      const u32x4 z = *reinterpret_cast<const u32x4*>(one + (lr + 8 * q) * kPitch + lc);
      const u32x4 u = *reinterpret_cast<const u32x4*>(two + (lr + 8 * q) * kPitch + lc);
      if (row < p.N) {
        uint16_t* const out = static_cast<uint16_t*>(p.dz) + row * 2 * p.ld_saved + col0 + lc;
        *reinterpret_cast<u32x4*>(out) = z;
        *reinterpret_cast<u32x4*>(out + p.ld_saved) = u;
      }
    }
    wave_exchange();
  };
  const int64_t across = (p.ld_saved + 255) / 256, down = (p.N + 15) / 16;
  if constexpr (PASS == kAgain) {
    for (int64_t t = blockIdx.x; t < across * down; t += gridDim.x) {
      const int64_t col0 = t % across * 256 + wave * 64;
      if (col0 < p.ld_saved) tile(t / across * 16, col0);
    }
  } else {
    const int64_t col0 = int64_t(blockIdx.x) * 256 + wave * 64;
    if (col0 < p.ld_saved)
      for (int64_t r = blockIdx.y; r < down; r += gridDim.y) tile(r * 16, col0);
  }
  if constexpr (PASS == kFirst) {
    __shared__ float tops[4];
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    if (threadIdx.x == 0)
      p.top[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] =
          fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  }
}

// A 64 x 64 tile of src [rows][cols] to dst = src^T, K-blocked with cols rows; source rows past
// the end are zeros.
__device__ __forceinline__ void turn_tile(const float* src, int64_t rows, int64_t cols, int64_t r0,
                                          int64_t c0, float* dst, float (&tile)[64][65]) {
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int u = 0; u < 16; ++u) {  // sixteen loads in flight
    const int k = ty + 4 * u;
    tile[k][tx] = r0 + k < rows && c0 + tx < cols ? src[(r0 + k) * cols + c0 + tx] : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int k = ty + 4 * u;
    if (c0 + k < cols) dst[kblk<32>(c0 + k, r0 + tx, cols)] = tile[tx][k];
  }
}

// fp32, whose products take K-blocked operands, all of them made in one launch: dz and du in
// tiles of 64 tokens x 64 columns, whole rows in, and out of LDS the same tile by columns (dz: the
// K of d_x) and by tokens (dzT), each a contiguous piece; then the weights' transposes and x's.
// Columns past F and tokens past N are zeros.  (In four launches, 201 x 288 x 771 took 27 us
// for these.)
__global__ __launch_bounds__(256) void k_gated_dz32(GatedDzArgs p) {
  __shared__ float tile[2][64][65];
  const int t = threadIdx.x;
  const int64_t nc = p.ld_saved / 64, nd = (p.D + 63) / 64, nt = (p.N + 63) / 64;
  int64_t b = blockIdx.x;
  if (b >= nc * nt) {
    b -= nc * nt;
    if (p.wt != nullptr) {
      if (b < 2 * nc * nd) {
        const bool up = b >= nc * nd;
        if (up) b -= nc * nd;
        turn_tile(static_cast<const float*>(up ? p.w_up : p.w_gate), p.F, p.D, b / nd * 64,
                  b % nd * 64, static_cast<float*>(p.wt) + (up ? p.ld_saved * p.D : 0), tile[0]);
        return;
      }
      b -= 2 * nc * nd;
    }
    turn_tile(static_cast<const float*>(p.x), p.N, p.D, b / nd * 64, b % nd * 64,
              static_cast<float*>(p.xt), tile[0]);
    return;
  }
  const int64_t r0 = b / nc * 64, c0 = b % nc * 64;
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // four rows of blocks, the lanes as in the kept blocks
    const int rl = q * 16 + (t & 15), cl = (t >> 4) * 4;
    const int64_t row = r0 + rl, col = c0 + cl, n = row < p.N ? p.F - col : 0;
    float a[4], b[4];
    if (n > 0)
      Kept<F32>::load4(static_cast<const char*>(p.saved) + Kept<F32>::block(row, col, p.ld_saved),
                       Kept<F32>::lane(row, col), a, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = e < n ? static_cast<const float*>(p.grad)[row * p.F + col + e] : 0.f;
      tile[0][rl][cl + e] = e < n ? g * b[e] : 0.f;
      tile[1][rl][cl + e] = e < n ? g * a[e] : 0.f;
    }
  }
  __syncthreads();
  const int64_t rows_t = 2 * p.ld_saved;
  float* const dz = static_cast<float*>(p.dz);
  float* const dzT = static_cast<float*>(p.dzT);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int64_t k0 = c0 + m * p.ld_saved;  // column of [dz | du], row of its transpose
#pragma unroll
    for (int pass = 0; pass < 16; ++pass) {
      const int a = (t >> 6) + 4 * pass, b = t & 63;
      if (dz != nullptr && r0 + a < p.N) dz[kblk<32>(r0 + a, k0 + b, p.N)] = tile[m][a][b];
      if (dzT != nullptr) dzT[kblk<32>(k0 + a, r0 + b, rows_t)] = tile[m][b][a];
    }
  }
}

// ---- 16-bit products of the backward -------------------------------------------------------------
//
// d_x = [dz | du] [Wg; Wu] (turned B), [d_Wg; d_Wu] = [dz | du]^T x (both turned: TURNED), over
// all of K or, in the grid's second dimension, over slabs of it whose fp32 sums go to p.acc.
template <class E, bool TURNED, int BM, int BN, int WM, int WN, bool SLABS>
__global__ __launch_bounds__(64 * WM * WN) void k_gated_gemm(GatedGemmArgs p) {
  constexpr int NW = WM * WN, RW = BM / WM, CW = BN / WN, NA = RW / 16, NB = CW / 16;
  using OpA = std::conditional_t<TURNED, TurnedOp<BM, NW, NA, false>, PlainOp<BM, NW, NA>>;
  using OpB = TurnedOp<BN, NW, NB, !TURNED>;
  using Ring = TrRing<E, OpA, OpB, NA, NB, NW>;
  extern __shared__ u32x4 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM, i = lane & 15, g = lane >> 4;
  const int64_t M = TURNED ? 2 * p.fp : p.rows, K = TURNED ? p.rows : 2 * p.fp;
  const int nbm = int((M + BM - 1) / BM), nbn = int((p.D + BN - 1) / BN);
  int tm, tn;
  tile_of<1>(blockIdx.x, nbm, nbn, tm, tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int64_t k0 = SLABS ? int64_t(blockIdx.y) * p.slab : 0;
  const int64_t kn = SLABS ? min(p.slab, K - k0) : K;
  OpA a;
  OpB b;
  const char* const dz = static_cast<const char*>(p.dz);
  const char* const x = static_cast<const char*>(p.x);
  if constexpr (TURNED) {
    a.init(dz, dz, 0, p.rows, 4 * p.fp, m0, M, k0, lane, wave, wm * NA);
    b.init(x, x, 0, p.rows, 2 * p.D, n0, p.D, k0, lane, wave, wn * NB);
  } else {
    a.init(dz + m0 * 4 * p.fp + k0 * 2, 4 * p.fp, M - m0, lane, wm * RW);
    b.init(static_cast<const char*>(p.w_gate), static_cast<const char*>(p.w_up), p.fp, p.F, 2 * p.D,
           n0, p.D, k0, lane, wave, wn * NB);
  }
  f32x4_t acc[NA][NB];
#pragma unroll
  for (int mb = 0; mb < NA; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Ring::run(acc, a, b, int((kn + kTrRows - 1) / kTrRows), smem, wave);
  if constexpr (std::is_same_v<E, F16> && !SLABS) {
    const float back = *p.back;
#pragma unroll
    for (int mb = 0; mb < NA; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[mb][nb] *= back;
  }
  if constexpr (SLABS) {
#pragma unroll
    for (int mb = 0; mb < NA; ++mb) {
      const int64_t m = m0 + wm * RW + mb * 16 + i;
      if (m >= M) continue;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int64_t n = n0 + wn * CW + nb * 16 + 4 * g;
        if (n < p.D)
          *reinterpret_cast<f32x4_t*>(p.acc + (int64_t(blockIdx.y) * M + m) * p.D + n) = acc[mb][nb];
      }
    }
  } else {
    // The tile is staged in the ring (rows of BN values plus 16 bytes) and written as 16-byte
    // chunks of whole rows; D is a multiple of 32, so every chunk lies inside one row.
    constexpr int kRowB = BN * 2 + 16, kCh = BN * 2 / 16;
    static_assert(size_t(BM) * kRowB <= Ring::kLds, "the staged tile fits the ring");
    char* lds = reinterpret_cast<char*>(smem);
    __syncthreads();  // every wave is done reading the ring
#pragma unroll
    for (int mb = 0; mb < NA; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int rl = wm * RW + mb * 16 + i, cl = wn * CW + nb * 16 + 4 * g;
        *reinterpret_cast<u32x2*>(lds + rl * kRowB + cl * 2) =
            u32x2{pack2<E>(acc[mb][nb][0], acc[mb][nb][1]), pack2<E>(acc[mb][nb][2], acc[mb][nb][3])};
      }
    __syncthreads();
    for (int idx = tid; idx < BM * kCh; idx += 64 * NW) {
      const int rl = idx / kCh, ch = idx - rl * kCh;
      const int64_t m = m0 + rl, n = n0 + ch * 8;
      const bool up = TURNED && m >= p.fp;
      const int64_t mo = up ? m - p.fp : m;
      uint16_t* const out = static_cast<uint16_t*>(up ? p.out2 : p.out);
      if (mo < (TURNED ? p.F : M) && n < p.D && out != nullptr)
        *reinterpret_cast<u32x4*>(out + mo * p.D + n) =
            *reinterpret_cast<const u32x4*>(lds + rl * kRowB + ch * 16);
    }
  }
}

// The slabs' fp32 sums added in ascending order and rounded once.
template <class E, bool TURNED>
__global__ __launch_bounds__(256) void k_gated_fold(GatedGemmArgs p, int slabs) {
  const int64_t M = TURNED ? 2 * p.fp : p.rows, n = M * p.D;  // a multiple of 32
  float back = 1.0f;
  if constexpr (std::is_same_v<E, F16>) back = *p.back;
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
       i += int64_t(gridDim.x) * 1024) {
    f32x4_t s = *reinterpret_cast<const f32x4_t*>(p.acc + i);
    for (int k = 1; k < slabs; ++k) s += *reinterpret_cast<const f32x4_t*>(p.acc + k * n + i);
    if constexpr (std::is_same_v<E, F16>) s *= back;
    if constexpr (TURNED) {
      const int64_t half = p.fp * p.D;
      const bool up = i >= half;
      const int64_t at = up ? i - half : i;
      void* const out = up ? p.out2 : p.out;
      if (at < p.F * p.D && out != nullptr) store4<E>(out, at, s);
    } else {
      store4<E>(p.out, i, s);
    }
  }
}

// ---- launchers ----------------------------------------------------------------------------------

template <class F>
hipError_t by_act(flp_activation act, F f) {
  if (act == FLP_ACT_GELU) return f(std::integral_constant<int, FLP_ACT_GELU>{});
  if (act == FLP_ACT_GELU_TANH) return f(std::integral_constant<int, FLP_ACT_GELU_TANH>{});
  return f(std::integral_constant<int, FLP_ACT_SILU>{});
}

template <class E, int BM, int BN, int WM, int WN, int NS, bool ODD>
hipError_t fwd_cfg(const GatedFwdArgs& a, hipStream_t s) {
  using Eng = Engine<E, BM, BN, WM, WN, NS>;
  return by_act(a.act, [&](auto act) {
    constexpr int kAct = decltype(act)::value;
    static std::atomic<int> ready[kMaxDevices];
    const hipError_t e = prepare(k_gated_fwd<E, BM, BN, WM, WN, NS, ODD, kAct>, Eng::kLds, ready);
    if (e != hipSuccess) return e;
    const int64_t blocks = ((a.N + BM - 1) / BM) * ((a.F + BN / 2 - 1) / (BN / 2));
    hipLaunchKernelGGL((k_gated_fwd<E, BM, BN, WM, WN, NS, ODD, kAct>), dim3(unsigned(blocks)),
                       dim3(Eng::NT), Eng::kLds, s, a);
    return hipGetLastError();
  });
}

// The largest tile that gives most compute units a workgroup.  D x F = 2688 x 7168 bf16, tiles of
// 256, 128 and 64 rows, us: 256 rows 53, 30, 34; 512 rows 57, 43, 59; 768 rows (168 tiles of 256)
// 58, 66, 86; 2048 rows 122, 150, 216.  Tiles of 32 rows are as fast as those of 64 up to 32 rows of
// bf16 (12.4) and faster in fp32 (27 and 47).
template <class E, bool ODD>
hipError_t fwd_rows(const GatedFwdArgs& a, hipStream_t s) {
  auto fills = [&](int64_t bm, int64_t cols) {
    return (a.N + bm - 1) / bm * ((a.F + cols - 1) / cols) >= 160;
  };
  if (a.N > 128 && fills(256, 128)) return fwd_cfg<E, 256, 256, 4, 2, 2, ODD>(a, s);
  if (a.N > 64 && fills(128, 64)) return fwd_cfg<E, 128, 128, 2, 2, 2, ODD>(a, s);
  if (a.N > 32) return fwd_cfg<E, 64, 64, 2, 2, 4, ODD>(a, s);
  return fwd_cfg<E, 32, 64, 2, 2, 4, ODD>(a, s);
}

template <class E>
hipError_t fwd_all(const GatedFwdArgs& a, hipStream_t s) {
  if constexpr (E::kSize == 2)  // 32 fp32 values are two stages
    if ((a.D * E::kSize / kStageBytes) % 2 == 1) return fwd_rows<E, true>(a, s);
  return fwd_rows<E, false>(a, s);
}

template <class E, bool TURNED, int BM, int BN, int WM, int WN, bool SLABS>
hipError_t gemm16_cfg(const GatedGemmArgs& a, int64_t slabs, hipStream_t s) {
  constexpr int NW = WM * WN, NA = BM / WM / 16, NB = BN / WN / 16;
  using OpA = std::conditional_t<TURNED, TurnedOp<BM, NW, NA, false>, PlainOp<BM, NW, NA>>;
  constexpr size_t kLds = TrRing<E, OpA, TurnedOp<BN, NW, NB, !TURNED>, NA, NB, NW>::kLds;
  static std::atomic<int> ready[kMaxDevices];
  const hipError_t e = prepare(k_gated_gemm<E, TURNED, BM, BN, WM, WN, SLABS>, kLds, ready);
  if (e != hipSuccess) return e;
  const int64_t M = TURNED ? 2 * a.fp : a.rows;
  const int64_t blocks = ((M + BM - 1) / BM) * ((a.D + BN - 1) / BN);
  hipLaunchKernelGGL((k_gated_gemm<E, TURNED, BM, BN, WM, WN, SLABS>),
                     dim3(unsigned(blocks), unsigned(slabs)), dim3(64 * NW), kLds, s, a);
  return hipGetLastError();
}

// The larger tile where it gives most compute units a workgroup (a chain over K is the same in
// both, so the tile does not change the bits).  2688 x 7168 bf16, large and small, us with dz: d_x of
// 200 rows 49 and 46, 512 rows 60 and 78, 4096 rows 338 and 404; weights' of 200 rows 40 and 37,
// 1000 rows 96 and 107, 4096 rows 319 and 405.
template <class E, bool TURNED>
hipError_t gemm16(const GatedGemmArgs& a, hipStream_t s) {
  const int64_t M = TURNED ? 2 * a.fp : a.rows, K = TURNED ? a.rows : 2 * a.fp;
  const int64_t slabs = a.slab > 0 ? (K + a.slab - 1) / a.slab : 1;
  const bool large = M > 128 && ((M + 255) / 256) * ((a.D + 223) / 224) * slabs >= kGatedTiles;
  if (slabs == 1)
    return large ? gemm16_cfg<E, TURNED, 256, 224, 4, 2, false>(a, 1, s)
                 : gemm16_cfg<E, TURNED, 128, 128, 2, 2, false>(a, 1, s);
  hipError_t e = hipSuccess;
  if constexpr (TURNED) {
    // at most kGatedTiles of the smaller tiles: fewer of the larger ones
    e = gemm16_cfg<E, TURNED, 128, 128, 2, 2, true>(a, slabs, s);
  } else {
    e = large ? gemm16_cfg<E, TURNED, 256, 224, 4, 2, true>(a, slabs, s)
              : gemm16_cfg<E, TURNED, 128, 128, 2, 2, true>(a, slabs, s);
  }
  if (e != hipSuccess) return e;
  const int64_t n = M * a.D;
  hipLaunchKernelGGL((k_gated_fold<E, TURNED>),
                     dim3(unsigned(std::min<int64_t>((n + 1023) / 1024, 4096))), dim3(256), 0, s, a,
                     int(slabs));
  return hipGetLastError();
}

template <class E>
hipError_t dz16(const GatedDzArgs& a, hipStream_t s) {
  const int64_t across = (a.ld_saved + 255) / 256, down = (a.N + 15) / 16;
  if constexpr (std::is_same_v<E, F16>) {
    hipLaunchKernelGGL((k_gated_dz<E, kFirst>), dim3(unsigned(across), unsigned(a.parts / across)),
                       dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // two workgroups per compute unit, which mostly have nothing to do
    hipLaunchKernelGGL((k_gated_dz<E, kAgain>), dim3(unsigned(std::min<int64_t>(across * down, 512))),
                       dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_gated_dz<E, kOnly>),
                       dim3(unsigned(across), unsigned(std::min<int64_t>(down, 65535))), dim3(256), 0,
                       s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_dx16(flp_dtype x, const GatedGemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DHIDDEN, s);
  return x == FLP_BF16 ? gemm16<BF16, false>(a, s) : gemm16<F16, false>(a, s);
}

hipError_t launch_gated_dw16(flp_dtype x, const GatedGemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DWEIGHT, s);
  return x == FLP_BF16 ? gemm16<BF16, true>(a, s) : gemm16<F16, true>(a, s);
}

// fp32: the largest tile that gives most compute units a workgroup.
hipError_t launch_gated_dw(const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DWEIGHT, s);
  auto fills = [&](int64_t bm, int64_t bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn) >= kGatedTiles;
  };
  if (fills(128, 128)) return gemm_cfg<F32, 128, 128, 2, 2, false, 0, 2, 2, false, true>(a, s);
  if (fills(64, 64)) return gemm_cfg<F32, 64, 64, 2, 2, false, 0, 4, 4, false, true>(a, s);
  return gemm_cfg<F32, 64, 32, 4, 1, false, 0, 8, 8, false, true>(a, s);
}

hipError_t launch_gated_dx(const GemmArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_DHIDDEN, s);
  if (a.k_slab == 0) return gemm_cfg<F32, 128, 128, 2, 2, false, 0>(a, s);
  const int64_t slabs = (a.K + a.k_slab - 1) / a.k_slab;
  auto fills = [&](int64_t bm, int64_t bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn) * slabs >= kGatedTiles;
  };
  hipError_t e;
  if (a.M > 64 && fills(128, 128))
    e = gemm_cfg<F32, 128, 128, 2, 2, false, 2, 2>(a, s);
  else if (a.M > 32 && fills(64, 64))
    e = gemm_cfg<F32, 64, 64, 2, 2, false, 2, 4>(a, s);
  else
    e = gemm_cfg<F32, 64, 32, 4, 1, false, 2, 8>(a, s);
  if (e != hipSuccess) return e;
  const int64_t n = a.M * a.N;
  hipLaunchKernelGGL(k_slab_fold<F32>, dim3(unsigned(std::min<int64_t>((n + 1023) / 1024, 4096))),
                     dim3(256), 0, s, a, int(slabs));
  return hipGetLastError();
}

hipError_t launch_gated_forward(flp_dtype x, const GatedFwdArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_GATED, s);
  if (x == FLP_BF16) return fwd_all<BF16>(a, s);
  return x == FLP_F16 ? fwd_all<F16>(a, s) : fwd_all<F32>(a, s);
}

hipError_t launch_gated_dz(flp_dtype x, const GatedDzArgs& a, hipStream_t s) {
  ProfScope ps(FLP_K_GATED, s);
  if (x == FLP_BF16) return dz16<BF16>(a, s);
  if (x == FLP_F16) return dz16<F16>(a, s);
  const int64_t nc = a.ld_saved / 64, nd = (a.D + 63) / 64, nt = (a.N + 63) / 64;
  const int64_t blocks = nc * nt + (a.wt ? 2 * nc * nd : 0) + (a.xt ? nt * nd : 0);
  hipLaunchKernelGGL(k_gated_dz32, dim3(unsigned(blocks)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace flp
